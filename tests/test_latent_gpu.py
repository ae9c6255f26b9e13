"""The latent attention operators on the GPU against plain 64-bit computations on the CPU
(latent_reference.py, which derives the bounds)."""
import math
import random

import pytest
import torch

import latent_reference as ref

pytestmark = pytest.mark.gpu
L, ROT, DIM, HEAD = 512, 64, 576, 128
SCALE = (HEAD + ROT) ** -0.5
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sk():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_skinny_addmm_amd as d
    d.ops.lib()
    return d


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(BF)


def inv_freq(base=10000.0):
    return base ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT)


# ------------------------------------------------------------------------------------ append

def append_case(sk, n, heads, page, interleaved, weight=True, seed=0, far=False, stride=0, spare=3):
    print("append", dict(n=n, heads=heads, page=page, interleaved=interleaved, weight=weight, seed=seed), flush=True)
    g = gen(seed)
    pages = -(-max(n, 1) // page) + spare
    kv = normal(g, n, DIM + stride)[:, :DIM]
    cache = normal(g, pages, page, DIM)
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[5::7] = -1
    slots[6::11] = pages * page + 3                       # past the cache: dropped too
    pos = torch.randint(0, 1 << 20, (n,), generator=g) if far else torch.arange(n)
    w = (1 + 0.1 * torch.randn(L, generator=g)).to(BF) if weight else None
    q = normal(g, n, heads, DIM)[:, :, L:]
    dev = dict(kv=kv.cuda(), cache=cache.cuda(), slots=slots.cuda(), pos=pos.cuda(), w=w.cuda() if weight else None)
    if stride:
        wide = torch.zeros(n, DIM + stride, dtype=BF, device="cuda")
        wide[:, :DIM] = dev["kv"]
        dev["kv"] = wide[:, :DIM]
    qd = torch.empty(n, heads, DIM, dtype=BF, device="cuda")
    qd[:, :, L:] = q.cuda()
    out = sk.latent_append(dev["kv"], dev["cache"], dev["slots"], dev["pos"], inv_freq().cuda(), norm_weight=dev["w"],
                           eps=1e-6, q=qd[:, :, L:] if heads else None, interleaved=interleaved)
    torch.cuda.synchronize()
    rows, bound = ref.append(kv, pos, inv_freq(), w, 1e-6, interleaved)
    kept = (slots >= 0) & (slots < pages * page)
    want = cache.double().view(-1, DIM).clone()
    want[slots[kept]] = rows[kept]
    limit = torch.zeros_like(want)
    limit[slots[kept]] = bound[kept]
    got = dev["cache"].cpu().double().view(-1, DIM)
    assert bool(((got - want).abs() <= limit).all()), (got - want).abs().max()
    if heads:
        y, m = ref.turned(q, pos, inv_freq(), interleaved)
        assert bool(((out.cpu().double() - y).abs() <= ref.HALF * y.abs() + (1 + ref.HALF) * m * 2.0 ** -21).all())
    else:
        assert out is None


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,page", [(1, 8, 64), (1, 0, 16), (3, 1, 1), (67, 5, 24), (130, 20, 16), (515, 128, 64)])
def test_append(sk, n, heads, page, interleaved):
    append_case(sk, n, heads, page, interleaved, far=n > 3, seed=n)


def test_append_without_norm_and_strided(sk):
    append_case(sk, 33, 4, 16, False, weight=False, far=True)
    append_case(sk, 33, 4, 16, True, stride=24, far=True)


def test_append_nothing(sk):
    cache = torch.ones(2, 4, DIM, dtype=BF, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert sk.latent_append(torch.empty(0, DIM, dtype=BF, device="cuda"), cache, none, none, inv_freq().cuda()) is None
    assert bool((cache == 1).all())


def test_append_queries_in_place(sk):
    g = gen(3)
    kv, q = normal(g, 19, DIM).cuda(), normal(g, 19, 12, DIM).cuda()
    slots, pos = torch.arange(19).cuda(), (torch.arange(19) * 1001).cuda()
    cache = torch.zeros(2, 16, DIM, dtype=BF, device="cuda")
    apart = sk.latent_append(kv, cache, slots, pos, inv_freq().cuda(), q=q[:, :, L:])
    before = q[:, :, :L].clone()
    sk.latent_append(kv, cache, slots, pos, inv_freq().cuda(), q=q[:, :, L:], q_out=q[:, :, L:])
    assert torch.equal(q[:, :, L:], apart) and torch.equal(q[:, :, :L], before)


# ------------------------------------------------------------------------------------ decode

def paged(g, lens, page, spare=2, extra_cols=0, scale=1.0):
    """A cache of random rows, a table of shuffled pages whose unused entries are nonsense, lens."""
    counts = [-(-n // page) for n in lens]
    order = torch.randperm(sum(counts) + spare, generator=g).int()
    table = torch.full((len(lens), max(counts + [1]) + extra_cols), 2 ** 30, dtype=torch.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    return (normal(g, sum(counts) + spare, page, DIM).float() * scale).to(BF), table, torch.tensor(lens, dtype=torch.int32)


def decode_case(sk, lens, heads, tokens, page, seed=0, scale=SCALE, spread=1.0):
    print("decode", dict(lens=lens[:8], heads=heads, tokens=tokens, page=page, seed=seed), flush=True)
    g = gen(seed)
    cache, table, n = paged(g, lens, page, scale=spread)
    q = normal(g, len(lens) * tokens, heads, DIM)
    out, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), scale, tokens=tokens)
    torch.cuda.synchronize()
    ref.check_decode(out, lse, q, cache, table, n, scale, tokens, "decode")


@pytest.mark.parametrize("page", [1, 16, 48, 64, 128])
def test_decode_lengths(sk, page):
    decode_case(sk, [1, 0, 31, 32, 33, 63, 64, 65, 127, 129, 500, 2], 8, 1, page, seed=page)


@pytest.mark.parametrize("heads,tokens", [(1, 1), (3, 1), (16, 1), (10, 2), (32, 1), (8, 4), (20, 2), (64, 1), (65, 1),
                                          (128, 1), (40, 4), (64, 3), (128, 2), (16, 16), (1, 7)])
def test_decode_shapes(sk, heads, tokens):
    decode_case(sk, [tokens, tokens + 1, 100, 333, 0, tokens - 1, 64 + tokens], heads, tokens, 16, seed=heads + tokens)


@pytest.mark.parametrize("heads", [8, 32, 64, 128])
def test_decode_long(sk, heads):
    """Many workgroups a request, partial sums joined; growing scores move the reference maximum."""
    decode_case(sk, [9001], heads, 1, 64, seed=heads)
    decode_case(sk, [3000, 17, 0, 5000], heads, 1, 64, seed=heads + 1, scale=0.5)


def test_decode_many_requests(sk):
    rng = random.Random(5)
    decode_case(sk, [rng.choice((0, 1, 3, 40, 95)) for _ in range(600)], 2, 1, 16, seed=5)


def test_decode_scores_of_all_sizes(sk):
    """Scores hundreds of steps apart, the largest first, last and in between."""
    g = gen(8)
    n, heads = 700, 16
    cache, table, lens = paged(g, [n] * 3, 64)
    rows = cache.view(-1, DIM)
    for i, big in enumerate((0, n - 1, n // 2)):
        rows[table[i, big // 64] * 64 + big % 64] *= 32
    q = normal(g, 3, heads, DIM)
    out, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), SCALE)
    ref.check_decode(out, lse, q, cache, table, lens, SCALE, 1, "sizes")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,tokens", [(2, 1), (2, 4), (8, 4), (16, 4), (32, 4)])
def test_decode_hidden_rows_may_hold_anything(sk, heads, tokens, bad):
    """Rows past a request's end in its last page, whole pages of others, and new tokens' rows that
    earlier tokens do not see: none may reach a row that does not see them."""
    g = gen(9)
    lens = [5, 70, 64, 1, 0, 33]
    cache, table, n = paged(g, lens, 64)
    used = torch.zeros(cache.shape[0], 64, dtype=torch.bool)
    for i, m in enumerate(lens):
        k = torch.arange(m)
        used[table[i, k // 64].long(), k % 64] = True
    cache[~used] = bad
    q = normal(g, len(lens) * tokens, heads, DIM)
    run = lambda: sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, tokens=tokens)
    out, lse = run()
    ref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, "past the end")
    if tokens == 1:
        return
    # the newest token's row: only the last token's queries see it
    for i, m in enumerate(lens):
        if m:
            cache[table[i, (m - 1) // 64], (m - 1) % 64, 17] = bad
    out, lse = run()
    o = out.view(len(lens), tokens, heads, L)
    for i, m in enumerate(lens):
        if m:
            assert not bool(torch.isfinite(o[i, -1, :, 17]).any())
    early = torch.arange(len(lens) * tokens) % tokens != tokens - 1
    want = ref.decode(q, cache, table, n, SCALE, tokens)
    for i, (answer, keys) in enumerate(want):
        rows = early[i * tokens:(i + 1) * tokens].repeat_interleave(heads)
        a = slice(i * tokens, (i + 1) * tokens)
        ref.check(out[a].reshape(tokens * heads, L).cpu()[rows], lse[a].reshape(-1).cpu()[rows],
                  tuple(x[rows] for x in answer), keys, "earlier tokens of request %d" % i)


def test_decode_strides(sk):
    g = gen(10)
    lens = [77, 130]
    cache, table, n = paged(g, lens, 32)
    q = normal(g, 2, 6, DIM)
    layers = torch.full((cache.shape[0], 3, 32, DIM + 8), math.nan, dtype=BF, device="cuda")
    layers[:, 1, :, :DIM] = cache.cuda()
    wide = torch.full((2, 9, DIM + 64), math.nan, dtype=BF, device="cuda")
    wide[:, 2:8, 64:] = q.cuda()
    tables = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    tables[:, :table.shape[1]] = table.cuda()
    store = torch.full((2, 8, L + 8), 7.0, dtype=BF, device="cuda")
    out, lse = sk.latent_decode(wide[:, 2:8, 64:], layers[:, 1, :, :DIM], tables[:, :table.shape[1]], n.cuda(), SCALE,
                                out=store[:, 1:7, :L])
    ref.check_decode(out, lse, q, cache, table, n, SCALE, 1, "strides")
    rest = torch.ones_like(store, dtype=torch.bool)
    rest[:, 1:7, :L] = False
    assert bool((store[rest] == 7).all())


def test_decode_beyond_32_bits(sk):
    """Pages that lie more than 4 GiB into the cache."""
    g = gen(11)
    small, table, lens = paged(g, [300, 77], 64)
    pages = 70000                                         # 64 * 1152 bytes each
    cache = torch.empty(pages, 64, DIM, dtype=BF, device="cuda")
    far = pages - small.shape[0]
    cache[far:] = small.cuda()
    moved = torch.where(table < small.shape[0], table + far, table)
    q = normal(g, 2, 16, DIM)
    out, lse = sk.latent_decode(q.cuda(), cache, moved.cuda(), lens.cuda(), SCALE)
    torch.cuda.synchronize()
    ref.check_decode(out, lse, q, small, table, lens, SCALE, 1, "far pages")


def test_decode_clamps_lengths_and_pages(sk):
    g = gen(12)
    cache, table, lens = paged(g, [64, 128, 20], 32)
    table[0, 1], table[1, 2] = -5, 10 ** 9
    lens[0], lens[2] = 10 ** 9, -3
    q = normal(g, 3, 8, DIM)
    out, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), SCALE)
    ref.check_decode(out, lse, q, cache, table, lens, SCALE, 1, "clamped")


def test_decode_another_stream_and_repeats(sk):
    g = gen(13)
    cache, table, lens = (t.cuda() for t in paged(g, [2000, 300, 41], 16))
    q = normal(g, 3, 24, DIM).cuda()
    work = sk.latent_decode_workspace(3, 1, 24)
    first = sk.latent_decode(q, cache, table, lens, SCALE, workspace=work)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        out, lse = sk.latent_decode(q, cache, table, lens, SCALE, workspace=work, stream=side)
        side.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_append_and_decode_in_a_graph(sk):
    """A captured decode step, replayed with new inputs and eager work in between."""
    g = gen(14)
    heads, page, B = 8, 16, 5
    cache, table, lens = (t.cuda() for t in paged(g, [90, 17, 33, 64, 200], page))
    rows = torch.tensor([89, 16, 32, 63, 199]).cuda()
    slots = (table.long()[torch.arange(B).cuda(), rows // page] * page + rows % page)
    kv, q = normal(g, B, DIM).cuda(), normal(g, B, heads, DIM).cuda()
    w, freq = torch.ones(L, dtype=BF, device="cuda"), inv_freq().cuda()
    out = torch.empty(B, heads, L, dtype=BF, device="cuda")
    lse = torch.empty(B, heads, device="cuda")
    work = sk.latent_decode_workspace(B, 1, heads)

    def step():
        sk.latent_append(kv, cache, slots, rows, freq, norm_weight=w, q=q[:, :, L:], q_out=q[:, :, L:])
        sk.latent_decode(q, cache, table, lens, SCALE, out=out, lse=lse, workspace=work)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        g = gen(100 + seed)
        nkv, nq = normal(g, B, DIM).cuda(), normal(g, B, heads, DIM).cuda()
        kv.copy_(nkv)
        q.copy_(nq)
        step()
        eager = out.clone(), lse.clone(), cache.clone()
        q.copy_(nq)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1]) and torch.equal(cache, eager[2])
    ref.check_decode(out, lse, q, cache, table, lens, SCALE, 1, "graph")


# ----------------------------------------------------------------------------------- prefill

def prefill_inputs(g, lq, lk, heads):
    kv = normal(g, sum(lk), heads, 2 * HEAD)
    return normal(g, sum(lq), heads, HEAD + ROT), kv[:, :, :HEAD], kv[:, :, HEAD:], normal(g, sum(lk), ROT)


def starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


def prefill_case(sk, lq, lk, heads, causal, seed=0, scale=SCALE):
    print("prefill", dict(lq=lq, lk=lk, heads=heads, causal=causal, seed=seed), flush=True)
    q, k, v, r = prefill_inputs(gen(seed), lq, lk, heads)
    kv = torch.cat((k, v), -1).cuda()
    out, lse = sk.latent_prefill(q.cuda(), kv[:, :, :HEAD], kv[:, :, HEAD:], r.cuda(), starts(lq), starts(lk), scale,
                                 causal=causal)
    torch.cuda.synchronize()
    ref.check_prefill(out, lse, q, k, v, r, lq, lk, scale, causal, "prefill")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([1], [1], 1), ([129], [129], 8), ([1, 2, 31, 32, 33], [1, 2, 31, 32, 33], 3),
    ([63, 64, 65, 127, 128], [63, 64, 65, 127, 128], 2), ([0, 5, 0, 300, 0], [0, 5, 7, 300, 0], 5),
    ([1, 7, 100], [500, 64, 163], 8), ([40, 1, 200], [3, 0, 130], 4), ([257], [1000], 16)])
def test_prefill(sk, lq, lk, heads, causal):
    prefill_case(sk, lq, lk, heads, causal, seed=sum(lq) + heads)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_split_keys(sk, causal):
    """Few queries, many keys: a row's keys go to several workgroups."""
    prefill_case(sk, [70], [5000], 2, causal, seed=1)
    prefill_case(sk, [3, 130], [4000, 3000], 1, causal, seed=2)
    prefill_case(sk, [10, 2000], [6000, 10], 1, causal, seed=4)
    prefill_case(sk, [64], [4096], 1, causal, seed=3, scale=0.7)


def test_prefill_many_sequences(sk):
    rng = random.Random(6)
    lens = [rng.choice((0, 1, 9, 40)) for _ in range(150)]
    prefill_case(sk, lens, [n + rng.choice((0, 3)) for n in lens], 2, True, seed=6)


def test_prefill_growing_scores(sk):
    lq = [300]
    q, k, v, r = prefill_inputs(gen(7), lq, lq, 2)
    k = (k.float() * torch.linspace(0.1, 12, 300)[:, None, None]).to(BF)
    out, lse = sk.latent_prefill(q.cuda(), k.cuda(), v.cuda(), r.cuda(), starts(lq), starts(lq), SCALE)
    ref.check_prefill(out, lse, q, k, v, r, lq, lq, SCALE, True, "growing")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,past", [(2, 0), (1, 5000)])
def test_prefill_hidden_values_may_be_anything(sk, heads, past, bad):
    """A value (and a key) that later queries see reaches none before them; those that see it get
    what is not finite."""
    lq, lk = [150], [150 + past]
    q, k, v, r = prefill_inputs(gen(8), lq, lk, heads)
    at = past + 101
    v[at, :, 5] = bad
    k[past + 140, :, 3] = math.nan
    kv = torch.cat((k, v), -1).cuda()
    out, lse = sk.latent_prefill(q.cuda(), kv[:, :, :HEAD], kv[:, :, HEAD:], r.cuda(), starts(lq), starts(lk), SCALE)
    out, lse = out.cpu(), lse.cpu()
    assert not bool(torch.isfinite(out[101:, :, 5]).any())
    assert bool(torch.isnan(out[140:]).all()) and bool(torch.isnan(lse[140:]).all())
    rest = [i for i in range(HEAD) if i != 5]
    keep = torch.arange(150) < 140
    clean = v.clone()
    clean[at, :, 5] = 0
    n = past + 140                                        # rows below 140 see none of the last 10 keys
    ref.check_prefill(out[keep][:, :, rest], lse[keep], q[keep], k[:n], clean[:n][:, :, rest], r[:n], [140], [n], SCALE,
                      True, "rest")
    n = past + 101
    ref.check_prefill(out[:101], lse[:101], q[:101], k[:n], v[:n], r[:n], [101], [n], SCALE, True, "before")


def test_prefill_strides(sk):
    g = gen(15)
    lq, lk, heads = [50, 20], [50, 90], 3
    q, k, v, r = prefill_inputs(g, lq, lk, heads)
    wide = torch.full((70, heads + 1, 200), math.nan, dtype=BF, device="cuda")
    wide[:, 1:, 8:] = q.cuda()
    vt = torch.full((heads, 140, HEAD + 8), math.nan, dtype=BF, device="cuda")
    vt[:, :, :HEAD] = v.cuda().transpose(0, 1)
    rows = torch.full((140, DIM), math.nan, dtype=BF, device="cuda")
    rows[:, L:] = r.cuda()
    store = torch.full((heads, 70, HEAD), 7.0, dtype=BF, device="cuda")
    out, lse = sk.latent_prefill(wide[:, 1:, 8:], k.contiguous().cuda(), vt[:, :, :HEAD].transpose(0, 1), rows[:, L:],
                                 starts(lq), starts(lk), SCALE, out=store.transpose(0, 1))
    ref.check_prefill(out, lse, q, k, v, r, lq, lk, SCALE, True, "strides")


def test_prefill_another_stream_graph_and_repeats(sk):
    g = gen(16)
    lq, lk, heads = [100, 3], [3000, 50], 2
    q, k, v, r = (t.cuda() for t in prefill_inputs(g, lq, lk, heads))
    cq, ck = starts(lq), starts(lk)
    work = sk.latent_prefill_workspace(103, 3050, 2, heads)
    assert work.numel() > 0                               # the keys are split
    out, lse = torch.empty(103, heads, HEAD, dtype=BF, device="cuda"), torch.empty(103, heads, device="cuda")
    call = lambda stream=None: sk.latent_prefill(q, k, v, r, cq, ck, SCALE, out=out, lse=lse, workspace=work, stream=stream)
    call()
    torch.cuda.synchronize()
    first = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


# ------------------------------------------------------- the two forms are the same attention

def test_prefill_and_decode_agree(sk):
    """Keys and values expanded from a cache's latents by projections: the expanded form of the last
    token and the absorbed form over the cache give the same attention (up to the roundings of the
    projections to bf16: 8 half steps of the values' size at these random weights)."""
    g = gen(17)
    n, heads = 200, 4
    cache, table, lens = paged(g, [n], 16)
    k = torch.arange(n)
    rows = cache[table[0, k // 16].long(), k % 16]
    up_k = torch.randn(heads, L, HEAD, generator=g, dtype=torch.float64) / L ** 0.5
    up_v = torch.randn(heads, L, HEAD, generator=g, dtype=torch.float64) / L ** 0.5
    q = normal(g, 1, heads, HEAD + ROT)
    z = rows[:, :L].double()
    keys = torch.stack([z @ up_k[h] for h in range(heads)], 1).to(BF)
    vals = torch.stack([z @ up_v[h] for h in range(heads)], 1).to(BF)
    o1, l1 = sk.latent_prefill(q.cuda(), keys.cuda(), vals.cuda(), rows[:, L:].contiguous().cuda(), starts([1]), starts([n]), SCALE)
    absorbed = torch.stack([q[0, h, :HEAD].double() @ up_k[h].T for h in range(heads)])
    qa = torch.cat((absorbed.to(BF), q[0, :, HEAD:]), -1)[None]
    o2, l2 = sk.latent_decode(qa.cuda(), cache.cuda(), table.cuda(), lens.cuda(), SCALE)
    got = torch.stack([o2[0, h].cpu().double() @ up_v[h] for h in range(heads)])
    assert (got - o1[0].cpu().double()).abs().max() <= 8 * ref.HALF * vals.double().abs().max()
    assert (l1 - l2).abs().max() <= 8 * ref.HALF


# ---------------------------------------------------------------------------------- refusals

def test_binding_refuses(sk):
    g = gen(18)
    cache, table, lens = (t.cuda() for t in paged(g, [20, 40], 16))
    q = normal(g, 2, 4, DIM).cuda()
    ok = dict(q=q, cache=cache, table=table, lens=lens, scale=SCALE)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q[:, :, :512]), dict(q=q.cpu()), dict(tokens=2), dict(tokens=0), dict(scale=0.0),
                dict(scale=math.inf), dict(scale=1e-60), dict(lens=lens.long()), dict(lens=lens[:1]), dict(table=table.long()),
                dict(cache=cache[:, :, :512]), dict(cache=cache[:0]), dict(table=table[:, :0]), dict(out=q[:, :, :512]),
                dict(out=torch.empty(2, 4, 512, device="cuda")), dict(lse=torch.empty(2, 8, device="cuda")[:, ::2]),
                dict(q=normal(g, 2, 4, DIM + 4).cuda()[:, :, 4:]), dict(q=normal(g, 2, 1, DIM).cuda().expand(2, 4, DIM)),
                dict(table=table.t().contiguous().t()), dict(rope_dim=32), dict(workspace=small.int()),
                dict(workspace=sk.latent_decode_workspace(2, 1, 4).cpu())):
        with pytest.raises(ValueError):
            sk.latent_decode(**{**ok, **bad})
    with pytest.raises(sk.ops.SkinnyError):
        sk.latent_decode(**ok, workspace=small)
    kv, slots = normal(g, 3, DIM).cuda(), torch.arange(3).cuda()
    f = inv_freq().cuda()
    ok = dict(kv=kv, cache=cache, slots=slots, positions=slots, inv_freq=f)
    q3 = normal(g, 3, 2, ROT).cuda()
    for bad in (dict(kv=cache[0, :3]), dict(kv=kv[:, :512]), dict(slots=slots.int()), dict(inv_freq=f.float()),
                dict(positions=slots[:2]), dict(eps=-1.0), dict(norm_weight=f), dict(q=q3[:2]), dict(q_out=q3),
                dict(q=q3, q_out=q3[:, :1]), dict(q=q3, q_out=q3.cpu()), dict(slots=torch.arange(6).cuda()[::2])):
        with pytest.raises(ValueError):
            sk.latent_append(**{**ok, **bad})
    q, k, v, r = (t.cuda() for t in prefill_inputs(g, [9], [9], 2))
    ok = dict(q=q, k=k, v=v, k_rot=r, cu_q=starts([9]), cu_k=starts([9]), scale=SCALE)
    for bad in (dict(q=q[:, :, :128]), dict(k=k[:8]), dict(v=v.float()), dict(k_rot=r[:, :32]), dict(cu_q=starts([9]).long()),
                dict(cu_k=starts([4, 5])), dict(out=v), dict(scale=-1.0), dict(lse=torch.empty(2, 9, device="cuda").t()),
                dict(workspace=small[::2])):
        with pytest.raises(ValueError):
            sk.latent_prefill(**{**ok, **bad})


# ------------------------------------------------- prompts long enough for the wide workgroups

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([192], [192], 1), ([255], [255], 3), ([256], [256], 8), ([257], [257], 2), ([511, 513], [511, 513], 2),
    ([700, 0, 900], [700, 3, 900], 3), ([600, 1], [200, 5], 2), ([1100], [1100], 8), ([300], [63], 1), ([400], [0], 2),
    ([260], [3000], 2), ([1000, 30, 64], [2500, 30, 65], 1)])
def test_prefill_wide(sk, lq, lk, heads, causal):
    prefill_case(sk, lq, lk, heads, causal, seed=sum(lk) + heads)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,past", [(2, 0), (1, 4000)])
def test_prefill_wide_hidden_values_may_be_anything(sk, heads, past, bad):
    n0 = 300
    lq, lk = [n0], [n0 + past]
    q, k, v, r = prefill_inputs(gen(21), lq, lk, heads)
    at = past + 170
    v[at, :, 5] = bad
    k[past + 290, :, 3] = math.nan
    kv = torch.cat((k, v), -1).cuda()
    out, lse = sk.latent_prefill(q.cuda(), kv[:, :, :HEAD], kv[:, :, HEAD:], r.cuda(), starts(lq), starts(lk), SCALE)
    out, lse = out.cpu(), lse.cpu()
    assert not bool(torch.isfinite(out[170:, :, 5]).any())
    assert bool(torch.isnan(out[290:]).all()) and bool(torch.isnan(lse[290:]).all())
    rest = [i for i in range(HEAD) if i != 5]
    clean = v.clone()
    clean[at, :, 5] = 0
    n = past + 290
    ref.check_prefill(out[:290][:, :, rest], lse[:290], q[:290], k[:n], clean[:n][:, :, rest], r[:n], [290], [n], SCALE,
                      True, "rest")
    n = past + 170
    ref.check_prefill(out[:170], lse[:170], q[:170], k[:n], v[:n], r[:n], [170], [n], SCALE, True, "before")


# ------------------------------------------------------------------ rows that do see such numbers

@pytest.mark.parametrize("at", [5, 66])                   # in a tile that all rows see whole, in the last
@pytest.mark.parametrize("place", [L + 3, 7])             # among the rotated numbers, among the latents
@pytest.mark.parametrize("heads,tokens", [(8, 1), (8, 4), (16, 4), (32, 4)])
def test_decode_infinite_keys(sk, heads, tokens, place, at):
    """A key with an infinite number scores +inf or -inf. Rows where it is +inf get NaN; for the
    others its weight is 0 (NaN in the output where the infinite number is a latent)."""
    g = gen(22)
    n = 70
    cache, table, lens = paged(g, [n], 16)
    q = normal(g, tokens, heads, DIM)
    q[:, :, place] = torch.where(q[:, :, place] >= 0, 1, -1).to(BF) * (q[:, :, place].abs() + 1)
    k = torch.arange(n)
    keys = cache[table[0, k // 16].long(), k % 16].double()
    cache[table[0, at // 16], at % 16, place] = math.inf
    out, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), SCALE, tokens=tokens)
    rows = q.reshape(-1, DIM).double()
    limit = (n - tokens + 1 + torch.arange(tokens)).repeat_interleave(heads)
    sees = limit > at
    seen = (k[None] < limit[:, None]) & (k != at)
    want = ref.attend(rows, keys, keys[:, :L], SCALE, seen)
    out, lse = out.reshape(-1, L).cpu(), lse.reshape(-1).cpu()
    up = sees & (rows[:, place] > 0)
    assert bool(up.any()) and bool((sees & ~up).any())
    assert bool(torch.isnan(out[up]).all()) and bool(torch.isnan(lse[up]).all())
    dims = torch.ones(L, dtype=torch.bool)
    if place < L:
        dims[place] = False
        assert bool(torch.isnan(out[sees & ~up][:, place]).all())
    e, el, d, pv, pv2 = (x[~up] for x in want)
    ref.check(out[~up][:, dims], lse[~up], (e[:, dims], el, d, pv[:, dims], pv2[:, dims]), n, "infinite key")


def test_workspace_of_a_call_belongs_to_its_stream(sk, monkeypatch):
    """Partial sums that a call allocates for itself are given back while it may still run on the
    stream it was given: the next tensor of the current stream must not get their memory."""
    g = gen(23)
    cache, table, lens = (t.cuda() for t in paged(g, [4000], 64))
    q = normal(g, 1, 8, DIM).cuda()
    p = [t.cuda() for t in prefill_inputs(g, [100], [3000], 2)]
    used = []
    module = sk.ops._latent()

    class Watch:
        decode = staticmethod(lambda *x: used.append((x[9].data_ptr(), x[9].numel())) or module.decode(*x))
        prefill = staticmethod(lambda *x: used.append((x[10].data_ptr(), x[10].numel())) or module.prefill(*x))

    monkeypatch.setattr(sk.ops, "_latent_module", Watch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = sk.latent_decode(q, cache, table, lens, SCALE, stream=side)
    at, size = used.pop()
    assert size > 0 and torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != at
    second = sk.latent_prefill(*p, starts([100]), starts([3000]), SCALE, stream=side)
    at, size = used.pop()
    assert size > 0 and torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != at
    torch.cuda.synchronize()
    monkeypatch.undo()
    for got, again in ((first, sk.latent_decode(q, cache, table, lens, SCALE)),
                       (second, sk.latent_prefill(*p, starts([100]), starts([3000]), SCALE))):
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


# ---------------------------------------------------------- the order of query tiles over sequences

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("count", [2, 64, 65, 256, 257, 700])
def test_prefill_sequences_of_all_lengths(sk, count, causal):
    """Tiles go by their number of keys; every one of them once, for batches below and past those that
    are ordered, with sequences of no queries, of no keys and of more keys than queries."""
    rng = random.Random(count)
    lq = [rng.choice((0, 1, 5, 130, 300)) if i % 16 == 3 else rng.choice((0, 1, 9, 33)) for i in range(count)]
    lk = [max(0, n + rng.choice((0, 0, 70, -4))) for n in lq]
    prefill_case(sk, lq, lk, 1, causal, seed=count)


def test_prefill_wide_sequences_of_all_lengths(sk):
    prefill_case(sk, [300, 0, 513, 1, 900, 256], [300, 9, 200, 0, 1500, 256], 8, True, seed=31)
    prefill_case(sk, [300, 0, 513, 1, 900, 256], [300, 9, 200, 0, 1500, 256], 3, False, seed=32)


def test_outputs_of_a_call_belong_to_its_stream(sk):
    """Of a call on another stream the caller takes the outputs and lets lse go, or takes nothing: the next
    tensors of the current stream must not get memory that the call may still write."""
    g = gen(27)
    cache, table, lens = (t.cuda() for t in paged(g, [4000], 64))
    q, kv = normal(g, 1, 8, DIM).cuda(), normal(g, 1, DIM).cuda()
    p = [t.cuda() for t in prefill_inputs(g, [100], [3000], 2)] + [starts([100]), starts([3000])]
    at, f = torch.tensor([4095]).cuda(), inv_freq().cuda()
    calls = (lambda s: (sk.latent_append(kv, cache, at, at, f, q=q[:, :, L:], stream=s),),
             lambda s: sk.latent_decode(q, cache, table, lens, SCALE, stream=s),
             lambda s: sk.latent_prefill(*p, SCALE, stream=s))
    side = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        got = call(side)
        kinds = [(t.shape, t.dtype, t.data_ptr()) for t in got]
        kept = got[0]
        del got
        for shape, dtype, where in kinds[1:]:
            assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != where
        side.synchronize()
        assert torch.equal(kept, want[0])
        shape, dtype, where = kinds[0]
        del kept
        assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != where


def test_overlapping_rows_are_refused(sk):
    """Rows that are written and share numbers with others are a ValueError; rows in another order, or
    apart from each other, are not."""
    g = gen(28)
    store = torch.zeros(1 << 16, dtype=BF, device="cuda")
    rows = lambda shape, strides: torch.as_strided(store, shape, strides)
    cache, table, lens = (t.cuda() for t in paged(g, [20, 40, 31], 16))
    q, kv = normal(g, 3, 4, DIM).cuda(), normal(g, 3, DIM).cuda()
    slots, f = torch.arange(3).cuda(), inv_freq().cuda()
    p = [t.cuda() for t in prefill_inputs(g, [9], [9], 2)] + [starts([9]), starts([9])]
    step = lambda **k: sk.latent_append(kv, k.pop("cache", cache), slots, slots, f, **k)
    for strides in ((L, L, 1), (3 * L, L, 1), (L, 2 * L, 1)):
        with pytest.raises(ValueError, match="overlap"):
            sk.latent_decode(q, cache, table, lens, SCALE, out=rows((3, 4, L), strides))
    for strides in ((HEAD, HEAD, 1), (HEAD, 8 * HEAD, 1)):
        with pytest.raises(ValueError, match="overlap"):
            sk.latent_prefill(*p, SCALE, out=rows((9, 2, HEAD), strides))
    for strides in ((DIM, DIM, 1), (DIM * 3, DIM, 1), (DIM, 2 * DIM, 1)):
        with pytest.raises(ValueError, match="overlap"):
            step(cache=rows((3, 4, DIM), strides))
    for strides in ((ROT, ROT, 1), (ROT, 2 * ROT, 1)):
        with pytest.raises(ValueError, match="overlap"):
            step(q=q[:, :, L:], q_out=rows((3, 4, ROT), strides))
    for out, strides, call in (((3, 4, L), (L, 3 * L, 1), lambda o: sk.latent_decode(q, cache, table, lens, SCALE, out=o)[0]),
                               ((9, 2, HEAD), (HEAD + 8, 9 * HEAD + 64, 1), lambda o: sk.latent_prefill(*p, SCALE, out=o)[0]),
                               ((3, 4, ROT), (ROT, 3 * ROT, 1), lambda o: step(q=q[:, :, L:], q_out=o))):
        assert torch.equal(call(rows(out, strides)), call(torch.empty(out, dtype=BF, device="cuda")))


# ----------------------------------------------------------------- tensors that share their memory

def test_lazy_clones_are_written_apart(sk):
    """A lazily cloned tensor shares its memory until it is written: what it was cloned from stays."""
    g = gen(26)
    lens = [2000, 17]
    cache, table, n = (t.cuda() for t in paged(g, lens, 16))
    heads = 8
    kept = []

    def lazy(t):
        kept.append((t, t.clone()))
        return t._lazy_clone()

    kv, q = normal(g, 5, DIM).cuda(), normal(g, 5, heads, ROT).cuda()
    slots, pos = torch.arange(5).cuda(), (torch.arange(5) * 100).cuda()
    f = inv_freq().cuda()
    want_cache = cache.clone()
    want_q = sk.latent_append(kv, want_cache, slots, pos, f, q=q)
    lazy_cache, lazy_q = lazy(cache), lazy(q)
    lazy_out = lazy(torch.zeros_like(q))
    sk.latent_append(kv, lazy_cache, slots, pos, f, q=q, q_out=lazy_out)
    assert torch.equal(lazy_cache, want_cache) and torch.equal(lazy_out, want_q)
    sk.latent_append(kv, lazy_cache, slots, pos, f, q=lazy_q, q_out=lazy_q)
    assert torch.equal(lazy_q, want_q)

    qd = normal(g, 2, heads, DIM).cuda()
    want = sk.latent_decode(qd, cache, table, n, SCALE)
    out, lse = lazy(torch.zeros_like(want[0])), lazy(torch.zeros_like(want[1]))
    work = lazy(torch.zeros_like(sk.latent_decode_workspace(2, 1, heads)))
    sk.latent_decode(qd, cache, table, n, SCALE, out=out, lse=lse, workspace=work)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])

    p = [t.cuda() for t in prefill_inputs(g, [100], [3000], 2)] + [starts([100]), starts([3000])]
    want = sk.latent_prefill(*p, SCALE)
    out, lse = lazy(torch.zeros_like(want[0])), lazy(torch.zeros_like(want[1]))
    work = lazy(torch.zeros_like(sk.latent_prefill_workspace(100, 3000, 1, 2)))
    assert work.numel() > 0
    sk.latent_prefill(*p, SCALE, out=out, lse=lse, workspace=work)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for origin, before in kept:
        assert torch.equal(origin, before)


# ------------------------------------------- the wide form without a split, joins of many requests

def wide_and_whole(lq, lk, heads, sk):
    """That a call of these sizes takes the wide form with its keys whole, as one long prompt of many
    heads does: the averages that the form is chosen by, and no workspace for partial sums."""
    assert sum(lq) // len(lq) >= 192 and sum(lk) // len(lk) >= 1024
    assert sk.latent_prefill_workspace(sum(lq), sum(lk), len(lq), heads).numel() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([1100, 1030], [1100, 1030], 16), ([1500, 0, 1800], [1500, 0, 1800], 9), ([1300, 200, 1800], [1500, 0, 1800], 9),
    ([257, 1, 700], [3000, 40, 700], 24), ([1100], [1100], 32)])
def test_prefill_wide_with_whole_keys(sk, lq, lk, heads, causal):
    wide_and_whole(lq, lk, heads, sk)
    prefill_case(sk, lq, lk, heads, causal, seed=sum(lk) + heads)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prefill_wide_whole_keys_hidden_values(sk, bad):
    n, heads, at = 1100, 32, 700
    wide_and_whole([n], [n], heads, sk)
    q, k, v, r = prefill_inputs(gen(25), [n], [n], heads)
    v[at, :, 5] = bad
    k[1000, :, 3] = math.nan
    out, lse = sk.latent_prefill(q.cuda(), k.cuda(), v.cuda(), r.cuda(), starts([n]), starts([n]), SCALE)
    out, lse = out.cpu(), lse.cpu()
    assert not bool(torch.isfinite(out[at:, :, 5]).any())
    assert bool(torch.isnan(out[1000:]).all()) and bool(torch.isnan(lse[1000:]).all())
    rest = [i for i in range(HEAD) if i != 5]
    clean = v.clone()
    clean[at, :, 5] = 0
    some = [0, 13, 31]
    ref.check_prefill(out[:1000, some][:, :, rest], lse[:1000, some], q[:1000, some], k[:1000, some],
                      clean[:1000, some][:, :, rest], r[:1000], [1000], [1000], SCALE, True, "rest")
    ref.check_prefill(out[:at, some], lse[:at, some], q[:at, some], k[:at, some], v[:at, some], r[:at], [at], [at], SCALE,
                      True, "before")


@pytest.mark.parametrize("heads,tokens", [(16, 1), (32, 1), (8, 4), (64, 1), (128, 1), (40, 4)])
def test_decode_many_cut_requests(sk, heads, tokens):
    """At least 64 requests, so that no more than four runs fall on one, long enough that most are cut."""
    rng = random.Random(heads + tokens)
    decode_case(sk, [rng.choice((0, 1, 33, 100, 170, 260)) for _ in range(70)], heads, tokens, 16, seed=heads + tokens)


# ----------------------------------------------------- infinities of both signs that some rows see

def both_infinities(sk, n, heads, at):
    """Key `at` has +inf, NaN, -inf in dims 5, 6, 7 of its value and the next key -inf, -inf, +inf: row
    `at` sees only the first of them, rows after it both, whose sum is NaN, and rows before neither."""
    print("both infinities", dict(n=n, heads=heads, at=at), flush=True)
    q, k, v, r = prefill_inputs(gen(24), [n], [n], heads)
    v[at, :, 5], v[at, :, 6], v[at, :, 7] = math.inf, math.nan, -math.inf
    v[at + 1, :, 5], v[at + 1, :, 6], v[at + 1, :, 7] = -math.inf, -math.inf, math.inf
    out, lse = sk.latent_prefill(q.cuda(), k.cuda(), v.cuda(), r.cuda(), starts([n]), starts([n]), SCALE)
    out, lse = out.cpu(), lse.cpu()
    assert bool((out[at, :, 5] == math.inf).all()) and bool((out[at, :, 7] == -math.inf).all())
    assert bool(torch.isnan(out[at, :, 6]).all())
    assert bool(torch.isnan(out[at + 1:, :, 5:8]).all())
    dims = [i for i in range(HEAD) if not 5 <= i < 8]
    some = slice(0, heads, max(1, heads // 2))
    ref.check_prefill(out[:, some][:, :, dims], lse[:, some], q[:, some], k[:, some], v[:, some][:, :, dims], r, [n], [n],
                      SCALE, True, "other numbers")
    ref.check_prefill(out[:at, some], lse[:at, some], q[:at, some], k[:at, some], v[:at, some], r[:at], [at], [at], SCALE,
                      True, "rows before")


@pytest.mark.parametrize("at", [101, 64, 76, 30])         # pairs of one matrix instruction's 16 keys
def test_prefill_infinities_of_both_signs(sk, at):
    both_infinities(sk, 150, 2, at)


@pytest.mark.parametrize("at", [700, 1050])
def test_prefill_wide_infinities_of_both_signs(sk, at):
    n, heads = 1100, 32
    wide_and_whole([n], [n], heads, sk)
    both_infinities(sk, n, heads, at)
