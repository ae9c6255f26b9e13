"""Latent attention at the limits of what its operands may hold, on the GPU: rows behind a request's end, few short
requests, weights with fewer columns than keys, lengths and page ids that are clamped, strided operands."""
import ctypes
import math

import pytest
import torch

import latent_reference as ref
import masked_reference as mref
from test_latent_gpu import BF, DIM, SCALE, gen, normal, paged, sk  # noqa: F401

pytestmark = pytest.mark.gpu


def shortest(*calls, each=20, rounds=12):
    """Each call's shortest time in us: graphs of `each` calls, replayed in turn."""
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(each):
                call()
        graphs.append(graph)
    best = [math.inf] * len(calls)
    for r in range(rounds):
        for i, graph in enumerate(graphs):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            if r > 1:
                best[i] = min(best[i], begin.elapsed_time(end) * 1e3 / each)
    return best


def decode_call(sk, q, cache, table, n, tokens=1):
    """A decode call on outputs and a workspace of its own; its outputs."""
    out, lse = torch.empty(*q.shape[:2], 512, dtype=BF, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    work = sk.latent_decode_workspace(len(n), tokens, q.shape[1])
    return (lambda: sk.latent_decode(q, cache, table, n, SCALE, tokens=tokens, out=out, lse=lse, workspace=work)), out, lse


@pytest.mark.parametrize("heads", [8, 32, 64, 128])
def test_rows_behind_the_end_cost_nothing(sk, heads):
    """A pool that was never written, as from torch.empty, may hold anything behind a request's last row: the outputs are
    the same bits, and the call takes as long. (In us, if numbers there are looked at: 8 heads 9.1 and 12.0 with
    NaN, 64 heads 16.3 and 27.9, 128 heads 20.2 and 31.0; repeats of the shortest time differ by 3%.)"""
    g = gen(heads)
    cache, table, n = (t.cuda() for t in paged(g, [33] * 64, 64))
    q = normal(g, 64, heads, DIM).cuda()
    spoiled = cache.clone()
    spoiled[:, 33:] = math.nan
    call, out, lse = decode_call(sk, q, cache, table, n)
    again, out_again, lse_again = decode_call(sk, q, spoiled, table, n)
    finite, odd = shortest(call, again)
    print("heads", heads, "finite", finite, "NaN behind the end", odd, flush=True)
    assert torch.equal(out, out_again) and torch.equal(lse, lse_again)
    assert odd < 1.15 * finite


@pytest.mark.parametrize("heads,keys,batch,most", [(32, 40, 3, 1.1), (64, 40, 3, 1.1), (64, 40, 8, 1.2), (128, 80, 3, 1.15)])
def test_a_few_short_requests_take_as_long_as_one(sk, heads, keys, batch, most):
    """Each of their tiles has a workgroup of its own, as one request's have. (One request and these, in us: 8.8 and 8.9, 10.0 and
    10.2, 10.0 and 11.0, 13.6 and 14.2; where tiles of a request shared one: 10.3, 12.9, 13.9 and 17.3.)"""
    g = gen(heads)
    cache, table, n = (t.cuda() for t in paged(g, [keys] * batch, 64))
    q = normal(g, batch, heads, DIM).cuda()
    one, out_one, lse_one = decode_call(sk, q[:1], cache, table[:1], n[:1])
    all_, out, lse = decode_call(sk, q, cache, table, n)
    alone, together = shortest(one, all_)
    print("heads", heads, "alone", alone, "together", together, flush=True)
    assert torch.equal(out[:1], out_one) and torch.equal(lse[:1], lse_one)
    ref.check_decode(out, lse, q, cache, table, n, SCALE, 1, "short")
    assert together < most * alone


# ---------------------------------------------------------------------------- fewer columns than keys

def draws(g, n, kind):
    """Weights: spread like sums of softmax weights, many zeros, or some negative."""
    w = torch.exp(2 * torch.randn(n, generator=g))
    if kind == "zeros":
        w[torch.rand(n, generator=g) < 0.7] = 0.0
    if kind == "signed":
        w *= torch.where(torch.rand(n, generator=g) < 0.5, -1.0, 1.0)
    return w


@pytest.mark.parametrize("kind", ["spread", "zeros", "signed"])
@pytest.mark.parametrize("columns,budget,sinks,recent", [(100, 40, 4, 8), (100, 150, 0, 0), (100, 99, 99, 0), (100, 120, 110, 10),
                                                         (300, 290, 3, 280), (300, 299, 0, 0), (1, 10, 0, 0), (0, 7, 2, 3),
                                                         (2000, 1900, 16, 64), (2000, 700, 0, 1)])
def test_select_of_keys_without_a_column(sk, columns, budget, sinks, recent, kind):
    """`recent` and the budget count from a request's true end, and keys without a column have the weight 0."""
    g = gen(columns + budget)
    lens = [0, 1, columns, columns + 1, columns + 37, budget, budget + 1, columns + budget, 5000, max(0, columns - 1)]
    w = torch.stack([draws(g, columns, kind) for _ in lens]) if columns else torch.empty(len(lens), 0)
    kept, counts = sk.latent_select(w.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, sinks=sinks, recent=recent)
    for i, n in enumerate(lens):
        full = w[i].tolist()[:n] + [0.0] * (n - columns)
        want = mref.select(full, n, budget, sinks, recent)
        assert int(counts[i]) == len(want), (i, n)
        assert kept[i].tolist() == want + [-1] * (budget - len(want)), (i, n)


def test_select_of_keys_far_past_the_columns(sk):
    """More columns than registers hold, and lengths that are cut to 2^30."""
    g = gen(7)
    w = torch.stack([draws(g, 70000, k) for k in ("spread", "zeros", "signed")])
    lens = torch.tensor([70001, 2 ** 31 - 1, 200000], dtype=torch.int32)
    kept, counts = sk.latent_select(w.cuda(), lens.cuda(), 60000, sinks=4, recent=100)
    assert counts.tolist() == [60000] * 3
    for i, n in enumerate((70001, 2 ** 30, 200000)):
        near = min(n - 100, 140000)                              # keys behind it have the weight 0, and earlier ones too
        full = w[i].tolist()[:near] + [0.0] * (near - 70000)
        want = mref.select(full, near, 59900, 4, 0) + list(range(n - 100, n))
        assert kept[i].tolist() == want, (i, n)


def test_select_and_keep_with_fewer_columns_than_keys(sk):
    """The newest rows stay, whatever the columns, and take the weight 0 along."""
    g = gen(8)
    lens, columns, budget, recent = [300, 90, 130, 0], 100, 64, 24
    cache, table, n = paged(g, lens, 16)
    q = normal(g, len(lens), 4, DIM)
    got = cache.cuda()
    _, lse = sk.latent_decode(q.cuda(), got, table.cuda(), n.cuda(), SCALE)
    weights = sk.latent_key_weights(q.cuda(), got, table.cuda(), n.cuda(), lse, torch.zeros(len(lens), columns, device="cuda"), SCALE)
    kept, counts = sk.latent_select(weights, n.cuda(), budget, sinks=4, recent=recent)
    left, fewer = sk.latent_keep(got, table.cuda(), n.cuda(), kept, counts, weights=weights)
    want = cache.clone()
    for i, m in enumerate(lens):
        full = weights[i].tolist()[:m] + [0.0] * (m - columns)
        numbers = mref.select(full, m, budget, 4, recent)
        mref.keep(want, table[i], m, numbers, 0)
        assert int(left[i]) == len(numbers)
        assert fewer[i].tolist() == [full[k] for k in numbers] + [0.0] * (columns - len(numbers)), i
        rows = mref.keys_of(got.cpu(), table, left.cpu(), i)
        newest = mref.keys_of(cache, table, n, i)[-recent:]
        assert torch.equal(rows[-len(newest):], newest), i
    assert torch.equal(got.cpu(), want)


# -------------------------------------------------------------------------------- lists that interleave

def test_keep_takes_lists_between_each_other(sk):
    """By the C entry: rows of weights and new weights, and the other lists, side by side in one array share no number."""
    from decode_skinny_addmm_amd import _lib
    g = gen(9)
    lens, columns = [90, 40, 64], 90
    cache, table, n = paged(g, lens, 16)
    kept = [sorted(torch.randperm(m, generator=g)[:m * 2 // 3].tolist()) for m in lens]
    most, pages = 60, table.shape[1]
    wide = torch.zeros(3, 2 * columns + most + pages + 3, dtype=torch.int32)
    w = torch.rand(3, columns, generator=g)
    wide[:, :columns] = w.view(torch.int32)
    for i, k in enumerate(kept):
        wide[i, 2 * columns:2 * columns + len(k)] = torch.tensor(k, dtype=torch.int32)
    wide[:, 2 * columns + most:2 * columns + most + pages] = table
    wide[1, -3:] = n                                              # behind a row's lists, before the next row's
    wide[0, -3:] = torch.tensor([len(k) for k in kept])
    got, lists = cache.cuda(), wide.cuda()
    at = lambda row, column: lists.data_ptr() + 4 * (row * wide.shape[1] + column)
    end = wide.shape[1] - 3
    args = _lib.SkinnyLatentKeepArgs(
        cache=got.data_ptr(), table=at(0, 2 * columns + most), lens=at(1, end), kept=at(0, 2 * columns), counts=at(0, end),
        new_lens=at(2, end), weights=at(0, 0), new_weights=at(0, columns), cache_page_stride=16 * DIM, cache_row_stride=DIM,
        table_stride=wide.shape[1], kept_stride=wide.shape[1], weights_stride=wide.shape[1], new_weights_stride=wide.shape[1],
        batch=3, tokens=0, most=most, pages=cache.shape[0], page=16, max_pages=pages, columns=columns, latent=512, rope=64)
    assert _lib.lib().skinny_latent_keep_bf16(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    want, lists = cache.clone(), lists.cpu()
    for i, m in enumerate(lens):
        left, moved = mref.keep(want, table[i], m, kept[i], 0, w[i])
        assert int(lists[2, end + i]) == left
        assert torch.equal(lists[i, columns:2 * columns], moved.view(torch.int32)), i
    assert torch.equal(got.cpu(), want)


# ---------------------------------------------------------------------- what is clamped, and strides

def clamped(g):
    """Lengths outside of 0 .. 48 and page ids outside of the pool of 10, of requests whose pages are their own."""
    lens = torch.tensor([41, 49, 2 ** 31 - 1, -5, -2 ** 31, 48], dtype=torch.int32)
    table = torch.tensor([[-3, 1, 2], [3, 4, 2 ** 30], [5, 6, 7], [8, 8, 8], [-1, -1, -1], [-2 ** 31, 1, 2 ** 31 - 1]], dtype=torch.int32)
    return normal(g, 10, 16, DIM), table, lens


@pytest.mark.parametrize("heads,tokens", [(2, 3), (8, 4), (16, 4), (32, 5)])
def test_masked_decode_clamps(sk, heads, tokens):
    g = gen(heads)
    cache, table, n = clamped(g)
    q = normal(g, len(n) * tokens, heads, DIM)
    parents = [[j - 1 if j % 3 else -1 for j in range(tokens)]] * len(n)
    above, depth = mref.ancestors(parents[0])
    mask, _ = sk.latent_tree_mask(torch.tensor(parents, dtype=torch.int32, device="cuda"))
    out, lse = sk.latent_tree_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), mask, SCALE)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, above=above), "tree")
    # depths are clamped to 0 .. tokens - 1 (those that the words do not speak of stand where they are told)
    far = torch.tensor([[-7 if j % 2 else 2 ** 31 - 1 for j in range(tokens)]] * len(n), dtype=torch.int32)
    out, lse = sk.latent_tree_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), mask, SCALE, window=11, sinks=2, depth=far.cuda())
    near = far[0].clamp(0, tokens - 1)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, 11, 2, above, near), "window")
    out, lse = sk.latent_window_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, 9, sinks=1, tokens=tokens)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, 9, 1), "chain")


@pytest.mark.parametrize("heads,tokens", [(2, 1), (16, 3), (64, 4)])
def test_key_weights_clamp(sk, heads, tokens):
    g = gen(heads)
    cache, table, n = clamped(g)
    q = normal(g, len(n) * tokens, heads, DIM)
    _, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, tokens=tokens)
    before = torch.rand(len(n), 60, generator=g)
    got = sk.latent_key_weights(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), lse, before.cuda(), SCALE, tokens=tokens)
    mref.check_weights(got, before, q, cache, table, n, lse, SCALE, tokens, "clamped")


@pytest.mark.parametrize("tokens", [0, 20])
def test_keep_clamps(sk, tokens):
    g = gen(10)
    cache, table, n = clamped(g)
    table, n = table[:5], n[:5]                                  # the last request shares pages with others
    kept = torch.tensor([sorted(torch.randperm(tokens or 48, generator=g)[:12].tolist()) for _ in n], dtype=torch.int32)
    counts = torch.tensor([2 ** 31 - 1, 12, 5, 7, -2 ** 31], dtype=torch.int32)
    weights = torch.rand(5, 60, generator=g)
    got = cache.cuda()
    left, fresh = sk.latent_keep(got, table.cuda(), n.cuda(), kept.cuda(), counts.cuda(), tokens=tokens, weights=weights.cuda())
    want = cache.clone()
    for i in range(5):
        m = max(0, min(int(n[i]), 48))
        length, moved = mref.keep(want, table[i], m, kept[i, :max(0, min(int(counts[i]), 12))].tolist(), tokens, weights[i])
        assert int(left[i]) == length, i
        assert torch.equal(fresh[i].cpu(), moved), i
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("heads,tokens", [(2, 3), (16, 2), (40, 4)])
def test_key_weights_of_strided_rows(sk, heads, tokens):
    """A cache whose rows and pages lie apart, queries that are a slice; then pages, rows and queries that lie so far apart that
    their offsets pass 31 and 32 bits."""
    g = gen(heads)
    lens, rows = [333, tokens, 90], 3 * tokens
    cache, table, n = paged(g, lens, 16)
    q = normal(g, rows, heads, DIM)
    before = torch.rand(3, 340, generator=g)

    def check(queries, pool, order, n, small, what):
        _, lse = sk.latent_decode(q.cuda(), small.cuda(), order.cuda(), n.cuda(), SCALE, tokens=tokens)
        got = sk.latent_key_weights(queries, pool, order.cuda(), n.cuda(), lse, before.cuda(), SCALE, tokens=tokens)
        mref.check_weights(got, before, q, small, order, n, lse, SCALE, tokens, what)

    apart = torch.full((cache.shape[0], 17, DIM + 16), math.nan, dtype=BF, device="cuda")[:, :16, :DIM]
    apart.copy_(cache)
    queries = torch.full((rows, heads + 1, DIM + 8), math.nan, dtype=BF, device="cuda")[:, 1:, :DIM]
    queries.copy_(q)
    check(queries, apart, table, n, cache, "strided")
    few, order = normal(g, 3, 16, DIM), torch.tensor([[2, 0, 1]] * 3, dtype=torch.int32)
    short = torch.tensor([48, tokens, 20 + tokens], dtype=torch.int32)
    for step, row in (((1 << 29) + 8, DIM), ((1 << 31) + 64, DIM + 8), (DIM + 8, (1 << 25) + 8)):
        far = torch.empty(2 * step + 15 * row + DIM, dtype=BF, device="cuda").as_strided((3, 16, DIM), (step, row, 1))
        far.copy_(few)
        check(queries, far, order, short, few, "far")
        del far
    step = (1 << 31) // (rows - 1) + 8 - (1 << 31) // (rows - 1) % 8
    far = torch.empty((rows - 1) * step + heads * DIM, dtype=BF, device="cuda").as_strided((rows, heads, DIM), (step, DIM, 1))
    far.copy_(q)
    check(far, apart, table, n, cache, "far queries")
