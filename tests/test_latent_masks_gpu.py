"""Latent attention over trees and windows, key weights, and which rows stay, on the GPU against plain 64-bit
computations on the CPU (masked_reference.py, which derives the bounds)."""
import math
import random

import pytest
import torch

import latent_reference as ref
import masked_reference as mref
from test_latent_gpu import BF, DIM, HEAD, L, SCALE, gen, inv_freq, normal, paged, prefill_inputs, sk, starts  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------- trees

def random_parents(g, tokens, deep=False):
    """Each token under any earlier one or the context; deep: mostly under the one before."""
    p = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for j in range(tokens)]
    return [j - 1 if deep and j % 7 else p[j] for j in range(tokens)]


@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 65, 100, 257, 512])
def test_tree_mask(sk, tokens):
    g = gen(tokens)
    trees = [random_parents(g, tokens), random_parents(g, tokens, deep=True), [j - 1 for j in range(tokens)], [-1] * tokens,
             [(j * 7) % (tokens + 3) - 2 for j in range(tokens)]]         # parents that are no earlier token
    mask, depth = sk.latent_tree_mask(torch.tensor(trees, dtype=torch.int32, device="cuda"))
    want = [mref.ancestors(p) for p in trees]
    assert torch.equal(mask.cpu(), mref.words_of(torch.stack([a for a, _ in want])))
    assert torch.equal(depth.cpu(), torch.stack([d for _, d in want]))


def tree_case(sk, lens, heads, tokens, page, window=0, sinks=0, seed=0, shared=False, deep=False):
    print("tree", dict(lens=lens, heads=heads, tokens=tokens, page=page, window=window, sinks=sinks, seed=seed), flush=True)
    g = gen(seed)
    cache, table, n = paged(g, lens, page)
    q = normal(g, len(lens) * tokens, heads, DIM)
    trees = [random_parents(g, tokens, deep) for _ in lens]
    if shared:
        trees = trees[:1] * len(lens)
    parents = torch.tensor(trees, dtype=torch.int32, device="cuda")
    mask, depth = sk.latent_tree_mask(parents[:1] if shared else parents)
    if shared:
        mask, depth = mask.expand(len(lens), -1, -1), depth.expand(len(lens), -1)
    out, lse = sk.latent_tree_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), mask, SCALE, window=window, sinks=sinks,
                                     depth=depth if window else None)
    torch.cuda.synchronize()
    paths = [mref.ancestors(p) for p in trees]
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens,
                      lambda i, m: mref.seen_of(m, tokens, window, sinks, *paths[i]), "tree")


@pytest.mark.parametrize("heads,tokens", [(1, 1), (8, 2), (3, 7), (1, 40), (16, 4), (2, 33), (8, 24), (5, 64), (1, 130)])
def test_tree_decode(sk, heads, tokens):
    """Drafts that begin and end anywhere in a tile and a page, requests of drafts only, and shorter than them."""
    tree_case(sk, [tokens, tokens + 1, 100 + tokens, 333, 0, tokens - 1, 64 + tokens, tokens // 2], heads, tokens, 16,
              seed=heads + tokens)


def test_tree_decode_largest(sk):
    tree_case(sk, [700, 512, 300], 1, 512, 64, seed=1, deep=True)


@pytest.mark.parametrize("page", [1, 48, 64])
def test_tree_decode_pages_and_shared_tree(sk, page):
    tree_case(sk, [500, 37, 1000], 4, 13, page, seed=page, shared=True)


def test_tree_decode_cut_requests(sk):
    """Requests cut between many workgroups, and row groups of 128 rows."""
    tree_case(sk, [5000, 41, 3500], 8, 20, 64, seed=3)
    tree_case(sk, [9000], 4, 4, 64, seed=4)


@pytest.mark.parametrize("page", [4, 12, 20])
@pytest.mark.parametrize("heads,tokens", [(2, 3), (8, 4), (16, 4), (16, 8), (5, 30)])
def test_tree_decode_pages_of_no_whole_groups(sk, heads, tokens, page):
    """8 rows in a row lie in up to three pages; row shapes of 16, 32, 64 and 128, and groups of them."""
    tree_case(sk, [700, tokens, 97, 0], heads, tokens, page, seed=page)
    tree_case(sk, [700, tokens, 97, 301], heads, tokens, page, window=90, sinks=21, seed=page + 1, deep=True)


@pytest.mark.parametrize("heads,tokens", [(2, 3), (16, 2), (16, 4), (16, 8)])
def test_tree_decode_of_strided_rows(sk, heads, tokens):
    """A cache whose rows and pages lie apart, queries that are a slice; then pages, rows and queries that lie so
    far apart that their offsets pass 31 and 32 bits."""
    g = gen(heads)
    lens, rows = [333, tokens, 90], 3 * tokens
    cache, table, n = paged(g, lens, 16)
    q = normal(g, rows, heads, DIM)
    parents = [random_parents(g, tokens) for _ in lens]
    mask, _ = sk.latent_tree_mask(torch.tensor(parents, dtype=torch.int32, device="cuda"))
    paths = [mref.ancestors(p) for p in parents]
    apart = torch.full((cache.shape[0], 17, DIM + 16), math.nan, dtype=BF, device="cuda")[:, :16, :DIM]
    apart.copy_(cache)
    queries = torch.full((rows, heads + 1, DIM + 8), math.nan, dtype=BF, device="cuda")[:, 1:, :DIM]
    queries.copy_(q)
    out, lse = sk.latent_tree_decode(queries, apart, table.cuda(), n.cuda(), mask, SCALE)
    seen = lambda i, m: mref.seen_of(m, tokens, above=paths[i][0])
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, seen, "strided")
    few, order = normal(g, 3, 16, DIM), torch.tensor([[2, 0, 1]] * 3, dtype=torch.int32)
    short = torch.tensor([48, tokens, 20 + tokens], dtype=torch.int32)
    queries = q.cuda()
    for step, row in (((1 << 29) - 8, DIM), ((1 << 29) + 8, DIM), ((1 << 31) + 64, DIM + 8), (DIM + 8, (1 << 25) + 8)):
        far = torch.empty(2 * step + 15 * row + DIM, dtype=BF, device="cuda").as_strided((3, 16, DIM), (step, row, 1))
        far.copy_(few)
        out, lse = sk.latent_tree_decode(queries, far, order.cuda(), short.cuda(), mask, SCALE)
        mref.check_decode(out, lse, q, few, order, short, SCALE, tokens, seen, "far")
        del far
    step = (1 << 29) // tokens + 8 - (1 << 29) // tokens % 8
    far = torch.empty((rows - 1) * step + heads * DIM, dtype=BF, device="cuda").as_strided((rows, heads, DIM), (step, DIM, 1))
    far.copy_(q)
    out, lse = sk.latent_tree_decode(far, apart, table.cuda(), n.cuda(), mask, SCALE)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, seen, "far queries")


@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("heads,tokens", [(8, 17), (128, 3), (64, 9), (128, 7), (32, 44), (128, 13), (128, 20),
                                          (128, 37), (256, 22)])
def test_decode_of_many_row_groups(sk, heads, tokens, page):
    """2 to 44 groups of 128 rows, side by side where they divide the chip well and else (37 and 44 over 256 CUs) behind
    each other, in few and in many runs, with requests shorter than a tile and empty ones between."""
    lens = [40, 0, tokens, 700, 3, 0, 0, 129]
    print("groups", heads, tokens, page, flush=True)
    g = gen(heads + tokens)
    cache, table, n = paged(g, lens, page)
    q = normal(g, len(lens) * tokens, heads, DIM)
    out, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, tokens=tokens)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens), "groups")
    window_case(sk, lens, heads, tokens, page, 90, 35, seed=1)


@pytest.mark.parametrize("lens", [[1], [5000], [31, 4000, 32], [1] * 40, [0] * 9, [2000] * 20, [64, 0] * 60])
@pytest.mark.parametrize("heads", [8, 24, 64, 100, 200])
def test_decode_lines(sk, lens, heads):
    """Runs that end and begin in the places ahead of a request, hold many requests, or a part of one."""
    window_case(sk, lens, heads, 1, 16, 3000, 10, seed=heads)


@pytest.mark.parametrize("batch", [511, 512, 513, 700])
def test_masked_decode_of_many_requests(sk, batch):
    """Around what each wave counts by itself, with empty requests and such shorter than their new tokens."""
    rng = random.Random(batch)
    lens = [rng.choice((0, 1, 2, 3, 31, 33, 70, 150)) for _ in range(batch)]
    window_case(sk, lens, 4, 2, 16, 20, 5, seed=batch)
    tree_case(sk, lens, 4, 3, 16, seed=batch)


@pytest.mark.parametrize("heads,tokens,window,sinks", [(8, 5, 5, 0), (8, 5, 40, 3), (2, 17, 100, 64), (16, 8, 33, 1),
                                                       (1, 64, 64, 32), (8, 24, 500, 4), (4, 3, 10 ** 9, 5)])
def test_tree_decode_windows(sk, heads, tokens, window, sinks):
    tree_case(sk, [tokens, 100 + tokens, 333, 0, tokens - 1, 900, 65 + window % 1000 + tokens], heads, tokens, 16, window, sinks,
              seed=heads + tokens, deep=True)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,tokens", [(2, 4), (8, 4), (16, 4), (32, 4)])
def test_tree_decode_hidden_rows_may_hold_anything(sk, heads, tokens, bad):
    """One branch's row holds numbers that are not finite: of the others no token sees it."""
    g = gen(5)
    lens, parents = [50, 97, 4, 64], [-1, 0, 0, 2]               # token 1 is on no other's path
    cache, table, n = paged(g, lens, 16)
    for i, m in enumerate(lens):
        cache[table[i, (m - 3) // 16], (m - 3) % 16] = bad
    q = normal(g, len(lens) * tokens, heads, DIM)
    mask, depth = sk.latent_tree_mask(torch.tensor([parents] * len(lens), dtype=torch.int32, device="cuda"))
    out, lse = sk.latent_tree_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), mask, SCALE)
    above = mref.ancestors(parents)[0]
    for i, m in enumerate(lens):
        keys = mref.keys_of(cache, table, n, i)
        for j in (0, 2, 3):
            mine = keys[mref.seen_of(m, tokens, above=above)[j]]
            answer = ref.attend(q[i * tokens + j].double(), mine, mine[:, :L], SCALE, torch.ones(heads, len(mine), dtype=torch.bool))
            ref.check(out[i * tokens + j], lse[i * tokens + j], answer, m, "request %d, token %d" % (i, j))
        if bad != -math.inf:
            assert not bool(torch.isfinite(out[i * tokens + 1]).all())


def test_a_chain_is_a_tree(sk):
    """The same sums in the same order: bit for bit what latent_decode gives."""
    g = gen(6)
    lens, tokens = [700, 64, 3, 5000], 4
    cache, table, n = (t.cuda() for t in paged(g, lens, 16))
    chain = torch.tensor([[-1, 0, 1, 2]], dtype=torch.int32, device="cuda")
    mask = sk.latent_tree_mask(chain)[0].expand(len(lens), -1, -1)
    for heads in (2, 8, 16, 40):
        q = normal(g, len(lens) * tokens, heads, DIM).cuda()
        want = sk.latent_decode(q, cache, table, n, SCALE, tokens=tokens)
        for got in (sk.latent_tree_decode(q, cache, table, n, mask, SCALE),
                    sk.latent_window_decode(q, cache, table, n, SCALE, 1 << 40, tokens=tokens)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tree_masks_of_any_bits(sk):
    """A mask need not be a tree's: tokens that see nothing, later ones, and bits past the last token."""
    g = gen(7)
    tokens, heads, lens = 6, 8, [6, 40, 3]
    cache, table, n = paged(g, lens, 16)
    q = normal(g, len(lens) * tokens, heads, DIM)
    words = torch.randint(-2 ** 31, 2 ** 31, (len(lens), tokens, 1), generator=g).int()
    words[:, 2] = 0
    out, lse = sk.latent_tree_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), words.cuda(), SCALE)
    above = (words.long() >> torch.arange(tokens)) & 1 == 1
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, above=above[i]), "bits")
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())


# ----------------------------------------------------------------------------------- windows

def window_case(sk, lens, heads, tokens, page, window, sinks, seed=0):
    print("window", dict(lens=lens, heads=heads, tokens=tokens, page=page, window=window, sinks=sinks), flush=True)
    g = gen(seed)
    cache, table, n = paged(g, lens, page)
    q = normal(g, len(lens) * tokens, heads, DIM)
    out, lse = sk.latent_window_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, window, sinks=sinks, tokens=tokens)
    torch.cuda.synchronize()
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, window, sinks), "window")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 40), (31, 0), (32, 4), (33, 32), (64, 33), (100, 100), (500, 4), (1000, 0)])
@pytest.mark.parametrize("heads,tokens", [(8, 1), (8, 3), (32, 2), (40, 4)])
def test_window_decode(sk, heads, tokens, window, sinks):
    window_case(sk, [0, 1, tokens, 31, 33, 64, 130, 257, 999], heads, tokens, 16, window, sinks, seed=window)


def test_window_decode_long(sk):
    window_case(sk, [20000, 5, 9999], 16, 1, 64, 4096, 4, seed=1)
    window_case(sk, [30001], 128, 1, 48, 5000, 70, seed=2)
    window_case(sk, [9000, 8000], 8, 9, 1, 3, 5, seed=3)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads,tokens", [(2, 1), (8, 2), (64, 1), (32, 4)])
def test_window_decode_hidden_keys_may_be_anything(sk, heads, tokens, bad):
    """Between the first keys and the window, in tiles and pages that are read in part."""
    g = gen(8)
    lens, window, sinks = [300, 75, 500], 45, 5
    cache, table, n = paged(g, lens, 64)
    for i, m in enumerate(lens):
        k = torch.arange(sinks, m - tokens - window + 1)
        cache[table[i, k // 64].long(), k % 64] = bad
    q = normal(g, len(lens) * tokens, heads, DIM)
    out, lse = sk.latent_window_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, window, sinks=sinks, tokens=tokens)
    mref.check_decode(out, lse, q, cache, table, n, SCALE, tokens, lambda i, m: mref.seen_of(m, tokens, window, sinks), "hidden")


def window_prefill_case(sk, lq, lk, heads, window, sinks, seed=0):
    print("window prefill", dict(lq=lq, lk=lk, heads=heads, window=window, sinks=sinks), flush=True)
    q, k, v, r = prefill_inputs(gen(seed), lq, lk, heads)
    kv = torch.cat((k, v), -1).cuda()
    out, lse = sk.latent_window_prefill(q.cuda(), kv[:, :, :HEAD], kv[:, :, HEAD:], r.cuda(), starts(lq), starts(lk), SCALE,
                                        window, sinks=sinks)
    torch.cuda.synchronize()
    mref.check_prefill(out, lse, q, k, v, r, lq, lk, SCALE, window, sinks, "window prefill")


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (63, 64), (64, 1), (65, 0), (130, 70), (10 ** 12, 10 ** 12)])
@pytest.mark.parametrize("lq,lk,heads", [([1], [1], 1), ([129], [129], 8), ([63, 0, 65, 400], [63, 9, 65, 400], 2),
                                         ([1, 7, 100], [500, 64, 900], 3), ([40, 1, 200], [3, 0, 130], 4)])
def test_window_prefill(sk, lq, lk, heads, window, sinks):
    window_prefill_case(sk, lq, lk, heads, window, sinks, seed=window % 1000)


@pytest.mark.parametrize("window,sinks", [(200, 4), (1000, 0), (1024, 130), (1900, 1)])
@pytest.mark.parametrize("lq,lk,heads", [([2500], [2500], 2), ([300, 900, 700], [2300, 2000, 3900], 2), ([256], [6000], 1)])
def test_window_prefill_long(sk, lq, lk, heads, window, sinks):
    """Both forms, tiles left out between the first keys and the window, split keys."""
    window_prefill_case(sk, lq, lk, heads, window, sinks, seed=window)


@pytest.mark.parametrize("window,sinks", [(2560, 0), (2700, 4), (3000, 130), (2561, 600)])
@pytest.mark.parametrize("lq,lk,heads", [([700], [4000], 2), ([3900], [3900], 1), ([200, 900, 300], [6100, 3600, 2700], 2),
                                         ([257, 511], [7001, 5000], 3)])
def test_window_prefill_of_long_windows(sk, lq, lk, heads, window, sinks):
    """Windows long enough for the wide form."""
    window_prefill_case(sk, lq, lk, heads, window, sinks, seed=window)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lq,lk,heads,window", [([700], [4000], 2, 2700), ([3700], [3700], 1, 2600)])
def test_long_windows_hide_anything(sk, lq, lk, heads, window, bad):
    test_window_prefill_hidden_values_may_be_anything(sk, lq, lk, heads, window, bad)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lq,lk,heads,window", [([200], [200], 2, 40), ([300], [4000], 1, 100), ([1500], [1500], 2, 1100),
                                                ([600], [4000], 8, 1300)])
def test_window_prefill_hidden_values_may_be_anything(sk, lq, lk, heads, window, bad):
    """A key and a value that are not finite reach the rows whose window holds them, and no others."""
    q, k, v, r = prefill_inputs(gen(9), lq, lk, heads)
    at = lk[0] - 50 - window // 2
    k, v = k.clone(), v.clone()
    v[at, :, 3] = bad
    k[at + 1] = bad
    out, lse = sk.latent_window_prefill(q.cuda(), k.cuda(), v.cuda(), r.cuda(), starts(lq), starts(lk), SCALE, window, sinks=7)
    mref.check_prefill(out, lse, q, k, v, r, lq, lk, SCALE, window, 7, "hidden")
    pos = lk[0] - lq[0] + torch.arange(lq[0])
    sees = (pos >= at) & (pos < at + window)
    assert bool(sees.any()) and not bool(torch.isfinite(out.cpu()[sees][:, :, 3]).any())


def test_whole_windows_are_no_windows(sk):
    """A window over everything: bit for bit what latent_prefill gives."""
    for lq, heads in (([100, 400, 7], 3), ([1300, 1100], 2)):
        p = [t.cuda() for t in prefill_inputs(gen(10), lq, lq, heads)] + [starts(lq), starts(lq)]
        want, got = sk.latent_prefill(*p, SCALE), sk.latent_window_prefill(*p, SCALE, 1 << 30, sinks=3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------- key weights

def weights_case(sk, lens, heads, tokens, page, seed=0, columns=None, scale=SCALE):
    print("weights", dict(lens=lens[:8], heads=heads, tokens=tokens, page=page, columns=columns), flush=True)
    g = gen(seed)
    cache, table, n = paged(g, lens, page)
    q = normal(g, len(lens) * tokens, heads, DIM)
    _, lse = sk.latent_decode(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), scale, tokens=tokens)
    columns = columns or max(max(lens) + 3, 1)
    wide = torch.rand(len(lens), columns + 5, generator=g) * 4
    got = wide.cuda()
    back = sk.latent_key_weights(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), lse, got[:, :columns], scale, tokens=tokens)
    torch.cuda.synchronize()
    assert back.data_ptr() == got.data_ptr() and torch.equal(got[:, columns:].cpu(), wide[:, columns:])
    mref.check_weights(back, wide[:, :columns], q, cache, table, n, lse, scale, tokens, "weights")


@pytest.mark.parametrize("page", [1, 16, 48, 64])
def test_key_weights_lengths(sk, page):
    weights_case(sk, [1, 0, 31, 32, 33, 63, 64, 65, 127, 129, 500, 2], 8, 1, page, seed=page)


@pytest.mark.parametrize("heads,tokens", [(1, 1), (3, 1), (16, 1), (10, 2), (32, 1), (33, 1), (8, 4), (64, 1), (65, 1), (128, 1),
                                          (40, 4), (128, 3), (16, 16), (1, 7), (1, 100)])
def test_key_weights_shapes(sk, heads, tokens):
    weights_case(sk, [tokens, tokens + 1, 100, 333, 0, tokens - 1, 64 + tokens, 700], heads, tokens, 16, seed=heads + tokens)


def test_key_weights_long_and_many(sk):
    weights_case(sk, [9001], 8, 1, 64, seed=1)
    weights_case(sk, [20000, 17, 0, 5000], 16, 1, 64, seed=2, scale=0.5)
    weights_case(sk, [3001, 2000], 32, 16, 48, seed=3)
    rng = random.Random(4)
    weights_case(sk, [rng.choice((0, 1, 3, 40, 95, 300)) for _ in range(900)], 2, 1, 16, seed=4)


def test_key_weights_columns(sk):
    """Keys without a column are left out, causality counts from the request's end all the same."""
    weights_case(sk, [300, 40, 129, 7], 4, 5, 16, seed=5, columns=100)
    weights_case(sk, [300, 40], 4, 2, 16, seed=6, columns=1)


def test_key_weights_odd_numbers(sk):
    """A key that is not finite has a weight that is not; no other key and no other request has."""
    g = gen(11)
    cache, table, n = paged(g, [200, 90], 16)
    cache[table[0, 3], 5] = math.nan
    cache[table[1, 5], 9] = math.nan                             # the newest token's, which the one before does not see
    q = normal(g, 4, 8, DIM)
    lse = torch.full((4, 8), 3.0)
    got = sk.latent_key_weights(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), lse.cuda(), torch.zeros(2, 200, device="cuda"), SCALE,
                                tokens=2).cpu()
    odd = torch.zeros(2, 200, dtype=torch.bool)
    odd[0, 53] = odd[1, 89] = True
    assert torch.equal(torch.isnan(got), odd) and bool(torch.isfinite(got[~odd]).all())


def test_key_weights_repeat(sk):
    """Twice the same call: the same bits added, also on another stream."""
    g = gen(12)
    cache, table, n = (t.cuda() for t in paged(g, [5000, 321], 64))
    q = normal(g, 2, 24, DIM).cuda()
    _, lse = sk.latent_decode(q, cache, table, n, SCALE)
    make = lambda s=None: sk.latent_key_weights(q, cache, table, n, lse, torch.zeros(2, 5000, device="cuda"), SCALE, stream=s)
    first = make()
    assert abs(float(first.sum()) - 48) < 1e-3                   # every row's weights are 1 in all
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        w = torch.zeros(2, 5000, device="cuda")
        torch.cuda.synchronize()
        sk.latent_key_weights(q, cache, table, n, lse, w, SCALE, stream=side)
        side.synchronize()
        assert torch.equal(w, first)


# ---------------------------------------------------------------------------- select and keep

def select_case(sk, rows, budget, sinks, recent):
    lens = [len(r) for r in rows]
    most = max(lens + [1])
    w = torch.full((len(rows), most + 7), 1e30)                  # what lies behind a request's keys counts for nothing
    for i, r in enumerate(rows):
        w[i, :len(r)] = torch.tensor(r)
    kept, counts = sk.latent_select(w.cuda()[:, :most], torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, sinks=sinks,
                                    recent=recent)
    for i, r in enumerate(rows):
        want = mref.select(w[i].tolist(), len(r), budget, sinks, recent)
        assert int(counts[i]) == len(want)
        assert kept[i].tolist() == want + [-1] * (budget - len(want)), (i, len(r))


@pytest.mark.parametrize("budget,sinks,recent", [(0, 0, 0), (1, 0, 0), (5, 5, 0), (5, 0, 5), (64, 3, 10), (100, 0, 1), (300, 16, 64)])
def test_select(sk, budget, sinks, recent):
    g = gen(budget)
    draw = lambda n: torch.exp(2 * torch.randn(n, generator=g)).tolist()
    select_case(sk, [draw(n) for n in (0, 1, 5, 6, 63, 64, 65, 101, 299, 301, 1000, 4097)], budget, sinks, recent)


def test_select_ties_and_odd_numbers(sk):
    """Equal weights, zeros of both signs, infinities, NaN, weights that differ in their last bit only, and negative ones."""
    g = gen(13)
    few = torch.tensor([0.0, -0.0, 1.0, 1.0 + 2.0 ** -23, 2.0 ** -149, -1.0, math.inf, -math.inf, math.nan])
    rows = [few[torch.randint(0, 9, (n,), generator=g)].tolist() for n in (50, 700, 3000)] + [[0.0] * 900, [3.5] * 77]
    for budget, sinks, recent in ((20, 0, 0), (41, 7, 5), (690, 4, 60)):
        select_case(sk, rows, budget, sinks, recent)


@pytest.mark.parametrize("n", [36000, 36864 + 70, 40001, 150000])
def test_select_many_keys(sk, n):
    """Around what fits LDS, and beyond."""
    g = gen(14)
    rows = [torch.exp(2 * torch.randn(m, generator=g)).tolist() for m in (n, n // 2)]
    select_case(sk, rows, 2048, 4, 64)
    select_case(sk, [[round(x, 1) for x in r] for r in rows], n // 3, 0, 0)


@pytest.mark.parametrize("n", [65535, 65536, 65537, 66000])
def test_select_around_what_registers_hold(sk, n):
    g = gen(n)
    rows = [torch.exp(2 * torch.randn(m, generator=g)).tolist() for m in (n, 9)]
    select_case(sk, rows, 3000 + n % 7, 4, 64)
    select_case(sk, [[float(int(x)) for x in r] for r in rows], n - 5, 0, 0)


def keep_case(sk, lens, kept, page, tokens=0, columns=None, seed=0, counts=None, most=None):
    """kept: a rising list a request."""
    print("keep", dict(lens=lens[:8], page=page, tokens=tokens, columns=columns), flush=True)
    g = gen(seed)
    cache, table, n = paged(g, lens, page)
    most = most or max(len(k) for k in kept) + 2
    lists = torch.full((len(lens), most), -1, dtype=torch.int32)
    for i, k in enumerate(kept):
        lists[i, :len(k)] = torch.tensor(k, dtype=torch.int32)
    count = torch.tensor([len(k) for k in kept] if counts is None else counts, dtype=torch.int32)
    w = torch.randn(len(lens), columns, generator=g) if columns else None
    got = cache.cuda()
    new_lens, new_w = sk.latent_keep(got, table.cuda(), n.cuda(), lists.cuda(), count.cuda(), tokens=tokens,
                                     weights=w.cuda() if columns else None)
    torch.cuda.synchronize()
    want = cache.clone()
    for i, m in enumerate(lens):
        left, moved = mref.keep(want, table[i], m, lists[i, :max(0, min(int(count[i]), most))].tolist(), tokens,
                                w[i] if columns else None)
        assert int(new_lens[i]) == left, i
        if columns:
            assert torch.equal(new_w[i].cpu(), moved), i
    assert torch.equal(got.cpu(), want)
    assert columns or new_w is None


@pytest.mark.parametrize("page", [1, 16, 48, 64])
def test_keep(sk, page):
    g = gen(page)
    lens = [0, 1, 7, 64, 65, 300, 1500, 2600]
    some = lambda n, m: sorted(torch.randperm(n, generator=g)[:m].tolist())
    keep_case(sk, lens, [some(n, n * 2 // 3) for n in lens], page, columns=2600, seed=1)
    keep_case(sk, lens, [list(range(n)) for n in lens], page, seed=2)                     # nothing moves
    keep_case(sk, lens, [list(range(n // 2, n)) for n in lens], page, columns=70, seed=3)  # everything by the same way
    keep_case(sk, lens, [[] for n in lens], page, columns=1, seed=4)


@pytest.mark.parametrize("batch", [63, 64, 70])
def test_keep_of_many_requests(sk, batch):
    """Lists longer than what a workgroup moves at once, in requests of every length."""
    g = gen(batch)
    lens = [int(x) for x in torch.randint(0, 1900, (batch,), generator=g)]
    lens[:4] = 1900, 0, 1, 64
    some = lambda n, m: sorted(torch.randperm(n, generator=g)[:m].tolist())
    keep_case(sk, lens, [some(n, n * 3 // 4) for n in lens], 16, columns=1900, seed=1)
    keep_case(sk, lens, [list(range(n // 3, n)) for n in lens], 48, columns=1000, seed=2)
    keep_case(sk, lens, [list(range(n)) for n in lens], 16, seed=3)


@pytest.mark.parametrize("most", [63, 64, 65])
def test_keep_around_short_lists(sk, most):
    g = gen(most)
    lens = [700, 64, 65, 66, 63, 0]
    some = lambda n, m: sorted(torch.randperm(n, generator=g)[:min(n, m)].tolist())
    keep_case(sk, lens, [some(n, most) for n in lens], 16, columns=700, most=most)


def test_keep_after_a_tree(sk):
    g = gen(15)
    for tokens in (1, 2, 24, 200):
        lens = [tokens, tokens + 1, 100 + tokens, 333, tokens - 1, 0, 64 + tokens]
        path = lambda n: sorted(torch.randperm(min(n, tokens), generator=g)[:max(1, min(n, tokens) // 3)].tolist())
        keep_case(sk, lens, [path(n) if n >= tokens else [] for n in lens], 16, tokens=tokens, columns=400, seed=tokens)


def test_keep_numbers_of_no_row(sk):
    """Numbers that do not rise, lie before their place, or are not a request's, and counts past everything."""
    keep_case(sk, [20, 40, 300], [[5, 3, 25, 2 ** 30, -7, 19], [1, 1, 1, 39, 39], [100] * 60], 16, columns=50)
    keep_case(sk, [20, 40, 3], [[5, 3, 25, 2 ** 30], [1, 0, 7], [2, 7, 0]], 16, tokens=8, columns=50)
    keep_case(sk, [20, 40, 9], [[3, 4], [7, 9, 30], [1]], 16, counts=[-5, 10 ** 9, 2], most=3)


def test_select_and_keep_far_pages(sk):
    """Pages that lie more than 4 GiB into the cache, a cache of strided rows."""
    g = gen(16)
    small, table, lens = paged(g, [300, 77], 64)
    pages = 66000
    far = pages - small.shape[0]
    cache = torch.empty(pages, 64, DIM, dtype=BF, device="cuda")
    cache[far:] = small.cuda()
    moved = torch.where(table < small.shape[0], table + far, table)
    kept = [list(range(0, 300, 2)), list(range(50, 77))]
    lists = torch.full((2, 150), -1, dtype=torch.int32)
    for i, k in enumerate(kept):
        lists[i, :len(k)] = torch.tensor(k)
    counts = torch.tensor([len(k) for k in kept], dtype=torch.int32)
    sk.latent_keep(cache, moved.cuda(), lens.cuda(), lists.cuda(), counts.cuda())
    want = small.clone()
    for i in range(2):
        mref.keep(want, table[i], int(lens[i]), kept[i], 0)
    assert torch.equal(cache[far:].cpu(), want)
    wide = torch.full((small.shape[0], 64, DIM + 8), 7.0, dtype=BF, device="cuda")
    wide[:, :, :DIM] = small.cuda()
    sk.latent_keep(wide[:, :, :DIM], table.cuda(), lens.cuda(), lists.cuda(), counts.cuda())
    assert torch.equal(wide[:, :, :DIM].cpu(), want) and bool((wide[:, :, DIM:] == 7).all())


# ------------------------------------------------------------------------------ a run of them

def test_a_speculative_step_with_eviction(sk):
    """A tree step: rows appended at their positions, attention, the accepted path kept, its weights added,
    and the cache cut to its budget; then attention over what is left."""
    g = gen(17)
    lens0, tokens, heads, page = [200, 90, 33], 6, 8, 16
    B = len(lens0)
    cache, table, _ = paged(g, [n + tokens for n in lens0], page)
    cache, table = cache.cuda(), table.cuda()
    context = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    lens = context + tokens
    parents = torch.tensor([[-1, 0, 0, 1, 2, 4]] * B, dtype=torch.int32, device="cuda")
    mask, depth = sk.latent_tree_mask(parents)
    row = (context[:, None] + torch.arange(tokens, device="cuda")).long()
    slots = table.long().gather(1, row // page) * page + row % page
    positions = (context[:, None] + depth).long()
    kv, q = normal(g, B * tokens, DIM).cuda(), normal(g, B * tokens, heads, DIM).cuda()
    freq = inv_freq().cuda()
    sk.latent_append(kv, cache, slots.flatten(), positions.flatten(), freq, q=q[:, :, L:], q_out=q[:, :, L:])
    out, lse = sk.latent_tree_decode(q, cache, table, lens, mask, SCALE)
    above, _ = mref.ancestors(parents[0].tolist())
    mref.check_decode(out, lse, q, cache, table, lens, SCALE, tokens, lambda i, n: mref.seen_of(n, tokens, above=above), "step")
    # a verified path: the same rows as a chain appended from the start
    path = torch.tensor([[0, 2, 4]] * B, dtype=torch.int32, device="cuda")
    counts = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    chain = cache.clone()
    chosen = torch.tensor([0, 2, 4], device="cuda")
    sk.latent_append(kv.view(B, tokens, DIM)[:, chosen].flatten(0, 1), chain, slots[:, :3].flatten(),
                     (context[:, None] + torch.arange(3, device="cuda")).long().flatten(), freq)
    lens, _ = sk.latent_keep(cache, table, lens, path, counts, tokens=tokens)
    assert torch.equal(lens, context + 3)
    mine = q.view(B, tokens, heads, DIM)[:, chosen].flatten(0, 1).contiguous()
    got, want = (sk.latent_decode(mine, c, table, lens, SCALE, tokens=3) for c in (cache, chain))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    weights = torch.zeros(B, 256, device="cuda")
    sk.latent_key_weights(mine, cache, table, lens, got[1], weights, SCALE, tokens=3)
    mref.check_weights(weights, torch.zeros(B, 256), mine, cache, table, lens, got[1], SCALE, 3, "step")
    kept, count = sk.latent_select(weights, lens, 64, sinks=4, recent=16)
    before = cache.clone()
    left, fewer = sk.latent_keep(cache, table, lens, kept, count, weights=weights)
    rows = before.cpu()
    for i in range(B):
        numbers = mref.select(weights[i].tolist(), int(lens[i]), 64, 4, 16)
        assert int(left[i]) == len(numbers)
        mref.keep(rows, table[i].cpu(), int(lens[i]), numbers, 0)
        assert torch.equal(fewer[i, :len(numbers)], weights[i, numbers]) and not bool(fewer[i, len(numbers):].any())
    assert torch.equal(rows, cache.cpu())
    out, lse = sk.latent_window_decode(mine[::3].contiguous(), cache, table, left, SCALE, 20, sinks=4)
    mref.check_decode(out, lse, mine[::3], cache, table, left, SCALE, 1, lambda i, n: mref.seen_of(n, 1, 20, 4), "after")


def test_a_step_in_a_graph(sk):
    """Captured and replayed with new inputs, eager work between, on the same workspace."""
    g = gen(18)
    lens, tokens, heads, page = [300, 70, 129], 5, 8, 16
    B = len(lens)
    store, table, n = (t.cuda() for t in paged(g, lens, page))
    parents = torch.tensor([random_parents(g, tokens) for _ in lens], dtype=torch.int32, device="cuda")
    q = normal(g, B * tokens, heads, DIM).cuda()
    work = sk.latent_decode_workspace(B, tokens, heads)
    cache, weights = store.clone(), torch.zeros(B, 320, device="cuda")
    made = {}

    def step():
        cache.copy_(store)
        weights.zero_()
        mask, depth = sk.latent_tree_mask(parents)
        made["tree"] = sk.latent_tree_decode(q, cache, table, n, mask, SCALE, window=64, sinks=2, depth=depth, workspace=work)
        made["window"] = sk.latent_window_decode(q, cache, table, n, SCALE, 50, sinks=1, tokens=tokens, workspace=work)
        lse = sk.latent_decode(q, cache, table, n, SCALE, tokens=tokens, workspace=work)[1]
        sk.latent_key_weights(q, cache, table, n, lse, weights, SCALE, tokens=tokens)
        kept, counts = sk.latent_select(weights, n, 100, sinks=1, recent=10)
        made["keep"] = sk.latent_keep(cache, table, n, kept, counts, weights=weights)
        return [t for pair in made.values() for t in pair] + [kept, counts, cache, weights]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(4):
        g = gen(200 + seed)
        parents.copy_(torch.tensor([random_parents(g, tokens) for _ in lens], dtype=torch.int32))
        q.copy_(normal(g, B * tokens, heads, DIM))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_binding_refuses(sk):
    g = gen(19)
    cache, table, n = (t.cuda() for t in paged(g, [40, 20], 16))
    q = normal(g, 6, 4, DIM).cuda()
    parents = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    mask, depth = sk.latent_tree_mask(parents)
    w, lse = torch.zeros(2, 40, device="cuda"), torch.zeros(6, 4, device="cuda")
    kept, counts = sk.latent_select(w, n, 10)
    tree = lambda **k: sk.latent_tree_decode(q, cache, table, n, k.pop("mask", mask), SCALE, **k)
    p = [t.cuda() for t in prefill_inputs(g, [9], [9], 2)] + [starts([9]), starts([9])]
    for match, call in (
            ("mask", lambda: tree(mask=mask.long())), ("mask", lambda: tree(mask=mask.cpu())), ("mask", lambda: tree(mask=mask[:1])),
            ("rows", lambda: tree(mask=mask[:, :2])), ("depth", lambda: tree(window=4)), ("window", lambda: tree(window=2, depth=depth)),
            ("window", lambda: tree(window=-1)), ("sinks", lambda: tree(sinks=-1)), ("depth", lambda: tree(depth=depth.t())),
            ("contiguous", lambda: tree(mask=torch.zeros(2, 6, 1, dtype=torch.int32, device="cuda")[:, ::2])),
            ("512", lambda: sk.latent_tree_mask(torch.zeros(1, 513, dtype=torch.int32, device="cuda"))),
            ("parents", lambda: sk.latent_tree_mask(parents.long())), ("overlap", lambda: sk.latent_tree_mask(parents, depth=parents)),
            ("window", lambda: sk.latent_window_decode(q, cache, table, n, SCALE, 0, tokens=3)),
            ("sinks", lambda: sk.latent_window_decode(q, cache, table, n, SCALE, 4, sinks=-1, tokens=3)),
            ("window", lambda: sk.latent_window_prefill(*p, SCALE, 0)), ("sinks", lambda: sk.latent_window_prefill(*p, SCALE, 4, sinks=-1)),
            ("scale", lambda: sk.latent_window_prefill(*p, -1.0, 4)), ("window", lambda: sk.latent_window_prefill(*p, SCALE, 2.5)),
            ("weights", lambda: sk.latent_key_weights(q, cache, table, n, lse, w.double(), SCALE, tokens=3)),
            ("apart", lambda: sk.latent_key_weights(q, cache, table, n, lse, w[:1].expand(2, -1), SCALE, tokens=3)),
            ("lse", lambda: sk.latent_key_weights(q, cache, table, n, lse[:, :2], w, SCALE, tokens=3)),
            ("rows", lambda: sk.latent_key_weights(q, cache, table, n, lse, w, SCALE, tokens=2)),
            ("scale", lambda: sk.latent_key_weights(q, cache, table, n, lse, w, 0.0, tokens=3)),
            ("overlap", lambda: sk.latent_key_weights(q, cache, table, n, w.flatten()[:24].view(6, 4), w, SCALE, tokens=3)),
            ("budget", lambda: sk.latent_select(w, n, -1)), ("budget", lambda: sk.latent_select(w, n, 2.5)), ("budget", lambda: sk.latent_select(w, n, 5, sinks=3, recent=3)),
            ("recent", lambda: sk.latent_select(w, n, 5, recent=-1)), ("lens", lambda: sk.latent_select(w, n.long(), 5)),
            ("overlap", lambda: sk.latent_select(w, n, 10, counts=n)),
            ("overlap", lambda: sk.latent_keep(cache, table, n, kept, counts, new_lens=n)),
            ("overlap", lambda: sk.latent_keep(cache, table, n, kept, counts, weights=w, new_weights=w)),
            ("weights", lambda: sk.latent_keep(cache, table, n, kept, counts, new_weights=w)),
            ("tokens", lambda: sk.latent_keep(cache, table, n, kept, counts, tokens=-1)),
            ("kept", lambda: sk.latent_keep(cache, table, n, kept.long(), counts)),
            ("counts", lambda: sk.latent_keep(cache, table, n, kept, counts[:1])),
            ("overlap", lambda: sk.latent_keep(cache.as_strided((3, 4, DIM), (DIM, DIM, 1)), table, n, kept, counts))):
        with pytest.raises(ValueError, match=match):
            call()


def test_nothing_to_do(sk):
    """Empty batches, no heads, no columns, no budget."""
    empty = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device="cuda")
    cache = torch.ones(2, 4, DIM, dtype=BF, device="cuda")
    mask, depth = sk.latent_tree_mask(empty(0, 3))
    assert mask.shape == (0, 3, 1) and depth.shape == (0, 3)
    out, _ = sk.latent_tree_decode(empty(0, 4, DIM, t=BF), cache, empty(0, 2), empty(0), mask, SCALE)
    assert out.shape == (0, 4, L)
    out, _ = sk.latent_window_decode(empty(0, 4, DIM, t=BF), cache, empty(0, 2), empty(0), SCALE, 4)
    assert out.shape == (0, 4, L)
    n, table = torch.tensor([3], dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(1, 8, device="cuda")
    sk.latent_key_weights(empty(1, 0, DIM, t=BF), cache, table, n, empty(1, 0, t=torch.float32), w, SCALE)
    sk.latent_key_weights(normal(gen(0), 1, 2, DIM).cuda(), cache, table, n, torch.zeros(1, 2, device="cuda"), w[:, :0], SCALE)
    kept, counts = sk.latent_select(w, n, 0)
    lens, fresh = sk.latent_keep(cache, table, n, kept, counts, weights=w)
    assert kept.shape == (1, 0) and int(counts) == 0 and int(lens) == 0 and not bool(fresh.any())
    assert bool((cache == 1).all()) and bool((w == 1).all())


def test_tensors_of_other_streams(sk):
    """What a call allocates on a named stream is that stream's, and its results are right there."""
    g = gen(20)
    cache, table, n = (t.cuda() for t in paged(g, [2000, 77], 16))
    q = normal(g, 4, 8, DIM).cuda()
    parents = torch.tensor([[-1, 0], [-1, -1]], dtype=torch.int32, device="cuda")
    mask, _ = sk.latent_tree_mask(parents)
    w = torch.rand(2, 2000, generator=g).cuda()
    kept, counts = sk.latent_select(w, n, 30)
    p = [t.cuda() for t in prefill_inputs(g, [100], [3000], 2)] + [starts([100]), starts([3000])]
    calls = (lambda s: sk.latent_tree_mask(parents, stream=s), lambda s: sk.latent_tree_decode(q, cache, table, n, mask, SCALE, stream=s),
             lambda s: sk.latent_window_decode(q, cache, table, n, SCALE, 100, tokens=2, stream=s),
             lambda s: sk.latent_window_prefill(*p, SCALE, 1000, stream=s), lambda s: sk.latent_select(w, n, 30, stream=s),
             lambda s: sk.latent_keep(copies.pop(), table, n, kept, counts, weights=w, stream=s))
    side, copies = torch.cuda.Stream(), [cache.clone(), cache.clone()]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        kinds = [(t.shape, t.dtype, t.data_ptr()) for t in got]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
        for shape, dtype, where in kinds:
            assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != where
