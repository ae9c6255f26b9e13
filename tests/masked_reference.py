"""Trees, windows and kept keys of the latent attention operators in 64 bits on the CPU. Outputs are checked
with the bounds of latent_reference.py, row set by row set, so that keys that a row does not see never enter
its sums.

Bound of key weights. A row's weight of a key is exp2(fma(s, c, -m)) with c = scale log2 e and m = lse log2 e,
each rounded at most twice, so its exponent is off by the score's own error (latent_reference.py: at most
576 * 2^-24 * scale * sum |q c|) and at most (|s| + |lse|) * 2^-22, and the exponential by 2^-21
relative. R of them and the earlier weight w, all of one sign, are added in fp32: at most R * 2^-24 relative to
their sum, and half a step of the result. With e the sum of the first two,

    |weights - exact| <= sum_r p_r (1.01 e_r + 2^-21 + R * 2^-24) + 2^-23 (w + sum_r p_r).
"""
import torch

import latent_reference as ref


def keys_of(cache, table, lens, i):
    """Request i's rows in 64 bits, lengths and page ids clamped."""
    page = cache.shape[1]
    n = max(0, min(int(lens[i]), table.shape[1] * page))
    at = torch.arange(n)
    return cache[table[i, at // page].long().clamp(0, cache.shape[0] - 1), at % page].double()


def ancestors(parents):
    """bool [tokens, tokens], and depth, from parents [tokens] walked one by one."""
    t = len(parents)
    above, depth = torch.zeros(t, t, dtype=torch.bool), torch.zeros(t, dtype=torch.int32)
    for j, p in enumerate(parents):
        if 0 <= p < j:
            above[j] = above[p]
            depth[j] = depth[p] + 1
        above[j, j] = True
    return above, depth


def words_of(above):
    """Bits [.., tokens] as int32 words [.., ceil(tokens / 32)]."""
    t = above.shape[-1]
    words = -(-t // 32)
    bits = torch.nn.functional.pad(above.long(), (0, words * 32 - t)).unflatten(-1, (words, 32))
    w = (bits << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def seen_of(n, tokens, window=0, sinks=0, above=None, depth=None):
    """bool [tokens, n]: the keys that each of a request's newest tokens sees."""
    base, k = n - tokens, torch.arange(n)[None]
    j = torch.arange(tokens)[:, None]
    at = base + (j if above is None or depth is None else depth[:, None])
    near = (k > at - window) | (k < sinks) if window else torch.ones(1, n, dtype=torch.bool)
    if above is None:
        return (k <= base + j) & near
    seen = ((k < base) & near).expand(tokens, n).clone()
    for d in range(max(0, -base), tokens):
        seen[:, base + d] = above[:, d]
    return seen


def check_decode(out, lse, q, cache, table, lens, scale, tokens, seen, what):
    """seen(i, n): bool [tokens, n] of request i."""
    out, lse, q, cache, table, lens = (t.cpu() for t in (out, lse, q, cache, table, lens))
    heads = q.shape[1]
    for i in range(len(lens)):
        keys = keys_of(cache, table, lens, i)
        rows = seen(i, len(keys))
        for j in range(tokens):
            r, mine = i * tokens + j, keys[rows[j]]
            answer = ref.attend(q[r].double(), mine, mine[:, :512], scale, torch.ones(heads, len(mine), dtype=torch.bool))
            ref.check(out[r], lse[r], answer, len(keys), "%s: request %d of %d keys, token %d" % (what, i, len(keys), j))


def check_prefill(out, lse, q, k, v, k_rot, lq, lk, scale, window, sinks, what):
    out, lse, q, k, v, k_rot = (t.cpu() for t in (out, lse, q, k, v, k_rot))
    a = b = 0
    for i, (m, n) in enumerate(zip(lq, lk)):
        at, key = (n - m + torch.arange(m))[:, None], torch.arange(n)[None]
        seen = (key <= at) & ((key > at - window) | (key < sinks))
        for h in range(q.shape[1]):
            keys = torch.cat((k[b:b + n, h], k_rot[b:b + n]), -1).double()
            vals = v[b:b + n, h].double()
            odd = ~(torch.isfinite(vals).all(-1) & torch.isfinite(keys).all(-1))
            # rows that see one of the odd keys are left to the test
            rows = (~(seen & odd[None]).any(-1)).nonzero().flatten()
            if rows.numel() == 0:
                continue
            keys, vals = keys.masked_fill(odd[:, None], 0), vals.masked_fill(odd[:, None], 0)
            answer = ref.attend(q[a + rows, h].double(), keys, vals, scale, seen[rows])
            ref.check(out[a + rows, h], lse[a + rows, h], answer, n, "%s: sequence %d (%d x %d), head %d" % (what, i, m, n, h))
        a, b = a + m, b + n


def check_weights(got, before, q, cache, table, lens, lse, scale, tokens, what):
    """got, before: weights [batch, columns] after and before the call."""
    got, before, q, cache, table, lens, lse = (t.cpu() for t in (got, before, q, cache, table, lens, lse))
    heads, columns = q.shape[1], got.shape[1]
    for i in range(len(lens)):
        keys = keys_of(cache, table, lens, i)
        n, m = len(keys), min(len(keys), columns)
        assert torch.equal(got[i, m:], before[i, m:]), "%s: columns behind request %d" % (what, i)
        rows = q[i * tokens:(i + 1) * tokens].reshape(tokens * heads, -1).double()
        s, mag = rows @ keys[:m].T * scale, rows.abs() @ keys[:m].abs().T * scale
        sums = lse[i * tokens:(i + 1) * tokens].reshape(-1, 1).double()
        limit = (n - tokens + torch.arange(tokens)).repeat_interleave(heads)[:, None]
        seen = torch.arange(m)[None] <= limit
        p = torch.where(seen, (s - sums).exp(), torch.zeros((), dtype=torch.float64))
        off = mag * 576 * 2.0 ** -24 + (s.abs() + torch.where(seen, sums.abs(), 0)) * 2.0 ** -22
        want, w = before[i, :m].double() + p.sum(0), before[i, :m].double().abs()
        bound = (p * (1.01 * off + 2.0 ** -21 + tokens * heads * 2.0 ** -24)).sum(0) + 2.0 ** -23 * (w + p.sum(0)) + 1e-37
        worst = ((got[i, :m].double() - want).abs() / bound).max().item() if m else 0.0
        assert worst <= 1, "%s: request %d off by %.2f of its bound" % (what, i, worst)


def select(weights, n, budget, sinks, recent):
    """Rising numbers of the keys that stay, of one request's weights (a list)."""
    if n <= budget:
        return list(range(n))
    size = lambda k: (0, 0.0) if weights[k] != weights[k] else (1, -weights[k])      # a NaN first
    between = sorted(range(sinks, n - recent), key=lambda k: (size(k), k))[:budget - sinks - recent]
    return sorted(list(range(sinks)) + between + list(range(n - recent, n)))


def keep(cache, table, n, kept, tokens, weights=None):
    """One request: its rows moved in `cache` (in place), its new length, its new weights."""
    page, first = cache.shape[1], n - tokens if tokens else 0
    base = max(0, first)
    kept = kept[:n - base]
    slot = lambda k: (int(table[k // page].clamp(0, cache.shape[0] - 1)), k % page)
    source = [first + k if base + j <= first + k < n else base + j for j, k in enumerate(kept)]
    rows = [cache[slot(k)].clone() for k in source]
    for j, row in enumerate(rows):
        cache[slot(base + j)] = row
    moved = None
    if weights is not None:
        moved = torch.zeros_like(weights)
        for j, k in enumerate(list(range(base)) + source):
            if j < len(moved) and k < len(moved):
                moved[j] = weights[k]
    return base + len(kept), moved
