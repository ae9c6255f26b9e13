"""The latent attention operators in 64 bits on the CPU, with the bounds that a bf16 kernel with
fp32 sums has to keep.

Bounds. HALF = 2^-8 is half a bf16 step relative to the value. One score is a sum of `dim` exact
products in fp32, off by at most dim * 2^-24 * sum |q c| in any order; `delta` is scale times the
largest such bound of a row (plus 2^-21 (1 + |s|) for its scaling and exponential), so a softmax
weight is off by at most 2 delta relative, the normaliser included. The weights are rounded once to
bf16 (HALF each) and the output once (HALF). So, for a row with weights p,

    |out - exact| <= HALF |exact| + (1 + HALF)(HALF + 2 delta + keys * 2^-24) sum_k p_k |v_k|
    |lse - exact| <= delta + 2^-20 (1 + |exact|)

and, roundings of different keys being independent, over a whole output

    ||out - exact|| <= HALF (||exact|| + ||sqrt(sum_k p_k^2 v_k^2)||) + 2 ||delta sum_k p_k |v_k| ||.
"""
import math

import torch

HALF = 2.0 ** -8


def attend(q, k, v, scale, seen):
    """One head's rows: q [r, d], k [n, d], v [n, e], seen bool [r, n], all float64. Returns out, lse,
    and the bounds' terms: delta [r], sum p |v| [r, e], sqrt(sum p^2 v^2) [r, e]. Values and keys
    that a row does not see never enter its sums."""
    r, n = seen.shape
    if n == 0:
        z = torch.zeros(r, v.shape[1], dtype=torch.float64)
        return z, torch.full((r,), -math.inf, dtype=torch.float64), torch.zeros(r, dtype=torch.float64), z, z
    s = (q @ k.T) * scale
    mag = (q.abs() @ k.abs().T) * scale
    s = s.masked_fill(~seen, -math.inf)
    lse = s.logsumexp(-1)
    p = torch.where(seen, (s - lse[:, None]).exp(), torch.zeros((), dtype=torch.float64)).nan_to_num(0.0)
    delta = (mag * q.shape[1] * 2.0 ** -24 + 2.0 ** -21 * (1 + s.abs())).masked_fill(~seen, 0.0).amax(-1)
    hidden = ~seen.any(0)
    v = v.masked_fill(hidden[:, None], 0.0)
    return p @ v, lse, delta, p @ v.abs(), ((p * p) @ (v * v)).sqrt()


def check(out, lse, ref, keys, what):
    """out bf16 [r, e] and lse fp32 [r] on any device against attend()'s answer."""
    e, el, delta, pv, pv2 = ref
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = el == -math.inf
    assert torch.equal(out[empty], torch.zeros_like(out[empty])), what + ": a row without keys is not zero"
    assert bool((lse[empty] == -math.inf).all()), what + ": lse of a row without keys"
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[~empty]).all()), what + ": not finite"
    d = delta[:, None]
    bound = HALF * e.abs() + (1 + HALF) * (HALF + 2 * d + keys * 2.0 ** -24) * pv + 1e-30
    worst = ((out - e).abs() / bound).max().item() if out.numel() else 0.0
    assert worst <= 1, "%s: out off by %.2f of its bound" % (what, worst)
    norm = HALF * (e.norm() + pv2.norm()) + 2 * (d * pv).norm() + 1e-30
    assert (out - e).norm() <= norm, "%s: out off by %.3g, bound %.3g" % (what, (out - e).norm(), norm)
    off = (lse - el).abs()[~empty]
    assert bool((off <= (delta + 2.0 ** -20 * (1 + el.abs()))[~empty]).all()), "%s: lse off by %.3g" % (what, off.max())


def decode(q, cache, table, lens, scale, tokens, latent=512):
    """Per request: attend()'s answers of all its rows (token major, then head), keys."""
    q, cache, table, lens = (t.cpu() for t in (q, cache, table, lens))
    heads, page = q.shape[1], cache.shape[1]
    answers = []
    for i, n in enumerate(lens.tolist()):
        n = max(0, min(n, table.shape[1] * page))
        ids = table[i, torch.arange(n) // page].long().clamp(0, cache.shape[0] - 1)
        keys = cache[ids, torch.arange(n) % page].double()
        rows = q[i * tokens:(i + 1) * tokens].reshape(tokens * heads, -1).double()
        limit = (n - tokens + 1 + torch.arange(tokens)).clamp_min(0).repeat_interleave(heads)
        seen = torch.arange(n)[None] < limit[:, None]
        # a key that only some rows see must not reach the others through a product with 0
        outs = [attend(rows[limit == m], keys[:m], keys[:m, :latent], scale, seen[limit == m][:, :m])
                for m in limit.unique().tolist()]
        answers.append((tuple(torch.cat([o[j] for o in outs]) for j in range(5)), n))
    return answers


def check_decode(out, lse, q, cache, table, lens, scale, tokens, what):
    heads = q.shape[1]
    for i, (ref, n) in enumerate(decode(q, cache, table, lens, scale, tokens)):
        rows = slice(i * tokens, (i + 1) * tokens)
        check(out[rows].reshape(tokens * heads, -1), lse[rows].reshape(-1), ref, n, "%s: request %d of %d keys" % (what, i, n))


def check_prefill(out, lse, q, k, v, k_rot, lq, lk, scale, causal, what):
    out, lse, q, k, v, k_rot = (t.cpu() for t in (out, lse, q, k, v, k_rot))
    a = b = 0
    for i, (m, n) in enumerate(zip(lq, lk)):
        limit = (n - m + 1 + torch.arange(m)).clamp(0, n) if causal else torch.full((m,), n)
        for h in range(q.shape[1]):
            keys = torch.cat((k[b:b + n, h], k_rot[b:b + n]), -1).double()
            vals = v[b:b + n, h].double()
            odd = not bool(torch.isfinite(vals).all() and torch.isfinite(keys).all())
            groups = limit.unique().tolist() if odd else [None]
            for g in groups:
                rows = torch.arange(m) if g is None else (limit == g).nonzero().flatten()
                e = n if g is None else g
                if rows.numel() == 0:
                    continue
                seen = torch.arange(e)[None] < limit[rows][:, None]
                ref = attend(q[a + rows, h].double(), keys[:e], vals[:e], scale, seen)
                check(out[a + rows, h], lse[a + rows, h], ref, n, "%s: sequence %d (%d x %d), head %d" % (what, i, m, n, h))
        a, b = a + m, b + n


def turned(x, positions, inv_freq, interleaved):
    """The rotation in 64 bits and, beside it, |a| + |b| of each number's pair (its error's measure)."""
    x = x.cpu().double()
    angle = positions.cpu().double()[:, None] * inv_freq.cpu()
    while angle.dim() < x.dim():
        angle = angle[:, None]
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y, z, m = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), a.abs() + b.abs()
    if interleaved:
        return torch.stack((y, z), -1).flatten(-2), torch.stack((m, m), -1).flatten(-2)
    return torch.cat((y, z), -1), torch.cat((m, m), -1)


def append(kv, positions, inv_freq, weight, eps, interleaved, latent=512):
    """Rows [n, 576] in 64 bits and the bound of a bf16 row with fp32 arithmetic: half a step of the
    value, and before it 2^-19 relative for the norm (a sum of 512 squares, all of one sign, of
    pairwise depth at most 14 roundings, root, division and two products) or 2^-21 (|a| + |b|) for a
    rotation (cosine, sine, two products, a sum)."""
    x = kv.cpu().double()
    z, rest = x[:, :latent], x[:, latent:]
    pre = torch.zeros_like(z)
    if weight is not None:
        z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * weight.cpu().double()
        pre = z.abs() * 2.0 ** -19
    r, m = turned(rest, positions, inv_freq, interleaved)
    rows = torch.cat((z, r), -1)
    pre = torch.cat((pre, m * 2.0 ** -21), -1)
    return rows, HALF * rows.abs() + (1 + HALF) * pre
