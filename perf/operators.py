"""The latent attention operators as a benchmark sees them: cases, inputs, one pass, its work.

Latent attention keeps one vector a token in the cache: a latent of LATENT numbers, from which
every head's keys and values follow by fixed projections, and ROT numbers of a rotated key that
all heads share. Three operators serve it:

  append   latents are normalised, rotated keys get their position, both go to their slot of a
           paged cache, and the queries' rotated parts get their position in the same pass
  decode   the absorbed form: queries already carry the key projection, so all heads attend to
           the cached vectors themselves; the sum over the latents is what comes out
  prefill  the expanded form for prompts: keys and values of each head next to the shared
           rotated key, ragged sequences, causal or not

`run` computes a case in elementary torch operations in 32 bits (`own` false), or calls this
repository's kernels (`own` true). `exact` gives the outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

LATENT = 512     # latent numbers a token
ROT = 64         # numbers of the shared rotated key
HEAD = 128       # numbers of a head's own key, and of its value
DIM = LATENT + ROT
THETA = 10000.0  # base of the rotation's frequencies
EPS = 1e-6
SCALE = 1.0 / math.sqrt(HEAD + ROT)
DEV = "cuda"


def listed():
    return [
        # one request's next token on a rank with 8 heads
        dict(name="append_single", op="append", n=1, heads=8, page=64, interleaved=False, pad=0),
        # a speculative step: 64 requests of 4 draft tokens, some rows padding of a captured batch
        dict(name="append_verify", op="append", n=256, heads=8, page=16, interleaved=True, pad=9),
        # a long prompt of a whole layer's heads (no tensor parallelism), an odd number of tokens
        dict(name="append_prompt", op="append", n=8191, heads=128, page=64, interleaved=False, pad=0),
        # one request early in its answer: latency
        dict(name="decode_single", op="decode", batch=1, tokens=1, heads=8, mean=500, spread=0.0, page=64),
        # a serving batch of short, ragged requests, single-token pages
        dict(name="decode_short", op="decode", batch=128, tokens=1, heads=16, mean=700, spread=0.9, page=1),
        # a speculative step at moderate context: 64 requests of 4 draft tokens, 8 heads a rank
        dict(name="decode_verify", op="decode", batch=64, tokens=4, heads=8, mean=4096, spread=0.5, page=64),
        # one request with a very long context, odd page size
        dict(name="decode_long", op="decode", batch=1, tokens=1, heads=32, mean=131071, spread=0.0, page=48),
        # a full batch with every head of the layer on this card
        dict(name="decode_full", op="decode", batch=96, tokens=1, heads=128, mean=4000, spread=0.3, page=64),
        # a short prompt alone
        dict(name="prefill_short", op="prefill", batch=1, heads=8, mean=129, spread=0.0, past=0, causal=True),
        # several ragged prompts in one batch
        dict(name="prefill_ragged", op="prefill", batch=6, heads=32, mean=1000, spread=0.9, past=0, causal=True),
        # a later chunk of a long prompt: its tokens attend to all earlier ones
        dict(name="prefill_chunk", op="prefill", batch=1, heads=8, mean=1024, spread=0.0, past=15000, causal=True),
        # one long prompt
        dict(name="prefill_long", op="prefill", batch=1, heads=32, mean=8192, spread=0.0, past=0, causal=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    top = max((c for c in listed() if c["op"] == op), key=lambda c: work(c)["bytes" if op == "append" else "flops"])
    limit = work(top)
    while True:
        if op == "append":
            case = dict(op=op, n=_spread(rng, 1, 16384), heads=rng.choice((1, 5, 8, 16, 20, 32, 64, 128)),
                        page=rng.choice((1, 16, 24, 64, 128)), interleaved=rng.random() < 0.5,
                        pad=rng.choice((0, 0, 7, 50)))
        elif op == "decode":
            case = dict(op=op, batch=_spread(rng, 1, 256), tokens=rng.choice((1, 1, 1, 2, 3, 4, 7)),
                        heads=rng.choice((1, 4, 8, 10, 16, 32, 40, 64, 128)), mean=_spread(rng, 16, 131072),
                        spread=rng.choice((0.0, 0.3, 0.9)), page=rng.choice((1, 16, 48, 64, 128)))
        else:
            case = dict(op=op, batch=_spread(rng, 1, 32), heads=rng.choice((1, 5, 8, 20, 32, 64)),
                        mean=_spread(rng, 16, 8192), spread=rng.choice((0.0, 0.3, 0.9)),
                        past=rng.choice((0, 0, 100, 4000)), causal=rng.random() < 0.8)
        cost = work(case)
        if cost["bytes"] <= limit["bytes"] and cost["flops"] <= limit["flops"]:
            return case


def _lengths(case):
    """The sequences' lengths: a rule of the case alone, uniform over mean * (1 -+ spread)."""
    rng = random.Random(case["batch"] * 7919 + case["mean"])
    low, high = case["mean"] * (1 - case["spread"]), case["mean"] * (1 + case["spread"])
    least = case.get("tokens", 1)
    return [max(least, int(round(rng.uniform(low, high)))) for _ in range(case["batch"])]


def _pairs(lq, lk, causal):
    """Query-key pairs that attend, the last query seeing the last key."""
    if not causal:
        return lq * lk
    first = lk - lq + 1                      # keys that the first query sees
    return lq * first + lq * (lq - 1) // 2


def work(case):
    if case["op"] == "append":
        n, heads = case["n"], case["heads"]
        kept = n - (n // case["pad"] if case["pad"] else 0)
        return {"bytes": n * (DIM * 2 + 16) + kept * DIM * 2 + n * heads * ROT * 4 + LATENT * 2 + ROT * 4,
                "flops": n * (LATENT * 4 + ROT * 3 * (heads + 1))}
    lens = _lengths(case)
    if case["op"] == "decode":
        heads, t = case["heads"], case["tokens"]
        rows = case["batch"] * t * heads
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": sum(lens) * DIM * 2 + rows * (DIM * 2 + LATENT * 2 + 4) + pages * 4 + len(lens) * 4,
                "flops": heads * sum(_pairs(t, n, True) for n in lens) * 2 * (DIM + LATENT)}
    heads = case["heads"]
    nq, nk = sum(lens), sum(lens) + case["past"] * len(lens)
    pairs = sum(_pairs(n, n + case["past"], case["causal"]) for n in lens)
    return {"bytes": nq * heads * ((HEAD + ROT) * 2 + HEAD * 2 + 4) + nk * (heads * HEAD * 4 + ROT * 2),
            "flops": heads * pairs * 2 * (HEAD + ROT + HEAD)}


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    state = _INPUTS[case["op"]](case, g)
    state["op"] = case["op"]
    return state


def _append_inputs(case, g):
    n, heads, page = case["n"], case["heads"], case["page"]
    pages = -(-n // page) + 3
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].contiguous()
    if case["pad"]:
        slots[case["pad"] - 1::case["pad"]] = -1             # padding rows write nothing
    return dict(kv=_normal(g, n, DIM), cache=_normal(g, pages, page, DIM), slots=slots,
                positions=torch.randint(0, 131072, (n,), generator=g, device=DEV),
                inv_freq=THETA ** (-torch.arange(0, ROT, 2, device=DEV, dtype=torch.float64) / ROT),
                weight=(1 + 0.1 * torch.randn(LATENT, generator=g, device=DEV)).to(torch.bfloat16),
                # the rotated part is the tail of each head's query
                q=_normal(g, n, heads, DIM)[:, :, LATENT:],
                q_out=torch.empty(n, heads, ROT, device=DEV, dtype=torch.bfloat16),
                interleaved=case["interleaved"])


def _decode_inputs(case, g):
    lens, page = _lengths(case), case["page"]
    counts = [-(-n // page) for n in lens]
    order = torch.randperm(sum(counts) + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), max(counts), dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    rows = case["batch"] * case["tokens"]
    state = dict(q=_normal(g, rows, case["heads"], DIM), cache=_normal(g, sum(counts) + 2, page, DIM), table=table,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), host_lens=lens, tokens=case["tokens"],
                 out=torch.empty(rows, case["heads"], LATENT, device=DEV, dtype=torch.bfloat16),
                 lse=torch.empty(rows, case["heads"], device=DEV, dtype=torch.float32), workspace=None)
    if own:
        import decode_skinny_addmm_amd as sk
        state["workspace"] = sk.latent_decode_workspace(case["batch"], case["tokens"], case["heads"], LATENT, DEV)
    return state


def _prefill_inputs(case, g):
    lq = _lengths(case)
    lk = [n + case["past"] for n in lq]
    starts = lambda lens: torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    heads, nq, nk = case["heads"], sum(lq), sum(lk)
    kv = _normal(g, nk, heads, 2 * HEAD)                     # one projection gives keys and values
    return dict(q=_normal(g, nq, heads, HEAD + ROT), k=kv[:, :, :HEAD], v=kv[:, :, HEAD:], k_rot=_normal(g, nk, ROT),
                cu_q=starts(lq), cu_k=starts(lk), host_q=lq, host_k=lk, causal=case["causal"],
                out=torch.empty(nq, heads, HEAD, device=DEV, dtype=torch.bfloat16),
                lse=torch.empty(nq, heads, device=DEV, dtype=torch.float32))


_INPUTS = {"append": _append_inputs, "decode": _decode_inputs, "prefill": _prefill_inputs}


# ---------------------------------------------------------------------------- one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _append_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_append(s["kv"], s["cache"], s["slots"], s["positions"], s["inv_freq"], norm_weight=s["weight"], eps=EPS,
                     q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"])
    return s["cache"], s["q_out"]


def _decode_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_decode(s["q"], s["cache"], s["table"], s["lens"], SCALE, tokens=s["tokens"], rope_dim=ROT, out=s["out"],
                     lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _prefill_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_prefill(s["q"], s["k"], s["v"], s["k_rot"], s["cu_q"], s["cu_k"], SCALE, causal=s["causal"],
                      out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _rotate(x, cos, sin, interleaved):
    """Pairs of x turned by their angles: neighbours, or the halves' same places."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, dim=-1)
    y, z = a * cos - b * sin, b * cos + a * sin
    return torch.stack((y, z), dim=-1).flatten(-2) if interleaved else torch.cat((y, z), dim=-1)


def _append_plain(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # 64 bits: far positions are many turns
    cos, sin = angle.cos().float(), angle.sin().float()
    kv = s["kv"].float()
    latent = kv[:, :LATENT]
    latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat((latent, _rotate(kv[:, LATENT:], cos, sin, s["interleaved"])), dim=-1).to(torch.bfloat16)
    kept = s["slots"] >= 0
    s["cache"].view(-1, DIM)[s["slots"][kept]] = row[kept]
    s["q_out"].copy_(_rotate(s["q"].float(), cos[:, None], sin[:, None], s["interleaved"]))
    return s["cache"], s["q_out"]


def _softmax_sum(score, seen, value):
    """softmax over the seen places of a row times value, and the log of its sum; no place seen: 0, -inf."""
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(score.dtype).min)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    return p @ value / total.clamp_min(torch.finfo(score.dtype).tiny), (top + total.log()).squeeze(-1)


def _decode_plain(s):
    t, heads = s["tokens"], s["q"].shape[1]
    page = s["cache"].shape[1]
    for i, n in enumerate(s["host_lens"]):
        keys = s["cache"][s["table"][i, :-(-n // page)]].view(-1, DIM)[:n].float()
        q = s["q"][i * t:(i + 1) * t].float().view(t * heads, DIM)
        last = torch.arange(n - t, n, device=DEV).repeat_interleave(heads)
        seen = torch.arange(n, device=DEV) <= last[:, None]
        out, lse = _softmax_sum(q @ keys.T * SCALE, seen, keys[:, :LATENT])
        s["out"][i * t:(i + 1) * t] = out.view(t, heads, LATENT)
        s["lse"][i * t:(i + 1) * t] = lse.view(t, heads)
    return s["out"], s["lse"]


def _prefill_plain(s):
    heads = s["q"].shape[1]
    q0 = k0 = 0
    for lq, lk in zip(s["host_q"], s["host_k"]):
        a, b = slice(q0, q0 + lq), slice(k0, k0 + lk)
        q0, k0 = q0 + lq, k0 + lk
        seen = torch.ones(lq, lk, dtype=torch.bool, device=DEV)
        if s["causal"]:
            seen = seen.tril(lk - lq)
        step = max(1, (1 << 28) // (lq * lk))                # heads at a time: a GiB of scores
        for h in range(0, heads, step):
            hs = slice(h, min(heads, h + step))
            count = hs.stop - hs.start
            keys = torch.cat((s["k"][b, hs].float(), s["k_rot"][b, None].float().expand(lk, count, ROT)), dim=-1)
            score = s["q"][a, hs].float().transpose(0, 1) @ keys.permute(1, 2, 0) * SCALE
            out, lse = _softmax_sum(score, seen, s["v"][b, hs].float().transpose(0, 1))
            s["out"][a, hs] = out.transpose(0, 1).to(torch.bfloat16)
            s["lse"][a, hs] = lse.transpose(0, 1)
    return s["out"], s["lse"]


_OWN = {"append": _append_own, "decode": _decode_own, "prefill": _prefill_own}
_PLAIN = {"append": _append_plain, "decode": _decode_plain, "prefill": _prefill_plain}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _append_exact(s):
    # pairs as complex numbers, turned by exp(i * position * frequency)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["inv_freq"])

    def turned(x, by):
        x = x.double()
        if s["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (ROT // 2, 2)).contiguous()) * by).flatten(-2)
        z = torch.complex(x[..., :ROT // 2], x[..., ROT // 2:]) * by
        return torch.cat((z.real, z.imag), dim=-1)

    cache = s["cache"].double().view(-1, DIM)
    latent = s["kv"][:, :LATENT].double()
    power = (latent * latent).sum(-1) / LATENT + EPS
    kept = (s["slots"] >= 0).nonzero().squeeze(-1)
    where = s["slots"][kept]
    cache[where, :LATENT] = (latent / power.sqrt()[:, None] * s["weight"].double())[kept]
    cache[where, LATENT:] = turned(s["kv"][:, LATENT:], turn)[kept]
    return cache.view(s["cache"].shape), turned(s["q"], turn[:, None])


def _decode_exact(s):
    t = s["tokens"]
    page = s["cache"].shape[1]
    out, lse = [], []
    for i, n in enumerate(s["host_lens"]):
        place = torch.arange(n, device=DEV)
        keys = s["cache"].flatten(0, 1)[s["table"][i].long()[place // page] * page + place % page].double()
        for j in range(t):
            upto = n - t + j + 1
            score = s["q"][i * t + j].double().mul(SCALE) @ keys[:upto].T.contiguous()
            lse.append(score.logsumexp(-1))
            out.append((score - lse[-1][:, None]).exp() @ keys[:upto, :LATENT])
    return torch.stack(out), torch.stack(lse)


def _prefill_exact(s):
    heads = s["q"].shape[1]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for lq, lk in zip(s["host_q"], s["host_k"]):
        hidden = torch.arange(lk, device=DEV)[None] > torch.arange(lk - lq, lk, device=DEV)[:, None]
        shared = s["k_rot"][k0:k0 + lk].double().T.contiguous()
        for h in range(heads):
            q = s["q"][q0:q0 + lq, h].double()
            score = q[:, :HEAD] @ s["k"][k0:k0 + lk, h].double().T.contiguous() + q[:, HEAD:] @ shared
            score *= SCALE
            if s["causal"]:
                score[hidden] = -math.inf
            lse[q0:q0 + lq, h] = score.logsumexp(-1)
            score -= lse[q0:q0 + lq, h, None]
            out[q0:q0 + lq, h] = score.exp_() @ s["v"][k0:k0 + lk, h].double().contiguous()
        q0, k0 = q0 + lq, k0 + lk
    return out, lse


_EXACT = {"append": _append_exact, "decode": _decode_exact, "prefill": _prefill_exact}
