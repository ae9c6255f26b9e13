"""Latent attention over long and speculative answers as a benchmark sees it: cases, inputs, one pass, its work.

The cache holds one row a token: LATENT numbers, from which every head's keys and values follow,
and ROT numbers of a rotated key that all heads share. These operators bound what a token reads of
it, what it holds, and let a step verify a whole tree of drafted tokens:

  tree     absorbed attention of a tree of drafted tokens: each sees the context and its ancestors
  window   absorbed attention of the newest tokens to the last `window` keys and the first `sinks`
  prompt   the same rule for prompts, over keys and values of each head
  weights  what the newest tokens' softmax weights of each key add up to
  evict    the keys with the largest sums stay: selection, and their rows move to the front
  commit   the accepted nodes of a verified tree move to the front of the drafted rows

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
SCALE = 1.0 / math.sqrt(HEAD + ROT)
DEV = "cuda"


def listed():
    return [
        # one request's step with a small tree early in its answer: latency
        dict(name="tree_single", op="tree", batch=1, tokens=7, heads=8, mean=500, spread=0.0, page=64, window=0, sinks=0),
        # a serving batch, trees of moderate size, 8 heads a rank
        dict(name="tree_batch", op="tree", batch=32, tokens=24, heads=8, mean=4096, spread=0.5, page=64, window=0, sinks=0),
        # the largest trees in use, twice the heads, odd pages
        dict(name="tree_wide", op="tree", batch=8, tokens=64, heads=16, mean=8000, spread=0.3, page=48, window=0, sinks=0),
        # a chain of drafts of few, long requests: window and first tokens at odd places
        dict(name="window_chain", op="window", batch=4, tokens=5, heads=8, mean=3000, spread=0.3, page=48, window=1000, sinks=33),
        # a batch of long answers on a bounded window
        dict(name="window_step", op="window", batch=64, tokens=1, heads=16, mean=20000, spread=0.5, page=64, window=4096, sinks=4),
        # ragged prompts
        dict(name="prompt_ragged", op="prompt", batch=6, heads=32, mean=1500, spread=0.9, past=0, window=500, sinks=17),
        # one long prompt
        dict(name="prompt_long", op="prompt", batch=1, heads=16, mean=16384, spread=0.0, past=0, window=1024, sinks=4),
        # every step of a batch adds its weights
        dict(name="weights_step", op="weights", batch=64, tokens=1, heads=16, mean=8000, spread=0.5, page=64),
        # a prompt's last tokens tell which of its keys matter
        dict(name="weights_prompt", op="weights", batch=2, tokens=32, heads=32, mean=16001, spread=0.2, page=64),
        # requests a little over their budget, some of them still under it
        dict(name="evict_step", op="evict", batch=64, mean=4200, spread=0.05, budget=4096, sinks=4, recent=512, page=64),
        # long prompts cut down to a small cache
        dict(name="evict_prompt", op="evict", batch=4, mean=32768, spread=0.3, budget=2048, sinks=16, recent=64, page=16),
        # the accepted path of every request's tree
        dict(name="commit_batch", op="commit", batch=64, tokens=24, accepted=5, mean=4096, spread=0.5, page=64),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "window", "prompt", "weights", "evict", "commit"))
    of = [work(c) for c in listed() if c["op"] == op]
    limit = {k: max(w[k] for w in of) for k in ("bytes", "flops")}
    heads = lambda: rng.choice((1, 4, 5, 8, 10, 16, 32, 64, 128))
    common = lambda most, longest: dict(batch=_spread(rng, 1, most), mean=_spread(rng, 16, longest),
                                        spread=rng.choice((0.0, 0.3, 0.9)), page=rng.choice((1, 16, 48, 64, 128)))
    while True:
        if op == "tree":
            tokens = _spread(rng, 1, 256)
            window = rng.choice((0, 0, 0, tokens + _spread(rng, 1, 4096)))
            case = dict(common(64, 65536), op=op, tokens=tokens, heads=heads(), window=window,
                        sinks=rng.choice((0, 1, 4, 70)) if window else 0)
        elif op == "window":
            case = dict(common(128, 65536), op=op, tokens=rng.choice((1, 1, 1, 2, 3, 5)), heads=heads(),
                        window=_spread(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 33, 100)))
        elif op == "prompt":
            case = dict(op=op, batch=_spread(rng, 1, 16), heads=rng.choice((1, 5, 8, 20, 32)), mean=_spread(rng, 16, 16384),
                        spread=rng.choice((0.0, 0.3, 0.9)), past=rng.choice((0, 0, 100, 4000)), window=_spread(rng, 64, 8192),
                        sinks=rng.choice((0, 1, 4, 17, 100)))
        elif op == "weights":
            case = dict(common(128, 65536), op=op, tokens=rng.choice((1, 1, 2, 5, 16, 64)), heads=heads())
        elif op == "evict":
            case = dict(common(128, 65536), op=op)
            case["sinks"], case["recent"] = rng.choice((0, 1, 4, 16)), rng.choice((0, 1, 32, 100))
            case["budget"] = case["sinks"] + case["recent"] + max(1, int(case["mean"] * rng.uniform(0.05, 0.95)))
        else:
            tokens = _spread(rng, 1, 256)
            case = dict(common(128, 16384), op=op, tokens=tokens, accepted=rng.randint(1, min(tokens, 12)))
        cost = work(case)
        if cost["bytes"] <= limit["bytes"] and cost["flops"] <= limit["flops"]:
            return case


def _lengths(case):
    """The sequences' lengths: a rule of the case alone, uniform over mean * (1 -+ spread)."""
    rng = random.Random(case["batch"] * 7919 + case["mean"])
    low, high = case["mean"] * (1 - case["spread"]), case["mean"] * (1 + case["spread"])
    least = case.get("tokens", 1)
    return [max(least, int(round(rng.uniform(low, high)))) for _ in range(case["batch"])]


def _seen(last, window, sinks):
    """Keys that a token at position `last` sees: the last `window` up to its own, and the first `sinks`."""
    return min(last + 1, window + min(sinks, max(0, last + 1 - window))) if window else last + 1


def work(case):
    op, lens = case["op"], _lengths(case)
    if op in ("tree", "window", "weights"):
        heads, t = case["heads"], case["tokens"]
        rows = len(lens) * t * heads
        window, sinks = case.get("window", 0), case.get("sinks", 0)
        read = sum(min(n, window + t - 1 + min(sinks, max(0, n - t + 1 - window))) if window else n for n in lens)
        tables = -(-read // case["page"]) * 4 + len(lens) * 4
        # a tree's nodes see some few of the others: counted as a chain whose nodes see the whole context
        # and half of the drafts
        pairs = sum(sum(_seen(n - t + j, window, sinks) for j in range(t)) for n in lens)
        if op == "weights":
            return {"bytes": read * (DIM * 2 + 8) + rows * (DIM * 2 + 4) + tables, "flops": heads * pairs * 2 * DIM}
        masks = len(lens) * t * (-(-t // 32) * 4 + 4) if op == "tree" else 0
        return {"bytes": read * DIM * 2 + rows * (DIM * 2 + LATENT * 2 + 4) + tables + masks,
                "flops": heads * pairs * 2 * (DIM + LATENT)}
    if op == "prompt":
        heads, past = case["heads"], case["past"]
        nq = sum(lens)
        # keys before the first query's window are read only where they are among the first
        nk = sum(min(n + past, n + case["window"] - 1 + case["sinks"]) for n in lens)
        pairs = sum(sum(_seen(past + x, case["window"], case["sinks"]) for x in range(n)) for n in lens)
        return {"bytes": nq * heads * ((HEAD + ROT) * 2 + HEAD * 2 + 4) + nk * (heads * HEAD * 4 + ROT * 2),
                "flops": heads * pairs * 2 * (HEAD + ROT + HEAD)}
    if op == "evict":
        # nearly all rows behind the first dropped one move
        moved = sum(case["budget"] - case["sinks"] for n in lens if n > case["budget"])
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": sum(lens) * 4 + kept * 12 + moved * DIM * 4, "flops": sum(lens) * 2}
    moved = len(lens) * case["accepted"]
    return {"bytes": moved * (DIM * 4 + 4) + len(lens) * 12, "flops": moved}


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    state = _INPUTS[case["op"]](case, g)
    state["op"] = case["op"]
    return state


def _paged(case, g):
    """A cache of random rows, its pages dealt to the requests in random order."""
    lens, page = torch.tensor(_lengths(case), device=DEV), case["page"]
    counts = (lens + page - 1) // page
    most, total = -(-max(_lengths(case)) // page), int(counts.sum())
    order = torch.randperm(total + 2, generator=g, device=DEV)
    column = torch.arange(most, device=DEV)
    number = (counts.cumsum(0) - counts)[:, None] + column
    table = torch.where(column < counts[:, None], order[number.clamp_max(total + 1)], 0).to(torch.int32)
    return dict(cache=_normal(g, total + 2, page, DIM), table=table, lens=lens.to(torch.int32), host_lens=_lengths(case))


def _queries(case, g):
    rows = case["batch"] * case["tokens"]
    return dict(q=_normal(g, rows, case["heads"], DIM), tokens=case["tokens"], workspace=None,
                out=torch.empty(rows, case["heads"], LATENT, device=DEV, dtype=torch.bfloat16),
                lse=torch.empty(rows, case["heads"], device=DEV, dtype=torch.float32))


def _tree_inputs(case, g):
    b, t = case["batch"], case["tokens"]
    # a token's parent is any earlier one, or the context
    parents = (torch.rand(b, t, generator=g, device=DEV) * torch.arange(1, t + 1, device=DEV)).long() - 1
    above = torch.eye(t, device=DEV) + torch.nn.functional.one_hot(parents + 1, t + 1)[:, :, 1:].float()
    for _ in range(t.bit_length()):                          # paths of 2, 4, 8 ... steps
        above = (above @ above).clamp_max(1)
    above = above > 0.5
    words = -(-t // 32)
    bit = torch.nn.functional.pad(above, (0, words * 32 - t)).view(b, t, words, 32).long() << torch.arange(32, device=DEV)
    mask = bit.sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return dict(_paged(case, g), **_queries(case, g), parents=parents.to(torch.int32), mask=mask,
                depth=(above.sum(-1) - 1).to(torch.int32), window=case["window"], sinks=case["sinks"])


def _window_inputs(case, g):
    return dict(_paged(case, g), **_queries(case, g), window=case["window"], sinks=case["sinks"])


def _prompt_inputs(case, g):
    lq = _lengths(case)
    lk = [n + case["past"] for n in lq]
    starts = lambda lens: torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV)
    heads, nq, nk = case["heads"], sum(lq), sum(lk)
    kv = _normal(g, nk, heads, 2 * HEAD)                     # one projection gives keys and values
    return dict(q=_normal(g, nq, heads, HEAD + ROT), k=kv[:, :, :HEAD], v=kv[:, :, HEAD:], k_rot=_normal(g, nk, ROT),
                cu_q=starts(lq), cu_k=starts(lk), host_q=lq, host_k=lk, past=case["past"], window=case["window"],
                sinks=case["sinks"], out=torch.empty(nq, heads, HEAD, device=DEV, dtype=torch.bfloat16),
                lse=torch.empty(nq, heads, device=DEV, dtype=torch.float32), workspace=None)


def _weights_inputs(case, g):
    state = dict(_paged(case, g), **_queries(case, g))
    # the attention's log sums of these queries, as its kernel leaves them, and what earlier steps added up to
    state["lse"].copy_(torch.cat([_softmax_of(state, i) for i in range(case["batch"])]))
    longest = max(state["host_lens"])
    state["weights"] = torch.rand(case["batch"], longest, generator=g, device=DEV) * case["heads"]
    return state


def _softmax_of(s, i):
    """The log sums of one request's rows, every one of which sees the keys up to its own."""
    t, n, page = s["tokens"], s["host_lens"][i], s["cache"].shape[1]
    keys = s["cache"][s["table"][i, :-(-n // page)]].view(-1, DIM)[:n].float()
    score = s["q"][i * t:(i + 1) * t].flatten(0, 1).float() @ keys.T.contiguous() * SCALE
    last = torch.arange(n - t, n, device=DEV).repeat_interleave(s["q"].shape[1])
    return score.masked_fill(torch.arange(n, device=DEV) > last[:, None], -math.inf).logsumexp(-1).view(t, -1)


def _evict_inputs(case, g):
    state = _paged(case, g)
    # sums of softmax weights: a few keys hold most of them
    state["weights"] = torch.exp(2 * torch.randn(case["batch"], max(state["host_lens"]), generator=g, device=DEV))
    return dict(state, budget=case["budget"], sinks=case["sinks"], recent=case["recent"])


def _commit_inputs(case, g):
    b, t, m = case["batch"], case["tokens"], case["accepted"]
    counts = torch.randint(1, m + 1, (b,), generator=g, device=DEV)
    chosen = torch.rand(b, t, generator=g, device=DEV).argsort(1)[:, :m]
    place = torch.arange(m, device=DEV)
    kept = chosen.masked_fill(place >= counts[:, None], t).sort(1).values
    kept = kept.masked_fill(place >= counts[:, None], -1)    # a path's nodes rise
    return dict(_paged(case, g), kept=kept.to(torch.int32), counts=counts.to(torch.int32), tokens=t)


_INPUTS = {"tree": _tree_inputs, "window": _window_inputs, "prompt": _prompt_inputs, "weights": _weights_inputs,
           "evict": _evict_inputs, "commit": _commit_inputs}


# ---------------------------------------------------------------------------- one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _workspace(s):
    """Kept by the program between its calls."""
    import decode_skinny_addmm_amd as sk
    if s["workspace"] is None:
        s["workspace"] = sk.latent_decode_workspace(s["lens"].shape[0], s["tokens"], s["q"].shape[1], LATENT, DEV)
    return s["workspace"]


def _tree_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_tree_decode(s["q"], s["cache"], s["table"], s["lens"], s["mask"], SCALE, window=s["window"],
                          sinks=s["sinks"], depth=s["depth"], rope_dim=ROT, out=s["out"], lse=s["lse"],
                          workspace=_workspace(s))
    return s["out"], s["lse"]


def _window_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_window_decode(s["q"], s["cache"], s["table"], s["lens"], SCALE, s["window"], sinks=s["sinks"],
                            tokens=s["tokens"], rope_dim=ROT, out=s["out"], lse=s["lse"], workspace=_workspace(s))
    return s["out"], s["lse"]


def _prompt_own(s):
    import decode_skinny_addmm_amd as sk
    if s["workspace"] is None:
        s["workspace"] = sk.latent_window_prefill_workspace(s["q"].shape[0], s["k"].shape[0], s["cu_q"].shape[0] - 1,
                                                            s["q"].shape[1], s["window"], s["sinks"], DEV)
    sk.latent_window_prefill(s["q"], s["k"], s["v"], s["k_rot"], s["cu_q"], s["cu_k"], SCALE, s["window"],
                             sinks=s["sinks"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _weights_own(s):
    import decode_skinny_addmm_amd as sk
    sk.latent_key_weights(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["weights"], SCALE, tokens=s["tokens"],
                          rope_dim=ROT)
    return s["weights"]


def _evict_own(s):
    import decode_skinny_addmm_amd as sk
    kept, counts = sk.latent_select(s["weights"], s["lens"], s["budget"], sinks=s["sinks"], recent=s["recent"])
    lens, weights = sk.latent_keep(s["cache"], s["table"], s["lens"], kept, counts, weights=s["weights"])
    return s["cache"], kept, lens, weights


def _commit_own(s):
    import decode_skinny_addmm_amd as sk
    lens, _ = sk.latent_keep(s["cache"], s["table"], s["lens"], s["kept"], s["counts"], tokens=s["tokens"])
    return s["cache"], lens


def _slots(s, key):
    """Where keys [batch, n] of the requests lie among all rows of the cache."""
    page = s["cache"].shape[1]
    return s["table"].long().gather(1, (key // page).clamp(0, s["table"].shape[1] - 1)) * page + key % page


def _softmax_sum(score, seen, value):
    """softmax over the seen places of a row times value, and the log of its sum; no place seen: 0, -inf."""
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(score.dtype).min)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    return p @ value / total.clamp_min(torch.finfo(score.dtype).tiny), (top + total.log()).squeeze(-1)


def _attend(s, key, seen):
    """Rows [batch, tokens] attend to keys [batch, n] of their request where seen [batch, tokens, n]."""
    b, heads = s["lens"].shape[0], s["q"].shape[1]
    keys = s["cache"].view(-1, DIM)[_slots(s, key)].float()
    q = s["q"].float().view(b, -1, DIM)
    out, lse = _softmax_sum(q @ keys.transpose(1, 2).contiguous() * SCALE, seen.repeat_interleave(heads, 1),
                            keys[:, :, :LATENT].contiguous())
    s["out"].copy_(out.view(s["out"].shape))
    s["lse"].copy_(lse.view(s["lse"].shape))
    return s["out"], s["lse"]


def _tree_plain(s):
    t = s["tokens"]
    key = torch.arange(max(s["host_lens"]), device=DEV)
    base = (s["lens"].long() - t)[:, None]
    seen = (key < base)[:, None].expand(-1, t, -1)
    if s["window"]:
        far = key <= (base + s["depth"] - s["window"])[:, :, None]
        seen = seen & ~(far & (key >= s["sinks"]))
    node = key - base
    j = node.clamp(0, t - 1)
    word = s["mask"].gather(2, (j // 32)[:, None].expand(-1, t, -1))
    above = ((word >> (j % 32)[:, None]) & 1).bool() & ((node >= 0) & (node < t))[:, None]
    return _attend(s, key.expand(base.shape[0], -1), seen | above)


def _window_plain(s):
    t, window = s["tokens"], min(s["window"], max(s["host_lens"]))
    first = torch.arange(s["sinks"], device=DEV)
    n = s["lens"].long()[:, None]
    near = n - t - window + 1 + torch.arange(window + t - 1, device=DEV)
    last = (n - t + torch.arange(t, device=DEV))[:, :, None]
    begin = last - s["window"]                               # the last key before a row's window
    seen = torch.cat(((first <= begin).expand(n.shape[0], t, -1),
                      (near[:, None] >= 0) & (near[:, None] <= last) & (near[:, None] > begin)), dim=-1)
    return _attend(s, torch.cat((first.expand(n.shape[0], -1), near), dim=1).clamp_min(0), seen)


def _prompt_plain(s):
    # blocks of queries, each with its window's keys and the first ones
    window = min(s["window"], max(s["host_k"]))
    block = max(64, min(512, window))
    lq, past = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), s["past"]
    x = torch.arange(-(-max(s["host_q"]) // block) * block, device=DEV).view(-1, block)
    first = torch.arange(s["sinks"], device=DEV)
    near = past + x[:, :1] - window + 1 + torch.arange(window + block - 1, device=DEV)
    key = torch.cat((first.expand(x.shape[0], -1), near), dim=1)                     # [blocks, keys]
    last = (past + x)[:, :, None]
    seen = torch.cat(((first <= last - s["window"]),
                      (near[:, None] >= 0) & (near[:, None] <= last) & (near[:, None] > last - s["window"])), dim=-1)
    rows = (s["cu_q"][:-1].long()[:, None, None] + x).clamp_max(s["q"].shape[0] - 1)  # [batch, blocks, block]
    keys = (s["cu_k"][:-1].long()[:, None, None] + key.clamp_min(0)).clamp_max(s["k"].shape[0] - 1)
    heads_first = lambda y: y.float().movedim(3, 2)
    k_rot = s["k_rot"][keys].float()[:, :, None].expand(-1, -1, s["k"].shape[1], -1, -1)
    k = torch.cat((heads_first(s["k"][keys]), k_rot), dim=-1)
    score = heads_first(s["q"][rows]) @ k.transpose(-1, -2).contiguous() * SCALE
    out, lse = _softmax_sum(score, seen[None, :, None], heads_first(s["v"][keys]).contiguous())
    there = (x < lq[:, None, None]).flatten()
    s["out"][rows.flatten()[there]] = out.movedim(2, 3).flatten(0, 2)[there].to(torch.bfloat16)
    s["lse"][rows.flatten()[there]] = lse.movedim(2, 3).flatten(0, 2)[there]
    return s["out"], s["lse"]


def _weights_plain(s):
    b, t, heads = s["lens"].shape[0], s["tokens"], s["q"].shape[1]
    key = torch.arange(s["weights"].shape[1], device=DEV)
    keys = s["cache"].view(-1, DIM)[_slots(s, key.expand(b, -1))].float()
    score = s["q"].float().view(b, -1, DIM) @ keys.transpose(1, 2).contiguous() * SCALE
    p = torch.exp(score - s["lse"].view(b, -1, 1))
    seen = key <= (s["lens"].long()[:, None] - t + torch.arange(t, device=DEV))[:, :, None]
    s["weights"] += p.masked_fill(~seen.repeat_interleave(heads, 1), 0).sum(1)
    return s["weights"]


def _moved(s, kept, counts, start):
    """Rows kept[i, j] of request i go to start[i] + j; its new lengths."""
    j = torch.arange(kept.shape[1], device=DEV)
    valid = j < counts[:, None]
    there, here = _slots(s, start[:, None] + j)[valid], _slots(s, kept.clamp_min(0))[valid]
    rows = s["cache"].view(-1, DIM)
    rows[there] = rows[here]
    return (start + counts).to(torch.int32)


def _evict_plain(s):
    n = s["lens"].long()
    key = torch.arange(s["weights"].shape[1], device=DEV)
    always = (key < s["sinks"]) | (key >= n[:, None] - s["recent"])
    rank = torch.where(always, math.inf, s["weights"]).masked_fill(key >= n[:, None], -math.inf)
    order = rank.sort(dim=1, descending=True, stable=True).indices[:, :s["budget"]]
    counts = n.clamp_max(s["budget"])
    j = torch.arange(order.shape[1], device=DEV)
    chosen = order.masked_fill(j >= counts[:, None], 1 << 40).sort(1).values
    kept = torch.full((n.shape[0], s["budget"]), -1, dtype=torch.int64, device=DEV)
    kept[:, :order.shape[1]] = chosen.masked_fill(j >= counts[:, None], -1)
    lens = _moved(s, kept, counts, torch.zeros_like(n))
    weights = torch.zeros_like(s["weights"])
    weights[:, :order.shape[1]] = s["weights"].gather(1, chosen.clamp_max(key.shape[0] - 1)).masked_fill(j >= counts[:, None], 0)
    return s["cache"], kept.to(torch.int32), lens, weights


def _commit_plain(s):
    base = s["lens"].long() - s["tokens"]
    return s["cache"], _moved(s, base[:, None] + s["kept"], s["counts"].long(), base)


_OWN = {"tree": _tree_own, "window": _window_own, "prompt": _prompt_own, "weights": _weights_own, "evict": _evict_own,
        "commit": _commit_own}
_PLAIN = {"tree": _tree_plain, "window": _window_plain, "prompt": _prompt_plain, "weights": _weights_plain,
          "evict": _evict_plain, "commit": _commit_plain}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _keys_of(s, i, n):
    place = torch.arange(n, device=DEV)
    page = s["cache"].shape[1]
    return s["cache"].flatten(0, 1)[s["table"][i].long()[place // page] * page + place % page].double()


def _paths(parents):
    """Each node with the nodes above it, followed parent by parent."""
    paths = []
    for j, parent in enumerate(parents):
        paths.append(([] if parent < 0 else paths[parent]) + [j])
    return paths


def _one_token(q, keys, which):
    """softmax(scale q . keys) of the keys in `which` times their latents, and the log of its sum."""
    keys = keys[which]
    score = q.double().mul(SCALE) @ keys.T.contiguous()
    lse = score.logsumexp(-1)
    return (score - lse[:, None]).exp() @ keys[:, :LATENT].contiguous(), lse


def _decode_exact(s, which):
    """Token by token over the keys that which(i, j, n) names."""
    t, answers = s["tokens"], []
    for i, n in enumerate(s["host_lens"]):
        keys = _keys_of(s, i, n)
        answers += [_one_token(s["q"][i * t + j], keys, which(i, j, n)) for j in range(t)]
    return torch.stack([a for a, _ in answers]), torch.stack([b for _, b in answers])


def _tree_exact(s):
    paths = [_paths(p) for p in s["parents"].tolist()]
    t = s["tokens"]

    def which(i, j, n):
        path = paths[i][j]
        begin = max(0, n - t + len(path) - s["window"]) if s["window"] else 0
        context = list(range(min(s["sinks"], begin))) + list(range(begin, n - t))
        return torch.tensor(context + [n - t + d for d in path], device=DEV)
    return _decode_exact(s, which)


def _window_exact(s):
    def which(i, j, n):
        end = n - s["tokens"] + j + 1
        begin = max(0, end - s["window"])
        return torch.tensor(list(range(min(s["sinks"], begin))) + list(range(begin, end)), device=DEV)
    return _decode_exact(s, which)


def _prompt_exact(s):
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for lq, lk in zip(s["host_q"], s["host_k"]):
        back = torch.arange(lk - lq, lk, device=DEV)[:, None] - torch.arange(lk, device=DEV)[None]
        hidden = (back < 0) | ((back >= s["window"]) & (torch.arange(lk, device=DEV) >= s["sinks"]))
        shared = s["k_rot"][k0:k0 + lk].double().T.contiguous()
        for h in range(s["q"].shape[1]):
            q = s["q"][q0:q0 + lq, h].double()
            score = q[:, :HEAD] @ s["k"][k0:k0 + lk, h].double().T.contiguous() + q[:, HEAD:] @ shared
            score *= SCALE
            score[hidden] = -math.inf
            lse[q0:q0 + lq, h] = score.logsumexp(-1)
            score -= lse[q0:q0 + lq, h, None]
            out[q0:q0 + lq, h] = score.exp_() @ s["v"][k0:k0 + lk, h].double().contiguous()
        q0, k0 = q0 + lq, k0 + lk
    return out, lse


def _weights_exact(s):
    t, weights = s["tokens"], s["weights"].double()
    for i, n in enumerate(s["host_lens"]):
        keys = _keys_of(s, i, n)
        for j in range(t):
            end = n - t + j + 1
            score = s["q"][i * t + j].double().mul(SCALE) @ keys[:end].T.contiguous()
            weights[i, :end] += (score - s["lse"][i * t + j].double()[:, None]).exp().sum(0)
    return weights


def _rows_to(s, i, rows, start):
    """Request i's rows to the places from start on: read all, then written."""
    page = s["cache"].shape[1]
    flat, place = s["cache"].flatten(0, 1), torch.arange(start, start + len(rows), device=DEV)
    rows = torch.as_tensor(rows, device=DEV)
    slot = lambda k: s["table"][i].long()[k // page] * page + k % page
    flat[slot(place)] = flat[slot(rows)].clone()


def _evict_exact(s):
    kept = torch.full((len(s["host_lens"]), s["budget"]), -1, dtype=torch.int32, device=DEV)
    weights, lens = torch.zeros_like(s["weights"], dtype=torch.float64), []
    for i, n in enumerate(s["host_lens"]):
        w = s["weights"][i].tolist()
        rows = list(range(n))
        if n > s["budget"]:
            fixed = list(range(s["sinks"])) + list(range(n - s["recent"], n))
            rows = sorted(range(s["sinks"], n - s["recent"]), key=lambda k: (-w[k], k))[:s["budget"] - len(fixed)]
            rows = sorted(rows + fixed)
        lens.append(len(rows))
        kept[i, :len(rows)] = torch.tensor(rows, dtype=torch.int32, device=DEV)
        weights[i, :len(rows)] = s["weights"][i, rows].double()
        _rows_to(s, i, rows, 0)
    return s["cache"].double(), kept, torch.tensor(lens, dtype=torch.int32, device=DEV), weights


def _commit_exact(s):
    lens = []
    for i, (n, count) in enumerate(zip(s["host_lens"], s["counts"].tolist())):
        base = n - s["tokens"]
        _rows_to(s, i, [base + d for d in s["kept"][i, :count].tolist()], base)
        lens.append(base + count)
    return s["cache"].double(), torch.tensor(lens, dtype=torch.int32, device=DEV)


_EXACT = {"tree": _tree_exact, "window": _window_exact, "prompt": _prompt_exact, "weights": _weights_exact,
          "evict": _evict_exact, "commit": _commit_exact}
