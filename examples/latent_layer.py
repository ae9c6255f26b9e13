"""A latent attention layer that serves requests: ragged prompts first, then tokens, over one paged
cache, with the layer's residual projection behind it.

    python examples/latent_layer.py --prompts 300 17 1024 --steps 8

Keys and values of all heads come from one cached row a token (512 latents and 64 rotated numbers).
A prompt expands its rows to each head's keys and values once (latent_prefill); a step of a few new
tokens leaves them as they are and moves the expansion to its queries and outputs (latent_decode).
Weights and inputs are synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import decode_skinny_addmm_amd as sk  # noqa: E402

LATENT, ROT, HEAD = 512, 64, 128
DIM = LATENT + ROT


class PagedCache:
    """Rows of all requests in one pool of pages, and each request's pages."""

    def __init__(self, requests: int, max_len: int, page: int = 64, device="cuda"):
        per = -(-max_len // page)
        self.page = page
        self.rows = torch.zeros(requests * per, page, DIM, dtype=torch.bfloat16, device=device)
        self.table = torch.randperm(requests * per, device=device).to(torch.int32).view(requests, per)

    def slots(self, request, position):
        """Where a request's position lives: both int64 tensors."""
        return self.table[request, position // self.page].long() * self.page + position % self.page


class LatentLayer:
    def __init__(self, hidden: int = 7168, heads: int = 28, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g, device=device) * fan ** -0.5).to(torch.bfloat16)

        self.heads = heads
        self.scale = (HEAD + ROT) ** -0.5
        self.w_q = weight(heads * (HEAD + ROT), hidden, fan=hidden)
        self.w_kv = weight(DIM, hidden, fan=hidden)
        self.w_k = weight(heads, HEAD, LATENT, fan=LATENT)       # a head's keys from latents: k = w_k z
        self.w_v = weight(heads, HEAD, LATENT, fan=LATENT)
        # both expansions as one product for prompts, and the values' laid out for steps
        self.w_up = torch.cat((self.w_k, self.w_v), dim=1).view(heads * 2 * HEAD, LATENT).contiguous()
        self.w_v_t = self.w_v.transpose(1, 2).contiguous()
        self.w_o = weight(hidden, heads * HEAD, fan=heads * HEAD)
        self.norm = torch.ones(LATENT, dtype=torch.bfloat16, device=device)
        self.inv_freq = 10000.0 ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device=device) / ROT)

    def _project(self, x, cache, slots, positions):
        """The tokens' queries [n, heads, 192], turned in place, and their rows into the cache."""
        q = torch.nn.functional.linear(x, self.w_q).view(-1, self.heads, HEAD + ROT)
        kv = torch.nn.functional.linear(x, self.w_kv)
        turned = q[:, :, HEAD:]
        sk.latent_append(kv, cache.rows, slots, positions, self.inv_freq, norm_weight=self.norm, q=turned, q_out=turned)
        return q

    def attend_prompts(self, x, cache, lens):
        """Heads' outputs [n, heads, 128] of whole prompts, one after the other in x [sum(lens), hidden]."""
        dev = x.device
        starts = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
        request = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(lens, device=dev),
                                          output_size=sum(lens))
        positions = torch.arange(sum(lens), device=dev) - starts.long()[request]
        slots = cache.slots(request, positions)
        q = self._project(x, cache, slots, positions)
        rows = cache.rows.view(-1, DIM)[slots]
        kv = torch.nn.functional.linear(rows[:, :LATENT], self.w_up).view(-1, self.heads, 2 * HEAD)
        return sk.latent_prefill(q, kv[:, :, :HEAD], kv[:, :, HEAD:], rows[:, LATENT:], starts, starts, self.scale)[0]

    def attend_step(self, x, cache, lens, tokens: int = 1, workspace=None):
        """The same for each request's `tokens` newest positions: x [batch * tokens, hidden], lens
        int32 [batch] on the device with the new tokens counted. workspace: the caller's
        sk.latent_decode_workspace(batch, tokens, heads), shared by steps that follow each other on one
        stream (of all layers); None: made for this step."""
        batch, dev = lens.shape[0], x.device
        request = torch.arange(batch, device=dev).repeat_interleave(tokens)
        positions = lens.long()[request] - tokens + torch.arange(tokens, device=dev).repeat(batch)
        q = self._project(x, cache, cache.slots(request, positions), positions)
        # q . (w_k z) = (w_k' q) . z: the queries carry the keys' expansion
        absorbed = torch.bmm(q[:, :, :HEAD].transpose(0, 1).contiguous(), self.w_k).transpose(0, 1)
        q = torch.cat((absorbed, q[:, :, HEAD:]), dim=-1)
        z = sk.latent_decode(q, cache.rows, cache.table, lens, self.scale, tokens=tokens, workspace=workspace)[0]
        return torch.bmm(z.transpose(0, 1).contiguous(), self.w_v_t).transpose(0, 1)

    def output(self, attended, x):
        """x + attended W', the residual projection."""
        return sk.addmm(attended.reshape(x.shape[0], -1), self.w_o, x)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--prompts", type=int, nargs="+", default=[300, 17, 1024, 513])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--tokens", type=int, default=1, help="new tokens a request and step")
    p.add_argument("--heads", type=int, default=28)
    p.add_argument("--hidden", type=int, default=7168)
    a = p.parse_args(argv)
    if min(a.prompts) < 1 or a.steps < 0 or a.tokens < 1:
        p.error("prompts and tokens must be at least 1, steps at least 0")
    torch.manual_seed(0)
    layer = LatentLayer(a.hidden, a.heads)
    cache = PagedCache(len(a.prompts), max(a.prompts) + a.steps * a.tokens)
    make = lambda n: torch.randn(n, a.hidden, device="cuda").to(torch.bfloat16)
    x = make(sum(a.prompts))
    y = layer.output(layer.attend_prompts(x, cache, a.prompts), x)
    print("prompts of %s tokens: output %s" % (a.prompts, tuple(y.shape)), flush=True)
    lens = torch.tensor(a.prompts, dtype=torch.int32, device="cuda")
    workspace = sk.latent_decode_workspace(len(a.prompts), a.tokens, a.heads)
    for i in range(a.steps):
        x = make(len(a.prompts) * a.tokens)
        lens += a.tokens
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = layer.output(layer.attend_step(x, cache, lens, a.tokens, workspace), x)
        torch.cuda.synchronize()
        print("step %d, lengths %s: %.0f us" % (i, lens.tolist(), 1e6 * (time.perf_counter() - t)), flush=True)
    return y


if __name__ == "__main__":
    main()
