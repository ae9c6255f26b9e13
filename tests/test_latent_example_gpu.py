"""The latent attention layer of examples/: prompts and steps over one cache give the same outputs.

A sequence attended to at once (expanded keys and values) and the same one in pieces (a prompt, then
steps of new tokens with absorbed queries) differ by roundings alone. The projections are made in 64
bits here, so that a token's are the same whatever goes with it. With u = 2^-8, the most that a
rounding to bf16 moves a number by (relative), and |.| the 2-norm:
  * a score's query or key is rounded once more on either side: the absorbed query (norm A, against
    latents of norm Z) and the expanded key (norm K, against a query of norm Q), so the two scores are
    at most d = scale * u * (A Z + Q K) apart; fp32 sums of at most 576 terms add less than 2^-14 of
    that. The softmax weights then differ by a factor within exp(+-2d).
  * the weights are rounded to bf16 for their product on both sides (2u of sum p|v|, v a value), and so
    are the expanded values (u) and both outputs (u each); the absorbed sum of latents (u) goes through
    w_v, which lengthens it by its largest singular value at most.
With V the largest norm of a head's value row and B = that singular value times Z, an output differs
by at most (exp(2d) - 1) V + u (5 V + B), taken up by a factor (1 + 2^-6) for second orders.
"""
import importlib.util
import math
import os

import pytest
import torch

import latent_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("prompts,tokens,steps", [([1, 70, 33], 1, 3), ([130, 5], 4, 2)])
def test_pieces_agree_with_the_whole(example, monkeypatch, prompts, tokens, steps):
    monkeypatch.setattr(torch.nn.functional, "linear", lambda x, w: (x.double() @ w.double().t()).to(x.dtype))
    torch.manual_seed(3)
    hidden, heads = 512, 6
    layer = example.LatentLayer(hidden, heads)
    total = [n + tokens * steps for n in prompts]
    x = [torch.randn(n, hidden, device="cuda").to(torch.bfloat16) for n in total]
    whole = layer.attend_prompts(torch.cat(x), example.PagedCache(len(total), max(total)), total).split(total)

    cache = example.PagedCache(len(total), max(total), page=16)
    pieces = [[o] for o in layer.attend_prompts(torch.cat([a[:n] for a, n in zip(x, prompts)]), cache, prompts).split(prompts)]
    for i in range(steps):
        lens = torch.tensor([n + (i + 1) * tokens for n in prompts], dtype=torch.int32, device="cuda")
        new = torch.cat([a[n + i * tokens:n + (i + 1) * tokens] for a, n in zip(x, prompts)])
        out = layer.attend_step(new, cache, lens, tokens)
        for o, part in zip(pieces, out.split(tokens)):
            o.append(part)

    w_k, w_v = layer.w_k.double().cpu(), layer.w_v.double().cpu()
    for i, n in enumerate(total):
        kv = torch.nn.functional.linear(x[i], layer.w_kv)[:, :example.LATENT].double().cpu()
        z = kv * torch.rsqrt(kv.square().mean(-1, keepdim=True) + 1e-6) * (1 + U)
        q = torch.nn.functional.linear(x[i], layer.w_q).view(n, heads, -1)[:, :, :example.HEAD].double().cpu()
        key = torch.matmul(z, w_k.transpose(1, 2).contiguous())          # heads, n, 128
        value = torch.matmul(z, w_v.transpose(1, 2).contiguous())
        absorbed = torch.matmul(q.transpose(0, 1).contiguous(), w_k)     # heads, n, 512
        norm = lambda t: t.norm(dim=-1).max().item()
        d = layer.scale * U * (norm(absorbed) * norm(z) + norm(q) * norm(key)) * (1 + 2.0 ** -6)
        top = torch.linalg.matrix_norm(w_v, 2).max().item()
        bound = (math.expm1(2 * d) * norm(value) + U * (5 * norm(value) + top * norm(z))) * (1 + 2.0 ** -6)
        got = torch.cat(pieces[i]).double().cpu()
        assert got.shape == whole[i].shape and bool(torch.isfinite(got).all())
        off = (got - whole[i].double().cpu()).norm(dim=-1).max().item()
        size = whole[i].double().cpu().norm(dim=-1).max().item()
        assert off <= bound, "request %d: off by %g, bound %g (outputs up to %g)" % (i, off, bound, size)
        assert bound < 0.5 * norm(value), "a bound that would pass other values' outputs"


def test_command(example, capsys):
    y = example.main(["--prompts", "40", "3", "--steps", "2", "--heads", "4", "--hidden", "512"])
    assert y.shape == (2, 512) and bool(torch.isfinite(y).all())
    assert "step 1, lengths [42, 5]" in capsys.readouterr().out


@pytest.mark.parametrize("prompts,tokens,steps", [([130, 5, 70, 33], 1, 2), ([70, 1, 130], 4, 2)])
def test_steps_against_64_bits(example, monkeypatch, prompts, tokens, steps):
    """A step of the layer stage by stage: the rows that the cache holds, the queries that it attends
    with, the sum over the latents of exactly these, and their way through w_v. Each stage is off by its
    own roundings alone (half a bf16 step, and 2^-24 relative for each term of an fp32 sum), so the
    bounds are far below the outputs' size."""
    monkeypatch.setattr(torch.nn.functional, "linear", lambda x, w: (x.double() @ w.double().t()).to(x.dtype))
    torch.manual_seed(4)
    hidden, heads = 512, 6
    layer = example.LatentLayer(hidden, heads)
    total = [n + tokens * steps for n in prompts]
    x = [torch.randn(n, hidden, device="cuda").to(torch.bfloat16) for n in total]
    cache = example.PagedCache(len(total), max(total), page=16)
    layer.attend_prompts(torch.cat([a[:n] for a, n in zip(x, prompts)]), cache, prompts)
    seen = []
    real = example.sk.latent_decode

    def watched(q, *args, **named):
        answer = real(q, *args, **named)
        seen.append((q, answer[0], answer[1]))
        return answer

    monkeypatch.setattr(example.sk, "latent_decode", watched, raising=False)
    w_k, w_v = layer.w_k.double().cpu(), layer.w_v.double().cpu()
    for i in range(steps):
        now = [n + (i + 1) * tokens for n in prompts]
        new = torch.cat([a[n - tokens:n] for a, n in zip(x, now)])
        out = layer.attend_step(new, cache, torch.tensor(now, dtype=torch.int32, device="cuda"), tokens).cpu().double()
        q, z, lse = (t.cpu() for t in seen.pop())
        assert not seen and out.shape == (len(new), heads, example.HEAD)
        positions = torch.cat([torch.arange(n - tokens, n) for n in now])
        made = torch.nn.functional.linear(new, layer.w_q).view(-1, heads, example.HEAD + example.ROT).cpu()
        want, m = ref.turned(made[:, :, example.HEAD:], positions, layer.inv_freq, False)
        assert bool(((q[:, :, example.LATENT:].double() - want).abs() <= U * want.abs() + (1 + U) * m * 2.0 ** -21).all())
        part = made[:, :, :example.HEAD].double().transpose(0, 1).contiguous()
        want = torch.matmul(part, w_k).transpose(0, 1)
        terms = torch.matmul(part.abs(), w_k.abs()).transpose(0, 1)
        off = (q[:, :, :example.LATENT].double() - want).abs()
        assert bool((off <= U * want.abs() + (1 + U) * example.HEAD * 2.0 ** -24 * terms).all())
        rows, table = cache.rows.cpu().view(-1, example.DIM), cache.table.cpu().long()
        for b, n in enumerate(now):
            place = torch.arange(n)
            held = rows[table[b, place // cache.page] * cache.page + place % cache.page]
            kv = torch.nn.functional.linear(x[b][:n], layer.w_kv)
            want, bound = ref.append(kv, place, layer.inv_freq, layer.norm, 1e-6, False)
            assert bool(((held.double() - want).abs() <= bound).all()), "rows of request %d" % b
            for j in range(tokens):
                t, sees = b * tokens + j, n - tokens + j + 1
                keys = held[:sees].double()
                answer = ref.attend(q[t].double(), keys, keys[:, :example.LATENT], layer.scale,
                                    torch.ones(heads, sees, dtype=torch.bool))
                ref.check(z[t], lse[t], answer, sees, "request %d, token %d" % (b, j))
        latents = z.double().transpose(0, 1).contiguous()
        to_heads = w_v.transpose(1, 2).contiguous()
        want = torch.matmul(latents, to_heads).transpose(0, 1)
        terms = torch.matmul(latents.abs(), to_heads.abs()).transpose(0, 1)
        assert bool(((out - want).abs() <= U * want.abs() + (1 + U) * example.LATENT * 2.0 ** -24 * terms).all())
        assert bool((want.norm(dim=-1) > 0.5).all())          # nothing above is satisfied by zeros
