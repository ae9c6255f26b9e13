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
