"""Latent attention at the limits of what its operands may hold, on the GPU: rows behind a request's end, few short
requests, weights with fewer columns than keys, lengths and page ids that are clamped, strided operands."""
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
