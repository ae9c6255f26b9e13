"""Refusals of the latent operators over trees, windows and kept keys, on the host: the C ABI answers before
anything is launched. And the references that the GPU tests use, against each other."""
import ctypes
import os

import pytest
import torch

import masked_reference as mref
from decode_skinny_addmm_amd import _lib, ops
from test_latent_host import ENOTSUP, EALIGN, EINVAL, OK, P, decode_args, prefill_args


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libskinny.so not built")
    return _lib.lib()


def mask(**over):
    d = dict(tree=P, depth=P, tree_stride=2, depth_stride=2, window=0, sinks=0)
    d.update(over)
    return _lib.SkinnyLatentMask(**d)


def weights_args(**over):
    d = dict(q=P, cache=P, table=P, lens=P, lse=P, weights=P, q_row_stride=8 * 576, q_head_stride=576,
             cache_page_stride=576 * 16, cache_row_stride=576, table_stride=9, weights_stride=100, batch=2, tokens=2,
             heads=8, pages=20, page=16, max_pages=9, columns=100, latent=512, rope=64, scale=0.1)
    d.update(over)
    return _lib.SkinnyLatentKeyWeightsArgs(**d)


def select_args(**over):
    d = dict(weights=P, lens=P, kept=P, counts=P, weights_stride=100, batch=2, columns=100, budget=10, sinks=4, recent=6)
    d.update(over)
    return _lib.SkinnyLatentSelectArgs(**d)


def keep_args(**over):
    d = dict(cache=P, table=P, lens=P, kept=P, counts=P, new_lens=P + 64, weights=P, new_weights=P + 64, cache_page_stride=576 * 16,
             cache_row_stride=576, table_stride=9, kept_stride=5, weights_stride=100, new_weights_stride=100, batch=2,
             tokens=0, most=5, pages=20, page=16, max_pages=9, columns=100, latent=512, rope=64)
    d.update(over)
    return _lib.SkinnyLatentKeepArgs(**d)


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(window=-1)), (EINVAL, dict(sinks=-1)), (EINVAL, dict(tree_stride=-2)), (EINVAL, dict(tree_stride=1)),
    (EINVAL, dict(tree_stride=1 << 50)), (EALIGN, dict(tree=P + 2)), (EALIGN, dict(depth=P + 2)), (EINVAL, dict(window=1)),
    (EINVAL, dict(window=5, depth=None)), (EINVAL, dict(window=5, depth_stride=1)), (EINVAL, dict(window=5, depth_stride=-1)),
    (EINVAL, dict(tree=None, window=-1)), (EINVAL, dict(tree=None, window=3, sinks=-2))])
def test_masked_decode_refuses_masks(L, want, over):
    call = lambda a: L.skinny_latent_masked_decode_bf16(ctypes.byref(a), ctypes.byref(mask(**over)), None)
    assert call(decode_args()) == want


@pytest.mark.parametrize("over", [{}, dict(tree_stride=0, depth_stride=0), dict(window=2, sinks=1 << 40), dict(window=1 << 60),
                                  dict(tree=None, depth=None, window=1), dict(tree=None, sinks=3)])
def test_masked_decode_takes_masks(L, over):
    a, m = decode_args(batch=0), mask(**over)
    assert L.skinny_latent_masked_decode_bf16(ctypes.byref(a), ctypes.byref(m), None) == OK


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(scale=0.0)), (ENOTSUP, dict(latent=448)), (EALIGN, dict(q=P + 8)),
    (EINVAL, dict(out_row_stride=512)), (ENOTSUP, dict(tokens=513)), (EINVAL, dict(lens=None))])
def test_masked_decode_refuses_what_decode_does(L, want, over):
    words = (over.get("tokens", 2) + 31) // 32 * over.get("tokens", 2)
    m = mask(tree_stride=words)
    assert L.skinny_latent_masked_decode_bf16(ctypes.byref(decode_args(**over)), ctypes.byref(m), None) == want


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(tokens=0)), (EINVAL, dict(heads=-1)), (EINVAL, dict(page=0)), (EINVAL, dict(pages=0)),
    (EINVAL, dict(columns=-1)), (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=float("nan"))), (EINVAL, dict(scale=float("inf"))),
    (ENOTSUP, dict(latent=256)), (ENOTSUP, dict(rope=32)), (EINVAL, dict(q=None)), (EINVAL, dict(cache=None)),
    (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(lse=None)), (EINVAL, dict(weights=None)),
    (EALIGN, dict(q=P + 8)), (EALIGN, dict(cache=P + 2)), (EALIGN, dict(weights=P + 2)), (EALIGN, dict(lse=P + 1)),
    (EALIGN, dict(q_head_stride=580)), (EINVAL, dict(cache_row_stride=512)), (EINVAL, dict(table_stride=8)),
    (EINVAL, dict(weights_stride=99)), (ENOTSUP, dict(batch=1 << 30)), (ENOTSUP, dict(tokens=1 << 14, heads=1 << 14)),
    (ENOTSUP, dict(max_pages=1 << 28, table_stride=1 << 28, page=1 << 20)), (OK, dict(batch=0)), (OK, dict(heads=0)),
    (OK, dict(columns=0)), (OK, dict(batch=0, q=None, pages=0))])
def test_key_weights_refuses(L, want, over):
    assert L.skinny_latent_key_weights_bf16(ctypes.byref(weights_args(**over)), None) == want


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(columns=-1)), (EINVAL, dict(budget=-1, sinks=0, recent=0)), (EINVAL, dict(sinks=-1)),
    (EINVAL, dict(recent=-1)), (EINVAL, dict(sinks=5)), (EINVAL, dict(sinks=11)), (EINVAL, dict(recent=1 << 62)),
    (EINVAL, dict(weights_stride=99)), (EINVAL, dict(weights=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(kept=None)),
    (EINVAL, dict(counts=None)), (EALIGN, dict(weights=P + 2)), (EALIGN, dict(kept=P + 1)), (ENOTSUP, dict(batch=1 << 21)),
    (ENOTSUP, dict(columns=1 << 31)), (ENOTSUP, dict(budget=1 << 31)), (OK, dict(batch=0))])
def test_select_refuses(L, want, over):
    assert L.skinny_latent_select(ctypes.byref(select_args(**over)), None) == want


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(tokens=-1)), (EINVAL, dict(most=-1)), (EINVAL, dict(page=0)), (EINVAL, dict(pages=0)),
    (EINVAL, dict(columns=-1)), (ENOTSUP, dict(latent=256)), (ENOTSUP, dict(rope=0)), (EINVAL, dict(cache=None)),
    (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(kept=None)), (EINVAL, dict(counts=None)),
    (EINVAL, dict(new_lens=None)), (EINVAL, dict(new_lens=P)), (EINVAL, dict(new_weights=P)),
    (EINVAL, dict(weights=None)), (EINVAL, dict(new_weights=None)),
    (EALIGN, dict(cache=P + 8)), (EALIGN, dict(kept=P + 2)), (EALIGN, dict(cache_page_stride=576 * 16 + 4)),
    (EINVAL, dict(cache_row_stride=568)), (EINVAL, dict(cache_page_stride=576)), (EINVAL, dict(table_stride=8)),
    (EINVAL, dict(kept_stride=4)), (EINVAL, dict(weights_stride=99)), (EINVAL, dict(new_weights_stride=99)),
    (ENOTSUP, dict(batch=1 << 16)), (ENOTSUP, dict(most=1 << 31)), (OK, dict(batch=0))])
def test_keep_refuses(L, want, over):
    assert L.skinny_latent_keep_bf16(ctypes.byref(keep_args(**over)), None) == want


@pytest.mark.parametrize("want,window,sinks,over", [
    (EINVAL, 0, 0, {}), (EINVAL, -1, 0, {}), (EINVAL, 5, -1, {}), (EINVAL, 5, 0, dict(causal=0)), (EINVAL, 5, 0, dict(nq=-1)),
    (EALIGN, 5, 0, dict(q=P + 8)), (EINVAL, 5, 0, dict(out_row_stride=128)), (OK, 5, 2, dict(nq=0)), (OK, 1 << 60, 1 << 60, dict(nq=0))])
def test_window_prefill_refuses(L, want, window, sinks, over):
    assert L.skinny_latent_window_prefill_bf16(ctypes.byref(prefill_args(**over)), window, sinks, None) == want


def test_other_refusals(L):
    n = ctypes.c_int64()
    assert L.skinny_latent_masked_decode_bf16(None, ctypes.byref(mask()), None) == EINVAL
    assert L.skinny_latent_masked_decode_bf16(ctypes.byref(decode_args()), None, None) == EINVAL
    assert L.skinny_latent_window_prefill_bf16(None, 1, 0, None) == EINVAL
    for f in (L.skinny_latent_key_weights_bf16, L.skinny_latent_select, L.skinny_latent_keep_bf16):
        assert f(None, None) == EINVAL
    assert L.skinny_latent_tree_mask(P, P, P, -1, 2, None) == EINVAL
    assert L.skinny_latent_tree_mask(P, P, P, 1, 513, None) == ENOTSUP
    assert L.skinny_latent_tree_mask(P, None, P, 1, 5, None) == EINVAL
    assert L.skinny_latent_tree_mask(P, P + 2, P, 1, 5, None) == EALIGN
    assert L.skinny_latent_tree_mask(None, None, None, 0, 5, None) == OK
    assert L.skinny_latent_window_prefill_workspace(1, 1, 1, 1, 0, 0, ctypes.byref(n)) == EINVAL
    assert L.skinny_latent_window_prefill_workspace(1, 1, 1, 1, 1, -1, ctypes.byref(n)) == EINVAL
    assert L.skinny_latent_window_prefill_workspace(1, 1, 1, 1, 1, 0, None) == EINVAL


def test_the_binding_wants_the_gpu():
    t, i, w = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    q, c, table = t.view(4, 1, 576), t.view(1, 4, 576), i.view(4, 1)
    for call in (lambda: ops.latent_tree_mask(table), lambda: ops.latent_tree_decode(q, c, table, i, i.view(4, 1, 1), 1.0),
                 lambda: ops.latent_window_decode(q, c, table, i, 1.0, 4), lambda: ops.latent_window_prefill(t, t, t, t, i, i, 1.0, 4),
                 lambda: ops.latent_key_weights(q, c, table, i, w, w, 1.0), lambda: ops.latent_select(w, i, 4),
                 lambda: ops.latent_keep(c, table, i, table, i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="window"):
        ops.latent_window_prefill(t, t, t, t, i, i, 1.0, 0)
    with pytest.raises(ValueError, match="mask"):
        ops.latent_tree_decode(q, c, table, i, i, 1.0)
    with pytest.raises(ValueError, match="Tensor"):
        ops.latent_select(None, i, 4)
    with pytest.raises(ValueError, match="GPU"):
        ops.latent_window_prefill_workspace(1, 1, 1, 1, 4, device="cpu")


def test_references_agree():
    """A chain is a tree; a window that holds everything hides nothing; every kept key keeps its row."""
    for n, t in ((9, 4), (4, 4), (2, 4), (40, 33)):
        above, depth = mref.ancestors([j - 1 for j in range(t)])
        assert torch.equal(mref.seen_of(n, t), mref.seen_of(n, t, above=above, depth=depth))
        assert torch.equal(mref.seen_of(n, t), mref.seen_of(n, t, window=n, sinks=0))
        assert torch.equal(mref.seen_of(n, t, window=t, sinks=2), mref.seen_of(n, t, window=t, sinks=2, above=above, depth=depth))
        w = mref.words_of(above)
        assert w.shape == (t, -(-t // 32)) and (int(w[t - 1, 0]) & 0xFFFFFFFF) == (1 << min(t, 32)) - 1
    cache = torch.randn(3, 4, 576)
    table, before = torch.tensor([2, 0, 1]), cache.clone()
    assert mref.keep(cache, table, 11, list(range(11)), 0)[0] == 11 and torch.equal(cache, before)
    assert mref.select([1.0, 5.0, float("nan"), 5.0, 0.0, 2.0], 6, 3, 1, 0) == [0, 1, 2]
