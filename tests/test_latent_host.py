"""Refusals of the latent attention operators, on the host: the C ABI answers before anything is
launched, and the binding's argument checks raise ValueError."""
import ctypes
import os

import pytest
import torch

from decode_skinny_addmm_amd import _lib, ops

OK, EINVAL, EALIGN, ENOTSUP = 0, 1, 2, 3
P = 1 << 20     # a plausible, aligned address: nothing below may reach a launch


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libskinny.so not built")
    return _lib.lib()


def append_args(**over):
    d = dict(kv=P, cache=P, slots=P, positions=P, inv_freq=P, norm_weight=P, q=P, q_out=P, kv_stride=576,
             cache_page_stride=576 * 16, cache_row_stride=576, q_row_stride=512, q_head_stride=64, q_out_row_stride=512,
             q_out_head_stride=64, n=4, heads=8, pages=3, page=16, latent=512, rope=64, eps=1e-6, interleaved=0)
    d.update(over)
    return _lib.SkinnyLatentAppendArgs(**d)


def decode_args(**over):
    d = dict(q=P, cache=P, table=P, lens=P, out=P, lse=P, workspace=P, workspace_bytes=1 << 40, q_row_stride=8 * 576,
             q_head_stride=576, cache_page_stride=576 * 16, cache_row_stride=576, table_stride=9, out_row_stride=8 * 512,
             out_head_stride=512, batch=2, tokens=2, heads=8, pages=20, page=16, max_pages=9, latent=512, rope=64,
             scale=0.1)
    d.update(over)
    return _lib.SkinnyLatentDecodeArgs(**d)


def prefill_args(**over):
    d = dict(q=P, k=P, v=P, k_rot=P, cu_q=P, cu_k=P, out=P, lse=P, workspace=P, workspace_bytes=1 << 40,
             q_row_stride=192 * 4, q_head_stride=192, k_row_stride=256 * 4, k_head_stride=256, v_row_stride=256 * 4,
             v_head_stride=256, k_rot_stride=64, out_row_stride=128 * 4, out_head_stride=128, nq=10, nk=20, batch=2,
             heads=4, head_dim=128, rope=64, scale=0.1, causal=1)
    d.update(over)
    return _lib.SkinnyLatentPrefillArgs(**d)


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(n=-1)), (EINVAL, dict(heads=-1)), (EINVAL, dict(page=0)), (EINVAL, dict(pages=-1)),
    (EINVAL, dict(eps=-1.0)), (EINVAL, dict(eps=float("nan"))), (ENOTSUP, dict(latent=256)), (ENOTSUP, dict(rope=32)),
    (EINVAL, dict(kv=None)), (EINVAL, dict(cache=None)), (EINVAL, dict(slots=None)), (EINVAL, dict(positions=None)),
    (EINVAL, dict(inv_freq=None)), (EINVAL, dict(q_out=None)), (EALIGN, dict(kv=P + 8)), (EALIGN, dict(cache=P + 2)),
    (EALIGN, dict(norm_weight=P + 8)), (EALIGN, dict(q=P + 4)), (EALIGN, dict(q_out=P + 4)), (EALIGN, dict(slots=P + 4)),
    (EALIGN, dict(inv_freq=P + 4)), (EALIGN, dict(kv_stride=580)), (EINVAL, dict(kv_stride=568)),
    (EINVAL, dict(cache_row_stride=512)), (EALIGN, dict(cache_page_stride=576 * 16 + 4)), (EINVAL, dict(q_head_stride=56)),
    (EINVAL, dict(q_out_row_stride=-64)), (EINVAL, dict(kv_stride=1 << 50)), (ENOTSUP, dict(heads=1 << 20)),
    (ENOTSUP, dict(n=1 << 40, kv_stride=576)), (OK, dict(n=0)), (OK, dict(n=0, kv=None, cache=None))])
def test_append_refuses(L, want, over):
    assert L.skinny_latent_append_bf16(ctypes.byref(append_args(**over)), None) == want


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(batch=-1)), (EINVAL, dict(tokens=0)), (EINVAL, dict(heads=-1)), (EINVAL, dict(page=0)),
    (EINVAL, dict(max_pages=-1)), (EINVAL, dict(pages=0)), (EINVAL, dict(max_pages=0)), (EINVAL, dict(scale=0.0)),
    (EINVAL, dict(scale=-0.1)), (EINVAL, dict(scale=float("inf"))), (EINVAL, dict(scale=float("nan"))),
    (ENOTSUP, dict(latent=448)), (ENOTSUP, dict(rope=0)), (EINVAL, dict(q=None)), (EINVAL, dict(cache=None)),
    (EINVAL, dict(table=None)), (EINVAL, dict(lens=None)), (EINVAL, dict(out=None)), (EALIGN, dict(q=P + 8)),
    (EALIGN, dict(cache=P + 8)), (EALIGN, dict(out=P + 2)), (EALIGN, dict(workspace=P + 4)), (EALIGN, dict(lse=P + 2)),
    (EALIGN, dict(table=P + 1)), (EALIGN, dict(q_head_stride=580)), (EINVAL, dict(q_head_stride=512)),
    (EINVAL, dict(out_head_stride=504)), (EINVAL, dict(cache_row_stride=0)), (EINVAL, dict(table_stride=8)),
    (ENOTSUP, dict(batch=1 << 30)), (ENOTSUP, dict(heads=1 << 20)), (ENOTSUP, dict(tokens=1 << 14, heads=1 << 14)),
    (ENOTSUP, dict(max_pages=1 << 28, table_stride=1 << 28, page=1 << 20)), (ENOTSUP, dict(batch=1 << 20, heads=1 << 10)),
    (OK, dict(batch=0)), (OK, dict(heads=0)), (OK, dict(batch=0, q=None, cache=None, pages=0))])
def test_decode_refuses(L, want, over):
    assert L.skinny_latent_decode_bf16(ctypes.byref(decode_args(**over)), None) == want


@pytest.mark.parametrize("want,over", [
    (EINVAL, dict(nq=-1)), (EINVAL, dict(nk=-1)), (EINVAL, dict(batch=-1)), (EINVAL, dict(heads=-1)),
    (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=float("nan"))), (ENOTSUP, dict(head_dim=64)), (ENOTSUP, dict(rope=32)),
    (EINVAL, dict(q=None)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)), (EINVAL, dict(k_rot=None)),
    (EINVAL, dict(cu_q=None)), (EINVAL, dict(cu_k=None)), (EINVAL, dict(out=None)), (EALIGN, dict(q=P + 8)),
    (EALIGN, dict(v=P + 8)), (EALIGN, dict(k_rot=P + 8)), (EALIGN, dict(out=P + 8)), (EALIGN, dict(cu_q=P + 2)),
    (EALIGN, dict(lse=P + 2)), (EALIGN, dict(v_row_stride=1028)), (EINVAL, dict(k_head_stride=64)),
    (EINVAL, dict(q_head_stride=128)), (EINVAL, dict(k_rot_stride=32)), (EINVAL, dict(out_row_stride=64)),
    (ENOTSUP, dict(nq=1 << 31)), (ENOTSUP, dict(nq=1 << 30, heads=1 << 16)), (OK, dict(nq=0)), (OK, dict(batch=0)),
    (OK, dict(heads=0)), (OK, dict(nq=0, q=None, out=None))])
def test_prefill_refuses(L, want, over):
    assert L.skinny_latent_prefill_bf16(ctypes.byref(prefill_args(**over)), None) == want


def test_null_arguments(L):
    for f in (L.skinny_latent_append_bf16, L.skinny_latent_decode_bf16, L.skinny_latent_prefill_bf16):
        assert f(None, None) == EINVAL
    n = ctypes.c_int64()
    assert L.skinny_latent_decode_workspace(1, 1, 1, None) == EINVAL
    assert L.skinny_latent_decode_workspace(-1, 1, 1, ctypes.byref(n)) == EINVAL
    assert L.skinny_latent_prefill_workspace(1, 1, 1, -1, ctypes.byref(n)) == EINVAL
    assert L.skinny_latent_prefill_workspace(1 << 40, 1, 1, 1, ctypes.byref(n)) == ENOTSUP


def test_the_binding_wants_the_gpu():
    t = torch.zeros(4, 576, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        ops.latent_append(t, t.view(1, 4, 576), i, i, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="GPU"):
        ops.latent_decode(t.view(4, 1, 576), t.view(1, 4, 576), i.int().view(4, 1), i.int(), 1.0)
    with pytest.raises(ValueError, match="GPU"):
        ops.latent_prefill(t, t, t, t, i.int(), i.int(), 1.0)
    with pytest.raises(ValueError, match="Tensor"):
        ops.latent_decode(None, t, i, i, 1.0)
    with pytest.raises(ValueError, match="GPU"):
        ops.latent_prefill_workspace(1, 1, 1, 1, device="cpu")
    with pytest.raises(ValueError, match="latent"):
        ops.latent_decode_workspace(1, 1, 1, 256)


def test_tensors_of_a_call_belong_to_its_stream(monkeypatch):
    """What a call allocates is memory of the stream that it was given: memory of the current stream could
    still be in use there, or go to another tensor while the call runs. Nothing is launched here."""
    named, inside, made = object(), [], []

    class Inside:
        def __init__(self, stream):
            assert stream is named

        def __enter__(self):
            inside.append(1)

        def __exit__(self, *x):
            inside.pop()

    empty = torch.empty

    def watched(*x, **k):
        made.append(bool(inside))
        return empty(*x, **k)

    class Module:
        append = decode = prefill = staticmethod(lambda *x: 0)

    class Library:
        skinny_latent_decode_workspace = skinny_latent_prefill_workspace = None

    monkeypatch.setattr(ops.torch.cuda, "stream", Inside)
    monkeypatch.setattr(ops.torch, "empty", watched)
    monkeypatch.setattr(ops, "lib", Library)
    monkeypatch.setattr(ops, "_latent", Module)
    monkeypatch.setattr(ops, "_gpu_of", lambda name, t: 0)
    monkeypatch.setattr(ops, "_call", lambda *x: None)
    monkeypatch.setattr(ops, "_workspace_bytes", lambda *x: 64)
    q, i = torch.zeros(2, 4, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    calls = ((1, lambda s: ops.latent_append(q[:, 0], q, i, i, i, q=q[:, :, 512:], stream=s)),
             (3, lambda s: ops.latent_decode(q, q, i.view(2, 1), i, 1.0, stream=s)),
             (3, lambda s: ops.latent_prefill(q[:, :, :192], q, q, q, i, i, 1.0, stream=s)))
    for count, call in calls:
        call(named)
        assert made == [True] * count and not inside
        made.clear()
        call(None)
        assert made == [False] * count
        made.clear()


# Rows that are written and share numbers: two tokens or heads would race on them.
@pytest.mark.parametrize("over", [
    dict(q_out_row_stride=64, q_out_head_stride=64), dict(q_out_row_stride=64 * 7), dict(q_out_row_stride=64, q_out_head_stride=128),
    dict(cache_page_stride=576), dict(cache_page_stride=576 * 15), dict(cache_page_stride=576, cache_row_stride=576 * 2),
    dict(cache_page_stride=576 * 16, cache_row_stride=576 + 64)])
def test_append_refuses_overlapping_rows(L, over):
    assert L.skinny_latent_append_bf16(ctypes.byref(append_args(**over)), None) == EINVAL


@pytest.mark.parametrize("over", [dict(out_row_stride=512), dict(out_row_stride=512 * 7), dict(out_row_stride=512, out_head_stride=512 * 3),
                                  dict(out_row_stride=(1 << 40) - 8, out_head_stride=1 << 40)])
def test_decode_refuses_overlapping_rows(L, over):
    assert L.skinny_latent_decode_bf16(ctypes.byref(decode_args(**over)), None) == EINVAL


@pytest.mark.parametrize("over", [dict(out_row_stride=128), dict(out_row_stride=128 * 3), dict(out_row_stride=128, out_head_stride=128 * 9)])
def test_prefill_refuses_overlapping_rows(L, over):
    assert L.skinny_latent_prefill_bf16(ctypes.byref(prefill_args(**over)), None) == EINVAL


def test_refuses_more_threads_than_a_launch_takes(L):
    """2^32 threads and more are no launch: the join of a decode call starts 128 a row (rows of a request
    filled up to 16, 32, 64 or a multiple of 128), append a wave a token."""
    for batch, tokens, heads in ((1 << 18, 1, 128), (1 << 20, 1, 17), (1 << 19, 1, 64), (1 << 17, 2, 65), (1 << 17, 1, 129)):
        a = decode_args(batch=batch, tokens=tokens, heads=heads, q_row_stride=heads * 576, out_row_stride=heads * 512)
        assert L.skinny_latent_decode_bf16(ctypes.byref(a), None) == ENOTSUP
    for n in ((1 << 26) - 3, 1 << 29):
        assert L.skinny_latent_append_bf16(ctypes.byref(append_args(n=n)), None) == ENOTSUP
