"""Python binding of the skinny residual GEMM: argument marshalling over the C ABI only.

Y = bf16(X @ W^T + R) for bf16 X[M,K], W[N,K], R[M,N] on the GPU; every step runs in the
HIP kernels of libskinny.so. torch supplies device memory and the current stream.
Argument errors raise ValueError before the library is called (as the launcher of the
vLLM API page "fused_add_multicast_skinny_gemm" does); library errors raise SkinnyError.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (CONFIG_FIELDS, FLAG_NO_NEG_ZERO, FLAG_ROUND_PRODUCT, SkinnyConfig, SkinnyError, SkinnyKdaArgs,  # noqa: F401
                   SkinnyResources, check, lib)


def _as_config(cfg) -> SkinnyConfig | None:
    if cfg is None:
        return None
    if isinstance(cfg, SkinnyConfig):
        return cfg
    if isinstance(cfg, dict):
        vals = [int(cfg.get(f, 0)) for f in CONFIG_FIELDS]
    else:
        vals = [int(v) for v in cfg] + [0] * (len(CONFIG_FIELDS) - len(cfg))
    return SkinnyConfig(*vals)


def _byte_span(t: torch.Tensor) -> tuple[int, int]:
    """[first, last) byte addresses of a tensor with non-negative strides."""
    if t.numel() == 0:
        return t.data_ptr(), t.data_ptr()
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _overlaps(a: torch.Tensor, b: torch.Tensor) -> bool:
    (a0, a1), (b0, b1) = _byte_span(a), _byte_span(b)
    return a0 < b1 and b0 < a1


def _check_aliasing(inputs, R, out):
    """The output may be R itself (same address, strides and dtype: every residual is read
    before its own output is written) but must not overlap the other inputs or any other
    part of R. Overlap is judged on byte spans, so two column blocks interleaved in one wide
    matrix count as overlapping (a conservative refusal, never a missed overlap)."""
    if any(_overlaps(out, t) for t in inputs):
        raise ValueError("out must not overlap the operands other than R")
    if _overlaps(out, R) and not (out.data_ptr() == R.data_ptr() and out.stride() == R.stride()
                                  and out.dtype == R.dtype):
        raise ValueError("out may be R itself but must not partially overlap it")


def _check_operands(X, W, R, out, out_dtype):
    for name, t in (("X", X), ("W", W), ("R", R), ("out", out)):
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s must be a torch.Tensor" % name)
        if t.device.type != "cuda":
            raise ValueError("%s must be on the GPU" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous (row-major)" % name)
        if t.dim() != 2:
            raise ValueError("%s must be 2-D" % name)
    for name, t in (("X", X), ("W", W), ("R", R)):
        if t.dtype != torch.bfloat16:
            raise ValueError("%s must be bfloat16" % name)
    if out.dtype != out_dtype:
        raise ValueError("out must be %s" % out_dtype)
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K] with K = X.shape[1] (got %s vs %s)" % (tuple(W.shape), tuple(X.shape)))
    if tuple(R.shape) != (M, N) or tuple(out.shape) != (M, N):
        raise ValueError("R and out must be [M, N] = [%d, %d]" % (M, N))
    devs = {t.device for t in (X, W, R, out)}
    if len(devs) != 1:
        raise ValueError("all operands must be on the same device")
    _check_aliasing((X, W), R, out)
    return M, N, K


def _stream_ptr(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return int(s.cuda_stream)


def addmm(X: torch.Tensor, W: torch.Tensor, R: torch.Tensor, out: torch.Tensor | None = None,
          config=None, stream=None) -> torch.Tensor:
    """Y = bf16(X @ W^T + R) via skinny_addmm_bf16_with_config. `out` may be R (in place)."""
    if out is None:
        out = torch.empty_like(R)
    M, N, K = _check_operands(X, W, R, out, torch.bfloat16)
    c = _as_config(config)
    with torch.cuda.device(X.device):
        st = lib().skinny_addmm_bf16_with_config(X.data_ptr(), W.data_ptr(), R.data_ptr(), out.data_ptr(),
                                                 M, N, K, ctypes.byref(c) if c is not None else None,
                                                 _stream_ptr(stream, X.device))
    check(st, "skinny_addmm_bf16")
    return out


def addmm_default(X, W, R, out, stream=None) -> torch.Tensor:
    """The plain entry point skinny_addmm_bf16 (configuration chosen by the library)."""
    M, N, K = _check_operands(X, W, R, out, torch.bfloat16)
    with torch.cuda.device(X.device):
        st = lib().skinny_addmm_bf16(X.data_ptr(), W.data_ptr(), R.data_ptr(), out.data_ptr(), M, N, K,
                                     _stream_ptr(stream, X.device))
    check(st, "skinny_addmm_bf16")
    return out


def addmm_acc_f32(X, W, R, out: torch.Tensor | None = None, config=None, stream=None) -> torch.Tensor:
    """fp32 value before rounding, fp32(sum) + fp32(R), from the same kernel (test entry)."""
    if out is None:
        out = torch.empty(R.shape, dtype=torch.float32, device=R.device)
    M, N, K = _check_operands(X, W, R, out, torch.float32)
    c = _as_config(config)
    with torch.cuda.device(X.device):
        st = lib().skinny_addmm_bf16_acc_f32(X.data_ptr(), W.data_ptr(), R.data_ptr(), out.data_ptr(),
                                             M, N, K, ctypes.byref(c) if c is not None else None,
                                             _stream_ptr(stream, X.device))
    check(st, "skinny_addmm_bf16_acc_f32")
    return out


def _check_shard_operands(X, W, R, out, out_dtype):
    """Like _check_operands, but R and out may be row-major views into wider matrices: each
    needs unit column stride and a row stride >= N (the leading dimension passed on)."""
    for name, t in (("X", X), ("W", W), ("R", R), ("out", out)):
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s must be a torch.Tensor" % name)
        if t.device.type != "cuda":
            raise ValueError("%s must be on the GPU" % name)
        if t.dim() != 2:
            raise ValueError("%s must be 2-D" % name)
    for name, t in (("X", X), ("W", W)):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous (row-major)" % name)
    for name, t in (("X", X), ("W", W), ("R", R)):
        if t.dtype != torch.bfloat16:
            raise ValueError("%s must be bfloat16" % name)
    if out.dtype != out_dtype:
        raise ValueError("out must be %s" % out_dtype)
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K] with K = X.shape[1]")
    if tuple(R.shape) != (M, N) or tuple(out.shape) != (M, N):
        raise ValueError("R and out must be [M, N] = [%d, %d]" % (M, N))
    for name, t in (("R", R), ("out", out)):
        if N > 1 and t.stride(1) != 1:
            raise ValueError("%s must have unit column stride" % name)
        if M > 1 and t.stride(0) < N:
            raise ValueError("%s row stride must be >= N" % name)
    if len({t.device for t in (X, W, R, out)}) != 1:
        raise ValueError("all operands must be on the same device")
    _check_aliasing((X, W), R, out)
    return M, N, K, (R.stride(0) if M > 1 else N), (out.stride(0) if M > 1 else N)


def _shard_flags(round_product: bool, no_neg_zero: bool) -> int:
    return (FLAG_ROUND_PRODUCT if round_product else 0) | (FLAG_NO_NEG_ZERO if no_neg_zero else 0)


def addmm_shard(X, W, R, out=None, round_product=False, no_neg_zero=False, config=None,
                stream=None) -> torch.Tensor:
    """Tensor-parallel shard form via skinny_addmm_bf16_shard: R and out may be column blocks
    of wider row-major matrices (their row strides are passed as leading dimensions).
    round_product: round the product sum to bf16 before adding R (two roundings);
    no_neg_zero: write +0 for a -0 result."""
    if out is None:
        out = torch.empty(R.shape, dtype=torch.bfloat16, device=R.device)
    M, N, K, ldr, ldy = _check_shard_operands(X, W, R, out, torch.bfloat16)
    c = _as_config(config)
    with torch.cuda.device(X.device):
        st = lib().skinny_addmm_bf16_shard(X.data_ptr(), W.data_ptr(), R.data_ptr(), ldr, out.data_ptr(), ldy,
                                           M, N, K, _shard_flags(round_product, no_neg_zero),
                                           ctypes.byref(c) if c is not None else None,
                                           _stream_ptr(stream, X.device))
    check(st, "skinny_addmm_bf16_shard")
    return out


def addmm_shard_acc_f32(X, W, R, out=None, round_product=False, config=None, stream=None) -> torch.Tensor:
    """Test entry of the shard form: the fp32 value each output is rounded from."""
    if out is None:
        out = torch.empty(R.shape, dtype=torch.float32, device=R.device)
    M, N, K, ldr, lda = _check_shard_operands(X, W, R, out, torch.float32)
    c = _as_config(config)
    with torch.cuda.device(X.device):
        st = lib().skinny_addmm_bf16_shard_acc_f32(X.data_ptr(), W.data_ptr(), R.data_ptr(), ldr, out.data_ptr(),
                                                   lda, M, N, K, _shard_flags(round_product, False),
                                                   ctypes.byref(c) if c is not None else None,
                                                   _stream_ptr(stream, X.device))
    check(st, "skinny_addmm_bf16_shard_acc_f32")
    return out


def _check_kbit(X, planes, absmax, codebook, kbits, R, out, out_dtype):
    for name, t in (("X", X), ("planes", planes), ("absmax", absmax), ("codebook", codebook), ("R", R),
                    ("out", out)):
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s must be a torch.Tensor" % name)
        if t.device.type != "cuda":
            raise ValueError("%s must be on the GPU" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if X.dtype != torch.bfloat16 or R.dtype != torch.bfloat16 or out.dtype != out_dtype:
        raise ValueError("X and R must be bfloat16, out %s" % out_dtype)
    if planes.dtype not in (torch.int32, torch.uint32) or absmax.dtype != torch.uint8 or codebook.dtype != torch.float32:
        raise ValueError("planes must be int32/uint32 bit words, absmax uint8, codebook float32")
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M, K = X.shape
    N = R.shape[0 if R.dim() == 1 else 1]
    if tuple(planes.shape) != (N, K // 32, kbits) or tuple(absmax.shape) != (N, K // 32):
        raise ValueError("planes must be [N, K/32, kbits] and absmax [N, K/32]")
    if tuple(codebook.shape) != (1 << kbits,):
        raise ValueError("codebook must have 2^kbits entries")
    if tuple(R.shape) != (M, N) or tuple(out.shape) != (M, N):
        raise ValueError("R and out must be [M, N]")
    _check_aliasing((X, planes, absmax, codebook), R, out)
    return M, N, K


def kbit_gemv(X, planes, absmax, codebook, kbits: int, R, out=None, stream=None) -> torch.Tensor:
    """Y = bf16(X @ What^T + R) with What the k-bit quantized weights (skinny_kbit_gemv_bf16)."""
    if out is None:
        out = torch.empty_like(R)
    M, N, K = _check_kbit(X, planes, absmax, codebook, kbits, R, out, torch.bfloat16)
    with torch.cuda.device(X.device):
        st = lib().skinny_kbit_gemv_bf16(X.data_ptr(), planes.data_ptr(), absmax.data_ptr(), codebook.data_ptr(),
                                         int(kbits), R.data_ptr(), out.data_ptr(), M, N, K,
                                         _stream_ptr(stream, X.device))
    check(st, "skinny_kbit_gemv_bf16")
    return out


def kbit_gemv_acc_f32(X, planes, absmax, codebook, kbits: int, R, out=None, stream=None) -> torch.Tensor:
    """Test entry: the fp32 value each output of kbit_gemv is rounded from."""
    if out is None:
        out = torch.empty(R.shape, dtype=torch.float32, device=R.device)
    M, N, K = _check_kbit(X, planes, absmax, codebook, kbits, R, out, torch.float32)
    with torch.cuda.device(X.device):
        st = lib().skinny_kbit_gemv_bf16_acc_f32(X.data_ptr(), planes.data_ptr(), absmax.data_ptr(),
                                                 codebook.data_ptr(), int(kbits), R.data_ptr(), out.data_ptr(),
                                                 M, N, K, _stream_ptr(stream, X.device))
    check(st, "skinny_kbit_gemv_bf16_acc_f32")
    return out


def kda_verify(inp: dict, T: int, H: int, HV: int, K: int, V: int, scale: float, snapshots: bool = True,
               ring: bool = False, out=None, stream=None) -> torch.Tensor:
    """One KDA chain-verify step (skinny_kda_verify_bf16) on device tensors named as on the
    sglang benchmark page: bf16 mixed [B*T, dim], w [dim, 4], bias [dim], conv_pool
    [lines, 3, dim], win_pool [lines, T, 3, dim], a [B*T, HV*K], b [B*T, HV]; float32 A_log
    [HV], dt_bias [HV*K], ssm [slots, HV, V, K], inter_ssm [lines, T, HV, V, K], ring
    buffers rawv [slots, HV, R, V], rawk [slots, H, R, K] (bf16), g [slots, HV, R, K], beta
    [slots, HV, R] (float32); int32 cache_indices, inter_indices [B]. Writes win_pool, and
    inter_ssm (snapshots) or the ring buffers (ring); returns o bf16 [B*T, HV, V]."""
    dim = 2 * H * K + HV * V
    B = int(inp["cache_indices"].shape[0])
    spec = {"mixed": (torch.bfloat16, (B * T, dim)), "w": (torch.bfloat16, (dim, 4)),
            "bias": (torch.bfloat16, (dim,)), "a": (torch.bfloat16, (B * T, HV * K)),
            "b": (torch.bfloat16, (B * T, HV)), "A_log": (torch.float32, (HV,)),
            "dt_bias": (torch.float32, (HV * K,)), "cache_indices": (torch.int32, (B,)),
            "inter_indices": (torch.int32, (B,))}
    lines = int(inp["conv_pool"].shape[0])
    slots = int(inp["ssm"].shape[0])
    spec["conv_pool"] = (torch.bfloat16, (lines, 3, dim))
    spec["win_pool"] = (torch.bfloat16, (lines, T, 3, dim))
    spec["ssm"] = (torch.float32, (slots, HV, V, K))
    R = 0
    if snapshots:
        spec["inter_ssm"] = (torch.float32, (lines, T, HV, V, K))
    if ring:
        R = int(inp["rawv"].shape[2])
        spec.update({"rawv": (torch.bfloat16, (slots, HV, R, V)), "rawk": (torch.bfloat16, (slots, H, R, K)),
                     "g": (torch.float32, (slots, HV, R, K)), "beta": (torch.float32, (slots, HV, R))})
    dev = inp["mixed"].device if isinstance(inp.get("mixed"), torch.Tensor) else None
    for name, (dt, shape) in spec.items():
        t = inp.get(name)
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError("%s must be a contiguous GPU tensor" % name)
        if t.device != dev:
            raise ValueError("%s is on %s, mixed on %s: all tensors must be on one GPU" % (name, t.device, dev))
        if t.dtype != dt or tuple(t.shape) != shape:
            raise ValueError("%s must be %s %s, got %s %s" % (name, dt, shape, t.dtype, tuple(t.shape)))
    if out is None:
        out = torch.empty((B * T, HV, V), dtype=torch.bfloat16, device=inp["mixed"].device)
    elif (out.dtype != torch.bfloat16 or tuple(out.shape) != (B * T, HV, V) or not out.is_contiguous()
          or out.device != dev):
        raise ValueError("out must be contiguous bf16 [B*T, HV, V] on the inputs' GPU")
    p = lambda name: inp[name].data_ptr() if name in spec else None
    args = SkinnyKdaArgs(mixed=p("mixed"), conv_w=p("w"), conv_b=p("bias"), conv_pool=p("conv_pool"),
                         cache_idx=p("cache_indices"), inter_idx=p("inter_indices"), a=p("a"), b=p("b"),
                         A_log=p("A_log"), dt_bias=p("dt_bias"), ssm=p("ssm"), conv_win=p("win_pool"),
                         snap=p("inter_ssm"), ring_v=p("rawv"), ring_k=p("rawk"), ring_g=p("g"),
                         ring_beta=p("beta"), out=out.data_ptr(), B=B, T=T, H=H, HV=HV, K=K, V=V,
                         lines=lines, slots=slots, ring_len=R, scale=float(scale))
    with torch.cuda.device(inp["mixed"].device):
        st = lib().skinny_kda_verify_bf16(ctypes.byref(args), _stream_ptr(stream, inp["mixed"].device))
    check(st, "skinny_kda_verify_bf16")
    return out


LATENT, ROPE, HEAD = 512, 64, 128  # the sizes that the latent attention kernels are built for

_latent_module = None


def _latent():
    """The native binding of the latent attention operators (csrc/binding.cpp), given the library's
    entry points: it checks the tensors (ValueError) and calls them."""
    global _latent_module
    if _latent_module is None:
        L = lib()
        try:
            from . import _latent as module
        except ImportError as e:
            raise RuntimeError("the _latent module is not built; run `python -m decode_skinny_addmm_amd.build` or "
                               "__graft_entry__.build()") from e
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (L.skinny_latent_append_bf16, L.skinny_latent_decode_bf16, L.skinny_latent_prefill_bf16,
                                L.skinny_latent_masked_decode_bf16, L.skinny_latent_tree_mask,
                                L.skinny_latent_window_prefill_bf16, L.skinny_latent_key_weights_bf16,
                                L.skinny_latent_select, L.skinny_latent_keep_bf16)))
        _latent_module = module
    return _latent_module


def _gpu_of(name, t) -> int:
    """Index of the GPU that tensor t is on."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    return t.get_device()


def _call(fn, what, gpu, stream, *args):
    raw = torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == gpu:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(gpu):
            st = fn(*args, raw)
    if st:
        check(st, what)


def _new(shape, dtype, dev, stream):
    """A tensor that a call allocates: memory of `stream` where one is named. The current stream's could
    still be in use there, and one that is let go before `stream` is done with it must come back to
    no other."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def latent_append(kv, cache, slots, positions, inv_freq, norm_weight=None, eps: float = 1e-6, q=None, q_out=None,
                  interleaved: bool = False, stream=None):
    """New tokens' rows into a paged latent cache (skinny_latent_append_bf16), in place.

    kv bf16 [n, 576]: each token's 512 latents and the 64 numbers of the key that all heads share.
    The latents are normalised (root mean square with eps, times norm_weight bf16 [512]; stored as
    they are where norm_weight is None), the shared key is turned by the token's position, and both
    go to slot slots[i] (int64 [n]: page * page_size + place; a slot outside the cache, such as -1
    for a padding row, writes nothing) of cache bf16 [pages, page_size, 576]. Pairs of numbers,
    (i, i + 32) or with interleaved (2i, 2i + 1), turn by positions (int64 [n]) * inv_freq (float64
    [32]). q bf16 [n, heads, 64], the rotated part of every head's query, is turned the same way
    into q_out (allocated where None; may be q itself). Returns q_out, or None without q. kv, cache,
    q and q_out may have strides (multiples of 8, contiguous last dimension). Here and below, what a
    call allocates with `stream` named belongs to that stream, as if made with it current."""
    gpu = _gpu_of("kv", kv)
    if q is not None and q_out is None:
        q_out = _new(tuple(q.shape) if isinstance(q, torch.Tensor) else 0, torch.bfloat16, kv.device, stream)
    _call(_latent().append, "skinny_latent_append_bf16", gpu, stream, kv, cache, slots, positions, inv_freq, norm_weight,
          eps, q, q_out, interleaved)
    return q_out


def _workspace_bytes(fn, what, dev, *sizes) -> int:
    n = ctypes.c_int64()
    if torch.cuda.current_device() == dev.index:
        st = fn(*sizes, ctypes.byref(n))
    else:
        with torch.cuda.device(dev):                         # the size follows the device
            st = fn(*sizes, ctypes.byref(n))
    if st:
        check(st, what)
    return n.value


def _workspace(fn, what, device, *sizes):
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("device must be a GPU")
    return torch.empty(_workspace_bytes(fn, what, dev, *sizes), dtype=torch.uint8, device=dev)


def _call_workspace(fn, what, dev, stream, *sizes):
    """Workspace of one call, None where it needs none."""
    n = _workspace_bytes(fn, what, dev, *sizes)
    return _new(n, torch.uint8, dev, stream) if n else None


def latent_decode_workspace(batch: int, tokens: int, heads: int, latent: int = LATENT, device="cuda") -> torch.Tensor:
    """Device memory for the partial sums of latent_decode calls of these sizes, whatever their
    lengths. Calls that follow each other on a stream may share it."""
    if latent != LATENT:
        raise ValueError("latent must be %d" % LATENT)
    return _workspace(lib().skinny_latent_decode_workspace, "skinny_latent_decode_workspace", device, batch, tokens, heads)


def latent_prefill_workspace(nq: int, nk: int, batch: int, heads: int, device="cuda") -> torch.Tensor:
    """Device memory for the partial sums of a latent_prefill call of these sizes (may be empty)."""
    return _workspace(lib().skinny_latent_prefill_workspace, "skinny_latent_prefill_workspace", device, nq, nk, batch,
                      heads)


def _decode_outputs(q, tokens, out, lse, workspace, stream):
    """The GPU of a decode call, and its out, lse and workspace, made for the call where None."""
    gpu = _gpu_of("q", q)
    if out is None or lse is None or workspace is None:
        dev = q.device
        if q.dim() != 3:
            raise ValueError("q must be 3-D")
        if tokens < 1:
            raise ValueError("tokens must be at least 1, got %d" % tokens)
        rows, heads = q.shape[:2]
        if out is None:
            out = _new((rows, heads, LATENT), torch.bfloat16, dev, stream)
        if lse is None:
            lse = _new((rows, heads), torch.float32, dev, stream)
        if workspace is None:
            workspace = _call_workspace(lib().skinny_latent_decode_workspace, "skinny_latent_decode_workspace", dev,
                                        stream, rows // tokens, tokens, heads)
    return gpu, out, lse, workspace


def latent_decode(q, cache, table, lens, scale: float, tokens: int = 1, rope_dim: int = ROPE, out=None, lse=None,
                  workspace=None, stream=None):
    """Absorbed latent attention of each request's newest tokens over a paged latent cache
    (skinny_latent_decode_bf16).

    q bf16 [batch * tokens, heads, 576]: queries that already carry the key projection, and their
    rotated parts. cache bf16 [pages, page_size, 576]; table int32 [batch, max_pages]: each
    request's pages; lens int32 [batch]: its cached tokens, the new ones among them. Token j of
    request i sees keys below lens[i] - tokens + j + 1; out bf16 [batch * tokens, heads, 512] is
    the softmax-weighted sum of the keys' latents, lse float32 [batch * tokens, heads] the log of
    the softmax's sum (zeros and -inf where a row sees no key). Lengths beyond the table and page
    ids outside the cache are clamped. q, cache and out may have strides (multiples of 8,
    contiguous last dimension). workspace: latent_decode_workspace(batch, tokens, heads), kept by
    the caller between calls; allocated for this call where None. Returns (out, lse)."""
    gpu, out, lse, workspace = _decode_outputs(q, tokens, out, lse, workspace, stream)
    _call(_latent().decode, "skinny_latent_decode_bf16", gpu, stream, q, cache, table, lens, scale, tokens, rope_dim, out,
          lse, workspace)
    return out, lse


def _prefill_outputs(q, k, cu_q, out, lse, workspace, stream, fn, what, *sizes):
    """The GPU of a prefill call, and its out, lse and workspace, made for the call where None."""
    gpu = _gpu_of("q", q)
    if out is None or lse is None or workspace is None:
        dev = q.device
        if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("q and k must be 3-D tensors")
        if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
            raise ValueError("cu_q must be a tensor [batch + 1]")
        nq, heads = q.shape[:2]
        if out is None:
            out = _new((nq, heads, HEAD), torch.bfloat16, dev, stream)
        if lse is None:
            lse = _new((nq, heads), torch.float32, dev, stream)
        if workspace is None:
            workspace = _call_workspace(fn, what, dev, stream, nq, k.shape[0], cu_q.shape[0] - 1, heads, *sizes)
    return gpu, out, lse, workspace


def latent_prefill(q, k, v, k_rot, cu_q, cu_k, scale: float, causal: bool = True, out=None, lse=None, workspace=None,
                   stream=None):
    """Expanded latent attention of prompts (skinny_latent_prefill_bf16).

    q bf16 [nq, heads, 192] (a head's 128 numbers, then its 64 rotated ones), k and v bf16 [nk,
    heads, 128], k_rot bf16 [nk, 64] shared by all heads; cu_q, cu_k int32 [batch + 1]: where each
    sequence's queries and keys start, rising from 0 to nq and nk. causal: a sequence's last query
    sees its last key, the one before it one key fewer, and so on. out bf16 [nq, heads, 128], lse
    float32 [nq, heads] (zeros and -inf where a row sees no key). q, k, v, k_rot and out may have
    strides (multiples of 8, contiguous last dimension). workspace: latent_prefill_workspace(nq,
    nk, batch, heads), allocated for this call where None. Returns (out, lse)."""
    gpu, out, lse, workspace = _prefill_outputs(q, k, cu_q, out, lse, workspace, stream,
                                                lib().skinny_latent_prefill_workspace, "skinny_latent_prefill_workspace")
    _call(_latent().prefill, "skinny_latent_prefill_bf16", gpu, stream, q, k, v, k_rot, cu_q, cu_k, scale, causal, out, lse,
          workspace)
    return out, lse


def _whole(name, value, least):
    if not hasattr(value, "__index__") or value < least:
        raise ValueError("%s must be a whole number of at least %d, got %s" % (name, least, value))


def latent_tree_mask(parents, mask=None, depth=None, stream=None):
    """Rows of trees of drafted tokens (skinny_latent_tree_mask), for latent_tree_decode.

    parents int32 [batch, tokens], at most 512 tokens: each token's parent among the earlier ones of its
    request; any other number (-1) where it follows the context. Returns mask int32 [batch, tokens,
    ceil(tokens / 32)], where bit d % 32 of word d / 32 says that a token sees token d (itself and those above
    it), and depth int32 [batch, tokens]: how many stand above it, so that it has position
    lens - tokens + depth. One call serves all layers of a step."""
    gpu = _gpu_of("parents", parents)
    if parents.dim() != 2:
        raise ValueError("parents must be a tensor [batch, tokens]")
    batch, tokens = parents.shape
    if mask is None:
        mask = _new((batch, tokens, (tokens + 31) // 32), torch.int32, parents.device, stream)
    if depth is None:
        depth = _new((batch, tokens), torch.int32, parents.device, stream)
    _call(_latent().tree_mask, "skinny_latent_tree_mask", gpu, stream, parents, mask, depth)
    return mask, depth


def latent_tree_decode(q, cache, table, lens, mask, scale: float, window: int = 0, sinks: int = 0, depth=None,
                       rope_dim: int = ROPE, out=None, lse=None, workspace=None, stream=None):
    """latent_decode of requests whose newest tokens are a tree (skinny_latent_masked_decode_bf16).

    mask int32 [batch, tokens, ceil(tokens / 32)], as from latent_tree_mask (its first dimension may have stride
    0: one tree for all): token j sees the context, which is the first lens[i] - tokens keys, and those of
    the new tokens whose bit is set. The number of new tokens, 512 at most, is the mask's. window (at least
    `tokens`; 0: none): of the context only the keys among the last `window` up to a token's own position, which
    depth (int32 [batch, tokens], as from latent_tree_mask) tells, and the first `sinks`. The rest as in
    latent_decode; workspace: latent_decode_workspace(batch, tokens, heads). Returns (out, lse)."""
    if not isinstance(mask, torch.Tensor) or mask.dim() != 3 or mask.shape[1] < 1:
        raise ValueError("mask must be a tensor [batch, tokens, ceil(tokens / 32)]")
    tokens = mask.shape[1]
    gpu, out, lse, workspace = _decode_outputs(q, tokens, out, lse, workspace, stream)
    _call(_latent().tree_decode, "skinny_latent_masked_decode_bf16", gpu, stream, q, cache, table, lens, scale, tokens,
          rope_dim, out, lse, workspace, mask, depth, window, sinks)
    return out, lse


def latent_window_decode(q, cache, table, lens, scale: float, window: int, sinks: int = 0, tokens: int = 1,
                         rope_dim: int = ROPE, out=None, lse=None, workspace=None, stream=None):
    """latent_decode with a sliding window (skinny_latent_masked_decode_bf16): a token at position p
    (its own key among those it sees) sees the last `window` keys, k > p - window, and the first `sinks`,
    k < sinks. Keys that no row of a request sees are not read. The rest as in latent_decode. Returns
    (out, lse)."""
    gpu, out, lse, workspace = _decode_outputs(q, tokens, out, lse, workspace, stream)
    _call(_latent().window_decode, "skinny_latent_masked_decode_bf16", gpu, stream, q, cache, table, lens, scale, tokens,
          rope_dim, out, lse, workspace, window, sinks)
    return out, lse


def latent_window_prefill_workspace(nq: int, nk: int, batch: int, heads: int, window: int, sinks: int = 0,
                                    device="cuda") -> torch.Tensor:
    """Device memory for the partial sums of a latent_window_prefill call of these sizes (may be empty)."""
    return _workspace(lib().skinny_latent_window_prefill_workspace, "skinny_latent_window_prefill_workspace", device, nq,
                      nk, batch, heads, window, sinks)


def latent_window_prefill(q, k, v, k_rot, cu_q, cu_k, scale: float, window: int, sinks: int = 0, out=None, lse=None,
                          workspace=None, stream=None):
    """Causal latent_prefill with a sliding window (skinny_latent_window_prefill_bf16): a query at position p of
    its sequence sees keys k <= p with k > p - window or k < sinks. The rest as in latent_prefill;
    workspace: latent_window_prefill_workspace(nq, nk, batch, heads, window, sinks). Returns (out, lse)."""
    _whole("window", window, 1)
    _whole("sinks", sinks, 0)
    gpu, out, lse, workspace = _prefill_outputs(q, k, cu_q, out, lse, workspace, stream,
                                                lib().skinny_latent_window_prefill_workspace,
                                                "skinny_latent_window_prefill_workspace", window, sinks)
    _call(_latent().window_prefill, "skinny_latent_window_prefill_bf16", gpu, stream, q, k, v, k_rot, cu_q, cu_k, scale,
          True, out, lse, workspace, window, sinks)
    return out, lse


def latent_key_weights(q, cache, table, lens, lse, weights, scale: float, tokens: int = 1, rope_dim: int = ROPE,
                       stream=None):
    """Adds to weights what latent_decode's softmax gave each key (skinny_latent_key_weights_bf16), in place.

    q, cache, table, lens, scale, tokens as in latent_decode, lse float32 [batch * tokens, heads] as it returned:
    weights float32 [batch, columns] (rows may lie apart) gets at [i, k] the sum over request i's rows
    that see key k of exp(scale * q . key - lse). Keys without a column are left out. The rows are a chain that sees all
    keys up to its own, `tokens` of every request: lse of latent_tree_decode or latent_window_decode gives no softmax
    weights here (take that of a latent_decode call of the rows that were accepted). With `tokens` the last ones
    of a prompt it tells which of the prompt's keys they look at. Returns weights."""
    gpu = _gpu_of("q", q)
    _call(_latent().key_weights, "skinny_latent_key_weights_bf16", gpu, stream, q, cache, table, lens, lse, weights, scale,
          tokens, rope_dim)
    return weights


def latent_select(weights, lens, budget: int, sinks: int = 0, recent: int = 0, kept=None, counts=None, stream=None):
    """Which keys of each request stay in the cache (skinny_latent_select).

    weights float32 [batch, columns], lens int32 [batch]. Of more than `budget` keys the first `sinks`, the last
    `recent` and the largest weights between them stay (of equal ones the first; a NaN is larger than any
    number; a key without a column, as latent_key_weights leaves out, has the weight 0); of fewer, all. Returns kept int32 [batch, budget], rising, -1 behind the last, and counts int32
    [batch], for latent_keep."""
    gpu = _gpu_of("weights", weights)
    if weights.dim() != 2:
        raise ValueError("weights must be a tensor [batch, columns]")
    _whole("budget", budget, 0)
    if kept is None:
        kept = _new((weights.shape[0], budget), torch.int32, weights.device, stream)
    if counts is None:
        counts = _new((weights.shape[0],), torch.int32, weights.device, stream)
    _call(_latent().select, "skinny_latent_select", gpu, stream, weights, lens, budget, sinks, recent, kept, counts)
    return kept, counts


def latent_keep(cache, table, lens, kept, counts, tokens: int = 0, weights=None, new_lens=None, new_weights=None,
                stream=None):
    """Moves the rows that stay in a paged latent cache together, in place (skinny_latent_keep_bf16).

    kept int32 [batch, most], rising, of which counts int32 [batch] count. With tokens 0 they are numbers of
    request i's lens[i] rows, and go to places 0, 1, ... (after latent_select). With tokens > 0 they count
    from the first of its newest `tokens` rows, all earlier rows stay, and they go to the places
    behind those: the accepted path of a tree. A number smaller than its place in the list, or of no row, leaves its new
    place's row as it is; rows behind the last kept one keep their numbers. The pages must be the request's own.
    weights float32 [batch, columns]: each key's, which go along into new_weights (0 behind the last). Returns
    (new_lens int32 [batch], new_weights or None); neither may be lens or weights itself."""
    gpu = _gpu_of("cache", cache)
    if new_lens is None:
        new_lens = _new(tuple(lens.shape) if isinstance(lens, torch.Tensor) else 0, torch.int32, cache.device, stream)
    if weights is not None and new_weights is None:
        new_weights = _new(tuple(weights.shape) if isinstance(weights, torch.Tensor) else 0, torch.float32, cache.device,
                           stream)
    _call(_latent().keep, "skinny_latent_keep_bf16", gpu, stream, cache, table, lens, kept, counts, tokens, new_lens, weights,
          new_weights)
    return new_lens, new_weights


def select_config(M: int, N: int = 7168, K: int = 3584) -> dict:
    c = SkinnyConfig()
    check(lib().skinny_select_config(M, N, K, ctypes.byref(c)), "skinny_select_config")
    return c.as_dict()


def configs() -> list[dict]:
    L = lib()
    out = []
    for i in range(L.skinny_num_configs()):
        c = SkinnyConfig()
        check(L.skinny_get_config(i, ctypes.byref(c)), "skinny_get_config")
        out.append(c.as_dict())
    return out


def config_resources(config) -> dict:
    c = _as_config(config)
    r = SkinnyResources()
    check(lib().skinny_config_resources(ctypes.byref(c), ctypes.byref(r)), "skinny_config_resources")
    return {f: int(getattr(r, f)) for f, _ in SkinnyResources._fields_}


def config_kernel(config) -> dict:
    """The kernel a plain call with this configuration launches at the tuned shape: its name as
    the HIP runtime reports it and the hash of its machine code in this build (kernel_code.json,
    written by the build); None for the hash when the build's map lacks the name."""
    import json
    import os
    c = _as_config(config)
    buf = ctypes.create_string_buffer(4096)
    check(lib().skinny_config_kernel_name(ctypes.byref(c), buf, len(buf)), "skinny_config_kernel_name")
    name = buf.value.decode()
    try:
        code = json.load(open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "kernel_code.json")))
    except (OSError, ValueError):
        code = {}
    return {"name": name, "code_sha256": code.get(name)}


def version() -> str:
    return lib().skinny_version().decode()
