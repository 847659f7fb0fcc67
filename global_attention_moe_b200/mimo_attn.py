"""Python binding of the C-ABI library ``libmimo_attn.so`` (include/mimo_attn.h).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the attention forward runs in the library's CUDA
kernels.  There is no CPU or eager fallback -- if the library is missing the
import of this module raises.
"""
from __future__ import annotations

import ctypes
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libmimo_attn.so")

LAYER_SWA = 0
LAYER_GLOBAL = 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_RANGE, ERR_BAD_SEQLENS, ERR_SCRATCH_LIMIT = range(8)

_BF16 = _F32 = _I32 = _raw_stream = None


def _use_torch():
    """Binds torch and what the entry points take from it to this module's names."""
    global torch, _BF16, _F32, _I32, _raw_stream
    import torch
    _BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
    # the current stream of a device as an integer: torch.cuda.current_stream() builds a Python stream object
    # (3.2 us of a 16 us call), this reads the handle (0.1 us); without it the object is built
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Torch:
    """Stands for torch until its first use: the raw-pointer entry points, the selections and the status calls
    work without it."""

    def __getattr__(self, name):
        _use_torch()
        return getattr(torch, name)


torch = _Torch()
if "torch" in sys.modules:
    _use_torch()

# Every symbol include/mimo_attn.h declares.
SYMBOLS = ("mimo_attn_fwd", "mimo_attn_host_workspace_size", "mimo_attn_fwd_host", "mimo_attn_check",
           "mimo_attn_selftest_wait_timeout", "mimo_attn_status_string", "mimo_attn_fwd_noalloc",
           "mimo_attn_noalloc_scratch_bytes", "mimo_attn_set_kernel", "mimo_attn_profile_start",
           "mimo_attn_profile_stop", "mimo_attn_profile_set_stride", "mimo_attn_decode", "mimo_attn_set_decode_kernel", "mimo_attn_version",
           "mimo_attn_bwd", "mimo_fp8_dequant_blockwise", "mimo_qkv_split", "mimo_moe_route",
           "mimo_linear_proj", "mimo_attn_set_bwd_kernel", "mimo_rms_norm", "mimo_rms_norm_bwd",
           "mimo_rms_norm_bwd_workspace_size", "mimo_moe_route_grouped", "mimo_moe_route_bwd",
           "mimo_decode_key_weights", "mimo_decode_key_weights_workspace_size", "mimo_kv_evict")
KERNEL_AUTO, KERNEL_SIMPLE, KERNEL_PIPELINED, KERNEL_WINDOW, KERNEL_WINDOW_PACKED = 0, 1, 2, 3, 4
DECODE_AUTO, DECODE_CUDA_CORES, DECODE_TENSOR = 0, 1, 2


class Dims(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32), ("max_seqlen", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim_qk", ctypes.c_int32), ("head_dim_v", ctypes.c_int32)]


class DecodeDims(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_kv", ctypes.c_int32),
                ("cache_rows", ctypes.c_int32), ("max_q_len", ctypes.c_int32), ("max_kv_len", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim_qk", ctypes.c_int32), ("head_dim_v", ctypes.c_int32)]


class MimoAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m global_attention_moe_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, D, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_float
    lib.mimo_attn_fwd.restype = I
    lib.mimo_attn_fwd.argtypes = [P, P, P, P, P, ctypes.POINTER(Dims), I, I, D, I, F, P, P, P]
    lib.mimo_attn_host_workspace_size.restype = ctypes.c_size_t
    lib.mimo_attn_host_workspace_size.argtypes = [ctypes.POINTER(Dims), I]
    lib.mimo_attn_fwd_host.restype = I
    lib.mimo_attn_fwd_host.argtypes = [P, P, P, P, P, ctypes.POINTER(Dims), I, I, D, I, F, P, P, P,
                                       ctypes.c_size_t, P]
    lib.mimo_attn_check.restype = I
    lib.mimo_attn_check.argtypes = [P]
    lib.mimo_attn_selftest_wait_timeout.restype = I
    lib.mimo_attn_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P]
    lib.mimo_attn_status_string.restype = ctypes.c_char_p
    lib.mimo_attn_status_string.argtypes = [I]
    lib.mimo_attn_fwd_noalloc.restype = I
    lib.mimo_attn_fwd_noalloc.argtypes = [P, P, P, P, P, ctypes.POINTER(Dims), I, I, D, I, F, P, P, P]
    lib.mimo_attn_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.mimo_attn_noalloc_scratch_bytes.argtypes = []
    lib.mimo_attn_profile_start.restype = I
    lib.mimo_attn_profile_start.argtypes = []
    lib.mimo_attn_profile_set_stride.restype = I
    lib.mimo_attn_profile_set_stride.argtypes = [I]
    lib.mimo_attn_profile_stop.restype = I
    lib.mimo_attn_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
    lib.mimo_attn_set_kernel.restype = I
    lib.mimo_attn_set_kernel.argtypes = [I]
    lib.mimo_attn_decode.restype = I
    lib.mimo_attn_decode.argtypes = [P, P, P, P, P, P, P, ctypes.POINTER(DecodeDims), I, I, D, I, F, P, P, P]
    lib.mimo_attn_bwd.restype = I
    lib.mimo_attn_bwd.argtypes = [P, P, P, P, P, ctypes.POINTER(Dims), I, I, D, I, F, P, P, P, P, P, P, P, P, P]
    L = ctypes.c_int64
    lib.mimo_fp8_dequant_blockwise.restype = I
    lib.mimo_fp8_dequant_blockwise.argtypes = [P, P, L, L, I, I, P, P]
    lib.mimo_qkv_split.restype = I
    lib.mimo_qkv_split.argtypes = [P, L, I, I, P, P, P, P]
    lib.mimo_attn_set_bwd_kernel.restype = I
    lib.mimo_attn_set_bwd_kernel.argtypes = [I]
    lib.mimo_linear_proj.restype = I
    lib.mimo_linear_proj.argtypes = [P, P, L, L, L, P, P]
    lib.mimo_moe_route.restype = I
    lib.mimo_moe_route.argtypes = [P, P, L, I, I, I, P, P, P]
    lib.mimo_rms_norm.restype = I
    lib.mimo_rms_norm.argtypes = [P, P, P, I, L, L, F, P, P, P, P, P]
    lib.mimo_rms_norm_bwd.restype = I
    lib.mimo_rms_norm_bwd.argtypes = [P, P, I, P, P, L, L, F, P, P, P, ctypes.c_size_t, P]
    lib.mimo_rms_norm_bwd_workspace_size.restype = ctypes.c_size_t
    lib.mimo_rms_norm_bwd_workspace_size.argtypes = [L, L]
    lib.mimo_moe_route_grouped.restype = I
    lib.mimo_moe_route_grouped.argtypes = [P, P, L, I, I, I, I, I, I, F, P, P, P]
    lib.mimo_moe_route_bwd.restype = I
    lib.mimo_moe_route_bwd.argtypes = [P, P, P, L, I, I, I, I, F, P, P]
    lib.mimo_decode_key_weights.restype = I
    lib.mimo_decode_key_weights.argtypes = [P, P, P, P, P, P, P, ctypes.POINTER(DecodeDims), I, I, D, I, P, P,
                                            ctypes.c_size_t, P]
    lib.mimo_decode_key_weights_workspace_size.restype = ctypes.c_size_t
    lib.mimo_decode_key_weights_workspace_size.argtypes = [ctypes.POINTER(DecodeDims)]
    lib.mimo_kv_evict.restype = I
    lib.mimo_kv_evict.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P, P, P]
    lib.mimo_attn_set_decode_kernel.restype = I
    lib.mimo_attn_set_decode_kernel.argtypes = [I]
    lib.mimo_attn_version.restype = I
    lib.mimo_attn_version.argtypes = []
    return lib


LIB = _load()


def status_string(status: int) -> str:
    return LIB.mimo_attn_status_string(int(status)).decode()


def version() -> tuple[int, int]:
    v = LIB.mimo_attn_version()
    return v >> 16, v & 0xFFFF


def set_kernel(choice: int) -> None:
    """Select the kernel mimo_attn_fwd launches (KERNEL_AUTO / _SIMPLE / _PIPELINED / _WINDOW / _WINDOW_PACKED)."""
    st = LIB.mimo_attn_set_kernel(int(choice))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_set_kernel")


def set_decode_kernel(choice: int) -> None:
    """Select the kernel mimo_attn_decode launches (DECODE_AUTO / _CUDA_CORES / _TENSOR)."""
    st = LIB.mimo_attn_set_decode_kernel(int(choice))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_set_decode_kernel")


def bwd(q, k, v, sink, cu_seqlens, max_seqlen, layer_kind, window, rope_base, out, lse, dout, dlse=None,
        rope_dims=64, v_scale=0.707, stream=None):
    """Gradients of the forward: q/k/v/out/dout bf16 CUDA tensors, lse / dlse fp32 [Hq, T] (dlse may be
    None).  Returns (dq fp32 [T, Hq, 192], dk fp32 [T, Hkv, 192], dv fp32 [T, Hkv, 128], dsink fp32 [Hq] or
    None)."""
    T, hq, dqk = q.shape
    hkv, dv_ = v.shape[1], v.shape[2]
    dq = torch.empty((T, hq, dqk), dtype=torch.float32, device=q.device)
    dk = torch.empty((T, hkv, dqk), dtype=torch.float32, device=q.device)
    dv = torch.empty((T, hkv, dv_), dtype=torch.float32, device=q.device)
    dsink = None if sink is None else torch.empty((hq,), dtype=torch.float32, device=q.device)
    dims = make_dims(cu_seqlens.numel() - 1, T, max_seqlen, hq, hkv)
    ptr = lambda t: None if t is None else t.data_ptr()
    st = LIB.mimo_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr(sink), cu_seqlens.data_ptr(),
                           ctypes.byref(dims), int(layer_kind), int(window), float(rope_base), int(rope_dims),
                           float(v_scale), out.data_ptr(), lse.data_ptr(), dout.data_ptr(), ptr(dlse),
                           dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ptr(dsink), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_bwd")
    return dq, dk, dv, dsink


def fp8_dequant_blockwise(codes, scale_inv, block=(128, 128), out=None, stream=None):
    """uint8 E4M3 codes [rows, cols] and fp32 scale_inv [ceil(rows/b0), ceil(cols/b1)] (CUDA) -> bf16."""
    rows, cols = codes.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=codes.device)
    st = LIB.mimo_fp8_dequant_blockwise(codes.data_ptr(), scale_inv.data_ptr(), rows, cols, int(block[0]),
                                        int(block[1]), out.data_ptr(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_fp8_dequant_blockwise")
    return out


def qkv_split(fused, num_q_heads, num_kv_heads, stream=None):
    """bf16 fused [T, Hkv * (Hq/Hkv*192 + 320)] (CUDA) -> q [T, Hq, 192], k [T, Hkv, 192], v [T, Hkv, 128]."""
    T = fused.shape[0]
    q = torch.empty((T, num_q_heads, 192), dtype=torch.bfloat16, device=fused.device)
    k = torch.empty((T, num_kv_heads, 192), dtype=torch.bfloat16, device=fused.device)
    v = torch.empty((T, num_kv_heads, 128), dtype=torch.bfloat16, device=fused.device)
    st = LIB.mimo_qkv_split(fused.data_ptr(), T, int(num_q_heads), int(num_kv_heads), q.data_ptr(), k.data_ptr(),
                            v.data_ptr(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_qkv_split")
    return q, k, v


BWD_AUTO, BWD_CUDA_CORES, BWD_TENSOR = 0, 1, 2


def set_bwd_kernel(choice: int) -> None:
    st = LIB.mimo_attn_set_bwd_kernel(int(choice))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_set_bwd_kernel")


def linear_proj(x, w, out=None, stream=None):
    """Output projection y = x . w^T: bf16 x [T, K] or the attention output [T, Hq, 128] (CUDA), bf16 w
    [N, K] (a Linear weight) -> bf16 y [T, N] (cuBLAS, FP32 accumulation)."""
    T = x.shape[0]
    feats = 1
    for d in x.shape[1:]:
        feats *= int(d)
    x2 = x.reshape(T, feats)  # explicit: reshape(T, -1) is ambiguous for zero tokens
    N, K = w.shape
    if x2.shape[1] != K:
        raise ValueError(f"x has {x2.shape[1]} features per token, w expects {K}")
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
    st = LIB.mimo_linear_proj(x2.data_ptr(), w.data_ptr(), T, K, N, out.data_ptr(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_linear_proj")
    return out


def moe_route(logits, bias, top_k=8, normalize=True, stream=None):
    """fp32 logits [T, E] and bias [E] (CUDA) -> ids int32 [T, top_k], weights fp32 [T, top_k]."""
    T, E = logits.shape
    ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    st = LIB.mimo_moe_route(logits.data_ptr(), bias.data_ptr(), T, int(E), int(top_k), int(bool(normalize)),
                            ids.data_ptr(), w.data_ptr(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_moe_route")
    return ids, w


def profile_start() -> None:
    """Record the attention kernel's duration on every following forward (see profile_stop)."""
    LIB.mimo_attn_profile_start()


def profile_set_stride(stride: int) -> None:
    """Record only every stride-th attention-kernel launch while profiling (1: every launch)."""
    st = LIB.mimo_attn_profile_set_stride(stride)
    if st != OK:
        raise MimoAttnError(st, "profile_set_stride")


def profile_stop() -> tuple[int, float]:
    """Stop recording; returns (attention-kernel launches, their summed milliseconds)."""
    n, ms = ctypes.c_int(0), ctypes.c_double(0.0)
    st = LIB.mimo_attn_profile_stop(ctypes.byref(n), ctypes.byref(ms))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_profile_stop")
    return n.value, ms.value


def make_dims(num_seqs, total_tokens, max_seqlen, hq, hkv, dqk=192, dv=128) -> Dims:
    return Dims(int(num_seqs), int(total_tokens), int(max_seqlen), int(hq), int(hkv), int(dqk), int(dv))


def _stream_handle(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def fwd_raw(q_ptr, k_ptr, v_ptr, sink_ptr, cu_ptr, dims: Dims, layer_kind, window, rope_base, rope_dims, v_scale,
            out_ptr, lse_ptr, stream_handle) -> int:
    """Direct C-ABI call with integer device pointers; returns the status code."""
    return LIB.mimo_attn_fwd(q_ptr, k_ptr, v_ptr, sink_ptr, cu_ptr, ctypes.byref(dims), int(layer_kind),
                             int(window), float(rope_base), int(rope_dims), float(v_scale), out_ptr, lse_ptr,
                             stream_handle)


def fwd(q, k, v, sink, cu_seqlens, max_seqlen, layer_kind, window, rope_base, rope_dims=64, v_scale=0.707,
        out=None, lse=None, stream=None):
    """Attention forward on CUDA tensors (bf16 q/k/v in THD layout, int32 cu_seqlens,
    fp32 sink or None).  Returns (out bf16 [T, Hq, 128], lse fp32 [Hq, T])."""
    T, hq, dqk = q.shape
    hkv, dv = k.shape[1], v.shape[2]
    for t in (q, k, v):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("q/k/v must be contiguous bf16 CUDA tensors")
    if out is None:
        out = torch.empty((T, hq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    dims = make_dims(cu_seqlens.numel() - 1, T, max_seqlen, hq, hkv, dqk, dv)
    st = fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), sink.data_ptr() if sink is not None else None,
                 cu_seqlens.data_ptr(), dims, layer_kind, window, rope_base, rope_dims, v_scale, out.data_ptr(),
                 lse.data_ptr(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_fwd")
    return out, lse


def fwd_noalloc(q, k, v, sink, cu_seqlens, max_seqlen, layer_kind, window, rope_base, out, lse, rope_dims=64,
                v_scale=0.707, stream=None):
    """Same as fwd() through mimo_attn_fwd_noalloc: for callers that cannot allocate
    device memory during the call (the caller passes out and lse; the library's
    scratch is a fixed array of noalloc_scratch_bytes())."""
    dims = make_dims(cu_seqlens.numel() - 1, q.shape[0], max_seqlen, q.shape[1], k.shape[1], q.shape[2], v.shape[2])
    st = LIB.mimo_attn_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   sink.data_ptr() if sink is not None else None, cu_seqlens.data_ptr(),
                                   ctypes.byref(dims), int(layer_kind), int(window), float(rope_base),
                                   int(rope_dims), float(v_scale), out.data_ptr(), lse.data_ptr(),
                                   _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_fwd_noalloc")
    return out, lse


def noalloc_scratch_bytes() -> int:
    return LIB.mimo_attn_noalloc_scratch_bytes()


def host_workspace_size(dims: Dims, has_sink: bool) -> int:
    return LIB.mimo_attn_host_workspace_size(ctypes.byref(dims), int(bool(has_sink)))


def fwd_host(q_host, k_host, v_host, sink_host, cu_host, dims: Dims, layer_kind, window, rope_base, rope_dims,
             v_scale, out_host, lse_host, workspace, stream=None):
    """End-to-end call from (pinned) host tensors through a caller-provided device workspace."""
    st = LIB.mimo_attn_fwd_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                sink_host.data_ptr() if sink_host is not None else None, cu_host.data_ptr(),
                                ctypes.byref(dims), int(layer_kind), int(window), float(rope_base), int(rope_dims),
                                float(v_scale), out_host.data_ptr(), lse_host.data_ptr(), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_fwd_host")


def check(stream=None) -> int:
    """Sync the stream and return (and clear) the device error status."""
    return LIB.mimo_attn_check(_stream_handle(stream))


def selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return LIB.mimo_attn_selftest_wait_timeout(int(limit_ns), _stream_handle(stream))


def make_decode_dims(num_seqs, total_q, total_kv, cache_rows, max_q_len, max_kv_len, hq, hkv, dqk=192,
                     dv=128) -> DecodeDims:
    return DecodeDims(int(num_seqs), int(total_q), int(total_kv), int(cache_rows), int(max_q_len),
                      int(max_kv_len), int(hq), int(hkv), int(dqk), int(dv))


def decode_raw(q_ptr, kc_ptr, vc_ptr, idx_ptr, indptr_ptr, cuq_ptr, sink_ptr, dims: DecodeDims, layer_kind, window,
               rope_base, rope_dims, v_scale, out_ptr, lse_ptr, stream_handle) -> int:
    """Direct C-ABI call of mimo_attn_decode with integer device pointers; returns the status code."""
    return LIB.mimo_attn_decode(q_ptr, kc_ptr, vc_ptr, idx_ptr, indptr_ptr, cuq_ptr, sink_ptr, ctypes.byref(dims),
                                int(layer_kind), int(window), float(rope_base), int(rope_dims), float(v_scale),
                                out_ptr, lse_ptr, stream_handle)


def decode(q, k_cache, v_cache, kv_indices, kv_indptr, cu_q, sink, max_q_len, max_kv_len, layer_kind, window,
           rope_base, rope_dims=64, v_scale=0.707, out=None, lse=None, stream=None):
    """New query tokens against a page-size-1 KV cache (CUDA tensors: bf16 q [Tq, Hq, 192], bf16 caches
    [rows, Hkv, 192] / [rows, Hkv, 128], int32 kv_indices / kv_indptr / cu_q, fp32 sink or None).
    Returns (out bf16 [Tq, Hq, 128], lse fp32 [Hq, Tq])."""
    Tq, hq, dqk = q.shape
    rows, hkv, dv = v_cache.shape
    for t in (q, k_cache, v_cache):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("q and the caches must be contiguous bf16 CUDA tensors")
    if out is None:
        out = torch.empty((Tq, hq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((hq, Tq), dtype=torch.float32, device=q.device)
    dims = make_decode_dims(cu_q.numel() - 1, Tq, kv_indices.numel(), rows, max_q_len, max_kv_len, hq, hkv, dqk, dv)
    st = decode_raw(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kv_indices.data_ptr(),
                    kv_indptr.data_ptr(), cu_q.data_ptr(), sink.data_ptr() if sink is not None else None, dims,
                    layer_kind, window, rope_base, rope_dims, v_scale, out.data_ptr(), lse.data_ptr(),
                    _stream_handle(stream))
    if st != OK:
        raise MimoAttnError(st, "mimo_attn_decode")
    return out, lse


def _refuse(name, t, dtype, shape, dev):
    dt = " or ".join(map(str, dtype)) if isinstance(dtype, tuple) else str(dtype)
    raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {tuple(shape)} on the current device cuda:{dev}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _check(name, t, dtype, shape, dev):
    """Contiguous CUDA tensors of the current device only: kernels are launched there, and rows are read as one
    dense block."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, dtype, shape, dev)


def _int32(*numbers):
    """Of a larger number ctypes would pass the low 32 bits.  Called where the numbers' bits, joined by `or`, are not
    all below 2^31 (which costs a call less than their maximum and minimum)."""
    if max(numbers) > 0x7FFFFFFF or min(numbers) < -0x80000000:
        raise ValueError(f"a size or choice beyond 32 bits among {numbers}")


def _norm_checks(x, name, weight):
    if x.dim() != 2:
        raise ValueError(f"{name} must be [tokens, features], got {tuple(x.shape)}")
    dev = torch.cuda.current_device()
    _check(name, x, _BF16, x.shape, dev)
    w32 = weight.dtype is _F32
    if not w32 and weight.dtype is not _BF16:
        _refuse("weight", weight, (_BF16, _F32), x.shape[1:], dev)
    _check("weight", weight, weight.dtype, x.shape[1:], dev)
    return dev, w32


# With a stream of the caller's, outputs and workspaces are allocated on that stream too (the calls below run
# again under it): memory that another stream still uses is never handed out.
def rms_norm(x, weight, residual=None, eps=1e-6, stream=None):
    """RMS norm of x (+ residual): bf16 x / residual [T, H] (CUDA), weight [H] bf16 or fp32.  Returns (y bf16
    [T, H], h bf16 [T, H]); h = bf16(x + residual) is the new residual stream (x itself without a residual)."""
    dev, w32 = _norm_checks(x, "x", weight)
    if residual is not None:
        _check("residual", residual, _BF16, x.shape, dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm(x, weight, residual, eps)
    T, H = x.shape
    y = torch.empty_like(x)
    h = x if residual is None else torch.empty_like(x)
    st = LIB.mimo_rms_norm(x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), w32, T, H,
                           eps, None if residual is None else h.data_ptr(), y.data_ptr(), None, None,
                           _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_rms_norm")
    return y, h


def rms_norm_fp8(x, weight, residual=None, eps=1e-6, with_bf16=False, stream=None):
    """The same with y as E4M3 bytes and one scale per 1 x 128 block (fp8_dequant_blockwise(codes, scale_inv,
    (1, 128)) gives it back).  Returns (codes uint8 [T, H], scale_inv fp32 [T, ceil(H/128)], h), and y in bf16
    as a fourth with with_bf16."""
    dev, w32 = _norm_checks(x, "x", weight)
    if residual is not None:
        _check("residual", residual, _BF16, x.shape, dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm_fp8(x, weight, residual, eps, with_bf16)
    T, H = x.shape
    codes = torch.empty_like(x, dtype=torch.uint8)
    scale = x.new_empty((T, (H + 127) // 128), dtype=_F32)
    h = x if residual is None else torch.empty_like(x)
    y = torch.empty_like(x) if with_bf16 else None
    st = LIB.mimo_rms_norm(x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), w32, T, H,
                           eps, None if residual is None else h.data_ptr(), y.data_ptr() if with_bf16 else None,
                           codes.data_ptr(), scale.data_ptr(), _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_rms_norm")
    return (codes, scale, h, y) if with_bf16 else (codes, scale, h)


def rms_norm_bwd(h, weight, dy, dh=None, eps=1e-6, stream=None):
    """Gradients of rms_norm: h as it returned it (bf16 [T, H]), dy = dL/dy and dh = dL/dh by h's other uses
    (None: 0), bf16.  Returns (dx bf16 [T, H], the gradient of x and of the residual; dweight fp32 [H])."""
    dev, w32 = _norm_checks(h, "h", weight)
    _check("dy", dy, _BF16, h.shape, dev)
    if dh is not None:
        _check("dh", dh, _BF16, h.shape, dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm_bwd(h, weight, dy, dh, eps)
    T, H = h.shape
    nbytes = LIB.mimo_rms_norm_bwd_workspace_size(T, H)
    dx = torch.empty_like(h)
    dw = torch.empty_like(weight, dtype=_F32)
    ws = h.new_empty((nbytes,), dtype=torch.uint8)
    st = LIB.mimo_rms_norm_bwd(h.data_ptr(), weight.data_ptr(), w32, dy.data_ptr(),
                               None if dh is None else dh.data_ptr(), T, H, eps, dx.data_ptr(), dw.data_ptr(),
                               ws.data_ptr(), nbytes, _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_rms_norm_bwd")
    return dx, dw


ROUTE_SIGMOID, ROUTE_SOFTMAX = 0, 1


def moe_route_grouped(logits, bias=None, top_k=8, num_groups=1, top_groups=1, score=ROUTE_SIGMOID, normalize=True,
                      scale=1.0, stream=None):
    """Routing with sigmoid or softmax scores, limited to the top_groups best of num_groups expert groups (a
    group's score: the sum of its two largest score + bias).  fp32 logits [T, E] and bias [E] or None (CUDA) ->
    ids int32 [T, top_k], weights fp32 [T, top_k] (scale times the scores, normalised to sum to one first)."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens, experts], got {tuple(logits.shape)}")
    T, E = logits.shape
    if (E | top_k | num_groups | top_groups | score) >> 31:
        _int32(E, top_k, num_groups, top_groups, score)
    dev = torch.cuda.current_device()
    _check("logits", logits, _F32, logits.shape, dev)
    if bias is not None:
        _check("bias", bias, _F32, logits.shape[1:], dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_route_grouped(logits, bias, top_k, num_groups, top_groups, score, normalize, scale)
    w = logits.new_empty((T, top_k if top_k > 0 else 0))
    ids = torch.empty_like(w, dtype=_I32)
    st = LIB.mimo_moe_route_grouped(logits.data_ptr(), None if bias is None else bias.data_ptr(), T, E, top_k,
                                    num_groups, top_groups, score, bool(normalize), scale, ids.data_ptr(),
                                    w.data_ptr(), _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_moe_route_grouped")
    return ids, w


def moe_route_bwd(logits, ids, dweights, score=ROUTE_SIGMOID, normalize=True, scale=1.0, stream=None):
    """Gradient of moe_route_grouped's weights (or, with the defaults, moe_route's) with respect to the logits:
    fp32 logits [T, E], int32 ids and fp32 dweights [T, top_k] (CUDA) -> dlogits fp32 [T, E].  An id outside
    [0, E) is an empty place."""
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError(f"logits and ids must be [tokens, ...], got {tuple(logits.shape)} and {tuple(ids.shape)}")
    T, E = logits.shape
    k = ids.shape[1]
    if (E | k | score) >> 31:
        _int32(E, k, score)
    dev = torch.cuda.current_device()
    _check("logits", logits, _F32, logits.shape, dev)
    _check("ids", ids, _I32, (T, k), dev)
    _check("dweights", dweights, _F32, (T, k), dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_route_bwd(logits, ids, dweights, score, normalize, scale)
    d = torch.empty_like(logits)
    st = LIB.mimo_moe_route_bwd(logits.data_ptr(), ids.data_ptr(), dweights.data_ptr(), T, E, k, score,
                                bool(normalize), scale, d.data_ptr(), _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_moe_route_bwd")
    return d


def decode_key_weights(q, k_cache, kv_indices, kv_indptr, cu_q, lse, max_q_len, max_kv_len, layer_kind, window,
                       rope_base, rope_dims=64, prev=None, out=None, stream=None):
    """Attention weight each cached key receives from a decode() step's new queries, summed over the query heads
    and the sequence's queries: arguments as decode (lse fp32 [Hq, Tq] as it returned it), prev fp32 [total_kv]
    or None is added.  Returns fp32 [total_kv], beside kv_indices (out, which may be prev, if given)."""
    if q.dim() != 3 or k_cache.dim() != 3 or kv_indices.dim() != 1 or cu_q.dim() != 1:
        raise ValueError(f"q and k_cache must be [rows, heads, 192] and the index lists flat, got {tuple(q.shape)}, "
                         f"{tuple(k_cache.shape)}, {tuple(kv_indices.shape)}, {tuple(cu_q.shape)}")
    Tq, hq, dqk = q.shape
    rows, hkv, _ = k_cache.shape
    total, B1 = kv_indices.shape[0], cu_q.shape[0]
    if (Tq | rows | total | B1 | max_q_len | max_kv_len | layer_kind | window + 1 | rope_dims) >> 31:
        _int32(Tq, rows, total, B1, max_q_len, max_kv_len, layer_kind, window, rope_dims)
    dev = torch.cuda.current_device()
    _check("q", q, _BF16, q.shape, dev)
    _check("k_cache", k_cache, _BF16, (rows, hkv, dqk), dev)
    _check("kv_indices", kv_indices, _I32, (total,), dev)
    _check("kv_indptr", kv_indptr, _I32, (B1,), dev)
    _check("cu_q", cu_q, _I32, (B1,), dev)
    _check("lse", lse, _F32, (hq, Tq), dev)
    for name, t in (("prev", prev), ("out", out)):
        if t is not None:
            _check(name, t, _F32, (total,), dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return decode_key_weights(q, k_cache, kv_indices, kv_indptr, cu_q, lse, max_q_len, max_kv_len, layer_kind,
                                      window, rope_base, rope_dims, prev, out)
    dims = DecodeDims(B1 - 1, Tq, total, rows, max_q_len, max_kv_len, hq, hkv, dqk, 128)
    ref = ctypes.byref(dims)
    nbytes = LIB.mimo_decode_key_weights_workspace_size(ref)
    if out is None:
        out = lse.new_empty((total,))
    ws = lse.new_empty((nbytes,), dtype=torch.uint8)
    st = LIB.mimo_decode_key_weights(q.data_ptr(), k_cache.data_ptr(), kv_indices.data_ptr(), kv_indptr.data_ptr(),
                                     cu_q.data_ptr(), lse.data_ptr(), None if prev is None else prev.data_ptr(), ref,
                                     layer_kind, window, rope_base, rope_dims, out.data_ptr(), ws.data_ptr(), nbytes,
                                     _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_decode_key_weights")
    return out


def kv_evict(weights, kv_indices, kv_indptr, max_kv_len, budget, keep_first=0, keep_recent=0, stream=None):
    """Eviction by accumulated attention weight: of each sequence longer than budget, the first keep_first, the
    last keep_recent and the heaviest of the rest stay.  fp32 weights and int32 kv_indices [total_kv], int32
    kv_indptr [B + 1] (CUDA).  Returns (new_indices, new_weights, new_indptr, freed): buffers of total_kv entries
    of which the first new_indptr[B] (freed: the first kv_indptr[B] - new_indptr[B]) are written."""
    if kv_indices.dim() != 1 or kv_indptr.dim() != 1:
        raise ValueError(f"the index lists must be flat, got {tuple(kv_indices.shape)} and {tuple(kv_indptr.shape)}")
    total, B1 = kv_indices.shape[0], kv_indptr.shape[0]
    if (total | B1 | max_kv_len) >> 31:
        _int32(total, B1, max_kv_len)
    dev = torch.cuda.current_device()
    _check("weights", weights, _F32, (total,), dev)
    _check("kv_indices", kv_indices, _I32, (total,), dev)
    _check("kv_indptr", kv_indptr, _I32, (B1,), dev)
    if stream is not None:
        with torch.cuda.stream(stream):
            return kv_evict(weights, kv_indices, kv_indptr, max_kv_len, budget, keep_first, keep_recent)
    # no sequence is longer than an int32, and what does not fit one is not to wrap
    budget, keep_first, keep_recent = (max(-1, min(n, 0x7FFFFFFF)) for n in (budget, keep_first, keep_recent))
    idx, freed = torch.empty_like(kv_indices), torch.empty_like(kv_indices)
    w, ptr = torch.empty_like(weights), torch.empty_like(kv_indptr)
    st = LIB.mimo_kv_evict(weights.data_ptr(), kv_indices.data_ptr(), kv_indptr.data_ptr(), B1 - 1, total, max_kv_len,
                           budget, keep_first, keep_recent, idx.data_ptr(), w.data_ptr(), ptr.data_ptr(),
                           freed.data_ptr(), _stream_handle(None))
    if st != OK:
        raise MimoAttnError(st, "mimo_kv_evict")
    return idx, w, ptr, freed
