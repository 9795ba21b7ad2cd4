"""Python binding of the C ABI in ``include/flint_attn.h`` (ctypes).

Argument marshalling only: tensors are allocated with torch on the current CUDA
device and passed as raw device pointers together with torch's current stream.
Every step of the computation runs in the library's CUDA kernels. There is no
CPU or PyTorch fallback: if the library is missing or a call fails, an error is
raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflint_attn.so")

FLINT_BF16 = 0
FLINT_FP32 = 1
CACHE_BF16 = 0
CACHE_E4M3 = 1

STATUS = {0: "FLINT_OK", 1: "FLINT_ERR_INVALID_ARG", 2: "FLINT_ERR_UNSUPPORTED",
          3: "FLINT_ERR_WORKSPACE", 4: "FLINT_ERR_CUDA", 5: "FLINT_ERR_TIMEOUT"}

EXPORTED = ["flint_attn_workspace_bytes", "flint_attn_fwd", "flint_attn_bwd",
            "flint_attn_check_status", "flint_status_string", "flint_attn_version",
            "flint_attn_profile_enable", "flint_attn_profile_collect",
            "flint_attn_profile_reset", "flint_attn_launch_count",
            "flint_attn_bwd_preprocess_static", "flint_attn_exp2_poly",
            "flint_attn_decode_workspace_bytes", "flint_attn_decode",
            "flint_attn_fwd_padded", "flint_attn_bwd_padded", "flint_attn_selftest_wait",
            "flint_attn_paged_append", "flint_attn_decode_paged_workspace_bytes",
            "flint_attn_decode_paged"]


class Params(ctypes.Structure):
    """Mirror of ``flint_attn_params_t``."""
    _fields_ = [
        ("total_tokens", ctypes.c_int32),
        ("num_docs", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("use_rope", ctypes.c_int32),
        ("rope_theta", ctypes.c_float),
        ("rms_eps", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("fp32_out", ctypes.c_int32),
        ("compute_f16", ctypes.c_int32),
    ]


class DecodeParams(ctypes.Structure):
    """Mirror of ``flint_decode_params_t``."""
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("cache_capacity", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("use_rope", ctypes.c_int32),
        ("rope_theta", ctypes.c_float),
        ("rms_eps", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("fp32_out", ctypes.c_int32),
    ]


class PagedCacheDesc(ctypes.Structure):
    """Mirror of ``flint_paged_cache_t``."""
    _fields_ = [
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("cache_dtype", ctypes.c_int32),
        ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("table_stride", ctypes.c_int64),
    ]


class PagedAppendParams(ctypes.Structure):
    """Mirror of ``flint_paged_append_params_t``."""
    _fields_ = [
        ("cache", PagedCacheDesc),
        ("num_seqs", ctypes.c_int32),
        ("total_tokens", ctypes.c_int32),
        ("use_rope", ctypes.c_int32),
        ("rope_theta", ctypes.c_float),
        ("rms_eps", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
    ]


class DecodePagedParams(ctypes.Structure):
    """Mirror of ``flint_decode_paged_params_t``."""
    _fields_ = [
        ("cache", PagedCacheDesc),
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("use_rope", ctypes.c_int32),
        ("rope_theta", ctypes.c_float),
        ("rms_eps", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("fp32_out", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
    ]


# The same two structures as packed by a call: a third of the time of building a
# ctypes structure.
_PACK_APPEND = struct.Struct("@6i4q3i2fi2q").pack
_PACK_DECODE = struct.Struct("@6i4q4i3f3i3q").pack


class FlintError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load (once) and return the ctypes handle; raises if the library is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"CUDA library not built: {path} (run python -m "
                          "sink_aware_sliding_head_b200.build)")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(Params)
    lib.flint_attn_workspace_bytes.argtypes = [P, ctypes.c_int]
    lib.flint_attn_workspace_bytes.restype = sz
    lib.flint_attn_fwd.argtypes = [P] + [vp] * 9 + [vp, sz, vp]
    lib.flint_attn_fwd.restype = ctypes.c_int
    lib.flint_attn_bwd.argtypes = [P] + [vp] * 16 + [vp, sz, vp]
    lib.flint_attn_bwd.restype = ctypes.c_int
    lib.flint_attn_fwd_padded.argtypes = [P] + [vp] * 10 + [vp, sz, vp]
    lib.flint_attn_fwd_padded.restype = ctypes.c_int
    lib.flint_attn_bwd_padded.argtypes = [P] + [vp] * 17 + [vp, sz, vp]
    lib.flint_attn_bwd_padded.restype = ctypes.c_int
    lib.flint_attn_check_status.argtypes = [vp, vp]
    lib.flint_attn_check_status.restype = ctypes.c_int
    lib.flint_status_string.argtypes = [ctypes.c_int]
    lib.flint_status_string.restype = ctypes.c_char_p
    lib.flint_attn_version.argtypes = []
    lib.flint_attn_version.restype = ctypes.c_char_p
    lib.flint_attn_profile_enable.argtypes = [ctypes.c_int]
    lib.flint_attn_profile_enable.restype = None
    lib.flint_attn_profile_collect.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                               ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(ctypes.c_longlong)]
    lib.flint_attn_profile_collect.restype = ctypes.c_int
    lib.flint_attn_profile_reset.argtypes = []
    lib.flint_attn_profile_reset.restype = None
    lib.flint_attn_launch_count.argtypes = []
    lib.flint_attn_launch_count.restype = ctypes.c_longlong
    lib.flint_attn_bwd_preprocess_static.argtypes = [P] + [vp] * 6 + [vp]
    lib.flint_attn_bwd_preprocess_static.restype = ctypes.c_int
    lib.flint_attn_exp2_poly.argtypes = [vp, vp, ctypes.c_int32, vp]
    lib.flint_attn_exp2_poly.restype = ctypes.c_int
    lib.flint_attn_selftest_wait.argtypes = [ctypes.c_int64, ctypes.c_int32, vp, vp]
    lib.flint_attn_selftest_wait.restype = ctypes.c_int
    DP = ctypes.POINTER(DecodeParams)
    lib.flint_attn_decode_workspace_bytes.argtypes = [DP]
    lib.flint_attn_decode_workspace_bytes.restype = sz
    lib.flint_attn_decode.argtypes = [DP] + [vp] * 11 + [vp, sz, vp]
    lib.flint_attn_decode.restype = ctypes.c_int
    # (the params of the paged calls: a structure by reference, or its bytes)
    lib.flint_attn_paged_append.argtypes = [vp] * 13
    lib.flint_attn_paged_append.restype = ctypes.c_int
    lib.flint_attn_decode_paged_workspace_bytes.argtypes = [vp]
    lib.flint_attn_decode_paged_workspace_bytes.restype = sz
    lib.flint_attn_decode_paged.argtypes = [vp] * 16 + [sz, vp]
    lib.flint_attn_decode_paged.restype = ctypes.c_int
    _lib = lib
    return lib


def make_params(total_tokens, num_docs, num_q_heads, num_kv_heads, window, use_rope,
                rope_theta, dtype, head_dim=128, rms_eps=1e-6, softmax_scale=0.0,
                fp32_out=False, compute_f16=False) -> Params:
    return Params(int(total_tokens), int(num_docs), int(num_q_heads), int(num_kv_heads),
                  int(head_dim), int(window), 1 if use_rope else 0, float(rope_theta),
                  float(rms_eps), float(softmax_scale), int(dtype), 1 if fp32_out else 0,
                  1 if compute_f16 else 0)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FLINT_BF16
    if t.dtype == torch.float32:
        return FLINT_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream_ptr(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise FlintError(code, where)


def params_for(q, k, cu_doc_lens, window, use_rope, rope_theta, rms_eps=1e-6,
               softmax_scale=0.0, fp32_out=False, compute_f16=False) -> Params:
    T, H, D = q.shape
    return make_params(T, cu_doc_lens.numel() - 1, H, k.shape[1], window, use_rope, rope_theta,
                       _dtype_code(q), head_dim=D, rms_eps=rms_eps, softmax_scale=softmax_scale,
                       fp32_out=fp32_out, compute_f16=compute_f16)


def workspace_bytes(params: Params, backward: bool) -> int:
    return int(load_library().flint_attn_workspace_bytes(ctypes.byref(params), int(backward)))


def alloc_workspace(params: Params, backward: bool, device=None) -> torch.Tensor:
    n = workspace_bytes(params, backward)
    if n == 0:
        raise FlintError(1, "flint_attn_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def fwd(q, k, v, q_norm_w, k_norm_w, sink, cu_doc_lens, window, use_rope, rope_theta,
        rms_eps=1e-6, softmax_scale=0.0, out=None, lse=None, workspace=None, stream=None,
        check_status=False, fp32_out=False, valid_lens=None, compute_f16=False):
    """Forward through ``flint_attn_fwd``. Returns (out [T,H,D], lse [H,T] fp32).

    ``fp32_out``: out is float32 (pass it unchanged to ``bwd`` with the same flag).
    ``valid_lens``: int32 [num_docs] on the device, the real tokens at the start of
    each document (trailing padding; ``flint_attn_fwd_padded``).
    ``compute_f16`` (float32 inputs): the fp16 attention boundary; out is float16
    unless ``fp32_out``.
    """
    lib = load_library()
    p = params_for(q, k, cu_doc_lens, window, use_rope, rope_theta, rms_eps, softmax_scale,
                   fp32_out, compute_f16)
    T, H, D = q.shape
    if out is None:
        odt = torch.float32 if fp32_out else (torch.float16 if compute_f16 else q.dtype)
        out = torch.empty(q.shape, dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty(H, T, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(p, False, q.device)
    st = _stream_ptr(stream)
    if valid_lens is None:
        code = lib.flint_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(q_norm_w),
                                  _ptr(k_norm_w), _ptr(sink), _ptr(cu_doc_lens), _ptr(out),
                                  _ptr(lse), _ptr(workspace), workspace.numel(), st)
    else:
        code = lib.flint_attn_fwd_padded(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(q_norm_w), _ptr(k_norm_w), _ptr(sink),
                                         _ptr(cu_doc_lens), _ptr(valid_lens), _ptr(out),
                                         _ptr(lse), _ptr(workspace), workspace.numel(), st)
    _check(code, "flint_attn_fwd")
    if check_status:
        _check(lib.flint_attn_check_status(_ptr(workspace), st), "flint_attn_fwd (device)")
    return out, lse


def bwd(q, k, v, q_norm_w, k_norm_w, sink, cu_doc_lens, out, lse, dout, window, use_rope,
        rope_theta, rms_eps=1e-6, softmax_scale=0.0, grads=None, workspace=None, stream=None,
        check_status=False, fp32_out=False, valid_lens=None, compute_f16=False):
    """Backward through ``flint_attn_bwd`` (``flint_attn_bwd_padded`` with ``valid_lens``).

    Returns a dict with dq, dk, dv (input dtype, or float32 with ``fp32_out``),
    dw_q, dw_k, dsink (fp32). ``out`` must be the forward's result with the same
    ``fp32_out``.
    """
    lib = load_library()
    p = params_for(q, k, cu_doc_lens, window, use_rope, rope_theta, rms_eps, softmax_scale,
                   fp32_out, compute_f16)
    T, H, D = q.shape
    gdt = torch.float32 if (fp32_out or q.dtype == torch.float32) else q.dtype
    if grads is None:
        grads = {
            "dq": torch.empty(q.shape, dtype=gdt, device=q.device),
            "dk": torch.empty(k.shape, dtype=gdt, device=q.device),
            "dv": torch.empty(v.shape, dtype=gdt, device=q.device),
            "dw_q": torch.empty(D, dtype=torch.float32, device=q.device),
            "dw_k": torch.empty(D, dtype=torch.float32, device=q.device),
            "dsink": torch.empty(H, dtype=torch.float32, device=q.device),
        }
    if workspace is None:
        workspace = alloc_workspace(p, True, q.device)
    st = _stream_ptr(stream)
    g = [_ptr(grads[n]) for n in ("dq", "dk", "dv", "dw_q", "dw_k", "dsink")]
    if valid_lens is None:
        code = lib.flint_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(q_norm_w),
                                  _ptr(k_norm_w), _ptr(sink), _ptr(cu_doc_lens), _ptr(out),
                                  _ptr(lse), _ptr(dout), *g, _ptr(workspace), workspace.numel(),
                                  st)
    else:
        code = lib.flint_attn_bwd_padded(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(q_norm_w), _ptr(k_norm_w), _ptr(sink),
                                         _ptr(cu_doc_lens), _ptr(valid_lens), _ptr(out),
                                         _ptr(lse), _ptr(dout), *g, _ptr(workspace),
                                         workspace.numel(), st)
    _check(code, "flint_attn_bwd")
    if check_status:
        _check(lib.flint_attn_check_status(_ptr(workspace), st), "flint_attn_bwd (device)")
    return grads


def profile_enable(on: bool = True):
    """Bracket each later kernel launch with CUDA events on its stream."""
    load_library().flint_attn_profile_enable(1 if on else 0)


def profile_reset():
    load_library().flint_attn_profile_reset()


def profile_collect():
    """{kernel name: (total ms, launches)} over the launches timed so far."""
    lib = load_library()
    n = 32
    names = (ctypes.c_char_p * n)()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    k = lib.flint_attn_profile_collect(n, names, ms, cnt)
    return {names[i].decode(): (ms[i], cnt[i]) for i in range(min(k, n))}


def launch_count() -> int:
    """Kernels the library has launched since it was loaded."""
    return int(load_library().flint_attn_launch_count())


def bwd_preprocess_static(out, dout, lse, sink, d_rowsum=None, dsink=None, stream=None):
    """D = rowsum(dout * out) [H,T] and d_sink [H] through the no-allocation entry point.

    For callers that cannot allocate device memory where they run: the library
    uses a fixed scratch array of its own instead of a caller workspace (see
    ``flint_attn_bwd_preprocess_static`` in include/flint_attn.h for its limits).
    The input type is dout's (bfloat16 or float32); out's type says how the
    forward stored it: bfloat16 inputs take a bfloat16 or float32 out (fp32_out),
    float32 inputs a float32 out, or float16 for the fp16 compute boundary
    (compute_f16).
    """
    lib = load_library()
    if out.dim() != 3 or dout.shape != out.shape:
        raise ValueError(f"out {tuple(out.shape)} and dout {tuple(dout.shape)} must both be [T,H,D]")
    T, H, D = out.shape
    if lse.shape != (H, T) or lse.dtype != torch.float32:
        raise ValueError(f"lse must be float32 [H,T] = [{H},{T}], got {lse.dtype} {tuple(lse.shape)}")
    if sink.shape != (H,) or sink.dtype != torch.float32:
        raise ValueError(f"sink must be float32 [H] = [{H}], got {sink.dtype} {tuple(sink.shape)}")
    allowed = {torch.bfloat16: (torch.bfloat16, torch.float32),
               torch.float32: (torch.float32, torch.float16)}
    if dout.dtype not in allowed or out.dtype not in allowed[dout.dtype]:
        raise TypeError(f"unsupported pair: dout {dout.dtype}, out {out.dtype}")
    fp32_out = out.dtype == torch.float32
    compute_f16 = out.dtype == torch.float16
    p = make_params(T, 1, H, 1, 0, False, 0.0, _dtype_code(dout), head_dim=D,
                    fp32_out=fp32_out, compute_f16=compute_f16)
    if d_rowsum is None:
        d_rowsum = torch.empty(H, T, dtype=torch.float32, device=dout.device)
    if dsink is None:
        dsink = torch.empty(H, dtype=torch.float32, device=dout.device)
    code = lib.flint_attn_bwd_preprocess_static(ctypes.byref(p), _ptr(out), _ptr(dout), _ptr(lse),
                                                _ptr(sink), _ptr(d_rowsum), _ptr(dsink),
                                                _stream_ptr(stream))
    _check(code, "flint_attn_bwd_preprocess_static")
    return d_rowsum, dsink


def decode_params(batch, cache_capacity, num_q_heads, num_kv_heads, window, use_rope,
                  rope_theta, rms_eps=1e-6, softmax_scale=0.0, fp32_out=False,
                  head_dim=128) -> DecodeParams:
    return DecodeParams(int(batch), int(cache_capacity), int(num_q_heads), int(num_kv_heads),
                        int(head_dim), int(window), 1 if use_rope else 0, float(rope_theta),
                        float(rms_eps), float(softmax_scale), FLINT_BF16,
                        1 if fp32_out else 0)


def decode(q, k, v, q_norm_w, k_norm_w, sink, cache_lens, k_cache, v_cache, window, use_rope,
           rope_theta, rms_eps=1e-6, softmax_scale=0.0, out=None, lse=None, workspace=None,
           stream=None, check_status=False, fp32_out=False):
    """One new token per sequence through ``flint_attn_decode``.

    q [B,H,D], k, v [B,Hk,D] bf16 (raw projections of the new tokens); cache_lens
    [B] int32 on the device; k_cache, v_cache [B,Hk,C,D] bf16, updated in place
    at slot cache_lens[b]. Returns (out [B,H,D], lse [B,H] fp32).
    """
    lib = load_library()
    B, H, D = q.shape
    Hk, C = k_cache.shape[1], k_cache.shape[2]
    p = decode_params(B, C, H, Hk, window, use_rope, rope_theta, rms_eps, softmax_scale,
                      fp32_out, D)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if fp32_out else q.dtype,
                          device=q.device)
    if lse is None:
        lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    if workspace is None:
        n = lib.flint_attn_decode_workspace_bytes(ctypes.byref(p))
        if n == 0:
            raise FlintError(1, "flint_attn_decode_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    st = _stream_ptr(stream)
    code = lib.flint_attn_decode(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(q_norm_w),
                                 _ptr(k_norm_w), _ptr(sink), _ptr(cache_lens), _ptr(k_cache),
                                 _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(workspace),
                                 workspace.numel(), st)
    _check(code, "flint_attn_decode")
    if check_status:
        _check(lib.flint_attn_check_status(_ptr(workspace), st), "flint_attn_decode (device)")
    return out, lse


# ---------------------------------------------------------------- paged KV cache
# A pool may be head-major [pages, Hk, P, D] or any strided view of that shape
# (a token-major pool transposed, one half of an interleaved K/V pool).

# (A call's checks run on the host every time: they are written to take as few
# tensor attributes as they can.)

def _same_device(index, names, tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            where = ", ".join(f"{n} on {x.device}" for n, x in zip(names.split(), tensors)
                              if x is not None)
            raise ValueError(f"the tensors must be on one CUDA device: {where}")


def _vector(t, name, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)}")


def _rows(t, name, n, heads, D):
    """Row stride of a bf16 [n, heads, D] tensor whose rows are contiguous."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.shape != (n, heads, D):
        raise ValueError(f"{name} must be [{n}, {heads}, {D}], got {list(t.shape)}")
    row, head, channel = t.stride()
    if (channel != 1 and D > 1) or (head != D and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous, got strides {t.stride()}")
    if n <= 1:
        return 0
    if row < heads * D:                          # 0 would mean "contiguous" to the library
        raise ValueError(f"{name}: rows must not overlap, got strides {t.stride()}")
    return row


def _pool_strides(t):
    # the stride of an axis of length 1 is never used and may be anything
    D = t.shape[3]
    return tuple(D if n == 1 else st for n, st in zip(t.shape[:3], t.stride())) + t.stride()[3:]


def _paged_cache(k_pages, v_pages, block_table, rows, k_scale, v_scale):
    """The fields of ``flint_paged_cache_t``, in order."""
    shape, dtype = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype is not dtype:
        raise ValueError("k_pages and v_pages must be [pages, Hk, page_size, D] of one type, got "
                         f"{k_pages.dtype} {list(k_pages.shape)} and {v_pages.dtype} "
                         f"{list(v_pages.shape)}")
    n, Hk, P, D = shape
    if dtype is torch.bfloat16:
        code = CACHE_BF16
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn caches")
    elif dtype is torch.float8_e4m3fn:
        code = CACHE_E4M3
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _vector(t, name, torch.float32, (Hk,))
    else:
        raise TypeError(f"unsupported cache dtype {dtype}")
    strides = k_pages.stride()
    if strides != v_pages.stride() or n == 1 or Hk == 1 or P == 1:
        strides = _pool_strides(k_pages)
        if strides != _pool_strides(v_pages):
            raise ValueError(f"k_pages and v_pages have different strides: {k_pages.stride()} and "
                             f"{v_pages.stride()}")
    page, head, slot, channel = strides
    if page < D or head < D or slot < D or channel != 1:
        raise ValueError(f"slots must be {D} contiguous channels and not overlap, got strides "
                         f"{k_pages.stride()}")
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != rows or block_table.dtype is not torch.int32:
        raise ValueError(f"block_table must be int32 [{rows}, max_pages], got {block_table.dtype} "
                         f"{list(shape)}")
    cols = shape[1]
    row, col = block_table.stride()
    if (col != 1 and cols > 1) or (row < cols and rows > 1):
        raise ValueError("block_table: the entries of a row must be contiguous and rows not "
                         f"overlap, got strides {block_table.stride()}")
    return n, P, cols, Hk, D, code, page, head, slot, row if rows > 1 else 0


def _addr(t):
    return None if t is None else t.data_ptr()


# the handle of a device's current stream, without a Stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(index, stream):
    """The context in which a call's allocations belong to its stream (or None where they
    do already), and the stream's handle."""
    if index < 0:
        raise ValueError("CUDA tensors expected")
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on "
                             f"cuda:{index}")
        return torch.cuda.stream(stream), stream.cuda_stream
    if index != torch.cuda.current_device():
        return torch.cuda.device(index), _raw_stream(index)
    return None, _raw_stream(index)


def paged_append(k, v, k_norm_w, cu_new_lens, cache_lens, block_table, k_pages, v_pages, use_rope,
                 rope_theta, rms_eps=1e-6, k_scale=None, v_scale=None, status=None, stream=None,
                 check_status=False):
    """New tokens' keys and values into a paged cache, through ``flint_attn_paged_append``.

    k, v [T,Hk,D] bf16 (raw projections; row stride free): rows cu_new_lens[b] ..
    cu_new_lens[b+1] belong to sequence b and get positions cache_lens[b], ...;
    keys are normalised and (``use_rope``) rotated on the way. cu_new_lens [N+1],
    cache_lens [N] and block_table [N, max_pages] are int32 on the device; a
    cache_lens of -1 leaves the sequence alone. k_pages, v_pages [pages, Hk,
    page_size, D] bf16 or float8_e4m3fn (with per-head float32 scales [Hk]) are
    written in place, whatever their page, head and token strides. ``status``: int32
    [64] zeroed once by the caller, where device-side errors collect (a fresh one if
    omitted); ``check_status`` synchronises and raises ``FlintError`` for them.
    """
    N, T = cache_lens.numel(), k.shape[0]
    desc = _paged_cache(k_pages, v_pages, block_table, N, k_scale, v_scale)
    Hk, D = desc[3], desc[4]
    params = _PACK_APPEND(*desc, N, T, 1 if use_rope else 0, rope_theta, rms_eps, FLINT_BF16,
                          _rows(k, "k", T, Hk, D), _rows(v, "v", T, Hk, D))
    _vector(k_norm_w, "k_norm_w", torch.bfloat16, (D,))
    _vector(cache_lens, "cache_lens", torch.int32, (N,))
    _vector(cu_new_lens, "cu_new_lens", torch.int32, (N + 1,))
    if status is not None:
        _vector(status, "status", torch.int32, (64,))
    index = k_pages.get_device()
    _same_device(index, "k v k_norm_w cu_new_lens cache_lens block_table k_pages v_pages k_scale "
                 "v_scale status", (k, v, k_norm_w, cu_new_lens, cache_lens, block_table, k_pages,
                                    v_pages, k_scale, v_scale, status))
    where, handle = _elsewhere(index, stream)
    if where is not None:
        with where:
            return _launch_append(params, k, v, k_norm_w, cu_new_lens, cache_lens, block_table,
                                  k_pages, v_pages, k_scale, v_scale, status, handle, check_status)
    return _launch_append(params, k, v, k_norm_w, cu_new_lens, cache_lens, block_table, k_pages,
                          v_pages, k_scale, v_scale, status, handle, check_status)


def _launch_append(params, k, v, k_norm_w, cu_new_lens, cache_lens, block_table, k_pages, v_pages,
                   k_scale, v_scale, status, handle, check_status):
    lib = load_library()
    if status is None:
        status = torch.zeros(64, dtype=torch.int32, device=k_pages.device)
    code = lib.flint_attn_paged_append(
        params, k.data_ptr(), v.data_ptr(), k_norm_w.data_ptr(), cu_new_lens.data_ptr(),
        cache_lens.data_ptr(), block_table.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        _addr(k_scale), _addr(v_scale), status.data_ptr(), handle)
    if code:
        raise FlintError(code, "flint_attn_paged_append")
    if check_status:
        _check(lib.flint_attn_check_status(status.data_ptr(), handle),
               "flint_attn_paged_append (device)")


def alloc_decode_paged_workspace(batch, num_q_heads, num_kv_heads, device=None) -> torch.Tensor:
    """A zeroed workspace for ``decode_paged`` calls of up to this many rows and KV heads.

    One workspace serves any number of calls one after the other; calls that may
    overlap on the GPU need one each.
    """
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        p = DecodePagedParams(PagedCacheDesc(1, 16, 1, num_kv_heads, 128, CACHE_BF16), batch,
                              num_q_heads)
        n = load_library().flint_attn_decode_paged_workspace_bytes(ctypes.byref(p))
        if n == 0:
            raise FlintError(1, "flint_attn_decode_paged_workspace_bytes")
        return torch.zeros(n, dtype=torch.uint8, device="cuda")


def decode_paged(q, k, v, q_norm_w, k_norm_w, sink, cache_lens, block_table, k_pages, v_pages,
                 window, use_rope, rope_theta, rms_eps=1e-6, softmax_scale=0.0, k_scale=None,
                 v_scale=None, out=None, lse=None, workspace=None, stream=None,
                 check_status=False, fp32_out=False):
    """One new token per sequence over a paged cache, through ``flint_attn_decode_paged``.

    q [B,H,D], k, v [B,Hk,D] bf16 (raw projections of the new tokens; row strides
    free); cache_lens [B] int32 on the device (-1: a row not in use, whose out and
    lse stay as they are); block_table, k_pages, v_pages, k_scale, v_scale as for
    ``paged_append``. The new key and value go into slot cache_lens[b]. Returns
    (out [B,H,D], lse [B,H] fp32). ``workspace``: from
    ``alloc_decode_paged_workspace``, kept between calls (a fresh one if omitted).
    """
    B, H = cache_lens.numel(), sink.numel()
    desc = _paged_cache(k_pages, v_pages, block_table, B, k_scale, v_scale)
    Hk, D = desc[3], desc[4]
    params = _PACK_DECODE(*desc, B, H, max(-1, min(window, 0x7fffffff)), 1 if use_rope else 0,
                          rope_theta, rms_eps, softmax_scale, FLINT_BF16, 1 if fp32_out else 0, 0,
                          _rows(q, "q", B, H, D), _rows(k, "k", B, Hk, D), _rows(v, "v", B, Hk, D))
    _vector(q_norm_w, "q_norm_w", torch.bfloat16, (D,))
    _vector(k_norm_w, "k_norm_w", torch.bfloat16, (D,))
    _vector(sink, "sink", torch.float32, (H,))
    _vector(cache_lens, "cache_lens", torch.int32, (B,))
    if out is not None:
        _vector(out, "out", torch.float32 if fp32_out else torch.bfloat16, (B, H, D))
    if lse is not None:
        _vector(lse, "lse", torch.float32, (B, H))
    if workspace is not None:
        _vector(workspace, "workspace", torch.uint8, (workspace.numel(),))
    index = k_pages.get_device()
    _same_device(index, "q k v q_norm_w k_norm_w sink cache_lens block_table k_pages v_pages "
                 "k_scale v_scale out lse workspace",
                 (q, k, v, q_norm_w, k_norm_w, sink, cache_lens, block_table, k_pages, v_pages,
                  k_scale, v_scale, out, lse, workspace))
    args = (params, q, k, v, q_norm_w, k_norm_w, sink, cache_lens, block_table, k_pages, v_pages,
            k_scale, v_scale, out, lse, workspace)
    where, handle = _elsewhere(index, stream)
    if where is not None:
        with where:
            return _launch_decode(*args, handle, check_status, fp32_out, (B, H, Hk, D))
    return _launch_decode(*args, handle, check_status, fp32_out, (B, H, Hk, D))


def _launch_decode(params, q, k, v, q_norm_w, k_norm_w, sink, cache_lens, block_table, k_pages,
                   v_pages, k_scale, v_scale, out, lse, workspace, handle, check_status, fp32_out,
                   sizes):
    lib = load_library()
    B, H, Hk, D = sizes
    if out is None:
        out = sink.new_empty(B, H, D) if fp32_out else q.new_empty(B, H, D)
    if lse is None:
        lse = sink.new_empty(B, H)
    if workspace is None:
        workspace = alloc_decode_paged_workspace(B, H, Hk)
    code = lib.flint_attn_decode_paged(
        params, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_norm_w.data_ptr(),
        k_norm_w.data_ptr(), sink.data_ptr(), cache_lens.data_ptr(), block_table.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), _addr(k_scale), _addr(v_scale), out.data_ptr(),
        lse.data_ptr(), workspace.data_ptr(), workspace.numel(), handle)
    if code:
        raise FlintError(code, "flint_attn_decode_paged")
    if check_status:
        _check(lib.flint_attn_check_status(workspace.data_ptr(), handle),
               "flint_attn_decode_paged (device)")
    return out, lse


def exp2_poly(x: torch.Tensor) -> torch.Tensor:
    """Diagnostic: the kernels' FMA-pipe 2^x evaluated on the device (fp32, even length)."""
    y = torch.empty_like(x)
    _check(load_library().flint_attn_exp2_poly(_ptr(x), _ptr(y), x.numel(), _stream_ptr()),
           "flint_attn_exp2_poly")
    return y


def selftest_wait(wait_cycles: int, arrive_first: bool, stream=None):
    """Bounded-wait self-test on the device: (flint_attn_check_status code, completed).

    A wait that nothing completes must give FLINT_ERR_TIMEOUT and completed = False.
    """
    lib = load_library()
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    st = _stream_ptr(stream)
    _check(lib.flint_attn_selftest_wait(int(wait_cycles), 1 if arrive_first else 0,
                                        _ptr(status), st), "flint_attn_selftest_wait")
    code = lib.flint_attn_check_status(_ptr(status), st)      # synchronises the stream
    return code, bool(status[1].item())


def version() -> str:
    return load_library().flint_attn_version().decode()
