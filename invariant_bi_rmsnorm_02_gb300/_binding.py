"""Thin ctypes binding over libbi.so (the C ABI in include/bi.h).

The functions named ``bi_*`` mirror the C entry points one to one: they take
torch tensors that already live on the GPU, pass their device pointers and the
current CUDA stream, and raise ``BiError`` on a non-OK status.  The short
names (``rmsnorm``, ``gemm``, ``attn_decode``, ``attn_prefill_chunk``,
``kv_write``) additionally allocate the outputs and the workspace with torch.
No arithmetic of the method happens here; every step runs in the CUDA
kernels, and a missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbi.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_BOUNDS, ERR_TIMEOUT = range(7)
INVARIANT, VARIANT = 0, 1
(ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU,
 ACT_SWIGLU) = range(6)                                               # bi_activation
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_LLAMA3, ROPE_YARN = range(5)   # bi_rope_scaling
NOALLOC_SCRATCH_BYTES = 32 << 20   # BI_NOALLOC_SCRATCH_BYTES in include/bi.h

__all__ = [
    "BiError", "INVARIANT", "VARIANT", "LIB_PATH", "load", "library_path", "OK",
    "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_WORKSPACE", "ERR_CUDA", "ERR_DEVICE_BOUNDS",
    "ERR_TIMEOUT",
    "bi_rmsnorm", "bi_rmsnorm_workspace_size", "bi_gemm", "bi_gemm_workspace_size",
    "bi_gemm_variant_splits", "bi_attn_decode", "bi_attn_decode_workspace_size",
    "bi_attn_prefill_chunk", "bi_kv_write", "bi_check_device_errors", "bi_status_string",
    "bi_version", "bi_attn_decode_noalloc", "bi_selftest_wait_timeout", "bi_add_rmsnorm",
    "bi_sample", "bi_gather_rows", "bi_rope_qkv", "bi_silu_mul", "bi_gemm_swiglu",
    "bi_kv_write_q8", "bi_kv_read_q8", "bi_attn_decode_q8", "bi_rope_frequencies",
    "bi_rope_qkv_scaled", "ROPE_NONE", "ROPE_LINEAR", "ROPE_NTK", "ROPE_LLAMA3", "ROPE_YARN",
    "bi_rmsnorm_q8", "bi_add_rmsnorm_q8", "bi_quantize_q8", "bi_gemm_epilogue", "bi_gemm_q8",
    "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_GELU_TANH", "ACT_SILU", "ACT_SWIGLU",
    "rmsnorm_q8", "add_rmsnorm_q8", "quantize_q8", "gemm_epilogue", "gemm_q8",
    "kv_q8_record_bytes", "kv_cache_q8", "kv_write_q8", "kv_read_q8", "attn_decode_q8",
    "rope_frequencies", "rope_high_turns", "rope_qkv_scaled",
    "NOALLOC_SCRATCH_BYTES", "rmsnorm", "add_rmsnorm", "gemm", "gemm_swiglu",
    "swiglu_interleave", "attn_decode", "attn_prefill_chunk", "kv_write", "sample",
    "gather_rows", "rope_qkv", "silu_mul", "EXPORTED_SYMBOLS",
]

# every function include/bi.h declares
EXPORTED_SYMBOLS = (
    "bi_rmsnorm", "bi_rmsnorm_workspace_size", "bi_gemm", "bi_gemm_workspace_size",
    "bi_gemm_variant_splits", "bi_attn_decode", "bi_attn_decode_workspace_size",
    "bi_attn_prefill_chunk", "bi_kv_write", "bi_check_device_errors", "bi_status_string",
    "bi_version", "bi_attn_decode_noalloc", "bi_selftest_wait_timeout", "bi_add_rmsnorm",
    "bi_sample", "bi_gather_rows", "bi_rope_qkv", "bi_silu_mul", "bi_gemm_swiglu",
    "bi_kv_write_q8", "bi_kv_read_q8", "bi_attn_decode_q8", "bi_rope_frequencies",
    "bi_rope_qkv_scaled", "bi_rmsnorm_q8", "bi_add_rmsnorm_q8", "bi_quantize_q8",
    "bi_gemm_epilogue", "bi_gemm_q8",
)


class BiError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, _status_text(status), status))


_lock = threading.Lock()
_lib = None

_vp, _i64, _i32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                             ctypes.c_size_t)
_f64 = ctypes.c_double


def library_path() -> str:
    return LIB_PATH


def load(build_if_missing: bool = True):
    """Load libbi.so (building it with nvcc first if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            if not build_if_missing:
                raise RuntimeError("libbi.so is not built (run the package's build step)")
            from . import build as _build
            _build.build()
        import torch.cuda  # noqa: F401  (loads the CUDA runtime torch ships)
        lib = ctypes.CDLL(LIB_PATH)
        sig = {
            "bi_rmsnorm": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _f32, _i32, _vp, _sz, _vp]),
            "bi_add_rmsnorm": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _i32, _vp, _sz,
                                      _vp]),
            "bi_rmsnorm_workspace_size": (_sz, [_i64, _i64, _i32]),
            "bi_gemm": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _sz, _vp]),
            "bi_gemm_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32]),
            "bi_gemm_variant_splits": (_i32, [_i64, _i64, _i64, _i32]),
            "bi_gemm_swiglu": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _sz,
                                      _vp]),
            "bi_attn_decode": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                      _i32, _i64, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _sz,
                                      _vp]),
            "bi_attn_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                                    _i32]),
            "bi_attn_prefill_chunk": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                             _i32, _i32, _i32, _i32, _i64, _i32, _i64, _i32,
                                             _i32, _i32, _f32, _i32, _i32, _vp, _sz, _vp]),
            "bi_kv_write": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32,
                                   _i64, _i32, _vp]),
            "bi_attn_decode_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                              _i32, _i32, _i32, _i64, _i32, _i32, _i32, _f32,
                                              _vp]),
            "bi_sample": (_i32, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
            "bi_gather_rows": (_i32, [_vp, _i64, _i64, _vp, _i64, _vp, _vp]),
            "bi_rope_qkv": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, ctypes.c_double, _vp, _vp,
                                   _vp, _vp]),
            "bi_silu_mul": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp]),
            "bi_kv_write_q8": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                                      _i64, _i32, _vp]),
            "bi_kv_read_q8": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp,
                                     _vp, _vp, _i64, _i32, _vp]),
            "bi_attn_decode_q8": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                         _i32, _i64, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _sz,
                                         _vp]),
            "bi_rope_frequencies": (_i32, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp,
                                           ctypes.POINTER(ctypes.c_float)]),
            "bi_rope_qkv_scaled": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _f32,
                                          _vp, _vp, _vp, _vp]),
            "bi_rmsnorm_q8": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _f32, _vp]),
            "bi_add_rmsnorm_q8": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _vp]),
            "bi_quantize_q8": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
            "bi_gemm_epilogue": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]),
            "bi_gemm_q8": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32,
                                  _vp]),
            "bi_check_device_errors": (_i32, [_vp]),
            "bi_selftest_wait_timeout": (_i32, [ctypes.c_uint32, _vp]),
            "bi_status_string": (ctypes.c_char_p, [_i32]),
            "bi_version": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _status_text(status: int) -> str:
    try:
        return load().bi_status_string(status).decode()
    except Exception:  # pragma: no cover - library not loadable
        return "status"


def _check(status: int, what: str) -> None:
    if status != OK:
        raise BiError(status, what)


# the current stream's handle without building a Stream object (a few
# microseconds per call, as long as a small kernel runs)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- raw entry points
def bi_rmsnorm(x, w, y, eps, mode=INVARIANT, workspace=None, stream=None, y_f32=None):
    M, H = x.shape
    wp, wb = _ws(workspace)
    _check(load().bi_rmsnorm(_ptr(x, torch.bfloat16, "x"), _ptr(w, torch.bfloat16, "w"),
                             _ptr(y, torch.bfloat16, "y"), _ptr(y_f32, torch.float32, "y_f32"),
                             M, H, float(eps), int(mode), wp, wb, _stream(stream)),
           "bi_rmsnorm")


def bi_add_rmsnorm(x, residual, w, y, eps, mode=INVARIANT, workspace=None, stream=None,
                   y_f32=None):
    """residual <- bf16(x + residual); y <- RMSNorm(residual) * w (include/bi.h)."""
    M, H = x.shape
    if tuple(residual.shape) != (M, H) or tuple(y.shape) != (M, H):
        raise ValueError("x, residual and y must have the same shape")
    wp, wb = _ws(workspace)
    _check(load().bi_add_rmsnorm(_ptr(x, torch.bfloat16, "x"),
                                 _ptr(residual, torch.bfloat16, "residual"),
                                 _ptr(w, torch.bfloat16, "w"), _ptr(y, torch.bfloat16, "y"),
                                 _ptr(y_f32, torch.float32, "y_f32"), M, H, float(eps),
                                 int(mode), wp, wb, _stream(stream)), "bi_add_rmsnorm")


def bi_rmsnorm_workspace_size(M, H, mode=INVARIANT) -> int:
    return int(load().bi_rmsnorm_workspace_size(M, H, int(mode)))


def bi_gemm(A, W, C, mode=INVARIANT, variant_splits=0, workspace=None, stream=None):
    M, K = A.shape
    N = W.shape[0]
    wp, wb = _ws(workspace)
    _check(load().bi_gemm(_ptr(A, torch.bfloat16, "A"), _ptr(W, torch.bfloat16, "W"),
                          _ptr(C, torch.bfloat16, "C"), M, N, K, int(mode), int(variant_splits),
                          wp, wb, _stream(stream)), "bi_gemm")


def bi_gemm_workspace_size(M, N, K, mode=INVARIANT, variant_splits=0) -> int:
    return int(load().bi_gemm_workspace_size(M, N, K, int(mode), int(variant_splits)))


def bi_gemm_variant_splits(M, N, K, num_sms) -> int:
    return int(load().bi_gemm_variant_splits(M, N, K, int(num_sms)))


def bi_gemm_swiglu(A, W, out, mode=INVARIANT, variant_splits=0, workspace=None, stream=None):
    M, K = A.shape
    F = W.shape[0] // 2
    if W.shape[0] % 2 or tuple(out.shape) != (M, F):
        raise ValueError("W must be [2F, K] and out [M, F]")
    wp, wb = _ws(workspace)
    _check(load().bi_gemm_swiglu(_ptr(A, torch.bfloat16, "A"), _ptr(W, torch.bfloat16, "W"),
                                 _ptr(out, torch.bfloat16, "out"), M, F, K, int(mode),
                                 int(variant_splits), wp, wb, _stream(stream)), "bi_gemm_swiglu")


def bi_attn_decode(q, k_cache, v_cache, block_table, kv_lens, out, out_f32=None, *,
                   max_kv_len, split_size, sm_scale, mode=INVARIANT, variant_splits=0,
                   workspace=None, stream=None):
    B, Hq, D = q.shape
    num_pages, Hkv, page, D2 = k_cache.shape
    wp, wb = _ws(workspace)
    _check(load().bi_attn_decode(
        _ptr(q, torch.bfloat16, "q"), _ptr(k_cache, torch.bfloat16, "k_cache"),
        _ptr(v_cache, torch.bfloat16, "v_cache"), _ptr(block_table, torch.int32, "block_table"),
        _ptr(kv_lens, torch.int32, "kv_lens"), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32"), B, Hq, Hkv, D, page, num_pages,
        block_table.shape[1], int(max_kv_len), int(split_size), float(sm_scale), int(mode),
        int(variant_splits), wp, wb, _stream(stream)), "bi_attn_decode")


def bi_attn_decode_noalloc(q, k_cache, v_cache, block_table, kv_lens, out, out_f32=None, *,
                           max_kv_len, split_size, sm_scale, stream=None):
    """Decode without a workspace argument (scratch from the library's fixed
    array); for callers that cannot allocate device memory."""
    B, Hq, D = q.shape
    num_pages, Hkv, page, _ = k_cache.shape
    _check(load().bi_attn_decode_noalloc(
        _ptr(q, torch.bfloat16, "q"), _ptr(k_cache, torch.bfloat16, "k_cache"),
        _ptr(v_cache, torch.bfloat16, "v_cache"), _ptr(block_table, torch.int32, "block_table"),
        _ptr(kv_lens, torch.int32, "kv_lens"), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32"), B, Hq, Hkv, D, page, num_pages,
        block_table.shape[1], int(max_kv_len), int(split_size), float(sm_scale),
        _stream(stream)), "bi_attn_decode_noalloc")


def bi_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, split_size, mode=INVARIANT,
                                  variant_splits=0) -> int:
    return int(load().bi_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, split_size,
                                                    int(mode), int(variant_splits)))


def bi_attn_prefill_chunk(q, cu_q, q_start_pos, k_cache, v_cache, block_table, kv_lens, out,
                          out_f32=None, *, max_q_len, max_kv_len, split_size, sm_scale,
                          mode=INVARIANT, variant_splits=0, workspace=None, stream=None):
    total_q, Hq, D = q.shape
    num_pages, Hkv, page, _ = k_cache.shape
    B = kv_lens.shape[0]
    wp, wb = _ws(workspace)
    _check(load().bi_attn_prefill_chunk(
        _ptr(q, torch.bfloat16, "q"), _ptr(cu_q, torch.int32, "cu_q"),
        _ptr(q_start_pos, torch.int32, "q_start_pos"), _ptr(k_cache, torch.bfloat16, "k_cache"),
        _ptr(v_cache, torch.bfloat16, "v_cache"), _ptr(block_table, torch.int32, "block_table"),
        _ptr(kv_lens, torch.int32, "kv_lens"), _ptr(out, torch.bfloat16, "out"),
        _ptr(out_f32, torch.float32, "out_f32"), B, Hq, Hkv, D, page, num_pages,
        block_table.shape[1], total_q, int(max_q_len), int(max_kv_len), int(split_size),
        float(sm_scale), int(mode), int(variant_splits), wp, wb, _stream(stream)),
        "bi_attn_prefill_chunk")


def bi_kv_write(k_new, v_new, seq, pos, k_cache, v_cache, block_table, stream=None):
    n, Hkv, D = k_new.shape
    num_pages, _, page, _ = k_cache.shape
    _check(load().bi_kv_write(
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(seq, torch.int32, "seq"), _ptr(pos, torch.int32, "pos"), n,
        _ptr(k_cache, torch.bfloat16, "k_cache"), _ptr(v_cache, torch.bfloat16, "v_cache"),
        _ptr(block_table, torch.int32, "block_table"), Hkv, D, page, num_pages,
        block_table.shape[1], _stream(stream)), "bi_kv_write")


def bi_sample(logits, temperature, seed, step, tokens, stream=None):
    """tokens[b] <- the token of row b of logits (include/bi.h).  seed and step
    are int64 tensors whose bits are read as uint64."""
    B, V = logits.shape
    for t, name in ((temperature, "temperature"), (seed, "seed"), (step, "step"),
                    (tokens, "tokens")):
        if tuple(t.shape) != (B,):
            raise ValueError("%s must have shape [B]" % name)
    _check(load().bi_sample(_ptr(logits, torch.bfloat16, "logits"), B, V,
                            _ptr(temperature, torch.float32, "temperature"),
                            _ptr(seed, torch.int64, "seed"), _ptr(step, torch.int64, "step"),
                            _ptr(tokens, torch.int32, "tokens"), _stream(stream)), "bi_sample")


def bi_gather_rows(src, idx, dst, stream=None):
    rows, H = src.shape
    n = idx.shape[0]
    if tuple(dst.shape) != (n, H):
        raise ValueError("dst must be [len(idx), H]")
    _check(load().bi_gather_rows(_ptr(src, torch.bfloat16, "src"), rows, H,
                                 _ptr(idx, torch.int32, "idx"), n,
                                 _ptr(dst, torch.bfloat16, "dst"), _stream(stream)),
           "bi_gather_rows")


def bi_rope_qkv(qkv, pos, Hq, Hkv, D, theta, q, k, v, stream=None):
    T = qkv.shape[0]
    if qkv.shape[1] != (Hq + 2 * Hkv) * D or pos.shape != (T,):
        raise ValueError("qkv must be [T, (Hq + 2 Hkv) D] and pos [T]")
    if q.shape != (T, Hq, D) or k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D):
        raise ValueError("q, k, v must be [T, H, D]")
    _check(load().bi_rope_qkv(_ptr(qkv, torch.bfloat16, "qkv"), _ptr(pos, torch.int32, "pos"), T,
                              Hq, Hkv, D, float(theta), _ptr(q, torch.bfloat16, "q"),
                              _ptr(k, torch.bfloat16, "k"), _ptr(v, torch.bfloat16, "v"),
                              _stream(stream)), "bi_rope_qkv")


def _dptr(t, dtype, dev, name):
    """_ptr for a tensor that has to be on the current device ``dev``: the
    library works there only, and a tensor of another device is refused here
    rather than read through a foreign pointer."""
    if t is None:
        return None
    try:
        on = t.get_device()
        if on == dev and t.dtype is dtype and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError("%s must be a CUDA tensor" % name) from None
    if on != dev:
        if on < 0:
            raise TypeError("%s must be a CUDA tensor" % name)
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, on, dev))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be contiguous" % name)


_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _here(stream):
    """(current device, the stream's handle), asking for the device once."""
    dev = torch.cuda.current_device()
    if stream is None and _raw_stream is not None:
        return dev, _raw_stream(dev)
    return dev, _stream(stream)


def _cache_q8(cache, Hkv, D) -> int:
    """The cache's page count, once its shape is what Hkv and D ask for."""
    s = cache.shape
    if len(s) != 3 or s[1] != Hkv or s[2] != 32 * D + 32:
        raise ValueError("cache must be [num_pages, %d, %d]" % (Hkv, kv_q8_record_bytes(D)))
    return s[0]


def bi_kv_write_q8(k_new, v_new, seq, pos, cache, block_table, stream=None):
    """Quantise K/V rows of new tokens into the paged cache (include/bi.h)."""
    shape = k_new.shape
    n, Hkv, D = shape
    if v_new.shape != shape or seq.shape != (n,) or pos.shape != (n,):
        raise ValueError("k_new, v_new must be [n, Hkv, D] and seq, pos [n]")
    pages = _cache_q8(cache, Hkv, D)
    num_seqs, max_blocks = block_table.shape
    dev = torch.cuda.current_device()
    _check(load().bi_kv_write_q8(
        _dptr(k_new, torch.bfloat16, dev, "k_new"), _dptr(v_new, torch.bfloat16, dev, "v_new"),
        _dptr(seq, torch.int32, dev, "seq"), _dptr(pos, torch.int32, dev, "pos"), n,
        _dptr(cache, torch.uint8, dev, "cache"),
        _dptr(block_table, torch.int32, dev, "block_table"), num_seqs, Hkv, D, 16, pages,
        max_blocks, _stream(stream)), "bi_kv_write_q8")


def bi_kv_read_q8(cache, block_table, kv_lens, k_out, v_out, out_table, *, max_kv_len,
                  stream=None):
    """Read the sequences' cached tokens back into bf16 pages (include/bi.h)."""
    num_out, Hkv, page, D = k_out.shape
    B = kv_lens.shape[0]
    if v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out must have the same shape")
    if block_table.dim() != 2 or block_table.shape[0] != B or out_table.dim() != 2 \
            or out_table.shape[0] != B:
        raise ValueError("block_table and out_table must be [B, blocks], kv_lens [B]")
    _cache_q8(cache, Hkv, D)
    dev = torch.cuda.current_device()
    _check(load().bi_kv_read_q8(
        _dptr(cache, torch.uint8, dev, "cache"),
        _dptr(block_table, torch.int32, dev, "block_table"),
        _dptr(kv_lens, torch.int32, dev, "kv_lens"), B, Hkv, D, page, cache.shape[0],
        block_table.shape[1], int(max_kv_len), _dptr(k_out, torch.bfloat16, dev, "k_out"),
        _dptr(v_out, torch.bfloat16, dev, "v_out"),
        _dptr(out_table, torch.int32, dev, "out_table"), num_out, out_table.shape[1],
        _stream(stream)), "bi_kv_read_q8")


def bi_attn_decode_q8(q, cache, block_table, kv_lens, out, out_f32=None, *, max_kv_len,
                      split_size, sm_scale, mode=INVARIANT, variant_splits=0, workspace=None,
                      stream=None):
    """Decode attention over the quantised cache (include/bi.h)."""
    shape = q.shape
    B, Hq, D = shape
    Hkv = cache.shape[1]
    pages = _cache_q8(cache, Hkv, D)
    if out.shape != shape or (out_f32 is not None and out_f32.shape != shape):
        raise ValueError("out must have q's shape")
    table = block_table.shape
    if len(table) != 2 or table[0] != B or kv_lens.shape != (B,):
        raise ValueError("block_table must be [B, max_blocks] and kv_lens [B]")
    dev = torch.cuda.current_device()
    if workspace is not None and workspace.get_device() != dev:
        raise ValueError("workspace must be on the current device")
    wp, wb = _ws(workspace)
    _check(load().bi_attn_decode_q8(
        _dptr(q, torch.bfloat16, dev, "q"), _dptr(cache, torch.uint8, dev, "cache"),
        _dptr(block_table, torch.int32, dev, "block_table"),
        _dptr(kv_lens, torch.int32, dev, "kv_lens"), _dptr(out, torch.bfloat16, dev, "out"),
        _dptr(out_f32, torch.float32, dev, "out_f32"), B, Hq, Hkv, D, 16, pages, table[1],
        int(max_kv_len), int(split_size), float(sm_scale), int(mode), int(variant_splits), wp, wb,
        _stream(stream)), "bi_attn_decode_q8")


def bi_rope_frequencies(rot_dim, theta, scaling, factor, trained_len, low_turns, high_turns,
                        freqs):
    """freqs (numpy float64 [rot_dim / 2], host) <- the rotation frequencies;
    returns the factor on cosine and sine (include/bi.h)."""
    if not isinstance(freqs, np.ndarray) or freqs.dtype != np.float64 \
            or not freqs.flags.c_contiguous or freqs.shape != (int(rot_dim) // 2,):
        raise TypeError("freqs must be a contiguous float64 array of rot_dim / 2 values")
    m = ctypes.c_float()
    _check(load().bi_rope_frequencies(int(rot_dim), float(theta), int(scaling), float(factor),
                                      float(trained_len), float(low_turns), float(high_turns),
                                      freqs.ctypes.data, ctypes.byref(m)), "bi_rope_frequencies")
    return m.value


def bi_rope_qkv_scaled(qkv, pos, Hq, Hkv, D, freqs, q, k, v, interleaved=False, attn_scale=1.0,
                       stream=None):
    """Rotary positions from a table of frequencies (device float64
    [rot_dim / 2]); include/bi.h."""
    T = qkv.shape[0]
    if qkv.shape != (T, (Hq + 2 * Hkv) * D) or pos.shape != (T,) or freqs.dim() != 1:
        raise ValueError("qkv must be [T, (Hq + 2 Hkv) D], pos [T] and freqs [rot_dim / 2]")
    if q.shape != (T, Hq, D) or k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D):
        raise ValueError("q, k, v must be [T, H, D]")
    dev = torch.cuda.current_device()
    _check(load().bi_rope_qkv_scaled(
        _dptr(qkv, torch.bfloat16, dev, "qkv"), _dptr(pos, torch.int32, dev, "pos"), T, Hq, Hkv,
        D, 2 * freqs.shape[0], 1 if interleaved else 0, _dptr(freqs, torch.float64, dev, "freqs"),
        float(attn_scale), _dptr(q, torch.bfloat16, dev, "q"),
        _dptr(k, torch.bfloat16, dev, "k"), _dptr(v, torch.bfloat16, dev, "v"),
        _stream(stream)), "bi_rope_qkv_scaled")


def bi_silu_mul(gate_up, out, block=None, stream=None):
    """block: features per gate/up block (None: F, i.e. the gate half then
    the up half; 128: the layout bi_gemm writes with bi_gemm_swiglu's
    weight)."""
    T, F2 = gate_up.shape
    if F2 % 2 or tuple(out.shape) != (T, F2 // 2):
        raise ValueError("gate_up must be [T, 2F] and out [T, F]")
    blk = F2 // 2 if block is None else int(block)
    _check(load().bi_silu_mul(_ptr(gate_up, torch.bfloat16, "gate_up"), T, F2 // 2, blk,
                              _ptr(out, torch.bfloat16, "out"), _stream(stream)), "bi_silu_mul")


def bi_rmsnorm_q8(x, w, y, y_scale, eps, stream=None):
    """y, y_scale <- RMSNorm(x) * w as e4m3 rows with a scale each (include/bi.h)."""
    shape = x.shape
    M, H = shape
    if y.shape != shape or w.shape != (H,) or y_scale.shape != (M,):
        raise ValueError("y must have x's shape, w [H] and y_scale [M]")
    dev, on = _here(stream)
    _check(load().bi_rmsnorm_q8(
        _dptr(x, _BF16, dev, "x"), _dptr(w, _BF16, dev, "w"),
        _dptr(y, _E4M3, dev, "y"), _dptr(y_scale, _F32, dev, "y_scale"),
        M, H, float(eps), on), "bi_rmsnorm_q8")


def bi_add_rmsnorm_q8(x, residual, w, h, y, y_scale, eps, stream=None):
    """h <- bf16(x + residual) (h may be residual or x); y, y_scale <-
    RMSNorm(h) * w as e4m3 rows with a scale each (include/bi.h)."""
    shape = x.shape
    M, H = shape
    if residual.shape != shape or h.shape != shape or y.shape != shape or w.shape != (H,) \
            or y_scale.shape != (M,):
        raise ValueError("residual, h and y must have x's shape, w [H] and y_scale [M]")
    dev, on = _here(stream)
    _check(load().bi_add_rmsnorm_q8(
        _dptr(x, _BF16, dev, "x"), _dptr(residual, _BF16, dev, "residual"),
        _dptr(w, _BF16, dev, "w"), _dptr(h, _BF16, dev, "h"),
        _dptr(y, _E4M3, dev, "y"), _dptr(y_scale, _F32, dev, "y_scale"),
        M, H, float(eps), on), "bi_add_rmsnorm_q8")


def bi_quantize_q8(x, y, y_scale, stream=None):
    """y, y_scale <- the rows of x as e4m3 with a scale each (include/bi.h)."""
    shape = x.shape
    M, K = shape
    if y.shape != shape or y_scale.shape != (M,):
        raise ValueError("y must have x's shape and y_scale [M]")
    dev, on = _here(stream)
    _check(load().bi_quantize_q8(
        _dptr(x, _BF16, dev, "x"), _dptr(y, _E4M3, dev, "y"),
        _dptr(y_scale, _F32, dev, "y_scale"), M, K, on), "bi_quantize_q8")


def _fused_shapes(A, W, C, bias, residual, activation):
    """(M, N, K) of a GEMM with an epilogue, once the tensors' shapes agree."""
    M, K = A.shape
    N, K2 = W.shape
    out = (M, N // 2 if activation == ACT_SWIGLU else N)
    if K2 != K or C.shape != out or (bias is not None and bias.shape != (N,)) \
            or (residual is not None and residual.shape != out):
        raise ValueError("W must be [N, K], bias [N], C and residual [M, N] ([M, N/2] for SwiGLU)")
    return M, N, K


def bi_gemm_epilogue(A, W, C, bias=None, residual=None, activation=ACT_NONE, stream=None):
    """C <- act(A W^T + bias) + residual (include/bi.h); residual may be C."""
    M, N, K = _fused_shapes(A, W, C, bias, residual, activation)
    dev, on = _here(stream)
    _check(load().bi_gemm_epilogue(
        _dptr(A, _BF16, dev, "A"), _dptr(W, _BF16, dev, "W"),
        _dptr(bias, _BF16, dev, "bias"), _dptr(residual, _BF16, dev, "residual"),
        _dptr(C, _BF16, dev, "C"), M, N, K, int(activation), on),
        "bi_gemm_epilogue")


def bi_gemm_q8(A, a_scale, W, w_scale, C, bias=None, residual=None, activation=ACT_NONE,
               stream=None):
    """C <- act((A W^T) a_scale w_scale + bias) + residual of e4m3 rows
    (include/bi.h); residual may be C."""
    M, N, K = _fused_shapes(A, W, C, bias, residual, activation)
    if a_scale.shape != (M,) or w_scale.shape != (N,):
        raise ValueError("a_scale must be [M] and w_scale [N]")
    dev, on = _here(stream)
    _check(load().bi_gemm_q8(
        _dptr(A, _E4M3, dev, "A"), _dptr(a_scale, _F32, dev, "a_scale"),
        _dptr(W, _E4M3, dev, "W"), _dptr(w_scale, _F32, dev, "w_scale"),
        _dptr(bias, _BF16, dev, "bias"), _dptr(residual, _BF16, dev, "residual"),
        _dptr(C, _BF16, dev, "C"), M, N, K, int(activation), on),
        "bi_gemm_q8")


def bi_check_device_errors(stream=None) -> int:
    return int(load().bi_check_device_errors(_stream(stream)))


def bi_selftest_wait_timeout(timeout_us: int, stream=None) -> int:
    """Launch the bounded-wait diagnostic (see include/bi.h); returns the
    launch status, the recorded one comes from bi_check_device_errors."""
    return int(load().bi_selftest_wait_timeout(int(timeout_us), _stream(stream)))


def bi_status_string(status: int) -> str:
    return load().bi_status_string(int(status)).decode()


def bi_version() -> str:
    return load().bi_version().decode()


# ---------------------------------------------------------- allocating helpers
def _workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    if nbytes == 2 ** 64 - 1:
        raise BiError(ERR_CUDA, "workspace size query")
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=device)


def rmsnorm(x, w, eps=1e-6, mode=INVARIANT, want_f32=False, stream=None):
    y = torch.empty_like(x)
    y32 = torch.empty(x.shape, dtype=torch.float32, device=x.device) if want_f32 else None
    ws = _workspace(bi_rmsnorm_workspace_size(x.shape[0], x.shape[1], mode), x.device)
    bi_rmsnorm(x, w, y, eps, mode, ws, stream, y_f32=y32)
    return (y, y32) if want_f32 else y


def add_rmsnorm(x, residual, w, eps=1e-6, mode=INVARIANT, want_f32=False, stream=None):
    """Updates residual in place (residual <- bf16(x + residual)) and returns
    RMSNorm(residual) * w (and its fp32 values with want_f32)."""
    y = torch.empty_like(x)
    y32 = torch.empty(x.shape, dtype=torch.float32, device=x.device) if want_f32 else None
    ws = _workspace(bi_rmsnorm_workspace_size(x.shape[0], x.shape[1], mode), x.device)
    bi_add_rmsnorm(x, residual, w, y, eps, mode, ws, stream, y_f32=y32)
    return (y, y32) if want_f32 else y


def gemm(A, W, mode=INVARIANT, variant_splits=0, stream=None):
    C = torch.empty(A.shape[0], W.shape[0], dtype=torch.bfloat16, device=A.device)
    ws = _workspace(bi_gemm_workspace_size(A.shape[0], W.shape[0], A.shape[1], mode,
                                           variant_splits), A.device)
    bi_gemm(A, W, C, mode, variant_splits, ws, stream)
    return C


def attn_decode(q, k_cache, v_cache, block_table, kv_lens, *, max_kv_len, split_size,
                sm_scale=None, mode=INVARIANT, variant_splits=0, want_f32=False, stream=None):
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    sm_scale = D ** -0.5 if sm_scale is None else sm_scale
    out = torch.empty_like(q)
    out32 = torch.empty(q.shape, dtype=torch.float32, device=q.device) if want_f32 else None
    ws = _workspace(bi_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, split_size, mode,
                                                  variant_splits), q.device)
    bi_attn_decode(q, k_cache, v_cache, block_table, kv_lens, out, out32,
                   max_kv_len=max_kv_len, split_size=split_size, sm_scale=sm_scale, mode=mode,
                   variant_splits=variant_splits, workspace=ws, stream=stream)
    return (out, out32) if want_f32 else out


def attn_prefill_chunk(q, cu_q, q_start_pos, k_cache, v_cache, block_table, kv_lens, *,
                       max_q_len, max_kv_len, split_size, sm_scale=None, mode=INVARIANT,
                       variant_splits=0, want_f32=False, stream=None):
    D = q.shape[2]
    sm_scale = D ** -0.5 if sm_scale is None else sm_scale
    out = torch.empty_like(q)
    out32 = torch.empty(q.shape, dtype=torch.float32, device=q.device) if want_f32 else None
    bi_attn_prefill_chunk(q, cu_q, q_start_pos, k_cache, v_cache, block_table, kv_lens, out,
                          out32, max_q_len=max_q_len, max_kv_len=max_kv_len,
                          split_size=split_size, sm_scale=sm_scale, mode=mode,
                          variant_splits=variant_splits, stream=stream)
    return (out, out32) if want_f32 else out


def sample(logits, temperature, seed, step, stream=None):
    """One token per row: seeded Gumbel-max at temperature > 0, argmax at 0."""
    tokens = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    bi_sample(logits, temperature, seed, step, tokens, stream)
    return tokens


def gather_rows(src, idx, stream=None):
    dst = torch.empty(idx.shape[0], src.shape[1], dtype=src.dtype, device=src.device)
    bi_gather_rows(src, idx, dst, stream)
    return dst


def rope_qkv(qkv, pos, Hq, Hkv, D, theta=500000.0, stream=None):
    T = qkv.shape[0]
    q = torch.empty(T, Hq, D, dtype=qkv.dtype, device=qkv.device)
    k = torch.empty(T, Hkv, D, dtype=qkv.dtype, device=qkv.device)
    v = torch.empty(T, Hkv, D, dtype=qkv.dtype, device=qkv.device)
    bi_rope_qkv(qkv, pos, Hq, Hkv, D, theta, q, k, v, stream)
    return q, k, v


def kv_q8_record_bytes(D: int) -> int:
    """Bytes of one (page, kv head) of the quantised cache: K and V of 16
    tokens, one byte per element, and 32 scale bytes."""
    return 32 * D + 32


def kv_cache_q8(num_pages, Hkv, D, device) -> torch.Tensor:
    """A zeroed quantised cache [num_pages, Hkv, kv_q8_record_bytes(D)]."""
    return torch.zeros(num_pages, Hkv, kv_q8_record_bytes(D), dtype=torch.uint8, device=device)


def kv_write_q8(k_new, v_new, seq, pos, cache, block_table, stream=None):
    bi_kv_write_q8(k_new, v_new, seq, pos, cache, block_table, stream)


def _alloc(stream, make):
    """make() -> tensors for a call on ``stream``: allocated in that stream's
    order (memory freed on the current stream may still be in use there) and
    held until the current stream, where the caller reads them, is past its
    uses too."""
    if stream is None:
        return make()
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    here = torch.cuda.current_stream()
    with torch.cuda.stream(s):
        ts = make()
    for t in ts:
        if t is not None:
            t.record_stream(here)
    return ts


def kv_read_q8(cache, D, block_table, kv_lens, *, max_kv_len, stream=None):
    """The cached tokens of each sequence as bf16 pages (k, v), under the
    cache's own page ids; every other slot is zero."""
    k, v = _alloc(stream, lambda: [torch.zeros(cache.shape[0], cache.shape[1], 16, D,
                                               dtype=torch.bfloat16, device=cache.device)
                                   for _ in range(2)])
    bi_kv_read_q8(cache, block_table, kv_lens, k, v, block_table, max_kv_len=max_kv_len,
                  stream=stream)
    return k, v


def attn_decode_q8(q, cache, block_table, kv_lens, *, max_kv_len, split_size, sm_scale=None,
                   mode=INVARIANT, variant_splits=0, want_f32=False, stream=None):
    B, Hq, D = q.shape
    sm_scale = D ** -0.5 if sm_scale is None else sm_scale
    nws = bi_attn_decode_workspace_size(B, Hq, cache.shape[1], D, max_kv_len, split_size, mode,
                                        variant_splits)
    out, out32, ws = _alloc(stream, lambda: (
        torch.empty_like(q),
        torch.empty(q.shape, dtype=torch.float32, device=q.device) if want_f32 else None,
        _workspace(nws, q.device)))
    bi_attn_decode_q8(q, cache, block_table, kv_lens, out, out32, max_kv_len=max_kv_len,
                      split_size=split_size, sm_scale=sm_scale, mode=mode,
                      variant_splits=variant_splits, workspace=ws, stream=stream)
    return (out, out32) if want_f32 else out


def rope_high_turns(scaling) -> float:
    """The published upper end of a scaling's ramp, in turns over the trained
    length: 32 for YaRN, 4 for Llama 3 (the others have no ramp)."""
    return 32.0 if scaling == ROPE_YARN else 4.0


def rope_frequencies(rot_dim, theta=500000.0, scaling=ROPE_NONE, factor=1.0, trained_len=8192,
                     low_turns=1.0, high_turns=None, device=None):
    """(freqs, attn_scale) of rotary positions: a float64 tensor of
    rot_dim / 2 rotation frequencies on ``device`` (the current CUDA device
    if None) and the factor on cosine and sine, both for rope_qkv_scaled.
    ``high_turns`` None: the scaling's published value (rope_high_turns)."""
    if high_turns is None:
        high_turns = rope_high_turns(scaling)
    f = np.empty(int(rot_dim) // 2, np.float64)
    m = bi_rope_frequencies(rot_dim, theta, scaling, factor, trained_len, low_turns, high_turns, f)
    return torch.from_numpy(f).to("cuda" if device is None else device), m


def rope_qkv_scaled(qkv, pos, Hq, Hkv, D, freqs, interleaved=False, attn_scale=1.0, stream=None):
    T = qkv.shape[0]
    q, k, v = _alloc(stream, lambda: [torch.empty(T, h, D, dtype=qkv.dtype, device=qkv.device)
                                      for h in (Hq, Hkv, Hkv)])
    bi_rope_qkv_scaled(qkv, pos, Hq, Hkv, D, freqs, q, k, v, interleaved, attn_scale, stream)
    return q, k, v


def _q8_rows(x, stream):
    """Outputs for rows of x held as e4m3."""
    return _alloc(stream, lambda: (
        torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device),
        torch.empty(x.shape[0], dtype=torch.float32, device=x.device)))


def rmsnorm_q8(x, w, eps=1e-6, stream=None):
    """RMSNorm(x) * w as (e4m3 rows, fp32 scale per row)."""
    y, scale = _q8_rows(x, stream)
    bi_rmsnorm_q8(x, w, y, scale, eps, stream)
    return y, scale


def add_rmsnorm_q8(x, residual, w, eps=1e-6, stream=None):
    """Updates residual in place (residual <- bf16(x + residual)) and returns
    RMSNorm(residual) * w as (e4m3 rows, fp32 scale per row)."""
    y, scale = _q8_rows(x, stream)
    bi_add_rmsnorm_q8(x, residual, w, residual, y, scale, eps, stream)
    return y, scale


def quantize_q8(x, stream=None):
    """The rows of x as (e4m3 rows, fp32 scale per row)."""
    y, scale = _q8_rows(x, stream)
    bi_quantize_q8(x, y, scale, stream)
    return y, scale


def _product(A, W, activation, stream):
    N = W.shape[0] // 2 if activation == ACT_SWIGLU else W.shape[0]
    return _alloc(stream, lambda: [torch.empty(A.shape[0], N, dtype=torch.bfloat16,
                                               device=A.device)])[0]


def gemm_epilogue(A, W, bias=None, residual=None, activation=ACT_NONE, stream=None):
    """act(A W^T + bias) + residual."""
    C = _product(A, W, activation, stream)
    bi_gemm_epilogue(A, W, C, bias, residual, activation, stream)
    return C


def gemm_q8(A, a_scale, W, w_scale, bias=None, residual=None, activation=ACT_NONE, stream=None):
    """act((A W^T) a_scale w_scale + bias) + residual of e4m3 rows."""
    C = _product(A, W, activation, stream)
    bi_gemm_q8(A, a_scale, W, w_scale, C, bias, residual, activation, stream)
    return C


def gemm_swiglu(A, W, mode=INVARIANT, variant_splits=0, stream=None):
    out = torch.empty(A.shape[0], W.shape[0] // 2, dtype=torch.bfloat16, device=A.device)
    ws = _workspace(bi_gemm_workspace_size(A.shape[0], W.shape[0], A.shape[1], mode,
                                           variant_splits), A.device)
    bi_gemm_swiglu(A, W, out, mode, variant_splits, ws, stream)
    return out


def swiglu_interleave(F: int, block: int = 128) -> np.ndarray:
    """Row order of bi_gemm_swiglu's weight (and of ACT_SWIGLU's with block =
    16): entry r is the row of a [gate; up] stacked weight (gate rows 0..F-1,
    up rows F..2F-1) that goes to row r (blocks of ``block`` features, the gate
    rows of a block before its up rows)."""
    if F % block:
        raise ValueError("F must be a multiple of %d" % block)
    j = np.arange(2 * F)
    blk, r = j // (2 * block), j % (2 * block)
    return np.where(r < block, blk * block + r, F + blk * block + (r - block)).astype(np.int32)


def silu_mul(gate_up, block=None, stream=None):
    out = torch.empty(gate_up.shape[0], gate_up.shape[1] // 2, dtype=gate_up.dtype,
                      device=gate_up.device)
    bi_silu_mul(gate_up, out, block, stream)
    return out


def kv_write(k_new, v_new, seq, pos, k_cache, v_cache, block_table, stream=None):
    bi_kv_write(k_new, v_new, seq, pos, k_cache, v_cache, block_table, stream)
