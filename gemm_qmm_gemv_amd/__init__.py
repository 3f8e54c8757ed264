"""Python binding of libqmm (quantized GEMV / GEMM with inline dequantization
for AMD MI355X, gfx950).

The functions here carry the C ABI's names (``include/qmm.h``) and only
marshal arguments: every step of the computation runs in the HIP kernels of
``libqmm.so``.  PyTorch supplies device memory and streams.  There is no
fallback: if the library is missing or fails to load, every call raises.

Arguments that are device buffers may be given as torch tensors (their
``data_ptr()`` is passed) or as raw integer addresses.  ``stream`` defaults to
torch's current stream on the current device.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "QmmError", "library_path", "load",
    "qmm_gemv", "qmm_gemm", "qmm_gemm_workspace_bytes", "qmm_moe_gemm", "qmm_unpack",
    "qmm_gemv_batch_prepare", "qmm_gemv_batched", "GemvDesc", "GemmMember", "qmm_gemv_swiglu",
    "qmm_gemm_f16out",
    "qmm_moe_swiglu", "qmm_gemv_residual", "qmm_moe_combine", "qmm_gemm_grouped",
    "qmm_gemm_grouped_workspace_bytes", "qmm_gemm_noalloc", "qmm_set_override", "overrides",
    "QMM_NOALLOC_SCRATCH_BYTES", "QMM_ATTN_COUNTER_BYTES",
    "KvCache", "qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_cache_workspace_bytes",
    "qmm_attn_prompt",
    "qmm_moe_route", "qmm_moe_route_workspace_bytes", "qmm_quantize_rows", "qmm_gemm_i8", "qmm_moe_gemm_i8",
    "qmm_moe_swiglu_i8", "qmm_moe_gather",
    "qmm_get_plan", "qmm_status_string", "qmm_last_error", "qmm_abi_version",
    "QMM_OK", "QMM_ERR_INVALID_ARGUMENT", "QMM_ERR_UNSUPPORTED", "QMM_ERR_MISALIGNED",
    "QMM_ERR_DEVICE", "EXPORTED_SYMBOLS",
]

QMM_OK = 0
QMM_ERR_INVALID_ARGUMENT = 1
QMM_ERR_UNSUPPORTED = 2
QMM_ERR_MISALIGNED = 3
QMM_ERR_DEVICE = 4
QMM_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # include/qmm.h
QMM_ATTN_COUNTER_BYTES = 64 * 1024  # include/qmm.h

EXPORTED_SYMBOLS = (
    "qmm_gemv", "qmm_gemm", "qmm_gemm_workspace_bytes", "qmm_moe_gemm", "qmm_unpack",
    "qmm_gemv_batch_prepare", "qmm_gemv_batched", "qmm_gemv_swiglu", "qmm_gemm_f16out",
    "qmm_moe_swiglu", "qmm_gemv_residual", "qmm_moe_combine", "qmm_gemm_grouped",
    "qmm_gemm_grouped_workspace_bytes", "qmm_gemm_noalloc", "qmm_set_override",
    "qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_cache_workspace_bytes", "qmm_attn_prompt",
    "qmm_moe_route", "qmm_moe_route_workspace_bytes", "qmm_quantize_rows", "qmm_gemm_i8", "qmm_moe_gemm_i8",
    "qmm_moe_swiglu_i8", "qmm_moe_gather",
    "qmm_call_words", "qmm_get_plan", "qmm_status_string", "qmm_last_error", "qmm_abi_version",
)

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libqmm.so"
_lib = None


class QmmError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__("%s failed with status %d: %s" % (func, status, detail))


class _Plan(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("lanes_per_row", ctypes.c_int32),
        ("units_per_lane", ctypes.c_int32),
        ("rows_per_iter", ctypes.c_int32),
        ("unit_codes", ctypes.c_int32),
        ("split_k", ctypes.c_int32),
        ("tile_m", ctypes.c_int32),
        ("tile_n", ctypes.c_int32),
        ("grid", ctypes.c_int64),
        ("block", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 5),
    ]


class GemvDesc(ctypes.Structure):
    """qmm_gemv_desc: one GEMV of a batched launch (64 bytes)."""
    _fields_ = [
        ("w_packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("mins", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("first_item", ctypes.c_int64),
    ]


assert ctypes.sizeof(GemvDesc) == 64


class GemmMember(ctypes.Structure):
    """qmm_gemm_member: one weight matrix of a grouped GEMM and its output."""
    _fields_ = [
        ("w_packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("mins", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("n", ctypes.c_int64),
    ]


assert ctypes.sizeof(GemmMember) == 40


class KvCache(ctypes.Structure):
    """qmm_kv_cache: a paged key/value cache (device tensors or addresses; the
    tensors have to outlive it and are kept alive by it)."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("k_mins", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("v_mins", ctypes.c_void_p),
        ("pages", ctypes.c_int64),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    def __init__(self, k, k_scales, k_mins, v, v_scales, v_mins, pages, kv_heads, head_dim, page_size, bits,
                 group_size):
        super().__init__(_addr(k), _addr(k_scales), _addr(k_mins), _addr(v), _addr(v_scales), _addr(v_mins),
                         int(pages), int(kv_heads), int(head_dim), int(page_size), int(bits), int(group_size), 0)
        self.keep = (k, k_scales, k_mins, v, v_scales, v_mins)


assert ctypes.sizeof(KvCache) == 80


def library_path() -> str:
    """In-tree libqmm.so, or the file named by $QMM_LIBRARY (tuning builds)."""
    return os.environ.get("QMM_LIBRARY") or os.path.join(_HERE, _LIB_NAME)


def load():
    """Load libqmm.so (built in-tree by ``python -m gemm_qmm_gemv_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            "libqmm.so is not built (%s); run `python -m gemm_qmm_gemv_amd.build`" % path)
    try:
        # torch first: its HIP runtime is then the one the library binds to.
        import torch  # noqa: F401
    except Exception:
        pass
    lib = ctypes.CDLL(path)
    p, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.qmm_gemv.argtypes = [p, p, p, p, p, i64, i64, ci, ci, p]
    lib.qmm_gemm.argtypes = [p, p, p, p, p, i64, i64, i64, ci, ci, p, sz, p]
    lib.qmm_gemv_swiglu.argtypes = [p, p, p, p, p, p, p, p, i64, i64, ci, ci, p]
    lib.qmm_gemv_residual.argtypes = [p, p, p, p, p, p, i64, i64, ci, ci, p]
    lib.qmm_gemm_f16out.argtypes = [p, p, p, p, p, i64, i64, i64, ci, ci, p, sz, p]
    lib.qmm_gemm_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, ci, ci, p]
    lib.qmm_set_override.argtypes = [ctypes.c_char_p, ci]
    lib.qmm_gemm_workspace_bytes.argtypes = [i64, i64, i64, ci, ci]
    lib.qmm_gemm_workspace_bytes.restype = sz
    lib.qmm_moe_gemm.argtypes = [p, p, p, p, p, i64, p, p, i64, i64, i64, i64, ci, ci, p]
    lib.qmm_moe_swiglu.argtypes = [p, p, p, p, p, p, p, p, i64, p, p, i64, i64, i64, i64, ci, ci, p]
    lib.qmm_moe_combine.argtypes = [p, p, p, p, p, i64, p, p, p, p, i64, i64, i64, i64, i64, ci, ci, p]
    lib.qmm_gemm_grouped.argtypes = [p, ci, p, i64, i64, ci, ci, p, ctypes.c_size_t, p]
    lib.qmm_gemm_grouped_workspace_bytes.argtypes = [p, ci, i64, i64, ci, ci]
    lib.qmm_gemm_grouped_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_unpack.argtypes = [p, p, i64, i64, ci, p]
    lib.qmm_gemv_batch_prepare.argtypes = [p, i64, ci, ci]
    lib.qmm_gemv_batched.argtypes = [p, p, i64, ci, ci, p]
    cf, pc = ctypes.c_float, ctypes.POINTER(KvCache)
    lib.qmm_norm_residual.argtypes = [p, ci, i64, p, p, i64, cf, p, p, p, p, i64, i64, cf, p]
    lib.qmm_kv_append.argtypes = [pc, p, p, p, ci, i64, i64, i64, p, p, cf, p, ci, ci, p, p, p, p, p, ci, i64, ci, p]
    lib.qmm_attn_cache.argtypes = [pc, p, p, i64, p, i64, p, i64, ci, ci, cf, p, sz, p]
    lib.qmm_attn_cache_workspace_bytes.argtypes = [pc, i64, ci, ci, i64]
    lib.qmm_attn_cache_workspace_bytes.restype = sz
    lib.qmm_attn_prompt.argtypes = [p, p, p, p, p, i64, i64, ci, ci, ci, i64, i64, i64, i64, cf, p]
    lib.qmm_moe_route.argtypes = [p, ci, i64, p, ci, ci, ci, ci, ci, ci, cf, p, p, p, p, p, p, p, p, sz, i64, ci, p]
    lib.qmm_moe_route_workspace_bytes.argtypes = [i64, ci, ci]
    lib.qmm_moe_route_workspace_bytes.restype = sz
    lib.qmm_quantize_rows.argtypes = [p, ci, i64, p, p, i64, i64, p]
    lib.qmm_gemm_i8.argtypes = [p, p, p, p, p, ci, i64, i64, i64, p]
    lib.qmm_moe_gemm_i8.argtypes = [p, p, p, p, p, i64, p, p, ci, i64, i64, i64, i64, p]
    lib.qmm_moe_swiglu_i8.argtypes = [p, p, p, p, p, p, p, i64, p, p, ci, i64, i64, i64, i64, p]
    lib.qmm_moe_gather.argtypes = [p, ci, p, p, p, p, i64, ci, i64, i64, p]
    lib.qmm_call_words.argtypes = [ci, ctypes.c_char_p]
    lib.qmm_get_plan.argtypes = [ci, i64, i64, i64, ci, ci, ci, sz, ctypes.POINTER(_Plan)]
    for f in ("qmm_gemv", "qmm_gemm", "qmm_moe_gemm", "qmm_unpack", "qmm_get_plan",
              "qmm_gemv_batch_prepare", "qmm_gemv_batched", "qmm_gemv_swiglu", "qmm_gemm_f16out", "qmm_moe_swiglu",
              "qmm_gemv_residual", "qmm_moe_combine", "qmm_gemm_grouped", "qmm_gemm_noalloc",
              "qmm_set_override", "qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_prompt",
              "qmm_moe_route", "qmm_quantize_rows", "qmm_gemm_i8", "qmm_moe_gemm_i8", "qmm_moe_swiglu_i8", "qmm_moe_gather",
              "qmm_call_words"):
        getattr(lib, f).restype = ci
    lib.qmm_status_string.argtypes = [ci]
    lib.qmm_status_string.restype = ctypes.c_char_p
    lib.qmm_last_error.restype = ctypes.c_char_p
    lib.qmm_abi_version.restype = ci
    _lib = lib
    return lib


def _addr(v):
    if v is None:
        return None
    if isinstance(v, int):
        return v
    return v.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # The handle alone: building a Stream object around it costs 2.3 us,
        # as much as the launch.
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, func: str) -> None:
    if status != QMM_OK:
        detail = load().qmm_last_error().decode()
        raise QmmError(status, func, detail)


def qmm_status_string(status: int) -> str:
    return load().qmm_status_string(int(status)).decode()


def qmm_last_error() -> str:
    return load().qmm_last_error().decode()


def qmm_abi_version() -> int:
    return load().qmm_abi_version()


def qmm_gemv(w_packed, scales, mins, x, y, n, k, bits, group_size, stream=None) -> None:
    """y[n] = sum_k (s*q + m)[n][k] x[k] (fp16 x, fp32 y); asynchronous."""
    _check(load().qmm_gemv(_addr(w_packed), _addr(scales), _addr(mins), _addr(x), _addr(y),
                           int(n), int(k), int(bits), int(group_size), _stream(stream)),
           "qmm_gemv")


def qmm_gemv_residual(w_packed, scales, mins, x, residual, y, n, k, bits, group_size,
                      stream=None) -> None:
    """y[n] = residual[n] + sum_k (s*q + m)[n][k] x[k] (residual may be y); asynchronous."""
    _check(load().qmm_gemv_residual(_addr(w_packed), _addr(scales), _addr(mins), _addr(x),
                                    _addr(residual), _addr(y), int(n), int(k), int(bits),
                                    int(group_size), _stream(stream)),
           "qmm_gemv_residual")


def qmm_gemv_swiglu(gate_w, gate_scales, gate_mins, up_w, up_scales, up_mins, x, h, n, k, bits,
                    group_size, stream=None) -> None:
    """h[n] = silu(g[n]) * u[n] with g = Wg x, u = Wu x (fp16 x, fp32 h); asynchronous."""
    _check(load().qmm_gemv_swiglu(_addr(gate_w), _addr(gate_scales), _addr(gate_mins), _addr(up_w),
                                  _addr(up_scales), _addr(up_mins), _addr(x), _addr(h), int(n),
                                  int(k), int(bits), int(group_size), _stream(stream)),
           "qmm_gemv_swiglu")


def qmm_gemm_f16out(w_packed, scales, mins, x, y, m, n, k, bits, group_size, workspace=None,
                    workspace_bytes=0, stream=None) -> None:
    """As qmm_gemm with y fp16 [m][n] (each sum rounded once); asynchronous."""
    _check(load().qmm_gemm_f16out(_addr(w_packed), _addr(scales), _addr(mins), _addr(x), _addr(y),
                                  int(m), int(n), int(k), int(bits), int(group_size), _addr(workspace),
                                  int(workspace_bytes), _stream(stream)),
           "qmm_gemm_f16out")


def qmm_gemm(w_packed, scales, mins, x, y, m, n, k, bits, group_size, workspace=None,
             workspace_bytes=0, stream=None) -> None:
    """y[m][n] = sum_k (s*q + m)[n][k] x[m][k]; asynchronous."""
    _check(load().qmm_gemm(_addr(w_packed), _addr(scales), _addr(mins), _addr(x), _addr(y),
                           int(m), int(n), int(k), int(bits), int(group_size), _addr(workspace),
                           int(workspace_bytes), _stream(stream)),
           "qmm_gemm")


def qmm_gemm_noalloc(w_packed, scales, mins, x, y, m, n, k, bits, group_size, stream=None) -> None:
    """As qmm_gemm with no workspace: the library's own fixed scratch array
    holds any K-split partial sums; asynchronous."""
    _check(load().qmm_gemm_noalloc(_addr(w_packed), _addr(scales), _addr(mins), _addr(x), _addr(y),
                                   int(m), int(n), int(k), int(bits), int(group_size), _stream(stream)),
           "qmm_gemm_noalloc")


def qmm_set_override(name: str, value: int) -> None:
    """Process-wide launch-plan override (value < 0 removes it)."""
    _check(load().qmm_set_override(name.encode(), int(value)), "qmm_set_override")


class overrides:
    """Context manager: ``with overrides(QMM_GEMM_TILE_M=64): ...`` sets the
    named launch-plan overrides and removes them on exit."""

    def __init__(self, **values):
        self.values = values

    def __enter__(self):
        for name, value in self.values.items():
            qmm_set_override(name, value)
        return self

    def __exit__(self, *exc):
        for name in self.values:
            qmm_set_override(name, -1)
        return False


def _members(members):
    arr = (GemmMember * len(members))()
    for d, (w, s, mn, y, n) in zip(arr, members):
        d.w_packed, d.scales, d.mins, d.y, d.n = _addr(w), _addr(s), _addr(mn), _addr(y), int(n)
    return arr


def qmm_gemm_grouped(members, x, m, k, bits, group_size, workspace=None, workspace_bytes=0,
                     stream=None) -> None:
    """members: [(w_packed, scales, mins, y, n)]; y_i = X W_i^T for all in one launch."""
    arr = _members(members)
    _check(load().qmm_gemm_grouped(ctypes.addressof(arr), len(members), _addr(x), int(m), int(k),
                                   int(bits), int(group_size), _addr(workspace), int(workspace_bytes),
                                   _stream(stream)),
           "qmm_gemm_grouped")


def qmm_gemm_grouped_workspace_bytes(members, m, k, bits, group_size) -> int:
    arr = _members(members)
    return int(load().qmm_gemm_grouped_workspace_bytes(ctypes.addressof(arr), len(members), int(m), int(k),
                                                       int(bits), int(group_size)))


def qmm_gemm_workspace_bytes(m, n, k, bits, group_size) -> int:
    return int(load().qmm_gemm_workspace_bytes(int(m), int(n), int(k), int(bits), int(group_size)))


def qmm_moe_gemm(w_packed, scales, mins, x, x_rows, x_rows_count, expert_offsets, y, p_rows,
                 n_experts, n, k, bits, group_size, stream=None) -> None:
    """Expert-grouped rows: y[p] = W_{e(p)} x[x_rows[p]]; asynchronous."""
    _check(load().qmm_moe_gemm(_addr(w_packed), _addr(scales), _addr(mins), _addr(x),
                               _addr(x_rows), int(x_rows_count), _addr(expert_offsets), _addr(y),
                               int(p_rows), int(n_experts), int(n), int(k), int(bits),
                               int(group_size), _stream(stream)),
           "qmm_moe_gemm")


def qmm_moe_combine(w_packed, scales, mins, x, x_rows, x_rows_count, expert_offsets, pair_token,
                    pair_weight, y, n_tokens, p_rows, n_experts, n, k, bits, group_size,
                    stream=None) -> None:
    """y[token[p]] += weight[p] * W_{e(p)} x[row(p)] (accumulates into y); asynchronous."""
    _check(load().qmm_moe_combine(_addr(w_packed), _addr(scales), _addr(mins), _addr(x),
                                  _addr(x_rows), int(x_rows_count), _addr(expert_offsets),
                                  _addr(pair_token), _addr(pair_weight), _addr(y), int(n_tokens),
                                  int(p_rows), int(n_experts), int(n), int(k), int(bits),
                                  int(group_size), _stream(stream)),
           "qmm_moe_combine")


def qmm_moe_swiglu(gate_w, gate_scales, gate_mins, up_w, up_scales, up_mins, x, x_rows,
                   x_rows_count, expert_offsets, h, p_rows, n_experts, n, k, bits, group_size,
                   stream=None) -> None:
    """h[p] = silu(Wg_{e(p)} x[row(p)]) * (Wu_{e(p)} x[row(p)]); asynchronous."""
    _check(load().qmm_moe_swiglu(_addr(gate_w), _addr(gate_scales), _addr(gate_mins), _addr(up_w),
                                 _addr(up_scales), _addr(up_mins), _addr(x), _addr(x_rows),
                                 int(x_rows_count), _addr(expert_offsets), _addr(h), int(p_rows),
                                 int(n_experts), int(n), int(k), int(bits), int(group_size),
                                 _stream(stream)),
           "qmm_moe_swiglu")


# The layer's operators go through qmm_call_words: ctypes converts every
# argument by a call of its own, which took 4.3 us for the append's 23 (packed:
# 2.1) where the kernel of a decode step takes 4.5.
_NORM_WORDS = struct.Struct("=6qd6qdq").pack
_APPEND_WORDS = struct.Struct("=10qd12q").pack
_CACHE_WORDS = struct.Struct("=10qd3q").pack
_PROMPT_WORDS = struct.Struct("=14qdq").pack
_ROUTE_WORDS = struct.Struct("=10qd12q").pack
_QUANTIZE_WORDS = struct.Struct("=8q").pack
_GEMM_I8_WORDS = struct.Struct("=10q").pack
_MOE_GEMM_I8_WORDS = struct.Struct("=14q").pack
_MOE_SWIGLU_I8_WORDS = struct.Struct("=16q").pack
_GATHER_WORDS = struct.Struct("=11q").pack


def _word(v):
    if v is None:
        return 0
    try:
        return v.data_ptr()
    except AttributeError:
        return v  # an address


_CachePointer = ctypes.POINTER(KvCache)


def _cache_word(cache):
    """Address of the struct (0 for None): a KvCache, or what ctypes takes where a pointer to one is declared."""
    if isinstance(cache, KvCache):
        return ctypes.addressof(cache)
    return ctypes.cast(_CachePointer.from_param(cache), ctypes.c_void_p).value or 0


def qmm_norm_residual(y, y_fp16, y_stride, post_weight, gate, gate_stride, scale, residual, h, pre_weight, x, rows, n,
                      eps, stream=None) -> None:
    """h = residual + scale * gate * rmsnorm(y); x = fp16(rmsnorm(h)); asynchronous."""
    status = load().qmm_call_words(0, _NORM_WORDS(_word(y), y_fp16, y_stride, _word(post_weight), _word(gate),
                                                  gate_stride, scale, _word(residual), _word(h), _word(pre_weight),
                                                  _word(x), rows, n, eps, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_norm_residual")


def qmm_kv_append(cache, q, k, v, in_fp16, q_stride, k_stride, v_stride, q_norm, k_norm, eps, inv_freq, rot_dim,
                  interleaved, positions, slots, q_out, k_out, v_out, out_cached, tokens, q_heads, stream=None) -> None:
    """Rotated queries, and keys and values into the cache's slots (``cache``: a ``KvCache``); asynchronous."""
    status = load().qmm_call_words(1, _APPEND_WORDS(_cache_word(cache), _word(q), _word(k), _word(v), in_fp16, q_stride,
                                                    k_stride, v_stride, _word(q_norm), _word(k_norm), eps,
                                                    _word(inv_freq), rot_dim, interleaved, _word(positions),
                                                    _word(slots), _word(q_out), _word(k_out), _word(v_out), out_cached,
                                                    tokens, q_heads, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_kv_append")


def qmm_attn_cache(cache, q, page_table, table_stride, kv_lens, max_kv_len, out, n_seqs, q_len, q_heads, scale,
                   workspace=None, workspace_bytes=0, stream=None) -> None:
    """Attention of each sequence's newest ``q_len`` tokens over its cached rows; asynchronous."""
    status = load().qmm_call_words(2, _CACHE_WORDS(_cache_word(cache), _word(q), _word(page_table), table_stride,
                                                   _word(kv_lens), max_kv_len, _word(out), n_seqs, q_len, q_heads,
                                                   scale, _word(workspace), workspace_bytes, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_attn_cache")


def qmm_attn_cache_workspace_bytes(cache, n_seqs, q_len, q_heads, max_kv_len) -> int:
    return int(load().qmm_attn_cache_workspace_bytes(cache, int(n_seqs), int(q_len), int(q_heads), int(max_kv_len)))


def qmm_attn_prompt(q, k, v, seq_offsets, out, tokens, n_seqs, q_heads, kv_heads, head_dim, q_stride, k_stride,
                    v_stride, out_stride, scale, stream=None) -> None:
    """Causal attention in each of the packed sequences; asynchronous."""
    status = load().qmm_call_words(3, _PROMPT_WORDS(_word(q), _word(k), _word(v), _word(seq_offsets), _word(out),
                                                    tokens, n_seqs, q_heads, kv_heads, head_dim, q_stride, k_stride,
                                                    v_stride, out_stride, scale, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_attn_prompt")


def qmm_moe_route(logits, logits_fp16, logits_stride, bias, sigmoid, n_groups, top_groups, group_best, top_k, renormalize,
                  scale, keep, expert_ids, weights, pair_row, expert_offsets, pair_token, pair_weight, workspace,
                  workspace_bytes, tokens, n_experts, stream=None) -> None:
    """Scores to experts and weights, and the rows grouped by expert; asynchronous."""
    status = load().qmm_call_words(4, _ROUTE_WORDS(_word(logits), logits_fp16, logits_stride, _word(bias), sigmoid, n_groups,
                                                   top_groups, group_best, top_k, renormalize, scale, _word(keep),
                                                   _word(expert_ids), _word(weights), _word(pair_row),
                                                   _word(expert_offsets), _word(pair_token), _word(pair_weight),
                                                   _word(workspace), workspace_bytes, tokens, n_experts, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_moe_route")


def qmm_moe_route_workspace_bytes(tokens, n_experts, top_k) -> int:
    return int(load().qmm_moe_route_workspace_bytes(int(tokens), int(n_experts), int(top_k)))


def qmm_quantize_rows(x, x_fp16, x_stride, codes, scales, rows, k, stream=None) -> None:
    """codes = round(x / scale), scale = max |x| / 127 of each row; asynchronous."""
    status = load().qmm_call_words(5, _QUANTIZE_WORDS(_word(x), x_fp16, x_stride, _word(codes), _word(scales), rows, k,
                                                      _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_quantize_rows")


def qmm_gemm_i8(w, w_scales, x, x_scales, y, y_fp16, m, n, k, stream=None) -> None:
    """y[m][n] = x_scales[m] w_scales[n] sum_k x[m][k] w[n][k] in 8-bit integers; asynchronous."""
    status = load().qmm_call_words(6, _GEMM_I8_WORDS(_word(w), _word(w_scales), _word(x), _word(x_scales), _word(y), y_fp16,
                                                     m, n, k, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_gemm_i8")


def qmm_moe_gemm_i8(w, w_scales, x, x_scales, x_rows, x_rows_count, expert_offsets, y, y_fp16, p_rows, n_experts, n, k,
                    stream=None) -> None:
    """The 8-bit product over rows grouped by expert; asynchronous."""
    status = load().qmm_call_words(7, _MOE_GEMM_I8_WORDS(_word(w), _word(w_scales), _word(x), _word(x_scales), _word(x_rows),
                                                         x_rows_count, _word(expert_offsets), _word(y), y_fp16, p_rows,
                                                         n_experts, n, k, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_moe_gemm_i8")


def qmm_moe_swiglu_i8(gate_w, gate_scales, up_w, up_scales, x, x_scales, x_rows, x_rows_count, expert_offsets, h, h_fp16,
                      p_rows, n_experts, n, k, stream=None) -> None:
    """h[p] = silu(gate[p]) * up[p] in 8-bit integers over rows grouped by expert; asynchronous."""
    status = load().qmm_call_words(8, _MOE_SWIGLU_I8_WORDS(_word(gate_w), _word(gate_scales), _word(up_w), _word(up_scales),
                                                           _word(x), _word(x_scales), _word(x_rows), x_rows_count,
                                                           _word(expert_offsets), _word(h), h_fp16, p_rows, n_experts, n,
                                                           k, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_moe_swiglu_i8")


def qmm_moe_gather(rows, rows_fp16, pair_row, weights, residual, y, tokens, top_k, p_rows, n, stream=None) -> None:
    """y[t] = residual[t] + sum_j weights[t][j] rows[pair_row[t][j]] in a fixed order; asynchronous."""
    status = load().qmm_call_words(9, _GATHER_WORDS(_word(rows), rows_fp16, _word(pair_row), _word(weights), _word(residual),
                                                    _word(y), tokens, top_k, p_rows, n, _stream(stream)))
    if status != QMM_OK:
        _check(status, "qmm_moe_gather")


def qmm_unpack(w_packed, codes, n, k, bits, stream=None) -> None:
    """codes[n][k] (uint8) = the packed codes; asynchronous."""
    _check(load().qmm_unpack(_addr(w_packed), _addr(codes), int(n), int(k), int(bits),
                             _stream(stream)),
           "qmm_unpack")


def qmm_gemv_batch_prepare(descs, bits, group_size) -> None:
    """Fill the library-owned fields of a ``GemvDesc`` array (host memory)."""
    _check(load().qmm_gemv_batch_prepare(ctypes.addressof(descs), len(descs), int(bits),
                                         int(group_size)),
           "qmm_gemv_batch_prepare")


def qmm_gemv_batched(descs_device, descs_host, bits, group_size, stream=None) -> None:
    """One launch over every GEMV of a prepared descriptor array.
    ``descs_device``: device copy (tensor or address); ``descs_host``: the
    ``GemvDesc`` array it was copied from."""
    _check(load().qmm_gemv_batched(_addr(descs_device), ctypes.addressof(descs_host),
                                   len(descs_host), int(bits), int(group_size), _stream(stream)),
           "qmm_gemv_batched")


def qmm_get_plan(op, m, n, k, bits, group_size, cu_count=0, workspace_bytes=0) -> dict:
    """The launch plan the library would use (op 0 gemv, 1 gemm, 2 moe,
    3 batched gemv with n = total rows and k = largest k)."""
    plan = _Plan()
    _check(load().qmm_get_plan(int(op), int(m), int(n), int(k), int(bits), int(group_size),
                               int(cu_count), int(workspace_bytes), ctypes.byref(plan)),
           "qmm_get_plan")
    return {f: getattr(plan, f) for f, _ in _Plan._fields_ if f != "reserved"} | {
        "multipass": bool(plan.reserved[0]), "staged": bool(plan.reserved[1]),
        "late": bool(plan.reserved[2])}
