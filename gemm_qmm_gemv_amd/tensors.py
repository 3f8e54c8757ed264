"""Torch-side plumbing around the C ABI: move numpy inputs to device memory
and allocate outputs.  No arithmetic of the method happens here; every
product is computed by the library's kernels.
"""
from __future__ import annotations

import ctypes
import functools
import math

import numpy as np
import torch

from . import (QMM_OK, GemvDesc, KvCache, _check, _stream, load, qmm_attn_cache, qmm_attn_cache_workspace_bytes,
               qmm_attn_prompt, qmm_gemm, qmm_gemm_f16out, qmm_gemm_workspace_bytes, qmm_gemv, qmm_gemv_batch_prepare,
               qmm_gemv_swiglu, qmm_moe_swiglu, qmm_gemv_residual, qmm_moe_combine, qmm_gemm_grouped,
               qmm_gemm_grouped_workspace_bytes,
               qmm_gemv_batched, qmm_kv_append, qmm_moe_gemm, qmm_norm_residual, qmm_unpack)


def device_tensor(a: np.ndarray, device="cuda") -> torch.Tensor:
    """Copy a numpy array to the device, keeping its bits (uint32 -> int32,
    float16 stays float16, uint16 -> int16 views)."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def upload_matrix(q: dict, device="cuda") -> dict:
    """dict(w, scales, mins, n, k, bits, group) with device tensors."""
    out = dict(q)
    for key in ("w", "scales", "mins"):
        out[key] = None if q[key] is None else device_tensor(q[key], device)
    return out


def gemv(dq: dict, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty(dq["n"], dtype=torch.float32, device=x.device)
    qmm_gemv(dq["w"], dq["scales"], dq["mins"], x, y, dq["n"], dq["k"], dq["bits"], dq["group"],
             stream=stream)
    return y


def gemv_residual(dq: dict, x: torch.Tensor, residual: torch.Tensor, y: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """y = residual + W x in one launch (residual may be y)."""
    if y is None:
        y = torch.empty(dq["n"], dtype=torch.float32, device=x.device)
    qmm_gemv_residual(dq["w"], dq["scales"], dq["mins"], x, residual, y, dq["n"], dq["k"], dq["bits"],
                      dq["group"], stream=stream)
    return y


def gemv_swiglu(dg: dict, du: dict, x: torch.Tensor, h: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """h = silu(Wg x) * (Wu x) in one launch (both matrices in one format)."""
    assert dg["n"] == du["n"] and dg["k"] == du["k"]
    assert dg["bits"] == du["bits"] and dg["group"] == du["group"]
    if h is None:
        h = torch.empty(dg["n"], dtype=torch.float32, device=x.device)
    qmm_gemv_swiglu(dg["w"], dg["scales"], dg["mins"], du["w"], du["scales"], du["mins"], x, h,
                    dg["n"], dg["k"], dg["bits"], dg["group"], stream=stream)
    return h


def gemm(dq: dict, x: torch.Tensor, y: torch.Tensor | None = None, workspace=None,
         stream=None, out_fp16: bool = False) -> torch.Tensor:
    """Y = X W^T: fp32 output, or fp16 (qmm_gemm_f16out) with out_fp16."""
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, dq["n"]), dtype=torch.float16 if out_fp16 else torch.float32,
                        device=x.device)
    if workspace is None:
        need = qmm_gemm_workspace_bytes(m, dq["n"], dq["k"], dq["bits"], dq["group"])
        # Zeroed: the split-K arrival counters at its start must read zero
        # before the first call (every call leaves them zero).
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=x.device) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    fn = qmm_gemm_f16out if out_fp16 else qmm_gemm
    fn(dq["w"], dq["scales"], dq["mins"], x, y, m, dq["n"], dq["k"], dq["bits"],
       dq["group"], workspace=workspace, workspace_bytes=ws_bytes, stream=stream)
    return y


def gemm_grouped(dqs: list, x: torch.Tensor, ys: list | None = None, workspace=None,
                 stream=None) -> list:
    """Y_i = X W_i^T for every matrix in dqs (same bits, group and K) in one launch."""
    m = x.shape[0]
    if ys is None:
        ys = [torch.empty((m, dq["n"]), dtype=torch.float32, device=x.device) for dq in dqs]
    members = [(dq["w"], dq["scales"], dq["mins"], y, dq["n"]) for dq, y in zip(dqs, ys)]
    bits, group, k = dqs[0]["bits"], dqs[0]["group"], dqs[0]["k"]
    if workspace is None:
        need = qmm_gemm_grouped_workspace_bytes(members, m, k, bits, group)
        # Zeroed: the arrival counters at its start must read zero at first use.
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=x.device) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    qmm_gemm_grouped(members, x, m, k, bits, group, workspace=workspace, workspace_bytes=ws_bytes,
                     stream=stream)
    return ys


def moe(dst: dict, x: torch.Tensor, x_rows: torch.Tensor | None, offsets: torch.Tensor,
        p_rows: int, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty((p_rows, dst["n"]), dtype=torch.float32, device=x.device)
    qmm_moe_gemm(dst["w"], dst["scales"], dst["mins"], x, x_rows, x.shape[0], offsets, y, p_rows,
                 dst["n_experts"], dst["n"], dst["k"], dst["bits"], dst["group"], stream=stream)
    return y


def moe_combine(dst: dict, x: torch.Tensor, x_rows: torch.Tensor | None, offsets: torch.Tensor,
                pair_token: torch.Tensor, pair_weight: torch.Tensor, p_rows: int, y: torch.Tensor,
                stream=None) -> torch.Tensor:
    """Expert rows with the routing-weighted combine: y[token[p]] += weight[p] * row p
    (y [tokens][n] fp32, accumulated in place)."""
    qmm_moe_combine(dst["w"], dst["scales"], dst["mins"], x, x_rows, x.shape[0], offsets, pair_token,
                    pair_weight, y, y.shape[0], p_rows, dst["n_experts"], dst["n"], dst["k"], dst["bits"],
                    dst["group"], stream=stream)
    return y


def moe_swiglu(dg: dict, du: dict, x: torch.Tensor, x_rows: torch.Tensor | None,
               offsets: torch.Tensor, p_rows: int, h: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Fused gate/up rows of the selected experts: h = silu(g) * u."""
    if h is None:
        h = torch.empty((p_rows, dg["n"]), dtype=torch.float32, device=x.device)
    qmm_moe_swiglu(dg["w"], dg["scales"], dg["mins"], du["w"], du["scales"], du["mins"], x, x_rows,
                   x.shape[0], offsets, h, p_rows, dg["n_experts"], dg["n"], dg["k"], dg["bits"],
                   dg["group"], stream=stream)
    return h


def unpack(dq: dict, stream=None) -> torch.Tensor:
    codes = torch.empty((dq["n"], dq["k"]), dtype=torch.uint8, device=dq["w"].device)
    qmm_unpack(dq["w"], codes, dq["n"], dq["k"], dq["bits"], stream=stream)
    return codes


def _rows(t: torch.Tensor) -> int:
    """Elements between the token rows of t; the rest of each row is dense."""
    if t.dim() == 2:
        (rows, n), (step, inner) = t.shape, t.stride()
        assert n == 1 or inner == 1, "rows must be dense"
        return step if rows > 1 else n
    dense = 1
    for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        assert size == 1 or step == dense, "rows must be dense"
        dense *= size
    return t.stride(0) if t.shape[0] > 1 else dense


def _output(shape: tuple, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """A tensor that a call on `stream` writes.  On another stream than the current one it comes from that stream's
    memory (a block of the current one may still be read by work behind which the call does not wait), and goes back
    only when the current stream, on which the caller may use it, is done with it too."""
    if stream is None or _stream(stream) == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _on_device(*ts) -> None:
    """Refuses tensors that are not all on the current GPU, where the call is launched (addresses are not looked at)."""
    here = None
    for t in ts:
        if not isinstance(t, torch.Tensor):
            continue
        at = t.get_device()  # -1: host memory
        if at != here:
            if at < 0 or here is not None or at != torch.cuda.current_device():
                raise ValueError("a tensor is on %s, not on the current GPU" % t.device)
            here = at


def _dense(name: str, t: torch.Tensor | None, dtype: torch.dtype, *shape: int) -> None:
    """Refuses what the kernels, which go by addresses, would take for something else: another type, gaps between
    elements, a last axis of another length, fewer rows than `shape` has."""
    if t is None or (t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise ValueError("%s is %s, not %s" % (name, t.dtype, dtype))
    flat = t.dim() == 1 and len(shape) > 1  # rows behind each other
    if not t.is_contiguous() or (t.shape[-1:] != shape[-1:] and not flat) or t.numel() < math.prod(shape):
        raise ValueError("%s of shape %s and strides %s is not dense or not %s"
                         % (name, tuple(t.shape), t.stride(), list(shape)))


def _vector(name: str, t: torch.Tensor | None, dtype: torch.dtype, size: int) -> None:
    """The same for `size` neighbouring values or more."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError("%s is %s, not %s" % (name, t.dtype, dtype))
    if not t.is_contiguous() or t.numel() < size:
        raise ValueError("%s of shape %s and strides %s is not dense or below %d values"
                         % (name, tuple(t.shape), t.stride(), size))


def _floating(name: str, t: torch.Tensor | None) -> None:
    if t is not None and t.dtype not in (torch.float16, torch.float32):
        raise ValueError("%s is %s, neither fp16 nor fp32" % (name, t.dtype))


def _gate_rows(gate: torch.Tensor | None, rows: int, n: int) -> int:
    """Elements between the gate rows of neighbouring rows, 0: one row for all."""
    if gate is None:
        return 0
    if gate.shape[-1:] != (n,) or (gate.numel() != n and (gate.dim() != 2 or gate.shape[0] < rows)):
        raise ValueError("a gate of shape %s for %d rows of %d" % (tuple(gate.shape), rows, n))
    if gate.numel() == n:
        _dense("gate", gate, torch.float32, n)
        return 0
    if gate.dtype != torch.float32:
        raise ValueError("gate is %s, not fp32" % gate.dtype)
    return _rows(gate)


def norm_residual(y: torch.Tensor | None, residual: torch.Tensor | None, pre: torch.Tensor | None, eps: float = 1e-6,
                  post: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  h: torch.Tensor | None = None, x: torch.Tensor | None = None, stream=None):
    """(h, x): h = residual + scale * gate * rmsnorm(y), x = fp16(rmsnorm(h) * pre), in one launch.

    y fp32 or fp16 rows (a column range of a wider tensor will do), None: h is
    the residual as it is; post None: y without a norm; gate [n], [1, n] or [rows, n];
    h may be the residual (updated in place)."""
    _on_device(y, residual, pre, post, gate, h, x)
    like = residual if y is None else y
    rows, n = like.shape
    if y is None:
        h = residual
    elif h is None:
        h = _output((rows, n), torch.float32, y.device, stream)
    if x is None:
        x = _output((rows, n), torch.float16, like.device, stream)
    _floating("y", y)
    _dense("residual", residual, torch.float32, rows, n)
    _dense("h", h, torch.float32, rows, n)
    _dense("x", x, torch.float16, rows, n)
    _dense("post", post, torch.float32, n)
    _dense("pre", pre, torch.float32, n)
    qmm_norm_residual(y, y is not None and y.dtype == torch.float16, 0 if y is None else _rows(y), post, gate,
                      0 if y is None else _gate_rows(gate, rows, n), scale, residual, None if y is None else h, pre, x, rows, n,
                      eps, stream=stream)
    return h, x


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, bits: int = 4, group: int = 64,
             device="cuda") -> KvCache:
    """A paged key/value cache of zeros (the handle keeps its tensors)."""
    def rows():
        return torch.zeros((pages, kv_heads, page_size, head_dim * bits // 32), dtype=torch.int32, device=device)

    def meta():
        if bits == 16:
            return None
        return torch.zeros((pages, kv_heads, head_dim // group, page_size), dtype=torch.float16, device=device)

    return KvCache(rows(), meta(), meta(), rows(), meta(), meta(), pages, kv_heads, head_dim, page_size, bits, group)


def kv_append(cache: KvCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
              slots: torch.Tensor | None, inv_freq: torch.Tensor | None = None, interleaved: bool = False,
              q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6,
              out: torch.Tensor | None = None, prompt_rows: bool = False, cached_values: bool = False, stream=None):
    """New tokens' rows q, k and v [tokens, heads * head_dim] (column ranges of one fused product will do): returns the
    normed and rotated queries [tokens, q_heads, head_dim] and stores keys and values in `slots` (int64; positions int32).
    With prompt_rows it returns (q, k, v) for attn_prompt, k and v as the cache stands for them if cached_values."""
    _on_device(q, k, v, positions, slots, inv_freq, q_norm, k_norm, out, *getattr(cache, "keep", ()))
    tokens, d = q.shape[0], cache.head_dim
    width = math.prod(q.shape[1:])
    q_heads = width // d
    _floating("q", q)
    assert q.dtype == k.dtype == v.dtype
    for name, t, heads in (("q", q, q_heads), ("k", k, cache.kv_heads), ("v", v, cache.kv_heads)):
        if t.shape != (tokens, heads * d) and (t.shape[0] < tokens or math.prod(t.shape[1:]) != heads * d):
            raise ValueError("%s of shape %s for %d tokens of %d heads of %d" % (name, tuple(t.shape), tokens, heads, d))
    _vector("out", out, torch.float16, tokens * width)
    _vector("inv_freq", inv_freq, torch.float32, 0)
    _vector("q_norm", q_norm, torch.float32, d)
    _vector("k_norm", k_norm, torch.float32, d)
    if out is None:
        out = _output((tokens, q_heads, d), torch.float16, q.device, stream)
    k_out = v_out = None
    if prompt_rows:
        k_out, v_out = (_output((tokens, cache.kv_heads, d), torch.float16, q.device, stream) for _ in range(2))
    if inv_freq is not None:
        _vector("positions", positions, torch.int32, tokens)
    _vector("slots", slots, torch.int64, tokens)
    qmm_kv_append(cache, q, k, v, q.dtype == torch.float16, _rows(q), _rows(k), _rows(v), q_norm, k_norm, eps,
                  inv_freq, 0 if inv_freq is None else 2 * inv_freq.numel(), interleaved, positions, slots, out,
                  k_out, v_out, cached_values, tokens, q_heads, stream=stream)
    return (out, k_out, v_out) if prompt_rows else out


def attn_workspace(cache: KvCache, n_seqs: int, q_len: int, q_heads: int, max_kv_len: int,
                   device="cuda") -> torch.Tensor:
    """Scratch for attn_cache calls up to this size, one after another on one stream."""
    need = qmm_attn_cache_workspace_bytes(cache, n_seqs, q_len, q_heads, max_kv_len)
    # Zeroed: the arrival counters at its start must read zero before the
    # first call (every call leaves them zero).
    return torch.zeros(max(need, 16), dtype=torch.uint8, device=device)


def attn_cache(cache: KvCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor, max_kv_len: int,
               scale: float | None = None, q_len: int = 1, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q [n_seqs * q_len, q_heads, head_dim], each sequence's newest q_len tokens, over the cache
    (page_table [n_seqs, pages of a sequence] and kv_lens [n_seqs] int32)."""
    _on_device(q, page_table, kv_lens, out, workspace, *getattr(cache, "keep", ()))
    n_seqs, q_heads = kv_lens.shape[0], q.shape[-2]
    _vector("kv_lens", kv_lens, torch.int32, n_seqs)
    if page_table.dtype != torch.int32:
        raise ValueError("page_table is %s, not torch.int32" % page_table.dtype)
    if page_table.dim() != 2 or page_table.shape[0] < n_seqs or (page_table.shape[1] > 1 and page_table.stride(1) != 1) \
            or page_table.shape[1] * cache.page_size < max_kv_len:
        raise ValueError("a page_table of shape %s and strides %s for %d sequences of up to %d rows"
                         % (tuple(page_table.shape), page_table.stride(), n_seqs, max_kv_len))
    _dense("q", q, torch.float16, n_seqs * q_len * q_heads, cache.head_dim)
    _vector("out", out, torch.float16, q.numel())
    assert q.is_contiguous() and q.numel() == n_seqs * q_len * q_heads * cache.head_dim
    if out is None:
        out = _output(tuple(q.shape), torch.float16, q.device, stream)
    if workspace is None:
        # Made and given back on the current stream.
        assert stream is None, "a call on another stream needs a workspace of its own"
        workspace = attn_workspace(cache, n_seqs, q_len, q_heads, max_kv_len, q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace is not dense")
    qmm_attn_cache(cache, q, page_table, page_table.stride(0) if n_seqs > 1 else page_table.shape[1], kv_lens,
                   max_kv_len, out, n_seqs, q_len, q_heads, cache.head_dim ** -0.5 if scale is None else scale,
                   workspace, workspace.numel() * workspace.element_size(), stream=stream)
    return out


def attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_offsets: torch.Tensor,
                scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention in each of the sequences packed in q [tokens, q_heads, d], k and v [tokens, kv_heads, d]
    (seq_offsets [sequences + 1] int32)."""
    _on_device(q, k, v, seq_offsets, out)
    tokens, q_heads, d = q.shape
    _vector("seq_offsets", seq_offsets, torch.int32, 1)
    for name, t, row in (("q", q, (q_heads, d)), ("k", k, (k.shape[1], d)), ("v", v, (k.shape[1], d)), ("out", out, (q_heads * d,))):
        if t is None or (t.dtype == torch.float16 and t.shape == (tokens, *row)):
            continue
        if t.dtype != torch.float16:
            raise ValueError("%s is %s, not fp16" % (name, t.dtype))
        got = t.shape[1:] if name != "out" else (math.prod(t.shape[1:]),)
        if t.shape[0] < tokens or got != row:
            raise ValueError("%s of shape %s for %d tokens of %s values" % (name, tuple(t.shape), tokens, row))
    if out is None:
        out = _output((tokens, q_heads, d), torch.float16, q.device, stream)
    qmm_attn_prompt(q, k, v, seq_offsets, out, tokens, seq_offsets.numel() - 1, q_heads, k.shape[1], d, _rows(q),
                    _rows(k), _rows(v), _rows(out), d ** -0.5 if scale is None else scale, stream=stream)
    return out


class GemvBatch:
    """A prepared batched launch: host descriptors plus their device copy.

    items: list of (device matrix dict, x tensor [k], y tensor [n]); every
    matrix must share bits and group size."""

    def __init__(self, items, bits: int, group: int, device="cuda"):
        self.bits, self.group = bits, group
        self.host = (GemvDesc * len(items))()
        for d, (dq, x, y) in zip(self.host, items):
            assert dq["bits"] == bits and dq["group"] == group
            ptr = lambda t: 0 if t is None else t.data_ptr()
            d.w_packed, d.scales, d.mins = ptr(dq["w"]), ptr(dq["scales"]), ptr(dq["mins"])
            d.x, d.y = x.data_ptr(), y.data_ptr()
            d.n, d.k = dq["n"], dq["k"]
        qmm_gemv_batch_prepare(self.host, bits, group)
        raw = np.frombuffer(bytes(self.host), dtype=np.uint8).copy()
        self.device = torch.from_numpy(raw).to(device)
        self.keep = items  # the buffers must outlive the batch
        # The call's fixed arguments, converted once: a launch then costs one
        # foreign call (the host time before the first launch of a timed
        # region counts in it).
        self._launch = functools.partial(load().qmm_gemv_batched, self.device.data_ptr(),
                                         ctypes.addressof(self.host), len(self.host), bits, group)

    def __call__(self, stream=None) -> None:
        status = self._launch(_stream(stream))
        if status != QMM_OK:
            _check(status, "qmm_gemv_batched")
