"""CPU oracle of the attention half of a decoder layer: the norm between two
products, the append to a paged cache, attention over the cache and over whole
prompts.  Plain definitions in numpy float64, one loop per thing that the
definition names; test infrastructure only, and no code shared with the
library.
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) [* weight] along the last axis."""
    x = np.asarray(x, dtype=np.float64)
    r = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return r if weight is None else r * np.asarray(weight, dtype=np.float64)


def norm_residual(y, post, gate, scale, residual, pre, eps):
    """(u, h, x) of the norm, gate and residual step (x not rounded)."""
    h = 0.0 if residual is None else np.asarray(residual, dtype=np.float64)
    u = None
    if y is not None:
        u = np.asarray(y, dtype=np.float64)
        if post is not None:
            u = rms_norm(u, post, eps)
        if gate is not None:
            u = u * np.asarray(gate, dtype=np.float64)
        h = h + scale * u
    return u, h, rms_norm(h, pre, eps)


def rotate(x, positions, inv_freq, rot, interleaved):
    """Rotation of the first `rot` elements of x [tokens][heads][d] by position."""
    x = np.array(x, dtype=np.float64)
    for t, pos in enumerate(positions):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            ang = float(pos) * float(inv_freq[i])
            xa, xb = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a] = xa * np.cos(ang) - xb * np.sin(ang)
            x[t, :, b] = xb * np.cos(ang) + xa * np.sin(ang)
    return x


def unpack_rows(words, bits):
    """Codes of uint32 rows: code d at stream bits [d * bits, (d + 1) * bits)."""
    w = np.ascontiguousarray(words).view(np.uint32)
    stream = np.unpackbits(w.view(np.uint8), axis=-1, bitorder="little")
    parts = stream.reshape(*w.shape[:-1], -1, bits).astype(np.int64)
    return (parts << np.arange(bits)).sum(-1)


def pack_rows(codes, bits):
    """The inverse of unpack_rows."""
    c = np.asarray(codes, dtype=np.int64)
    flat = ((c[..., None] >> np.arange(bits)) & 1).astype(np.uint8).reshape(*c.shape[:-1], -1)
    return np.packbits(flat, axis=-1, bitorder="little").view(np.uint32)


def cache_values(rows, scales, mins, bits, group):
    """float64 values [pages][heads][page][d] that a side of a cache stands for."""
    if bits == 16:
        return np.ascontiguousarray(rows).view(np.float16).astype(np.float64)
    codes = unpack_rows(rows, bits).astype(np.float64)
    s = np.repeat(np.swapaxes(scales.astype(np.float64), -1, -2), group, axis=-1)
    m = np.repeat(np.swapaxes(mins.astype(np.float64), -1, -2), group, axis=-1)
    return codes * s + m


def sequence_rows(values, table, length):
    """Rows [length][heads][d] of one sequence through its page-table row."""
    page = values.shape[2]
    return np.stack([values[table[t // page], :, t % page] for t in range(length)]) if length else \
        np.zeros((0,) + (values.shape[1], values.shape[3]))


def attend(q, k, v, limits, scale):
    """Rows of q [n][d] over k, v [m][d], row i seeing the first limits[i] of them.

    Returns (o, a, l, smax): outputs, sum of weight * |v|, the softmax's sum
    (of exponentials of the distance to the maximum) and the largest
    scale * sum |q k|, from which tests derive their bounds.  A row that sees
    nothing is zero."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, d = q.shape
    o, a = np.zeros((n, d)), np.zeros((n, d))
    total, smax = np.ones(n), np.zeros(n)
    for i in range(n):
        m = int(limits[i])
        if m <= 0:
            continue
        s = scale * (k[:m] @ q[i])
        e = np.exp(s - s.max())
        total[i] = e.sum()
        o[i] = (e / total[i]) @ v[:m]
        a[i] = (e / total[i]) @ np.abs(v[:m])
        smax[i] = abs(scale) * (np.abs(k[:m]) @ np.abs(q[i])).max()
    return o, a, total, smax
