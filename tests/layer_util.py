"""Inputs and bounds shared by the tests of the attention half of a decoder layer."""
from __future__ import annotations

import numpy as np
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer

E32 = 2.0 ** -24   # half a step of fp32, relative
E16 = 2.0 ** -11   # half a step of fp16, relative
TINY16 = 2.0 ** -25  # half a step of fp16 below its normal range


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).cuda()


def empty_cache(rng, pages, heads, d, page, bits, group, garbage=False):
    """Host arrays of a cache; `garbage`: every scale, min or fp16 value that no row sets is NaN."""
    words = d * bits // 32
    out = {}
    for side in "kv":
        if bits == 16:
            rows = rng.standard_normal((pages, heads, page, d)).astype(np.float16)
            if garbage:
                rows[:] = np.nan
            out[side] = rows.view(np.uint32)
            out[side + "s"] = out[side + "m"] = None
            continue
        out[side] = rng.integers(0, 1 << 32, size=(pages, heads, page, words), dtype=np.uint32)
        shape = (pages, heads, d // group, page)
        span = 4.6 + 0.5 * rng.standard_normal(shape)
        out[side + "s"] = (span / (2 ** bits - 1)).astype(np.float16)
        out[side + "m"] = (-0.5 * span + 0.2 * rng.standard_normal(shape)).astype(np.float16)
        if garbage:
            out[side + "s"][:] = np.nan
            out[side + "m"][:] = np.inf
    return out


class DeviceCache:
    def __init__(self, host, pages, heads, d, page, bits, group):
        self.t = {k: None if v is None else dev(v) for k, v in host.items()}
        self.shape = (pages, heads, d, page, bits, group)
        t = self.t
        self.handle = qmm.KvCache(t["k"], t["ks"], t["km"], t["v"], t["vs"], t["vm"], pages, heads, d, page, bits, group)

    def host(self):
        out = {}
        for k, v in self.t.items():
            out[k] = None if v is None else v.cpu().numpy()
            if k in "kv":
                out[k] = out[k].view(np.uint32)
        return out


def held(host, side, bits, group):
    return layer.cache_values(host[side], host[side + "s"], host[side + "m"], bits, group)


def attention_bound(o, a, total, smax, terms, vmax, d, v_rounded, p_rounded):
    """How far outputs may be from the float64 ones.

    A score is a sum of d products and, over a quantized cache, of its groups'
    factors: below d + 8 roundings of terms whose magnitudes add up to smax
    (codes and mins apart they may add up to three times as much, as a code's
    share and its min can cancel), so es = 3 (d + 8) E32 smax, plus the
    exponential's own 2^-21 or so.  That error enters every weight and the sum
    of weights: 2 (es + 2^-21) a.  The sums over `terms` rows are fp32 in any
    order of tiles: at most 64 + terms / 32 additions deep.  Values rounded to
    fp16 add E16 a, probabilities rounded to fp16 E16 a and, below fp16's
    normal range, TINY16 each: terms * TINY16 * vmax / total.  The output is
    rounded once."""
    es = 3 * (d + 8) * E32 * smax[:, None] + 2.0 ** -21
    b = 2 * np.expm1(es) * a + 2 * (64 + terms / 32) * E32 * a
    if v_rounded:
        b = b + E16 * a
    if p_rounded:
        b = b + E16 * a
    b = b + terms * TINY16 * vmax / total[:, None]
    return b + E16 * np.abs(o) * 1.01 + TINY16


def check(got, ref, bound, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), "%s: %d values not finite" % (what, (~np.isfinite(got)).sum())
    err = np.abs(got - ref)
    bad = err > bound
    if bad.any():
        i = np.unravel_index(np.argmax(err - bound), err.shape)
        raise AssertionError("%s: %d of %d outside; worst at %s: %r for %r, bound %r"
                             % (what, bad.sum(), bad.size, i, got[i], ref[i], np.broadcast_to(bound, err.shape)[i]))
    if err.size:
        print("[parity] %s: worst error / bound %.3f" % (what, float((err / bound).max())), flush=True)
