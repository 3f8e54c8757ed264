"""qmm_attn_prompt against the float64 definition."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import attention_bound, check, dev

pytestmark = pytest.mark.gpu


def expect(q, k, v, offsets, scale, rows=None):
    """Outputs and bounds of the given rows (all by default) as dicts row -> [heads][d]."""
    t, hq, d = q.shape
    g = hq // k.shape[1]
    o, b = {}, {}
    for i in range(len(offsets) - 1):
        lo, hi = offsets[i], offsets[i + 1]
        mine = [r for r in range(lo, hi) if rows is None or r in rows]
        if not mine:
            continue
        oo, bb = np.zeros((len(mine), hq, d)), np.zeros((len(mine), hq, d))
        for h in range(hq):
            vs = v[lo:hi, h // g].astype(np.float64)
            r = layer.attend(q[mine, h], k[lo:hi, h // g], vs, [x - lo + 1 for x in mine], scale)
            oo[:, h] = r[0]
            bb[:, h] = attention_bound(*r, hi - lo, np.abs(vs).max(), d, False, True)
        for n, x in enumerate(mine):
            o[x], b[x] = oo[n], bb[n]
    return o, b


def call(qd, kd, vd, offsets, scale, out):
    t, hq, d = qd.shape
    qmm.qmm_attn_prompt(qd, kd, vd, dev(np.asarray(offsets, np.int32)), out, t, len(offsets) - 1, hq, kd.shape[1], d, qd.stride(0),
                        kd.stride(0), vd.stride(0), out.stride(0), scale)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def inputs(rng, t, hq, hkv, d):
    return tuple(rng.standard_normal((t, h, d)).astype(np.float16) for h in (hq, hkv, hkv))


def compare(got, o, b, what):
    rows = sorted(o)
    check(got[rows], np.stack([o[r] for r in rows]), np.stack([b[r] for r in rows]), what)


CASES = [
    # lengths, hq, hkv, d
    ([1], 1, 1, 64), ([1], 4, 2, 128), ([2, 1, 1, 3], 4, 4, 64), ([64], 2, 1, 128), ([63, 65], 2, 2, 64),
    ([127, 1, 128], 4, 2, 128), ([129, 0, 31, 0, 0, 200], 3, 1, 64), ([300], 16, 8, 128), ([257, 40], 8, 8, 64),
    ([16] * 20, 4, 1, 128), ([1] * 130, 2, 2, 64), ([5, 250, 3, 3, 390], 10, 5, 128),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join([str(len(c[0])), str(sum(c[0]))] + [str(x) for x in c[1:]]))
def test_against_float64(c):
    lens, hq, hkv, d = c
    announce("prompt attention", c)
    rng = np.random.default_rng([sum(lens), hq, d])
    offsets = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = inputs(rng, sum(lens), hq, hkv, d)
    o, b = expect(q, k, v, offsets, d ** -0.5)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    compare(call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out), o, b, "prompt %s" % (c,))


@pytest.mark.parametrize("d,n", [(64, 1700), (128, 2311)])
def test_long_prompts_at_sampled_rows(d, n):
    announce("long prompt", d, n)
    rng = np.random.default_rng([d, n])
    offsets = [0, n - 900, n]
    q, k, v = inputs(rng, n, 8, 2, d)
    rows = set(int(x) for x in rng.integers(0, n, 40)) | {0, 1, n - 901, n - 900, n - 1}
    o, b = expect(q, k, v, offsets, d ** -0.5, rows)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    compare(call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out), o, b, "long prompt")


def test_strided_rows_and_rows_that_no_sequence_covers():
    # q, k and v are parts of one fused product, out is wider than its heads;
    # rows before the first and behind the last sequence stay as they were,
    # whatever their inputs hold.
    rng = np.random.default_rng(31)
    hq, hkv, d, t = 4, 2, 64, 211
    fused = rng.standard_normal((t, (hq + 2 * hkv) * d + 24)).astype(np.float16)
    offsets = [5, 100, 203]
    fused[:5] = np.nan
    fused[203:] = np.inf
    whole = dev(fused)
    q = whole[:, :hq * d].unflatten(1, (hq, d))
    k = whole[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = whole[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    buf = torch.full((t, hq * d + 8), 7.0, dtype=torch.float16, device="cuda")
    out = buf[:, :hq * d].unflatten(1, (hq, d))
    announce("strided prompt")
    got = call(q, k, v, offsets, 0.2, out)
    o, b = expect(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), offsets, 0.2)
    compare(got, o, b, "strided")
    host = buf.cpu().numpy()
    assert (host[:5] == 7).all() and (host[203:] == 7).all() and (host[:, hq * d:] == 7).all()


def test_non_finite_values_reach_only_the_rows_that_see_them():
    rng = np.random.default_rng(32)
    lens = [90, 70, 100]
    offsets = np.concatenate([[0], np.cumsum(lens)])
    for d in (64, 128):
        q, k, v = inputs(rng, 260, 4, 2, d)
        v[40, 0, 3] = np.nan       # rows 40..89, heads 0 and 1
        v[130, 1, 7] = np.inf      # rows 130..159, heads 2 and 3
        k[200, 0, 0] = np.nan      # rows 200..259, heads 0 and 1
        q[10, 3] = np.inf          # row 10, head 3
        out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        announce("non-finite prompt", d)
        got = call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out)
        spoiled = np.zeros((260, 4), dtype=bool)
        spoiled[40:90, :2] = spoiled[130:160, 2:] = spoiled[200:260, :2] = True
        spoiled[10, 3] = True
        finite = np.isfinite(got).all(-1)
        assert np.array_equal(finite, ~spoiled)
        k[200, 0, 0] = 0
        v[40, 0, 3] = v[130, 1, 7] = 0
        q[10, 3] = 0
        o, b = expect(q, k, v, offsets, d ** -0.5)
        o, b = np.stack([o[r] for r in range(260)]), np.stack([b[r] for r in range(260)])
        check(got[~spoiled], o[~spoiled], b[~spoiled], "the rows that do not see them")


def test_large_and_equal_scores():
    rng = np.random.default_rng(33)
    offsets = [0, 150]
    q, k, v = inputs(rng, 150, 2, 2, 64)
    k[:, 1] = 0.5
    announce("large scores")
    for scale in (5.0, 0.0, -0.25):
        o, b = expect(q, k, v, offsets, scale)
        out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        compare(call(dev(q), dev(k), dev(v), offsets, scale, out), o, b, "scale %g" % scale)


def test_offsets_that_are_no_packing_touch_nothing_outside():
    # Decreasing, negative and far offsets: results mean nothing, but guard
    # rows around the buffers stay as they were and the call ends.
    rng = np.random.default_rng(34)
    t, h, d = 130, 2, 64
    q, k, v = (dev(x) for x in inputs(rng, t, h, h, d))
    for offsets in ([0, 400], [-50, 60], [90, 20, 130], [2 ** 31 - 1, -2 ** 31, 0], [130, 130]):
        buf = torch.full((t + 64, h, d), 3.0, dtype=torch.float16, device="cuda")
        announce("odd offsets", offsets)
        call(q, k, v, offsets, 0.1, buf[32:32 + t])
        assert (buf[:32] == 3).all() and (buf[32 + t:] == 3).all()


def test_graph_replays_and_another_stream():
    rng = np.random.default_rng(35)
    q, k, v = (dev(x) for x in inputs(rng, 333, 8, 2, 128))
    off = dev(np.array([0, 100, 333], np.int32))
    announce("prompt replays")
    want = torch.empty_like(q)

    def go(out, stream=None):
        qmm.qmm_attn_prompt(q, k, v, off, out, 333, 2, 8, 2, 128, 1024, 256, 256, 1024, 0.1, stream=stream)
    go(want)
    torch.cuda.synchronize()
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(out)
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        other = torch.zeros_like(out)
        torch.cuda.synchronize()
        g.replay()
        go(other, side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)
