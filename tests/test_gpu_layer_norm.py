"""qmm_norm_residual against the float64 definition."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16, check, dev

pytestmark = pytest.mark.gpu

EPS = 1e-6


def bounds(u, h, x, scale, pre, r_steps=64):
    """A row's root mean square is off by the depth of its sum (at most 32 + 6 + 16 additions, halved by the root) and a
    few roundings, the elements by a few more: below 64 steps of E32 in all.  x inherits h's error through the norm."""
    eu = 0.0 if u is None else r_steps * E32 * np.abs(scale * u)
    eh = eu + 2 * E32 * np.abs(h)
    gain = np.abs(x) / np.maximum(np.abs(h), 1e-300)
    rms = np.sqrt(np.mean(h * h, axis=-1, keepdims=True))
    er = np.sqrt(np.mean(np.square(eh), axis=-1, keepdims=True)) / np.maximum(rms, 1e-300)
    ex = eh * gain + np.abs(x) * (er + r_steps * E32)
    return eh + 1e-37, ex + E16 * np.abs(x) * 1.01 + TINY16


def case(rng, rows, n, y16, post, gate, with_y=True, with_res=True):
    y = rng.standard_normal((rows, n)).astype(np.float16 if y16 else np.float32) if with_y else None
    pw = (1 + 0.1 * rng.standard_normal(n)).astype(np.float32) if post else None
    g = None
    if gate != "none":
        g = (1 / (1 + np.exp(-rng.standard_normal((1 if gate == "shared" else rows, n))))).astype(np.float32)
    res = (3 * rng.standard_normal((rows, n))).astype(np.float32) if with_res else None
    pre = (1 + 0.1 * rng.standard_normal(n)).astype(np.float32)
    return y, pw, g, res, pre


def run(y, y16, pw, g, scale, res, pre, rows, n, h=None, x=None, keep_h=True, keep_x=True):
    if keep_h and h is None:
        h = torch.full((rows, n), float("nan"), device="cuda")
    if keep_x and x is None:
        x = torch.full((rows, n), float("nan"), dtype=torch.float16, device="cuda")
    gs = 0 if g is None or g.shape[0] == 1 else g.stride(0)
    qmm.qmm_norm_residual(y, y16, 0 if y is None else y.stride(0), pw, g, gs, scale, res, h, pre, x, rows, n, EPS)
    torch.cuda.synchronize()
    return h, x


def ten(a):
    return None if a is None else dev(a)


@pytest.mark.parametrize("rows,n,y16,post,gate", [
    (1, 1, False, True, "none"), (3, 7, True, True, "rows"), (1, 1024, False, False, "none"),
    (5, 1023, False, True, "shared"), (2, 1025, True, False, "rows"), (37, 2048, False, True, "shared"),
    (4, 2052, True, True, "rows"), (9, 4096, True, True, "rows"), (3, 5120, False, True, "none"),
    (2, 8192, True, False, "shared"), (2, 8193, False, True, "rows"), (2, 32768, True, True, "rows"),
    (1, 32767, False, True, "shared"), (700, 64, False, True, "rows"),
])
def test_against_float64(rows, n, y16, post, gate):
    announce("norm", rows, n, y16, post, gate)
    rng = np.random.default_rng([rows, n, 1])
    y, pw, g, res, pre = case(rng, rows, n, y16, post, gate)
    u, h, x = layer.norm_residual(y, pw, g, 0.7, res, pre, EPS)
    hd, xd = run(ten(y), y16, ten(pw), ten(g), 0.7, ten(res), ten(pre), rows, n)
    eh, ex = bounds(u, h, x, 0.7, pre)
    check(hd.cpu().numpy(), h, eh, "norm h %d x %d" % (rows, n))
    check(xd.cpu().numpy(), x, ex, "norm x %d x %d" % (rows, n))


def test_without_y_the_residual_is_normed_and_not_written():
    rng = np.random.default_rng(2)
    _, _, _, res, pre = case(rng, 6, 640, False, False, "none")
    rd = ten(res)
    _, xd = run(None, False, None, None, 1.0, rd, ten(pre), 6, 640, keep_h=False)
    _, h, x = layer.norm_residual(None, None, None, 1.0, res, pre, EPS)
    _, ex = bounds(None, h, x, 1.0, pre)
    check(xd.cpu().numpy(), x, ex, "norm of the residual")
    assert np.array_equal(rd.cpu().numpy(), res)


def test_no_residual_no_weight_and_one_output_only():
    rng = np.random.default_rng(3)
    y, _, _, _, _ = case(rng, 5, 96, False, False, "none")
    u, h, x = layer.norm_residual(y, None, None, 2.5, None, None, EPS)
    eh, ex = bounds(u, h, x, 2.5, None)
    hd, _ = run(ten(y), False, None, None, 2.5, None, None, 5, 96, keep_x=False)
    check(hd.cpu().numpy(), h, eh, "h alone")
    _, xd = run(ten(y), False, None, None, 2.5, None, None, 5, 96, keep_h=False)
    check(xd.cpu().numpy(), x, ex, "x alone")


@pytest.mark.parametrize("n", [512, 515])
def test_residual_in_place_strided_and_unaligned(n):
    # h is the residual itself; y and gate are column ranges of wider arrays,
    # and every pointer is aligned to its elements only.
    rng = np.random.default_rng([4, n])
    rows = 11
    y, pw, g, res, pre = case(rng, rows, n, True, True, "rows")
    wide = torch.zeros((rows, n + 37), dtype=torch.float16, device="cuda")
    yd = wide[:, 5:5 + n]
    yd.copy_(dev(y))
    gw = torch.zeros((rows, n + 3), device="cuda")
    gd = gw[:, 1:1 + n]
    gd.copy_(dev(g))
    hbuf = torch.zeros(rows * n + 1, device="cuda")
    hd = hbuf[1:].view(rows, n)
    hd.copy_(dev(res))
    xbuf = torch.zeros(rows * n + 1, dtype=torch.float16, device="cuda")
    xd = xbuf[1:].view(rows, n)
    run(yd, True, ten(pw), gd, -0.3, hd, ten(pre), rows, n, h=hd, x=xd)
    u, h, x = layer.norm_residual(y, pw, g, -0.3, res, pre, EPS)
    eh, ex = bounds(u, h, x, -0.3, pre)
    check(hd.cpu().numpy(), h, eh, "in-place h")
    check(xd.cpu().numpy(), x, ex, "in-place x")
    assert xbuf[0] == 0 and hbuf[0] == 0


def test_zero_rows_of_zeros_and_non_finite():
    # A row of zeros stays zero (eps keeps the root from zero); a NaN stays in its row.
    rng = np.random.default_rng(5)
    res = rng.standard_normal((3, 256)).astype(np.float32)
    res[0] = 0
    res[1, 7] = np.nan
    _, xd = run(None, False, None, None, 1.0, dev(res), None, 3, 256, keep_h=False)
    x = xd.cpu().numpy()
    assert (x[0] == 0).all() and np.isnan(x[1]).all() and np.isfinite(x[2]).all()


def test_graph_replays_and_another_stream():
    rng = np.random.default_rng(6)
    y, pw, g, res, pre = (ten(a) for a in case(rng, 33, 1536, False, True, "rows"))
    h0, x0 = run(y, False, pw, g, 0.5, res, pre, 33, 1536)
    h, x = torch.empty_like(h0), torch.empty_like(x0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qmm.qmm_norm_residual(y, False, 1536, pw, g, 1536, 0.5, res, h, pre, x, 33, 1536, EPS)
    s.synchronize()
    assert torch.equal(h, h0) and torch.equal(x, x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_norm_residual(y, False, 1536, pw, g, 1536, 0.5, res, h, pre, x, 33, 1536, EPS)
    for _ in range(4):
        h.zero_()
        x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h0) and torch.equal(x, x0)
