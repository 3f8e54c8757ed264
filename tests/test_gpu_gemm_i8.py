"""qmm_gemm_i8, qmm_moe_gemm_i8 and qmm_moe_swiglu_i8: exact sums of 8-bit codes, scaled."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16, dev

pytestmark = pytest.mark.gpu


def codes(rng, *shape):
    return rng.integers(-128, 128, shape).astype(np.int8)


def scales(rng, *shape):
    return ((0.5 + rng.random(shape)) * 2.0 ** -12).astype(np.float32)


def check(got, want, bound, covered, what):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got[covered]), np.isnan(want[covered])), what
    ok = covered[:, None] & ~np.isnan(want)
    err = np.abs(got - want)[ok]
    assert (err <= bound[ok]).all(), "%s: %d of %d outside, worst %.2f of the bound" % (
        what, (err > bound[ok]).sum(), err.size, (err / bound[ok]).max())


def plain_bound(y, f16):
    """The sum is exact; its conversion and the two scales round once each, an fp16 output once more."""
    return 3.01 * E32 * np.abs(y) + (E16 * 1.01 * np.abs(y) + TINY16 if f16 else 0) + 1e-40


def gated_bound(g, u, h, f16):
    """g and u to 3 E32 each.  silu's relative slope is 1 + g (1 - sigmoid(g)), at most 1 + |g|; the exponential is good to
    4 E32, its sum, the quotient and the product with u round once each, and e^-g past fp32 leaves nothing of |g| e^g."""
    b = E32 * np.abs(h) * (3 * (1 + np.abs(g)) + 3 + 4 + 4) + 1e-35 * np.abs(u) + 1e-40
    return b + (E16 * 1.01 * np.abs(h) + TINY16 if f16 else 0)


def dense(m, n, k, f16, seed=0, extremes=False):
    rng = np.random.default_rng(m * 7 + n * 3 + k + seed)
    announce("gemm_i8", m, n, k, "fp16" if f16 else "fp32", "extremes" if extremes else "")
    w, x, ws, xs = codes(rng, n, k), codes(rng, m, k), scales(rng, n), scales(rng, m)
    if extremes:
        w[:], x[:] = -128, -128
        w[::2] = 127
    y = torch.full((m + 1, n), 77.0, dtype=torch.float16 if f16 else torch.float32, device="cuda")
    qmm.qmm_gemm_i8(dev(w), dev(ws), dev(x), dev(xs), y, f16, m, n, k)
    torch.cuda.synchronize()
    assert (y[m] == 77).all()
    want = moe.product_i8(w, ws, x, xs)
    check(y[:m].float().cpu().numpy(), want, plain_bound(want, f16), np.ones(m, dtype=bool), "gemm_i8")


@pytest.mark.parametrize("m", [1, 2, 3, 15, 16, 17, 31, 33, 48, 64, 65, 100, 127, 128, 129, 200, 257, 300, 513])
@pytest.mark.parametrize("n,k", [(64, 64), (130, 96), (256, 1024), (1000, 544)])
def test_sizes(m, n, k):
    dense(m, n, k, m % 2 == 0)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 15, 16, 17, 31, 33, 63, 65, 127, 129, 255, 257, 383, 1001])
@pytest.mark.parametrize("m", [1, 20, 70, 140, 600])
def test_columns(m, n):
    dense(m, n, 160, n % 2 == 0)


@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 192, 224, 256, 288, 480, 512, 544, 1056, 2048, 4128, 8192, 32768])
@pytest.mark.parametrize("m", [1, 40, 150])
def test_depths(m, k):
    dense(m, 72, k, k % 64 == 0)


@pytest.mark.parametrize("m", [1, 30, 130, 300])
def test_largest_sums(m):
    # 128 * 128 * 32768 = 2^29.
    dense(m, 40, 32768, False, extremes=True)


@pytest.mark.parametrize("m,n,k", [(1, 8192, 2048), (37, 8192, 2048), (128, 2048, 8192), (1024, 2048, 1024), (700, 4099, 512), (2048, 1000, 256)])
def test_larger(m, n, k):
    dense(m, n, k, True)


def on_device(x, xs, w, ws):
    """float64 [rows][n] on the GPU: sums below 2^53 are exact."""
    return (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()[None, :]


@pytest.mark.parametrize("m,n,k,f16", [(4096, 4096, 256, True), (4099, 5001, 160, False), (2500, 16384, 128, True), (1000, 8192, 512, False),
                                       (520, 4096, 2048, True), (300, 16384, 96, False), (8192, 2048, 32, True)])
def test_many_tiles(m, n, k, f16):
    # Every tile size, several tiles for each work-group, one and more steps of K.
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    announce("gemm_i8 many tiles", m, n, k)
    w = torch.randint(-128, 128, (n, k), device="cuda", dtype=torch.int8, generator=g)
    x = torch.randint(-128, 128, (m, k), device="cuda", dtype=torch.int8, generator=g)
    ws, xs = torch.rand(n, device="cuda", generator=g) * 1e-4, torch.rand(m, device="cuda", generator=g)
    y = torch.full((m + 1, n), 77.0, dtype=torch.float16 if f16 else torch.float32, device="cuda")
    qmm.qmm_gemm_i8(w, ws, x, xs, y, f16, m, n, k)
    torch.cuda.synchronize()
    assert (y[m] == 77).all()
    want = on_device(x, xs, w, ws)
    bound = 3.01 * E32 * want.abs() + (E16 * 1.01 * want.abs() + TINY16 if f16 else 0) + 1e-40
    assert ((y[:m].double() - want).abs() <= bound).all()


# A few tiles more than the work-groups take at once, of 64, 128 and 256 rows and columns, of full and of few rows.
@pytest.mark.parametrize("m,n", [(4500, 4096), (4100, 4096), (4353, 4096), (8200, 8192), (3000, 2900), (2049, 4096), (1700, 1950), (1600, 2000)])
@pytest.mark.parametrize("k", [96, 256, 1056])
def test_a_last_round_of_few_tiles(m, n, k):
    test_many_tiles(m, n, k, k == 256)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("experts,n,k,mean", [(3, 1000, 160, 700), (40, 512, 96, 90), (128, 520, 64, 30), (2, 2048, 128, 3000), (8, 768, 2048, 500), (100, 256, 32, 200)])
def test_many_grouped_tiles(glu, experts, n, k, mean):
    rng = np.random.default_rng(experts)
    counts = rng.integers(0, 2 * mean + 1, experts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    p = int(offsets[-1])
    g = torch.Generator(device="cuda")
    g.manual_seed(experts)
    announce("moe_i8 many tiles", experts, p, n, k, "glu" if glu else "")
    xr = p // 2 + 1
    w = torch.randint(-128, 128, (experts, n, k), device="cuda", dtype=torch.int8, generator=g)
    w2 = torch.randint(-128, 128, (experts, n, k), device="cuda", dtype=torch.int8, generator=g)
    x = torch.randint(-128, 128, (xr, k), device="cuda", dtype=torch.int8, generator=g)
    ws, ws2 = torch.rand((experts, n), device="cuda", generator=g) * 1e-4, torch.rand((experts, n), device="cuda", generator=g) * 1e-4
    xs = torch.rand(xr, device="cuda", generator=g)
    rows = torch.randint(0, xr, (p,), device="cuda", dtype=torch.int32, generator=g)
    y = torch.full((p + 1, n), 77.0, device="cuda")
    off = dev(offsets.astype(np.int32))
    if glu:
        qmm.qmm_moe_swiglu_i8(w, ws, w2, ws2, x, xs, rows, xr, off, y, False, p, experts, n, k)
    else:
        qmm.qmm_moe_gemm_i8(w, ws, x, xs, rows, xr, off, y, False, p, experts, n, k)
    torch.cuda.synchronize()
    assert (y[p] == 77).all()
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        at = rows[a:b].long()
        v = on_device(x[at], xs[at], w[e], ws[e])
        bound = 3.01 * E32 * v.abs() + 1e-40
        if glu:
            u = on_device(x[at], xs[at], w2[e], ws2[e])
            h = v * torch.sigmoid(v) * u
            bound = E32 * h.abs() * (3 * (1 + v.abs()) + 11) + 1e-35 * u.abs() + 1e-40
            v = h
        assert ((y[a:b].double() - v).abs() <= bound).all(), e


def test_scales_that_are_not_finite_stay_in_their_rows_and_columns():
    rng = np.random.default_rng(9)
    for m, n in ((3, 50), (40, 50), (200, 90)):
        w, x, ws, xs = codes(rng, n, 64), codes(rng, m, 64), scales(rng, n), scales(rng, m)
        ws[5], xs[1] = np.nan, np.nan
        y = torch.empty((m, n), device="cuda")
        announce("gemm_i8 nan scales", m, n)
        qmm.qmm_gemm_i8(dev(w), dev(ws), dev(x), dev(xs), y, False, m, n, 64)
        bad = torch.isnan(y).cpu().numpy()
        want = np.zeros((m, n), dtype=bool)
        want[1], want[:, 5] = True, True
        assert np.array_equal(bad, want)


def test_nothing_to_do():
    y = torch.full((4, 4), 5.0, device="cuda")
    w, s = torch.zeros((4, 32), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    qmm.qmm_gemm_i8(w, s, w, s, y, False, 0, 4, 32)
    qmm.qmm_gemm_i8(w, s, w, s, y, False, 4, 0, 32)
    qmm.qmm_moe_gemm_i8(w, s, w, s, None, 4, None, y, False, 0, 1, 4, 32)
    qmm.qmm_moe_gemm_i8(None, None, None, None, None, 0, None, y, False, 4, 0, 4, 32)
    assert (y == 5).all()


# ---- rows grouped by expert ------------------------------------------------


def grouped(experts, counts, n, k, f16, glu, x_rows="some", behind=0, seed=0):
    rng = np.random.default_rng(experts * 31 + n + k + seed + sum(counts))
    p = int(sum(counts))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = p + behind
    announce("moe_i8", experts, "rows", total, n, k, "fp16" if f16 else "fp32", "glu" if glu else "", x_rows)
    xr = max(1, total // 3) if x_rows != "own" else total
    rows = None if x_rows == "own" else rng.integers(0, xr, total).astype(np.int32)
    if x_rows == "bad":
        rows[::5] = -1
        rows[1::7] = xr
        rows[2::11] = 2 ** 31 - 1
    w, x, ws, xs = codes(rng, experts, n, k), codes(rng, xr, k), scales(rng, experts, n), scales(rng, xr)
    w2, ws2 = codes(rng, experts, n, k), scales(rng, experts, n)
    y = torch.full((total + 1, n), 33.0, dtype=torch.float16 if f16 else torch.float32, device="cuda")
    d_rows, d_off = None if rows is None else dev(rows), dev(offsets)
    if glu:
        qmm.qmm_moe_swiglu_i8(dev(w), dev(ws), dev(w2), dev(ws2), dev(x), dev(xs), d_rows, xr, d_off, y, f16, total, experts, n, k)
    else:
        qmm.qmm_moe_gemm_i8(dev(w), dev(ws), dev(x), dev(xs), d_rows, xr, d_off, y, f16, total, experts, n, k)
    torch.cuda.synchronize()
    got = y.float().cpu().numpy()
    assert (got[p:] == 33).all()
    g, covered = moe.moe_product_i8(w, ws, x, xs, rows, offsets, total)
    if not glu:
        check(got[:total], g, plain_bound(g, f16), covered, "moe_gemm_i8")
        return
    u, _ = moe.moe_product_i8(w2, ws2, x, xs, rows, offsets, total)
    nan = np.isnan(g)
    g, u = np.nan_to_num(g), np.nan_to_num(u)
    h = moe.silu(g) * u
    h[nan] = np.nan
    check(got[:total], h, gated_bound(g, u, np.nan_to_num(h), f16), covered, "moe_swiglu_i8")


COUNTS = [[1], [5], [0], [40], [300], [3, 0, 1, 7], [0, 0, 0, 2], [16, 17, 15, 1, 0, 33], [64, 65, 1], [130, 0, 200, 128], [600, 1, 0, 2]]


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("x_rows", ["own", "some", "bad"])
def test_groups(counts, glu, x_rows):
    grouped(len(counts), counts, 96, 160, sum(counts) % 2 == 0, glu, x_rows, behind=3)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,k", [(1, 32), (33, 64), (130, 96), (257, 128), (768, 256), (1001, 1056)])
@pytest.mark.parametrize("per", [1, 20, 90])
def test_groups_of_other_sizes(glu, n, k, per):
    grouped(3, [per, 0, per + 5], n, k, True, glu)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("experts,n,k,mean", [(128, 768, 96, 256), (128, 700, 160, 100), (64, 1001, 64, 300), (16, 2048, 288, 520), (16, 2200, 128, 500)])
def test_last_rounds_of_grouped_tiles(glu, experts, n, k, mean):
    for shift in (0, 40, 90):
        test_many_grouped_tiles(glu, experts, n, k, mean + shift)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("experts,per", [(60, 1), (64, 3), (65, 2), (130, 1), (200, 9), (128, 40)])
def test_many_experts(glu, experts, per):
    rng = np.random.default_rng(experts)
    grouped(experts, rng.integers(0, 2 * per + 1, experts).tolist(), 32, 64, False, glu)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("per", [2, 50, 300])
def test_offsets_that_hold_nonsense_stay_inside_the_rows(glu, per):
    # Whatever the offsets hold, only the given rows are written, and weights and activations are read in bounds.
    rng = np.random.default_rng(per)
    n, k, p = 40, 64, 4 * per
    w, x, ws, xs = dev(codes(rng, 4, n, k)), dev(codes(rng, p, k)), dev(scales(rng, 4, n)), dev(scales(rng, p))
    for offsets in ([0, -5, 3, 2, p + 100], [p + 7] * 5, [-9] * 5, [0, p, 0, p, 0], [5, 4, 3, 2, 1], [2 ** 31 - 1, -2 ** 31, 0, 2 ** 31 - 1, p]):
        announce("moe_i8 offsets", offsets, "glu" if glu else "")
        y = torch.full((p + 2, n), 33.0, device="cuda")
        off = dev(np.array(offsets, dtype=np.int64).astype(np.int32))
        mid = y[1:p + 1]
        if glu:
            qmm.qmm_moe_swiglu_i8(w, ws, w, ws, x, xs, None, p, off, mid, False, p, 4, n, k)
        else:
            qmm.qmm_moe_gemm_i8(w, ws, x, xs, None, p, off, mid, False, p, 4, n, k)
        torch.cuda.synchronize()
        assert (y[0] == 33).all() and (y[p + 1] == 33).all()


@pytest.mark.parametrize("rows", [1, 7, 30, 90, 200])
@pytest.mark.parametrize("glu", [False, True])
def test_one_expert_without_offsets(rows, glu):
    rng = np.random.default_rng(rows)
    n, k = 136, 224
    announce("moe_i8 dense", rows, "glu" if glu else "")
    w, x, ws, xs = codes(rng, 1, n, k), codes(rng, rows, k), scales(rng, 1, n), scales(rng, rows)
    w2, ws2 = codes(rng, 1, n, k), scales(rng, 1, n)
    y = torch.empty((rows, n), device="cuda")
    g = moe.product_i8(w[0], ws[0], x, xs)
    if glu:
        qmm.qmm_moe_swiglu_i8(dev(w), dev(ws), dev(w2), dev(ws2), dev(x), dev(xs), None, rows, None, y, False, rows, 1, n, k)
        u = moe.product_i8(w2[0], ws2[0], x, xs)
        h = moe.silu(g) * u
        check(y.cpu().numpy(), h, gated_bound(g, u, h, False), np.ones(rows, dtype=bool), "dense glu")
    else:
        qmm.qmm_moe_gemm_i8(dev(w), dev(ws), dev(x), dev(xs), None, rows, None, y, False, rows, 1, n, k)
        check(y.cpu().numpy(), g, plain_bound(g, False), np.ones(rows, dtype=bool), "dense")


def test_results_repeat():
    rng = np.random.default_rng(1)
    w, x, ws, xs = dev(codes(rng, 700, 512)), dev(codes(rng, 300, 512)), dev(scales(rng, 700)), dev(scales(rng, 300))
    for m in (5, 50, 300):
        ys = []
        for _ in range(3):
            y = torch.empty((m, 700), device="cuda")
            qmm.qmm_gemm_i8(w, ws, x, xs, y, False, m, 700, 512)
            ys.append(y)
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
        # A row's sums are exact: the same whatever stands next to it.
        one = torch.empty((1, 700), device="cuda")
        qmm.qmm_gemm_i8(w, ws, x, xs, one, False, 1, 700, 512)
        assert torch.equal(one[0], ys[0][0])
