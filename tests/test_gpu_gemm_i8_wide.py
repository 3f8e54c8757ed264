"""8-bit products with more work-groups than one launch has of the kernel that is quickest by time: another one takes them."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16, dev
from tests.test_gpu_moe_far import codes, generator

pytestmark = pytest.mark.gpu


def right(y, x, xs, w, ws, u=None, us=None):
    """fp16 outputs within the bounds of a product, or of a gated one, as for smaller ones."""
    v = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()[None, :]
    bound = 3.01 * E32 * v.abs()
    if u is not None:
        t = (x.double() @ u.double().T) * xs.double()[:, None] * us.double()[None, :]
        h = v * torch.sigmoid(v) * t
        bound, v = E32 * h.abs() * (3 * (1 + v.abs()) + 11) + 1e-35 * t.abs(), h
    bound = bound + E16 * 1.01 * v.abs() + TINY16 + 1e-40
    return ((y.double() - v).abs() <= bound).all()


@pytest.mark.parametrize("glu", [False, True])
def test_few_rows_of_many_columns(glu):
    m, n, k = 100, 33554560, 32
    announce("gemm_i8 wide", m, n, k, "glu" if glu else "")
    g = generator(m)
    w, x = codes(g, n, k), codes(g, m, k)
    u = codes(g, n, k) if glu else None
    ws, us = (torch.rand(n, device="cuda", generator=g) * 1e-4 for _ in range(2))
    xs = torch.rand(m, device="cuda", generator=g)
    y = torch.full((m + 1, n), 77.0, dtype=torch.float16, device="cuda")
    if glu:
        qmm.qmm_moe_swiglu_i8(w, ws, u, us, x, xs, None, m, None, y, True, m, 1, n, k)
    else:
        qmm.qmm_gemm_i8(w, ws, x, xs, y, True, m, n, k)
    torch.cuda.synchronize()
    assert (y[m] == 77).all()
    for c in range(0, n, 1 << 20):
        part = slice(c, min(n, c + (1 << 20)))
        assert right(y[:m, part], x, xs, w[part], ws[part], u[part] if glu else None, us[part]), c


@pytest.mark.parametrize("glu", [False, True])
def test_a_row_for_each_expert_of_many_columns(glu):
    experts, n, k = 64, 3950000, 32
    announce("moe_i8 wide", experts, n, k, "glu" if glu else "")
    g = generator(experts)
    w, x = codes(g, experts, n, k), codes(g, experts, k)
    u = w.flip(0) if glu else None
    ws, us = (torch.rand((experts, n), device="cuda", generator=g) * 1e-4 for _ in range(2))
    xs = torch.rand(experts, device="cuda", generator=g)
    counts = np.ones(experts, dtype=np.int64)
    counts[[3, 9, 40]] = [0, 3, 0]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    y = torch.full((experts + 1, n), 77.0, dtype=torch.float16, device="cuda")
    off = dev(offsets.astype(np.int32))
    if glu:
        qmm.qmm_moe_swiglu_i8(w, ws, u, us, x, xs, None, experts, off, y, True, experts, experts, n, k)
    else:
        qmm.qmm_moe_gemm_i8(w, ws, x, xs, None, experts, off, y, True, experts, experts, n, k)
    torch.cuda.synchronize()
    assert (y[experts] == 77).all()
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            assert right(y[a:b], x[a:b], xs[a:b], w[e], ws[e], u[e] if glu else None, us[e]), e


def test_many_rows_of_few_columns():
    # More tiles of 128 rows than work-groups that have one tile each.
    experts, rows, n, k, xr = 3, (1 << 29) + 3001, 8, 4096, 700
    announce("moe_i8 long", experts, rows, n, k)
    g = generator(n)
    w, x = codes(g, experts, n, k), codes(g, xr, k)
    ws, xs = torch.rand((experts, n), device="cuda", generator=g) * 1e-5, torch.rand(xr, device="cuda", generator=g)
    at = torch.randint(0, xr, (rows,), device="cuda", dtype=torch.int32, generator=g)
    offsets = [0, 1000, rows // 2 + 77, rows]
    y = torch.full((rows + 1, n), 77.0, dtype=torch.float16, device="cuda")
    qmm.qmm_moe_gemm_i8(w, ws, x, xs, at, xr, dev(np.array(offsets, dtype=np.int32)), y, True, rows, experts, n, k)
    torch.cuda.synchronize()
    assert (y[rows] == 77).all()
    for e in range(experts):
        want = (x.double() @ w[e].double().T) * xs.double()[:, None] * ws[e].double()[None, :]
        bound = 3.01 * E32 * want.abs() + E16 * 1.01 * want.abs() + TINY16 + 1e-40
        for a in range(offsets[e], offsets[e + 1], 1 << 24):
            part = slice(a, min(offsets[e + 1], a + (1 << 24)))
            r = at[part].long()
            assert ((y[part].double() - want[r]).abs() <= bound[r]).all(), (e, a)
