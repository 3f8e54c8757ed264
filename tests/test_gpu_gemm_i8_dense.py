"""8-bit products of one matrix, plain and gated, over rows, columns and depths that take every kernel for them: from one row to
thousands, narrow and wide matrices, short and long K."""
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16
from tests.test_gpu_gemm_i8 import on_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k", [(1000, 544), (2048, 512), (8200, 96), (8195, 256), (8192, 2048), (1024, 4096), (4096, 4096), (16400, 2080)])
@pytest.mark.parametrize("f16", [False, True])
def test_rows(n, k, f16):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + k)

    def codes(rows):
        return torch.randint(-128, 128, (rows, k), device="cuda", dtype=torch.int8, generator=g)

    def scales(rows):
        return (0.5 + torch.rand(rows, device="cuda", generator=g)) * 2.0 ** -12

    w, u, ws, us = codes(n), codes(n), scales(n), scales(n)
    for m in (1, 9, 16, 17, 25, 32, 33, 40, 48, 49, 64, 100, 128, 129, 200, 300, 513, 1024, 2048, 4100):
        announce("one matrix", m, n, k, "fp16" if f16 else "fp32")
        x, xs = codes(m), scales(m)
        y, h = (torch.full((m + 1, n), 77.0, dtype=torch.float16 if f16 else torch.float32, device="cuda") for _ in range(2))
        qmm.qmm_gemm_i8(w, ws, x, xs, y, f16, m, n, k)
        qmm.qmm_moe_swiglu_i8(w, ws, u, us, x, xs, None, m, None, h, f16, m, 1, n, k)
        torch.cuda.synchronize()
        assert (y[m] == 77).all() and (h[m] == 77).all()
        v, t = on_device(x, xs, w, ws), on_device(x, xs, u, us)
        bound = 3.01 * E32 * v.abs() + (E16 * 1.01 * v.abs() + TINY16 if f16 else 0) + 1e-40
        assert ((y[:m].double() - v).abs() <= bound).all(), ("plain", m)
        # silu's slope, its exponential, quotient and products, as for rows grouped by expert.
        want = v * torch.sigmoid(v) * t
        bound = E32 * want.abs() * (3 * (1 + v.abs()) + 11) + 1e-35 * t.abs() + (E16 * 1.01 * want.abs() + TINY16 if f16 else 0) + 1e-40
        assert ((h[:m].double() - want).abs() <= bound).all(), ("gated", m)
