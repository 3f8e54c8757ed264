"""qmm_quantize_rows against the definition: scales to the bit, codes the whole numbers next to the quotients in 64 bits."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import dev

pytestmark = pytest.mark.gpu


def run(x, pad_stride=0):
    rows, k = x.shape
    announce("quantize", rows, k, x.dtype, pad_stride)
    wide = torch.full((rows, k + pad_stride), 3e4, dtype=x.dtype, device="cuda")
    wide[:, :k] = x
    codes = torch.full((rows + 1, k), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((rows + 1,), 99.0, device="cuda")
    qmm.qmm_quantize_rows(wide, x.dtype == torch.float16, wide.stride(0), codes, scales, rows, k)
    torch.cuda.synchronize()
    assert (codes[rows] == 99).all() and scales[rows] == 99
    want, unit = moe.quantize_rows(x.float().cpu().numpy())
    got = scales[:rows].cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(unit))
    ok = ~np.isnan(unit)
    assert np.array_equal(got[ok], unit[ok])
    assert np.array_equal(codes[:rows].cpu().numpy().astype(np.int64), want)
    return want, unit


@pytest.mark.parametrize("k", [32, 64, 96, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 16384, 16416, 32768])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_sizes(k, dtype):
    rng = np.random.default_rng(k)
    for rows in (1, 2, 37):
        run(dev(rng.standard_normal((rows, k)).astype(np.float32)).to(dtype))


@pytest.mark.parametrize("pad", [1, 2, 4, 8, 13])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_rows_apart(pad, dtype):
    rng = np.random.default_rng(pad)
    run(dev(rng.standard_normal((19, 416)).astype(np.float32)).to(dtype), pad)


def test_quotients_on_and_next_to_a_border():
    # Scale 2^e and values of whole and half codes, and their neighbours: 0.5 to even, all else to the nearer.
    rng = np.random.default_rng(1)
    rows = []
    for e in (-20, -3, 0, 9):
        half = (rng.integers(-253, 254, 512) / 2.0).astype(np.float32) * np.float32(2.0 ** e)
        for way in (0, -np.inf, np.inf):
            r = half if way == 0 else np.nextafter(half, np.float32(way), dtype=np.float32)
            r = np.clip(r, -127 * 2.0 ** e, 127 * 2.0 ** e).astype(np.float32)
            r[0] = 127 * 2.0 ** e
            rows.append(r)
    run(dev(np.stack(rows)))
    # Scales of 24 bits: values next to (code + 1/2) scale.
    rows = []
    for _ in range(64):
        top = np.float32(rng.uniform(0.5, 2.0))
        unit = np.float32(float(top) / 127)
        half = ((rng.integers(-126, 126, 512) + 0.5) * float(unit)).astype(np.float32)
        r = np.nextafter(half, np.where(rng.random(512) < 0.5, np.float32(-9), np.float32(9)).astype(np.float32), dtype=np.float32)
        r = np.where(rng.random(512) < 0.4, half, r).astype(np.float32)
        r[1] = top
        rows.append(r)
    run(dev(np.stack(rows)))


def test_zero_small_large_and_bad_rows():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((24, 256)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2, 100:] = 0
    x[3] *= 1e-30
    x[4] *= 1e-36
    x[5] *= 1e38 / 4
    x[6, 17] = np.inf
    x[7, 18] = -np.inf
    x[8, 255] = np.nan
    x[9] = np.nan
    x[10] = 7.0
    x[11, 0] = 1e30  # the others' codes are 0
    x[12, 3] = np.finfo(np.float32).max
    x[13] = np.inf
    want, unit = run(dev(x))
    assert unit[0] == 0 and (want[0] == 0).all() and (want[10] == 127).all()
    run(dev(x).half())


def test_scales_below_the_normal_range():
    # The scale has few bits there, and the codes are the quotients by what it is held as.
    rng = np.random.default_rng(6)
    x = (rng.standard_normal((40, 64)) * (10.0 ** rng.uniform(-44, -36, (40, 1)))).astype(np.float32)
    run(dev(x))
