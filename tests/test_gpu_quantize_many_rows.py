"""qmm_quantize_rows over thousands of rows of up to 1024 values, where a wave has a row for itself, against the definition."""
import numpy as np
import pytest
import torch

from tests.layer_util import dev
from tests.test_gpu_quantize_rows import run

pytestmark = pytest.mark.gpu


def rows_of_every_kind(rng, rows, k, f16):
    """Normal rows, and among them zeros, tiny, large and not finite ones, and values on and next to a border between codes."""
    x = rng.standard_normal((rows, k)).astype(np.float32)
    kind = rng.integers(0, 24, rows)
    kind[-5:] = [0, 5, 6, 2, 7]
    x[kind == 0] = 0
    x[kind == 1] *= 1e-6 if f16 else 1e-37
    x[kind == 2] *= 1e3 if f16 else 1e37
    x[kind == 3, k - 1] = np.inf
    x[kind == 4, k // 2] = np.nan
    for r in np.flatnonzero((kind >= 5) & (kind < 8)):
        # Whole and half codes of a scale of few bits, and their neighbours.
        unit = 2.0 ** int(rng.integers(-6, 7))
        half = (rng.integers(-253, 254, k) / 2.0 * unit).astype(np.float16 if f16 else np.float32)
        way = np.array(rng.choice([-np.inf, np.inf], k), dtype=half.dtype)
        x[r] = np.clip(np.where(rng.random(k) < 0.5, half, np.nextafter(half, way)), -127 * unit, 127 * unit)
        x[r, int(rng.integers(k))] = 127 * unit
    if not f16:
        for r in np.flatnonzero(kind == 8):
            # Values next to (code + 1/2) scale, scales of 24 bits.
            top = np.float32(rng.uniform(0.5, 2.0))
            unit = float(np.float32(float(top) / 127))
            x[r] = ((rng.integers(-126, 126, k) + 0.5) * unit).astype(np.float32)
            x[r, int(rng.integers(k))] = -top
    return dev(x).half() if f16 else dev(x)


@pytest.mark.parametrize("k", [32, 64, 96, 480, 512, 544, 768, 992, 1024, 1056])
@pytest.mark.parametrize("rows", [2047, 2048, 2049, 2051, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_sizes(k, rows, dtype):
    run(rows_of_every_kind(np.random.default_rng(k + rows), rows, k, dtype == torch.float16))


# Rows apart by a multiple of eight values, of four and of neither.
@pytest.mark.parametrize("pad", [8, 40, 4, 12, 1, 2])
@pytest.mark.parametrize("k", [96, 768])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_rows_apart(pad, k, dtype):
    run(rows_of_every_kind(np.random.default_rng(k + pad), 2050, k, dtype == torch.float16), pad)
