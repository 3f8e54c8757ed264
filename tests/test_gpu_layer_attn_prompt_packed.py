"""qmm_attn_prompt on packed batches around the numbers of work-groups at which their size changes, against the float64
definition."""
import numpy as np
import pytest
import torch

from tests.gpu_util import announce
from tests.layer_util import dev
from tests.test_gpu_layer_attn_prompt import call, compare, expect, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,most,hq", [(16, 128, 32), (15, 128, 32), (13, 120, 32), (12, 120, 32), (2, 1000, 32), (3, 801, 32),
                                       (9, 400, 16), (1, 2500, 32)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("even", [True, False])
def test_packed_batches(n, most, hq, d, even):
    rng = np.random.default_rng([51, n, most, hq, d])
    lens = [most if even else int(rng.integers(1, most + 1)) for _ in range(n)]
    offsets = np.concatenate([[0], np.cumsum(lens)])
    t = int(offsets[-1]) + 5
    q, k, v = inputs(rng, t, hq, 2, d)
    announce("packed prompts", lens, hq, d)
    rows = set(int(x) for x in rng.integers(0, t - 5, 40)) | {int(x) for x in offsets[:-1]} | {int(x) - 1 for x in offsets[1:]}
    o, b = expect(q, k, v, offsets, d ** -0.5, rows)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out)
    assert np.isfinite(got).all() and (got[t - 5:] == 7).all()
    compare(got, o, b, "packed prompts")
