"""qmm_attn_prompt rounds its probabilities to the nearest fp16, half a step at most."""
import numpy as np
import pytest
import torch

from tests.gpu_util import announce
from tests.layer_util import E16, TINY16, check, dev
from tests.test_gpu_layer_attn_prompt import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq", [2, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part", [0.02, 0.4, 0.6, 0.98])
def test_probabilities_are_off_by_half_a_step(part, d, hq):
    # The last row of a sequence sees n keys of score 0 and value 0, and one whose probability lies `part` of a step above
    # one half, with value 1: o = p / (n + p).  A probability off by a relative e moves o by (1 - o) e o: half a step next to
    # one half is E16.  The output is rounded once more; scores and sums are right to 2^-19 or better.
    p = 0.5 * (1 + part * 2.0 ** -10)
    counts = list(range(1, 61))
    offsets = np.concatenate([[0], np.cumsum([n + 1 for n in counts])])
    t = int(offsets[-1])
    q, k, v = np.zeros((t, hq, d), np.float16), np.zeros((t, 1, d), np.float16), np.zeros((t, 1, d), np.float16)
    q[:, :, 0] = 1
    last = offsets[1:] - 1
    k[last, 0, 0] = -1
    v[last, 0] = 1
    announce("rounded probabilities", part, d, hq)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), offsets, -np.log(p), out)[last]
    o = (p / (np.array(counts) + p))[:, None, None] * np.ones((1, hq, d))
    check(got, o, o * (E16 * (1 - o) + E16 * 1.01 + 2.0 ** -19), "half a step")


@pytest.mark.parametrize("hq", [2, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("log2p", [-14, -15, -18, -20])
def test_probabilities_below_the_normal_range_count_on_both_sides(log2p, d, hq):
    # One key of score 0 and value 0 and many of probability 2^log2p, exact in fp16, and value 1: o = n p / (1 + n p).
    # Scores and sums are right to 2^-19 or better, the output is rounded once.
    p = 2.0 ** log2p
    n = 1900
    q, k, v = np.zeros((n + 1, hq, d), np.float16), np.zeros((n + 1, 1, d), np.float16), np.ones((n + 1, 1, d), np.float16)
    q[:, :, 0] = 1
    k[1:, 0, 0] = -1
    v[0] = 0
    announce("small probabilities", log2p, d, hq)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), [0, n + 1], -log2p * np.log(2), out)
    rows = np.arange(n + 1)
    o = (rows * p / (1 + rows * p))[:, None, None] * np.ones((1, hq, d))
    check(got, o, o * (E16 * 1.01 + 2.0 ** -19) + TINY16, "small probabilities")
