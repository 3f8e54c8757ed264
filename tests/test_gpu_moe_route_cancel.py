"""qmm_moe_route where the two best c of a group have opposite signs: the sum is small, and what 32 bits lose of its terms is not."""
import numpy as np
import pytest

from tests.layer_util import dev
from tests.test_gpu_moe_route import run

pytestmark = pytest.mark.gpu


def signs(experts):
    return np.where(np.arange(experts) % 2 == 0, 1.0, -1.0).astype(np.float32)


def test_worked_examples():
    # Sums of 0.78167 and 0.78144, in fp32 0.78149 and 0.78174.
    l = np.array([[-0.55, -0.34, 0.05, -1.0]], dtype=np.float32)
    run(dev(l), "cancel", top_k=2, kind="sigmoid", groups=2, top_groups=1, best=2, bias=dev(4096 * signs(4)))
    # Of 0.982303 and 0.982309 one has to go, in fp32 0.98236 and 0.98230.
    l = np.array([[-1.81413, -0.33443, 0.54865, -0.62572, 0.92902, -1.01791, -0.81125, 1.34987]], dtype=np.float32)
    for experts in (l, np.repeat(l, 70, 0)):
        run(dev(experts), "cancel", top_k=2, kind="sigmoid", groups=4, top_groups=2, best=2, bias=dev(1000 * signs(8)))


# Groups of two (every sum cancels) and of more, whose two best do; in one step over all groups, and one group after the other.
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(8, 4, 2, 2), (64, 32, 4, 6), (64, 16, 3, 4), (128, 64, 8, 8), (60, 20, 6, 5), (256, 64, 9, 8)])
@pytest.mark.parametrize("size", [16.0, 100.0, 4096.0, 1e6])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_biases_of_both_signs(experts, groups, top_groups, top_k, size, kind):
    rng = np.random.default_rng(experts + int(size))
    each = experts // groups
    bias = np.full(experts, -4 * size, dtype=np.float32)
    bias[::each], bias[1::each] = size, -size
    run(dev(rng.standard_normal((1500, experts)).astype(np.float32)), "cancel", top_k=top_k, kind=kind, groups=groups, top_groups=top_groups,
        best=2, bias=dev(bias))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(16, 5), (32, 12)])
def test_sizes_that_differ_between_groups(kind, groups, top_groups):
    # A group that is not next to the border by its sum may be by what 32 bits lose of its terms; groups and experts that are
    # switched off by a bias far below or of -inf.
    rng = np.random.default_rng(groups)
    experts = 64
    each = experts // groups
    l = rng.standard_normal((2000, experts)).astype(np.float32)
    for off in (None, -1e9, -np.inf):
        bias = np.repeat((10.0 ** rng.integers(-1, 7, groups)).astype(np.float32), each) * signs(experts)
        if each > 2:
            bias.reshape(groups, each)[:, 2:] = -1e8
        if off is not None:
            bias.reshape(groups, each)[::5] = off
            bias[7] = off
        run(dev(l), "cancel", top_k=6, kind=kind, groups=groups, top_groups=top_groups, best=2, bias=dev(bias))
    huge = signs(experts) * np.float32(3e38)  # sums of two of one sign are past fp32
    huge[::8] = 3.2e38
    huge[1::8] = 3.3e38
    huge[4:8] = -3e38
    run(dev(l[:100]), "past fp32", top_k=6, kind=kind, groups=groups, top_groups=top_groups, best=2, bias=dev(huge))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups", [(64, 16, 5), (40, 8, 3), (128, 16, 4)])
def test_long_batches(kind, experts, groups, top_groups):
    # Sixteen lanes a token: some of a wave's four tokens are clear in fp32.
    rng = np.random.default_rng(experts)
    each = experts // groups
    bias = np.full(experts, -4000, dtype=np.float32)
    bias[::each], bias[1::each] = 700, -700
    run(dev((2 * rng.standard_normal((4099, experts))).astype(np.float32)), "cancel", top_k=4, kind=kind, groups=groups, top_groups=top_groups,
        best=2, bias=dev(bias))
