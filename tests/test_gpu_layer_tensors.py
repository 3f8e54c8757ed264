"""The torch-side calls of the layer's operators against the float64 definitions."""
import numpy as np
import pytest
import torch

from gemm_qmm_gemv_amd import tensors
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import check, dev
from tests.test_gpu_layer_norm import EPS, bounds, case

pytestmark = pytest.mark.gpu


def test_one_gate_row_for_several_rows():
    rng = np.random.default_rng(71)
    rows, n = 7, 192
    y, pw, g, res, pre = case(rng, rows, n, True, True, "shared")
    u, h, x = layer.norm_residual(y, pw, g, 0.5, res, pre, EPS)
    eh, ex = bounds(u, h, x, 0.5, pre)
    # Whatever lies behind the gate is no part of it.
    buf = torch.full((rows, n), float("nan"), device="cuda")
    buf[0] = dev(g)[0]
    for gate in (buf[:1], buf[0], buf[:1].expand(rows, n)):
        announce("one gate row", tuple(gate.shape))
        hd, xd = tensors.norm_residual(dev(y), dev(res), dev(pre), EPS, dev(pw), gate, 0.5)
        check(hd.cpu().numpy(), h, eh, "h")
        check(xd.cpu().numpy(), x, ex, "x")
