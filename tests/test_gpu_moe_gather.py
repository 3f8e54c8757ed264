"""qmm_moe_gather against the sum in 64 bits."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import E32, check, dev

pytestmark = pytest.mark.gpu


def run(rows, pair_row, weights, residual, in_place=False, offset=0):
    """The sum of top_k products and a residual: each fused step and the last addition round once, of what has been added
    so far: (top_k + 2) roundings of the sum of magnitudes."""
    tokens, top_k = pair_row.shape
    p, n = rows.shape
    announce("gather", tokens, top_k, p, n, rows.dtype, "residual" if residual is not None else "", offset)
    y = torch.full((tokens + 2, n), 55.0, device="cuda")
    out = y.view(-1)[offset:offset + tokens * n].view(tokens, n)
    res = None if residual is None else dev(residual)
    if in_place:
        out.copy_(res)
        res = out
    r = torch.empty(p * n + 8, dtype=rows.dtype, device="cuda")[offset:offset + p * n].view(p, n)
    r.copy_(rows)
    qmm.qmm_moe_gather(r, rows.dtype == torch.float16, dev(pair_row), dev(weights), res, out, tokens, top_k, p, n)
    torch.cuda.synchronize()
    assert (y.view(-1)[:offset] == 55).all() and (y.view(-1)[offset + tokens * n:] == 55).all()
    want, mag = moe.gather(rows.cpu().numpy(), pair_row, weights, residual)
    check(out.cpu().numpy(), want, (top_k + 2) * E32 * mag + 1e-40, "gather")


def make(rng, tokens, top_k, n, dtype=torch.float32, spare=0):
    p = tokens * top_k + spare
    rows = dev(rng.standard_normal((p, n)).astype(np.float32)).to(dtype)
    return rows, rng.permutation(p)[:tokens * top_k].astype(np.int32).reshape(tokens, top_k), rng.random((tokens, top_k)).astype(np.float32)


@pytest.mark.parametrize("n", [1, 3, 4, 8, 100, 1001, 1024, 2048, 2880, 4100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(n, dtype, residual):
    rng = np.random.default_rng(n)
    for tokens, top_k in ((1, 1), (3, 8), (21, 5), (9, 13)):
        rows, at, w = make(rng, tokens, top_k, n, dtype, spare=3)
        run(rows, at, w, 3 * rng.standard_normal((tokens, n)).astype(np.float32) if residual else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_in_place_and_odd_addresses(dtype):
    rng = np.random.default_rng(2)
    for offset in (0, 1, 2, 4):
        rows, at, w = make(rng, 7, 4, 512, dtype)
        run(rows, at, w, rng.standard_normal((7, 512)).astype(np.float32), in_place=True, offset=offset)


def test_rows_that_are_not_there_add_nothing():
    rng = np.random.default_rng(3)
    rows, at, w = make(rng, 12, 6, 260)
    at[1] = -1
    at[2, ::2] = [-5, 12 * 6, 2 ** 31 - 1]
    at[3, 1] = -2 ** 31
    w[1] = np.nan
    run(rows, at, w, None)
    run(rows, at, w, rng.standard_normal((12, 260)).astype(np.float32))


def test_the_same_row_twice_and_values_that_are_not_finite():
    rng = np.random.default_rng(4)
    rows, at, w = make(rng, 5, 3, 64)
    at[0] = 4
    run(rows, at, w, None)
    rows[at[2, 1], 7] = float("nan")
    rows[at[2, 1], 8] = float("inf")
    y = torch.empty((5, 64), device="cuda")
    qmm.qmm_moe_gather(rows, False, dev(at), dev(w), None, y, 5, 3, rows.shape[0], 64)
    y = y.cpu().numpy()
    assert np.isnan(y[2, 7]) and np.isinf(y[2, 8]) and np.isfinite(np.delete(y, 2, 0)).all()


def test_no_choice_leaves_the_residual():
    y = torch.full((3, 40), 9.0, device="cuda")
    res = torch.randn((3, 40), device="cuda")
    qmm.qmm_moe_gather(None, False, None, None, res, y, 3, 0, 0, 40)
    assert torch.equal(y, res)
    qmm.qmm_moe_gather(None, False, None, None, None, y, 3, 0, 0, 40)
    assert (y == 0).all()
