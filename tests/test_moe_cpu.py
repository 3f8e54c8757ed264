"""Expert routing, 8-bit integer products and the gather of expert rows without a GPU: what the entry points refuse, before
any device is touched, what the torch-side calls hand over and refuse, and the oracle's own pins."""
import math
import os

import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from gemm_qmm_gemv_amd import tensors
from oracle import moe_block as moe

A16 = 0x10000  # a 16-byte aligned stand-in address; never dereferenced here
INV, UNS, MIS, OK = qmm.QMM_ERR_INVALID_ARGUMENT, qmm.QMM_ERR_UNSUPPORTED, qmm.QMM_ERR_MISALIGNED, qmm.QMM_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(qmm.library_path()):
        from gemm_qmm_gemv_amd import build
        build.build()
    return qmm.load()


def status(fn, *args, **kw):
    try:
        fn(*args, stream=0, **kw)
    except qmm.QmmError as e:
        assert qmm.qmm_last_error() != ""
        return e.status
    return OK


def route(logits=A16, f16=False, stride=64, bias=None, sigmoid=False, groups=1, top_groups=1, best=1, top_k=4, renorm=True, scale=1.0,
          keep=None, ids=A16, weights=A16, pair_row=A16, offsets=A16, token=A16, weight=A16, ws=A16, nws=1 << 30, tokens=100, experts=64):
    return status(qmm.qmm_moe_route, logits, f16, stride, bias, sigmoid, groups, top_groups, best, top_k, renorm, scale, keep, ids, weights,
                  pair_row, offsets, token, weight, ws, nws, tokens, experts)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INV), (dict(tokens=1 << 24), UNS), (dict(experts=0), INV), (dict(experts=-3), INV), (dict(experts=1025, stride=1025), UNS),
    (dict(top_k=0), INV), (dict(top_k=-1), INV), (dict(top_k=65), INV), (dict(top_k=65, experts=128, stride=128), UNS),
    (dict(groups=0), INV), (dict(groups=7), INV), (dict(groups=128, experts=128, stride=128), UNS), (dict(groups=8, top_groups=0), INV),
    (dict(groups=8, top_groups=9), INV), (dict(best=0), INV), (dict(best=3), INV), (dict(groups=64, top_groups=8, best=2), INV),
    (dict(groups=16, top_groups=1, top_k=5), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(logits=None), INV),
    (dict(ids=None), INV), (dict(weights=None), INV), (dict(stride=63), INV), (dict(stride=1 << 36), INV), (dict(logits=A16 + 2), MIS),
    (dict(logits=A16 + 1, f16=True), MIS), (dict(bias=A16 + 2), MIS), (dict(ids=A16 + 1), MIS), (dict(weights=A16 + 2), MIS),
    (dict(pair_row=A16 + 2), MIS), (dict(offsets=A16 + 2), MIS), (dict(token=A16 + 3), MIS), (dict(weight=A16 + 2), MIS),
    (dict(ws=A16 + 8), MIS), (dict(ws=None), INV), (dict(ws=None, nws=0), INV), (dict(nws=8), INV),
    (dict(tokens=0, offsets=None, logits=None), OK),
])
def test_route_refusals(kw, want):
    assert route(**kw) == want


def test_route_workspace():
    need = qmm.qmm_moe_route_workspace_bytes(100, 64, 4)
    assert need > 0 and route(nws=need - 1) == INV
    assert qmm.qmm_moe_route_workspace_bytes(1, 64, 4) == 0 and qmm.qmm_moe_route_workspace_bytes(-1, 64, 4) == 0
    sizes = [qmm.qmm_moe_route_workspace_bytes(t, 64, 4) for t in (16, 17, 4096, 16384, 16385, 1 << 20)]
    assert sizes[0] == 0 and all(s > 0 for s in sizes[1:])


def test_route_workspace_serves_fewer_tokens():
    sizes = [qmm.qmm_moe_route_workspace_bytes(t, 100, 4) for t in (*range(1, 300), 2047, 2048, 2049, 2064, 4095, 4096, 4097, 8192, 16384, 16448, 1 << 18)]
    assert sizes == sorted(sizes)


def quantize(x=A16, f16=True, stride=64, codes=A16, scales=A16, rows=3, k=64):
    return status(qmm.qmm_quantize_rows, x, f16, stride, codes, scales, rows, k)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(rows=1 << 22), UNS), (dict(k=0), INV), (dict(k=48), INV), (dict(k=-32), INV), (dict(k=32800, stride=32800), UNS),
    (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(stride=63), INV), (dict(stride=1 << 40), INV),
    (dict(x=A16 + 1), MIS), (dict(x=A16 + 2, f16=False), MIS), (dict(codes=A16 + 8), MIS), (dict(scales=A16 + 2), MIS),
    (dict(rows=0, x=None), OK),
])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


def product(kind, w=A16, ws=A16, w2=A16, ws2=A16, x=A16, xs=A16, x_rows=None, xr=8, offsets=A16, y=A16, f16=False, rows=8, experts=4, n=64, k=64):
    if kind == "dense":
        return status(qmm.qmm_gemm_i8, w, ws, x, xs, y, f16, rows, n, k)
    if kind == "glu":
        return status(qmm.qmm_moe_swiglu_i8, w, ws, w2, ws2, x, xs, x_rows, xr, offsets, y, f16, rows, experts, n, k)
    return status(qmm.qmm_moe_gemm_i8, w, ws, x, xs, x_rows, xr, offsets, y, f16, rows, experts, n, k)


@pytest.mark.parametrize("kind", ["dense", "plain", "glu"])
@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(rows=-1, xr=-1), INV), (dict(k=0), INV), (dict(k=16), INV), (dict(k=33), INV), (dict(k=65536), UNS),
    (dict(n=1 << 26, k=64), UNS), (dict(rows=1 << 26, xr=1 << 26, k=64), UNS), (dict(w=None), INV), (dict(ws=None), INV), (dict(x=None), INV),
    (dict(xs=None), INV), (dict(y=None), INV), (dict(w=A16 + 4), MIS), (dict(x=A16 + 8), MIS), (dict(y=A16 + 4), MIS), (dict(ws=A16 + 2), MIS),
    (dict(xs=A16 + 1), MIS), (dict(rows=0, xr=0, w=None), OK), (dict(n=0, y=None), OK),
])
def test_product_refusals(kind, kw, want):
    assert product(kind, **kw) == want


@pytest.mark.parametrize("kind", ["plain", "glu"])
@pytest.mark.parametrize("kw,want", [
    (dict(experts=-1), INV), (dict(experts=1025), UNS), (dict(offsets=None), INV), (dict(x_rows=A16 + 2), MIS), (dict(offsets=A16 + 2), MIS),
    (dict(xr=7), INV), (dict(xr=-1, x_rows=A16), INV), (dict(rows=1 << 31, x_rows=A16), UNS), (dict(experts=0, offsets=None, w=None), OK),
])
def test_grouped_product_refusals(kind, kw, want):
    assert product(kind, **kw) == want


@pytest.mark.parametrize("kw,want", [(dict(w2=None), INV), (dict(ws2=None), INV), (dict(w2=A16 + 4), MIS), (dict(ws2=A16 + 2), MIS)])
def test_gated_product_refusals(kw, want):
    assert product("glu", **kw) == want


def gather(rows=A16, f16=False, pair_row=A16, weights=A16, residual=A16, y=A16, tokens=3, top_k=2, p=6, n=64):
    return status(qmm.qmm_moe_gather, rows, f16, pair_row, weights, residual, y, tokens, top_k, p, n)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INV), (dict(n=-1), INV), (dict(p=-1), INV), (dict(top_k=-1), INV), (dict(top_k=65), UNS), (dict(tokens=1 << 24), UNS),
    (dict(n=1 << 22), UNS), (dict(p=1 << 31), UNS), (dict(rows=None), INV), (dict(pair_row=None), INV), (dict(weights=None), INV),
    (dict(y=None), INV), (dict(rows=A16 + 2), MIS), (dict(rows=A16 + 1, f16=True), MIS), (dict(pair_row=A16 + 2), MIS),
    (dict(weights=A16 + 1), MIS), (dict(residual=A16 + 2), MIS), (dict(y=A16 + 2), MIS), (dict(tokens=0, y=None), OK), (dict(n=0), OK),
])
def test_gather_refusals(kw, want):
    assert gather(**kw) == want


# ---- the torch-side calls ----------------------------------------------------

F16, F32, I8, I32, U8 = torch.float16, torch.float32, torch.int8, torch.int32, torch.uint8


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, which are not made; tensors may be on the host."""
    seen = []
    monkeypatch.setattr(tensors, "_on_device", lambda *ts: None)
    for f in ("qmm_moe_route", "qmm_moe_gather", "qmm_quantize_rows", "qmm_gemm_i8", "qmm_moe_gemm_i8", "qmm_moe_swiglu_i8"):
        monkeypatch.setattr(tensors, f, lambda *a, **kw: seen.append(a))
    return seen


def z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


OPERANDS = {
    "moe_route": dict(logits=z(5, 16), top_k=2, bias=z(16), keep=z(5, dtype=U8)),
    "moe_gather": dict(rows=z(10, 32), pair_row=z(5, 2, dtype=I32), weights=z(5, 2), residual=z(5, 32), y=z(5, 32)),
    "quantize_rows": dict(x=z(5, 64), codes=z(5, 64, dtype=I8), scales=z(5)),
    "gemm_i8": dict(w=z(24, 64, dtype=I8), w_scales=z(24), x=z(5, 64, dtype=I8), x_scales=z(5), y=z(5, 24)),
    "moe_i8": dict(w=z(3, 24, 64, dtype=I8), w_scales=z(3, 24), x=z(5, 64, dtype=I8), x_scales=z(5), x_rows=z(9, dtype=I32),
                   offsets=z(4, dtype=I32), y=z(9, 24)),
    "moe_swiglu_i8": dict(gate=z(3, 24, 64, dtype=I8), gate_scales=z(3, 24), up=z(3, 24, 64, dtype=I8), up_scales=z(3, 24),
                          x=z(5, 64, dtype=I8), x_scales=z(5), x_rows=z(9, dtype=I32), offsets=z(4, dtype=I32), h=z(9, 24, dtype=F16)),
}


@pytest.mark.parametrize("name,kw", [
    ("moe_route", {}), ("moe_route", dict(logits=z(5, 40)[:, 8:24], bias=None, keep=None)), ("moe_route", dict(logits=z(5, 16, dtype=F16))),
    ("moe_route", dict(keep=z(5, dtype=torch.bool))), ("moe_route", dict(grouped=False)),
    ("moe_gather", {}), ("moe_gather", dict(rows=z(10, 32, dtype=F16), residual=None, y=None)),
    ("quantize_rows", {}), ("quantize_rows", dict(x=z(5, 96, dtype=F16)[:, 32:], codes=None, scales=None)),
    ("gemm_i8", {}), ("gemm_i8", dict(y=None, out_fp16=True)), ("moe_i8", {}), ("moe_i8", dict(x_rows=None, y=None)), ("moe_swiglu_i8", {}),
])
def test_calls_are_made(calls, name, kw):
    getattr(tensors, name)(**{**OPERANDS[name], **kw})
    assert len(calls) == 1


@pytest.mark.parametrize("name,arg,t", [
    ("moe_route", "logits", z(5, 16, dtype=torch.bfloat16)), ("moe_route", "bias", z(15)), ("moe_route", "bias", z(16, dtype=F16)),
    ("moe_route", "keep", z(4, dtype=U8)), ("moe_route", "keep", z(5, dtype=I32)), ("moe_route", "keep", z(10, dtype=U8)[::2]),
    ("moe_route", "workspace", z(64, dtype=U8)[::2]),
    ("moe_gather", "rows", z(10, 40)[:, :32]), ("moe_gather", "rows", z(10, 32, dtype=torch.bfloat16)), ("moe_gather", "pair_row", z(5, 2, dtype=torch.int64)),
    ("moe_gather", "weights", z(5, 3)), ("moe_gather", "weights", z(5, 2, dtype=F16)), ("moe_gather", "residual", z(4, 32)), ("moe_gather", "y", z(5, 32, dtype=F16)),
    ("quantize_rows", "x", z(5, 64, dtype=torch.float64)), ("quantize_rows", "codes", z(5, 64, dtype=U8)), ("quantize_rows", "codes", z(4, 64, dtype=I8)),
    ("quantize_rows", "scales", z(4)), ("gemm_i8", "w", z(24, 64)), ("gemm_i8", "w", z(24, 80, dtype=I8)[:, :64]), ("gemm_i8", "w_scales", z(23)),
    ("gemm_i8", "x", z(5, 32, dtype=I8)), ("gemm_i8", "x_scales", z(5, dtype=F16)), ("gemm_i8", "y", z(4, 24)), ("gemm_i8", "y", z(5, 24, dtype=I32)),
    ("moe_i8", "w_scales", z(3, 23)), ("moe_i8", "x_rows", z(9, dtype=torch.int64)), ("moe_i8", "offsets", z(3, dtype=I32)), ("moe_i8", "y", z(8, 24)),
    ("moe_swiglu_i8", "up", z(2, 24, 64, dtype=I8)), ("moe_swiglu_i8", "up_scales", z(3, 24, dtype=F16)), ("moe_swiglu_i8", "h", z(9, 25)),
])
def test_operands_of_another_kind_are_refused(calls, name, arg, t):
    with pytest.raises(ValueError):
        getattr(tensors, name)(**{**OPERANDS[name], arg: t})
    assert not calls


def test_rows_that_are_not_dense_are_refused(calls):
    for name, arg, t in (("moe_route", "logits", z(16, 5).t()), ("quantize_rows", "x", z(64, 5).t())):
        with pytest.raises(AssertionError):
            getattr(tensors, name)(**{**OPERANDS[name], arg: t})
    assert not calls


# ---- the oracle's pins -------------------------------------------------------


def test_oracle_routes_a_worked_example():
    l = np.array([[1.0, 3.0, 2.0, 3.0], [0.0, 0.0, 0.0, 0.0]])
    ids, w, pair_row, offsets, token, weight = moe.route(l, "softmax", None, 1, 1, 1, 2, True, 1.0)
    assert ids.tolist() == [[1, 3], [0, 1]] and np.allclose(w, 0.5)
    assert offsets.tolist() == [0, 1, 3, 3, 4] and token.tolist() == [1, 0, 1, 0] and pair_row.tolist() == [[1, 3], [0, 2]]
    ids, w, *_ = moe.route(l, "softmax", np.array([0.5, 0, 0, 0]), 2, 1, 2, 2, False, 2.0)
    p = np.exp(l[0]) / np.exp(l[0]).sum()
    assert ids.tolist() == [[0, 1], [0, 1]]  # 0.5 + p0 + p1 against p2 + p3; of the group both, the higher first
    assert np.allclose(w[0], 2 * p[[0, 1]]) and np.allclose(w[1], 0.5)


def test_oracle_quantizes_a_worked_example():
    codes, scales = moe.quantize_rows([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1, np.inf, 0, 0]])
    assert codes.tolist() == [[127, -64, 0, 2], [0] * 4, [0] * 4] and scales[0] == 1 and scales[1] == 0 and np.isnan(scales[2])


def test_oracle_notices_planted_mistakes():
    # A wrong order among equals, an unstable grouping and a dropped scale all change what the tests compare.
    l = np.zeros((3, 4))
    ids, w, pair_row, offsets, token, _ = moe.route(l, "sigmoid", None, 1, 1, 1, 2, True, 1.0)
    assert ids.tolist() == [[0, 1]] * 3 and token.tolist() == [0, 1, 2, 0, 1, 2]
    wrong = np.sort(ids, 1)[:, ::-1]
    assert not np.array_equal(ids, wrong)
    x = np.array([[1, 2]]); wq = np.array([[3, 4]])
    assert moe.product_i8(wq, [0.5], x, [2.0])[0, 0] == 11.0 != (x @ wq.T)[0, 0] * 0.5
