"""perf/more_operators.py: its flag `own` is set after it is imported, its calls then reach the library with the arguments
that the entry points take, and both sides agree with the 64-bit form."""
import importlib.util
import inspect
import os
import random

import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")

ROUTE = dict(op="route", tokens=37, experts=24, top_k=3, score="softmax", bias=False, groups=1, top_groups=1, best=1, renorm=True, scale=1.0,
             f16=False, pad=0)
CASES = [
    (["qmm_moe_route"], ROUTE),
    (["qmm_moe_route"], dict(ROUTE, score="sigmoid", bias=True, groups=4, top_groups=2, best=2, scale=2.5, pad=3, f16=True)),
    (["qmm_quantize_rows", "qmm_gemm_i8"], dict(op="product", m=5, n=40, k=96, x16=True, y16=False)),
    (["qmm_quantize_rows", "qmm_gemm_i8"], dict(op="product", m=130, n=33, k=160, x16=False, y16=True)),
    (["qmm_quantize_rows", "qmm_moe_swiglu_i8"], dict(op="experts", glu=True, tokens=9, experts=6, top_k=2, n=40, k=64, x16=True, y16=True)),
    (["qmm_quantize_rows", "qmm_moe_gemm_i8"], dict(op="experts", glu=False, tokens=70, experts=6, top_k=2, n=40, k=64, x16=False, y16=False)),
    (["qmm_moe_gather"], dict(op="gather", tokens=9, top_k=3, n=72, f16=True, residual=True, pad=2)),
]
NAMES = ("qmm_moe_route", "qmm_quantize_rows", "qmm_gemm_i8", "qmm_moe_gemm_i8", "qmm_moe_swiglu_i8", "qmm_moe_gather")


def module():
    spec = importlib.util.spec_from_file_location("more_operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_listed_and_drawn_cases_state_their_work():
    m = module()
    rng = random.Random(3)
    cases = m.listed() + [m.draw(rng) for _ in range(200)]
    assert len({c["name"] for c in m.listed()}) == len(m.listed())
    for c in cases:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0, c


@pytest.mark.parametrize("names,case", CASES)
def test_calls_reach_the_entry_points(monkeypatch, names, case):
    m = module()
    m.own, m.DEV = True, "cpu"
    seen = []
    for f in NAMES:
        takes = inspect.signature(getattr(qmm, f))
        monkeypatch.setattr(qmm, f, lambda *a, f=f, takes=takes, **kw: seen.append((f, takes.bind(*a, **kw))))
    m.run(m.prepare(case, 1))
    assert [f for f, _ in seen] == names


@pytest.mark.parametrize("names,case", CASES)
def test_the_plain_form_against_64_bits(names, case):
    # 32-bit sums of a few hundred terms, rounded to fp16 at the end where the case says so: below four half steps of it.
    m = module()
    m.DEV = "cpu"
    compare(m.run(m.prepare(case, 5)), m.exact(case, 5))


def compare(got, want):
    pairs = [(got, want)] if torch.is_tensor(got) else [(got[k], want[k]) for k in want]
    for g, w in pairs:
        assert g.shape == w.shape
        if not g.dtype.is_floating_point:
            assert torch.equal(g.long(), w.long())
            continue
        g, w = g.double(), w.double()
        assert float((g - w).norm()) <= 2.0 ** -9 * float(w.norm()) + 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("names,case", CASES)
def test_the_library_against_64_bits(names, case):
    announce("operator case", case)
    want = module().exact(case, 5)
    m = module()
    m.own = True
    got = m.run(m.prepare(case, 5))
    torch.cuda.synchronize()
    compare(got, want)
