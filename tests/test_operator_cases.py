"""perf/operators.py: its flag `own` is set after it is imported, and its calls then reach the library with the arguments
that the entry points take."""
import importlib.util
import inspect
import os

import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")

CASES = [
    ("qmm_norm_residual", dict(op="norm", rows=5, n=96, y16=True, y=True, post=True, gate="shared")),
    ("qmm_norm_residual", dict(op="norm", rows=3, n=33, y16=False, y=False, post=False, gate="none")),
    ("qmm_kv_append", dict(op="append", tokens=21, seqs=3, hq=4, hkv=2, d=64, bits=16, group=32, page=16, in16=False, fused=True,
                           qknorm=True, rot=64, inter=False, far=500, pad=2)),
    ("qmm_kv_append", dict(op="append", tokens=9, seqs=2, hq=2, hkv=1, d=128, bits=8, group=64, page=16, in16=True, fused=False,
                           qknorm=False, rot=64, inter=True, far=0, pad=0)),
    ("qmm_attn_cache", dict(op="cache", seqs=3, lo=0, hi=300, q_len=2, hq=4, hkv=2, d=64, bits=4, group=32, page=16)),
    ("qmm_attn_prompt", dict(op="prompt", seqs=3, lo=1, hi=70, hq=4, hkv=2, d=128, tail=3)),
]


def module():
    spec = importlib.util.spec_from_file_location("operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_listed_and_drawn_cases_state_their_work():
    import random
    m = module()
    rng = random.Random(3)
    cases = m.listed() + [m.draw(rng) for _ in range(200)]
    assert len({c["name"] for c in m.listed()}) == len(m.listed())
    for c in cases:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0, c


@pytest.mark.parametrize("name,case", CASES)
def test_calls_reach_the_entry_points(monkeypatch, name, case):
    m = module()
    m.own, m.DEV = True, "cpu"
    seen = []
    for f in ("qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_prompt"):
        takes = inspect.signature(getattr(qmm, f))
        monkeypatch.setattr(qmm, f, lambda *a, f=f, takes=takes, **kw: seen.append((f, takes.bind(*a, **kw))))
    m.run(m.prepare(case, 1))
    assert [f for f, _ in seen] == [name]


@pytest.mark.gpu
@pytest.mark.parametrize("name,case", CASES)
def test_the_library_and_the_plain_form_against_64_bits(name, case):
    # Outputs are fp16 (or fp32) roundings of a few roundings: below four half steps of fp16 in the 2-norm.  A code next to
    # a border may go either way, one in 10^4 or fewer of 2^8 steps a group, which 2^-9 covers as well.
    announce("operator case", case)
    want = module().exact(case, 5)
    for own in (False, True):
        m = module()
        m.own = own
        got = m.run(m.prepare(case, 5))
        torch.cuda.synchronize()
        pairs = [(got, want)] if torch.is_tensor(got) else [(got[k], want[k]) for k in want]
        for g, w in pairs:
            g, w = g.double(), w.double()
            assert g.shape == w.shape
            assert float((g - w).norm()) <= 2.0 ** -9 * float(w.norm()) + 1e-12, own
