"""The torch-side calls of the layer's operators without a GPU: what they hand to the library and what they refuse."""
import pytest
import torch

from gemm_qmm_gemv_amd import tensors

F16, F32, I32, I64 = torch.float16, torch.float32, torch.int32, torch.int64


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, which are not made."""
    seen = []
    for f in ("qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_prompt"):
        monkeypatch.setattr(tensors, f, lambda *a, **kw: seen.append(a))
    return seen


def norm(rows=3, n=64, **kw):
    a = dict(y=torch.zeros(rows, n), residual=torch.zeros(rows, n), pre=torch.zeros(n))
    a.update(kw)
    return tensors.norm_residual(**a)


GATE_STRIDE = 5  # its place among qmm_norm_residual's arguments


@pytest.mark.parametrize("gate,stride", [
    (None, 0), (torch.zeros(64), 0), (torch.zeros(1, 64), 0), (torch.zeros(3, 64), 64), (torch.zeros(3, 80)[:, 8:72], 80),
    (torch.zeros(1, 64).expand(3, 64), 0), (torch.zeros(5, 64), 64),
])
def test_rows_of_a_gate(calls, gate, stride):
    norm(gate=gate)
    assert calls[0][GATE_STRIDE] == stride


@pytest.mark.parametrize("gate", [torch.zeros(2, 64), torch.zeros(3, 63), torch.zeros(63), torch.zeros(64, 1), torch.zeros(1, 3, 64)])
def test_gates_of_another_shape_are_refused(calls, gate):
    with pytest.raises(ValueError, match="gate"):
        norm(gate=gate)
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(y=torch.zeros(3, 96)[:, 8:72]), dict(y=torch.zeros(3, 64, dtype=F16)), dict(y=None), dict(residual=None),
    dict(residual=torch.zeros(1, 3, 64)), dict(h=torch.zeros(8, 64)), dict(x=torch.zeros(3, 64, dtype=F16)), dict(pre=None),
    dict(pre=torch.zeros(1, 64), post=torch.zeros(64)),
])
def test_operands_of_the_norm(calls, kw):
    norm(**kw)
    assert len(calls) == 1


@pytest.mark.parametrize("name,t", [
    ("y", torch.zeros(3, 64, dtype=torch.bfloat16)), ("y", torch.zeros(3, 64, dtype=torch.float64)),
    ("residual", torch.zeros(3, 64, dtype=F16)), ("residual", torch.zeros(3, 80)[:, :64]), ("residual", torch.zeros(2, 64)),
    ("residual", torch.zeros(3, 65)), ("residual", torch.zeros(1, 64).expand(3, 64)), ("h", torch.zeros(3, 64, dtype=torch.float64)),
    ("h", torch.zeros(3, 80)[:, :64]), ("h", torch.zeros(64, 3).t()), ("x", torch.zeros(3, 64)),
    ("x", torch.zeros(3, 80, dtype=F16)[:, :64]), ("x", torch.zeros(2, 64, dtype=F16)), ("pre", torch.zeros(64, dtype=F16)),
    ("pre", torch.zeros(63)), ("pre", torch.zeros(128)[::2]), ("post", torch.zeros(64, dtype=F16)), ("post", torch.zeros(1)),
    ("gate", torch.zeros(64, dtype=F16)), ("gate", torch.zeros(3, 64, dtype=F16)), ("gate", torch.zeros(128)[::2]),
])
def test_operands_that_the_norm_would_misread_are_refused(calls, name, t):
    with pytest.raises(ValueError, match=name):
        norm(**{name: t})
    assert not calls


def test_a_residual_alone_is_looked_at_too(calls):
    for t in (torch.zeros(3, 64, dtype=F16), torch.zeros(3, 80)[:, :64]):
        with pytest.raises(ValueError, match="residual"):
            norm(y=None, residual=t)
    assert not calls
