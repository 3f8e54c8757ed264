"""The torch-side calls of the layer's operators without a GPU: what they hand to the library and what they refuse."""
import pytest
import torch

from gemm_qmm_gemv_amd import tensors

F16, F32, I32, I64 = torch.float16, torch.float32, torch.int32, torch.int64


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, which are not made; tensors may be on the host."""
    seen = []
    monkeypatch.setattr(tensors, "_on_device", lambda *ts: None)
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
    dict(pre=torch.zeros(1, 64), post=torch.zeros(64)), dict(residual=torch.zeros(192), h=torch.zeros(192), x=torch.zeros(200, dtype=F16)),
])
def test_operands_of_the_norm(calls, kw):
    norm(**kw)
    assert len(calls) == 1


@pytest.mark.parametrize("name,t", [
    ("y", torch.zeros(3, 64, dtype=torch.bfloat16)), ("y", torch.zeros(3, 64, dtype=torch.float64)),
    ("residual", torch.zeros(3, 64, dtype=F16)), ("residual", torch.zeros(3, 80)[:, :64]), ("residual", torch.zeros(2, 64)),
    ("residual", torch.zeros(3, 65)), ("residual", torch.zeros(191)), ("h", torch.zeros(384)[::2]), ("residual", torch.zeros(1, 64).expand(3, 64)), ("h", torch.zeros(3, 64, dtype=torch.float64)),
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


def cache(bits=4, group=32, pages=4, hkv=2, d=64, page=16):
    return tensors.kv_cache(pages, hkv, d, page, bits, group, device="cpu")


def append(tokens=3, hq=4, hkv=2, d=64, **kw):
    a = dict(cache=cache(hkv=hkv, d=d), q=torch.zeros(tokens, hq * d, dtype=F16), k=torch.zeros(tokens, hkv * d, dtype=F16),
             v=torch.zeros(tokens, hkv * d, dtype=F16), positions=torch.zeros(tokens, dtype=I32), slots=torch.zeros(tokens, dtype=I64),
             inv_freq=torch.zeros(d // 2))
    a.update(kw)
    return tensors.kv_append(**a)


def attend(n=3, q_len=2, hq=4, hkv=2, d=64, **kw):
    a = dict(cache=cache(hkv=hkv, d=d), q=torch.zeros(n * q_len, hq, d, dtype=F16), page_table=torch.zeros(n, 4, dtype=I32),
             kv_lens=torch.zeros(n, dtype=I32), max_kv_len=64, q_len=q_len, workspace=torch.zeros(16, dtype=torch.uint8))
    a.update(kw)
    return tensors.attn_cache(**a)


def prompt(tokens=10, hq=4, hkv=2, d=64, **kw):
    a = dict(q=torch.zeros(tokens, hq, d, dtype=F16), k=torch.zeros(tokens, hkv, d, dtype=F16),
             v=torch.zeros(tokens, hkv, d, dtype=F16), seq_offsets=torch.tensor([0, 4, 10], dtype=I32))
    a.update(kw)
    return tensors.attn_prompt(**a)


@pytest.mark.parametrize("call,name,t", [
    (append, "positions", torch.zeros(3, dtype=I64)), (append, "positions", torch.zeros(3)), (append, "positions", torch.zeros(2, dtype=I32)),
    (append, "positions", torch.zeros(6, dtype=I32)[::2]), (append, "slots", torch.zeros(3, dtype=I32)),
    (append, "slots", torch.zeros(2, dtype=I64)), (append, "slots", torch.zeros(1, dtype=I64).expand(3)),
    (append, "slots", torch.zeros(6, dtype=I64)[::2]), (attend, "kv_lens", torch.zeros(3, dtype=I64)),
    (attend, "kv_lens", torch.zeros(6, dtype=I32)[::2]), (attend, "page_table", torch.zeros(3, 4, dtype=I64)),
    (attend, "page_table", torch.zeros(3, 4, dtype=torch.int16)), (prompt, "seq_offsets", torch.tensor([0, 4, 10])),
    (prompt, "seq_offsets", torch.zeros(6, dtype=I32)[::2]), (prompt, "seq_offsets", torch.zeros(0, dtype=I32)),
])
def test_indices_of_another_type_or_with_gaps_are_refused(calls, call, name, t):
    with pytest.raises(ValueError, match=name):
        call(**{name: t})
    assert not calls


@pytest.mark.parametrize("call,kw", [
    (append, {}), (append, dict(positions=torch.zeros(9, dtype=I32), slots=torch.zeros(9, dtype=I64))), (append, dict(slots=None)),
    (append, dict(positions=None, inv_freq=None)), (append, dict(positions=torch.zeros(3, dtype=I64), inv_freq=None)),
    (append, dict(tokens=0)), (attend, {}), (attend, dict(n=1)), (attend, dict(page_table=torch.zeros(3, 9, dtype=I32)[:, 2:6])),
    (attend, dict(n=0)), (prompt, {}), (prompt, dict(seq_offsets=torch.tensor([0], dtype=I32))),
    (prompt, dict(tokens=0, seq_offsets=torch.tensor([0, 0], dtype=I32))),
])
def test_calls_that_are_handed_on(calls, call, kw):
    call(**kw)
    assert len(calls) == 1


@pytest.mark.parametrize("call,name,t", [
    (attend, "q", torch.zeros(6, 4, 64)), (attend, "q", torch.zeros(6, 2, 128, dtype=F16)), (attend, "out", torch.zeros(6, 4, 64)),
    (attend, "out", torch.zeros(6, 8, 64, dtype=F16)[:, :4]), (attend, "out", torch.zeros(5, 4, 64, dtype=F16)),
    (attend, "page_table", torch.zeros(4, 3, dtype=I32).t()), (attend, "page_table", torch.zeros(3, 8, dtype=I32)[:, ::2]),
    (attend, "page_table", torch.zeros(2, 4, dtype=I32)), (attend, "page_table", torch.zeros(4, dtype=I32)),
    # Rows are wide enough, but not what belongs to a sequence.
    (attend, "page_table", torch.zeros(3, 8, dtype=I32)[:, 5:]), (attend, "workspace", torch.zeros(64, dtype=torch.uint8)[::2]),
    (prompt, "q", torch.zeros(10, 4, 64)), (prompt, "k", torch.zeros(10, 2, 64)), (prompt, "v", torch.zeros(10, 2, 64, dtype=torch.bfloat16)),
    (prompt, "k", torch.zeros(9, 2, 64, dtype=F16)), (prompt, "v", torch.zeros(9, 2, 64, dtype=F16)),
    (prompt, "v", torch.zeros(10, 1, 64, dtype=F16)), (prompt, "k", torch.zeros(10, 2, 128, dtype=F16)),
    (prompt, "v", torch.zeros(10, 4, 32, dtype=F16)), (prompt, "out", torch.zeros(10, 4, 64)),
    (prompt, "out", torch.zeros(9, 4, 64, dtype=F16)), (prompt, "out", torch.zeros(10, 4, 32, dtype=F16)),
])
def test_operands_that_attention_would_misread_are_refused(calls, call, name, t):
    with pytest.raises(ValueError, match=name):
        call(**{name: t})
    assert not calls


@pytest.mark.parametrize("call,kw", [
    (attend, dict(out=torch.zeros(6, 4 * 64, dtype=F16))), (attend, dict(q=torch.zeros(3, 2, 4, 64, dtype=F16))),
    (attend, dict(page_table=torch.zeros(5, 4, dtype=I32))), (attend, dict(page_table=torch.zeros(3, 1, dtype=I32), max_kv_len=16)),
    (prompt, dict(out=torch.zeros(10, 4 * 64, dtype=F16))), (prompt, dict(out=torch.zeros(10, 4 * 64 + 8, dtype=F16)[:, :256])),
    (prompt, dict(k=torch.zeros(16, 2, 64, dtype=F16), v=torch.zeros(16, 2, 64, dtype=F16))),
    (prompt, dict(k=torch.zeros(10, 8, 64, dtype=F16)[:, 2:4])),
])
def test_other_layouts_of_attention_are_handed_on(calls, call, kw):
    call(**kw)
    assert len(calls) == 1


@pytest.mark.parametrize("name,t", [
    ("q", torch.zeros(3, 260, dtype=F16)), ("k", torch.zeros(2, 128, dtype=F16)), ("k", torch.zeros(3, 64, dtype=F16)),
    ("k", torch.zeros(3, 256, dtype=F16)), ("v", torch.zeros(3, 130, dtype=F16)), ("v", torch.zeros(1, 128, dtype=F16)),
    ("out", torch.zeros(3, 4, 64)), ("out", torch.zeros(2, 4, 64, dtype=F16)), ("out", torch.zeros(3, 8, 64, dtype=F16)[:, :4]),
    ("inv_freq", torch.zeros(32, dtype=torch.float64)), ("inv_freq", torch.zeros(64)[::2]), ("q_norm", torch.zeros(64, dtype=F16)),
    ("q_norm", torch.zeros(32)), ("k_norm", torch.zeros(128)[::2]), ("k_norm", torch.zeros(64, dtype=torch.float64)),
])
def test_operands_that_the_append_would_misread_are_refused(calls, name, t):
    with pytest.raises(ValueError, match=name):
        append(**{name: t})
    assert not calls


def test_rows_of_bfloat16_are_refused(calls):
    rows = {x: torch.zeros(3, w, dtype=torch.bfloat16) for x, w in (("q", 256), ("k", 128), ("v", 128))}
    with pytest.raises(ValueError, match="q is"):
        append(**rows)
    assert not calls


Q_HEADS = 21  # its place among qmm_kv_append's arguments


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 4, 64, dtype=F16), k=torch.zeros(3, 2, 64, dtype=F16)), dict(out=torch.zeros(3, 256, dtype=F16)),
    dict(out=torch.zeros(9, 4, 64, dtype=F16)), dict(q_norm=torch.zeros(64), k_norm=torch.zeros(64)),
    {x: torch.zeros(3, 512)[:, a:b] for x, a, b in (("q", 0, 256), ("k", 256, 384), ("v", 384, 512))},
    dict(k=torch.zeros(8, 128, dtype=F16), v=torch.zeros(8, 128, dtype=F16)),
    dict(tokens=0, q=torch.zeros(0, 4, 64, dtype=F16)),
])
def test_other_layouts_of_the_append_are_handed_on(calls, kw):
    append(**kw)
    assert len(calls) == 1 and calls[0][Q_HEADS] == 4


@pytest.mark.parametrize("call", [norm, append, attend, prompt])
def test_tensors_in_host_memory_are_refused(monkeypatch, call):
    for f in ("qmm_norm_residual", "qmm_kv_append", "qmm_attn_cache", "qmm_attn_prompt"):
        monkeypatch.setattr(tensors, f, None)
    with pytest.raises(ValueError, match="on cpu"):
        call()


def test_every_operand_is_looked_at(monkeypatch):
    seen = []

    def note(*ts):
        seen.extend(ts)
        raise ValueError
    monkeypatch.setattr(tensors, "_on_device", note)
    given = {n: torch.zeros(1) for n in ("y", "residual", "pre", "post", "gate", "h", "x")}
    named = {n: torch.zeros(1) for n in ("q", "k", "v", "positions", "slots", "inv_freq", "q_norm", "k_norm", "out")}
    held = cache()
    for call, ts in ((tensors.norm_residual, given), (tensors.kv_append, named | dict(cache=held))):
        seen.clear()
        with pytest.raises(ValueError):
            call(**ts)
        for t in ts.values():
            for u in (t.keep if t is held else (t,)):
                assert any(u is s for s in seen)
    named = {n: torch.zeros(1) for n in ("q", "page_table", "kv_lens", "out", "workspace")}
    seen.clear()
    with pytest.raises(ValueError):
        tensors.attn_cache(held, max_kv_len=1, **named)
    assert all(any(u is s for s in seen) for u in list(named.values()) + list(held.keep))
    named = {n: torch.zeros(1) for n in ("q", "k", "v", "seq_offsets", "out")}
    seen.clear()
    with pytest.raises(ValueError):
        tensors.attn_prompt(**named)
    assert all(any(u is s for s in seen) for u in named.values())


class _On:
    """Stands in for a tensor on some device."""
    def __init__(self, at):
        self.at, self.device = at, "cuda:%d" % at

    def get_device(self):
        return self.at


def test_tensors_of_another_gpu_are_refused(monkeypatch):
    monkeypatch.setattr(torch, "Tensor", _On)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    tensors._on_device(_On(1), None, 4096, _On(1))
    for ts in ((_On(0),), (_On(1), _On(0)), (_On(1), _On(-1)), (_On(-1), _On(1))):
        with pytest.raises(ValueError, match="not on the current GPU"):
            tensors._on_device(*ts)
