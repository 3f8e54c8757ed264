"""The entry points of the attention half of a decoder layer without a GPU: what they refuse, before any device is
touched, and the oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest

import gemm_qmm_gemv_amd as qmm
from oracle import layer

A16 = 0x10000  # a 16-byte aligned stand-in address; never dereferenced here
INV, UNS, MIS = qmm.QMM_ERR_INVALID_ARGUMENT, qmm.QMM_ERR_UNSUPPORTED, qmm.QMM_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qmm.library_path()):
        from gemm_qmm_gemv_amd import build
        build.build()
    return qmm.load()


def status(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except qmm.QmmError as e:
        assert qmm.qmm_last_error() != ""
        return e.status
    return qmm.QMM_OK


def cache(**kw):
    a = dict(k=A16, k_scales=A16, k_mins=A16, v=A16, v_scales=A16, v_mins=A16, pages=4, kv_heads=2, head_dim=128, page_size=16,
             bits=4, group_size=64)
    a.update(kw)
    return qmm.KvCache(**a)


def norm(y=A16, y16=False, ys=64, post=A16, gate=A16, gs=64, scale=1.0, res=A16, h=A16, pre=A16, x=A16, rows=2, n=64, eps=1e-6):
    return status(qmm.qmm_norm_residual, y, y16, ys, post, gate, gs, scale, res, h, pre, x, rows, n, eps, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(n=-1), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(n=32769, ys=32769, gs=0), UNS), (dict(rows=1 << 22), UNS), (dict(y=None, res=None), INV), (dict(h=None, x=None), INV),
    (dict(y=None, x=None), INV), (dict(ys=63), INV), (dict(gs=63), INV), (dict(ys=1 << 40), INV), (dict(y=A16 + 2), MIS),
    (dict(y=A16 + 1, y16=True), MIS), (dict(post=A16 + 1), MIS), (dict(gate=A16 + 2), MIS), (dict(res=A16 + 2), MIS),
    (dict(h=A16 + 2), MIS), (dict(pre=A16 + 2), MIS), (dict(x=A16 + 1), MIS),
    (dict(rows=0, y=None, res=None), qmm.QMM_OK), (dict(n=0), qmm.QMM_OK),
])
def test_norm_refusals(lib, kw, want):
    assert norm(**kw) == want


def append(c=None, q=A16, k=A16, v=A16, in16=True, qs=512, ks=256, vs=256, qn=None, kn=None, eps=1e-6, inv=A16, rot=128,
           pos=A16, slots=A16, qo=A16, ko=A16, vo=A16, tokens=3, hq=4):
    return status(qmm.qmm_kv_append, cache() if c is None else c, q, k, v, in16, qs, ks, vs, qn, kn, eps, inv, rot, False, pos, slots, qo, ko, vo,
                  True, tokens, hq, stream=0)


BAD_CACHES = [
    (dict(bits=7), UNS), (dict(bits=2), UNS), (dict(bits=5), UNS), (dict(bits=1), INV), (dict(bits=32), INV), (dict(head_dim=96), UNS),
    (dict(head_dim=256), UNS), (dict(head_dim=0), INV), (dict(head_dim=-64), INV), (dict(kv_heads=0), INV), (dict(kv_heads=4097), INV),
    (dict(page_size=0), INV), (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=1 << 17), UNS),
    (dict(group_size=0), INV), (dict(group_size=16), INV), (dict(group_size=96), INV), (dict(group_size=256), INV), (dict(pages=-1), INV),
    (dict(pages=1 << 31), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(k_scales=None), INV), (dict(v_mins=None), INV),
    (dict(k=A16 + 8), MIS), (dict(v_scales=A16 + 2), MIS),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused_by_both(lib, kw, want):
    c = cache(**kw)
    assert append(c) == want
    assert attend(c) == want


def test_a_null_cache(lib):
    assert append(ctypes.POINTER(qmm.KvCache)()) == INV
    assert attend(ctypes.POINTER(qmm.KvCache)()) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INV), (dict(tokens=1 << 24), UNS), (dict(hq=-1), INV), (dict(hq=4097, qs=1 << 20), INV), (dict(q=None), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(qo=None), INV), (dict(qs=504), INV), (dict(ks=248), INV), (dict(vs=0), INV),
    (dict(qs=516), MIS), (dict(in16=False, qs=514), MIS), (dict(q=A16 + 8), MIS), (dict(k=A16 + 4), MIS), (dict(rot=8), INV),
    (dict(rot=144), INV), (dict(rot=-16), INV), (dict(inv=None), INV), (dict(pos=None), INV), (dict(eps=float("nan")), INV),
    (dict(qo=A16 + 8), MIS), (dict(ko=A16 + 2), MIS), (dict(vo=A16 + 2), MIS), (dict(slots=A16 + 4), MIS), (dict(pos=A16 + 2), MIS),
    (dict(inv=A16 + 2), MIS), (dict(qn=A16 + 2), MIS), (dict(tokens=0, q=None), qmm.QMM_OK),
])
def test_append_refusals(lib, kw, want):
    assert append(**kw) == want


def attend(c=None, q=A16, table=A16, stride=4, lens=A16, mx=64, out=A16, n=2, q_len=1, hq=4, scale=0.1, ws=None, wsb=0):
    return status(qmm.qmm_attn_cache, cache() if c is None else c, q, table, stride, lens, mx, out, n, q_len, hq, scale, ws, wsb, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(q_len=0), INV), (dict(q_len=257), INV), (dict(hq=3), INV), (dict(hq=0), INV), (dict(mx=-1), INV),
    (dict(mx=65), INV), (dict(mx=1 << 30, stride=1 << 30), INV), (dict(stride=-1), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(q=None), INV), (dict(out=None), INV), (dict(lens=None), INV), (dict(table=None), INV),
    (dict(wsb=64), INV), (dict(ws=A16 + 8, wsb=64), MIS), (dict(q=A16 + 8), MIS), (dict(out=A16 + 2), MIS), (dict(table=A16 + 2), MIS),
    (dict(lens=A16 + 2), MIS), (dict(n=1 << 24), UNS), (dict(n=1 << 23, q_len=256), UNS), (dict(n=0, q=None), qmm.QMM_OK),
])
def test_attn_cache_refusals(lib, kw, want):
    assert attend(**kw) == want


def test_a_cache_without_pages_is_refused(lib):
    assert attend(cache(pages=0)) == INV


def test_attn_cache_workspace(lib):
    c = cache()
    need = qmm.qmm_attn_cache_workspace_bytes(c, 1, 1, 16, 8192)
    assert need > 0
    # Enough sequences fill the device on their own; short ones are not split.
    assert qmm.qmm_attn_cache_workspace_bytes(c, 4096, 1, 16, 8192) == 0
    assert qmm.qmm_attn_cache_workspace_bytes(c, 1, 1, 16, 64) == 0
    assert qmm.qmm_attn_cache_workspace_bytes(c, 0, 1, 16, 8192) == 0
    assert qmm.qmm_attn_cache_workspace_bytes(cache(bits=7), 1, 1, 16, 8192) == 0
    assert qmm.qmm_attn_cache_workspace_bytes(c, 1, 1, 3, 8192) == 0


def prompt(q=A16, k=A16, v=A16, off=A16, out=A16, t=10, n=2, hq=4, hkv=2, d=64, qs=256, ks=128, vs=128, os_=256, scale=0.1):
    return status(qmm.qmm_attn_prompt, q, k, v, off, out, t, n, hq, hkv, d, qs, ks, vs, os_, scale, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(d=0), INV), (dict(d=80), UNS), (dict(hq=0), INV), (dict(hkv=0), INV), (dict(hq=5), INV), (dict(hq=8192), INV), (dict(t=-1), INV),
    (dict(n=-1), INV), (dict(t=1 << 31), UNS), (dict(t=1 << 30, hq=64, qs=1 << 20), UNS), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(out=None), INV), (dict(off=None), INV), (dict(qs=248), INV), (dict(ks=127), INV), (dict(os_=255), INV), (dict(qs=260), MIS),
    (dict(q=A16 + 8), MIS), (dict(out=A16 + 4), MIS), (dict(off=A16 + 2), MIS), (dict(scale=float("nan")), INV),
    (dict(t=0, q=None), qmm.QMM_OK), (dict(n=0, q=None), qmm.QMM_OK),
])
def test_prompt_refusals(lib, kw, want):
    assert prompt(**kw) == want


def test_valid_calls_without_a_device_report_one(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (norm, append, attend, prompt):
        assert f() == qmm.QMM_ERR_DEVICE


# ---- the oracle's pins


def test_oracle_packing_round_trip_and_hand_worked_words():
    rng = np.random.default_rng(1)
    for bits in (4, 8):
        codes = rng.integers(0, 2 ** bits, size=(3, 64))
        assert np.array_equal(layer.unpack_rows(layer.pack_rows(codes, bits), bits), codes)
    assert layer.pack_rows(np.arange(8)[None], 4)[0, 0] == 0x76543210
    assert layer.pack_rows(np.array([[1, 2, 3, 255]]), 8)[0, 0] == 0xFF030201


def test_oracle_attend_against_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((9, 4)), rng.standard_normal((9, 4))
    o, a, l, _ = layer.attend(np.zeros((3, 4)), k, v, [9, 4, 0], 1.0)
    assert np.allclose(o[0], v.mean(0)) and np.allclose(o[1], v[:4].mean(0)) and (o[2] == 0).all()
    assert np.allclose(a[0], np.abs(v).mean(0)) and l[0] == 9
    # One key far ahead of the rest takes all the weight.
    k[5] = 100
    o = layer.attend(np.ones((1, 4)), k, v, [9], 1.0)[0]
    assert np.allclose(o[0], v[5])


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 64))
    inv = 1e4 ** (-np.arange(16) / 16)
    for inter in (False, True):
        y = layer.rotate(x, np.arange(5) * 1000, inv, 32, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.array_equal(y[0], x[0])
        # Products of rotated rows depend on the distance of their positions alone.
        a = layer.rotate(x[:1], [7], inv, 32, inter) * layer.rotate(x[1:2], [3], inv, 32, inter)
        b = layer.rotate(x[:1], [107], inv, 32, inter) * layer.rotate(x[1:2], [103], inv, 32, inter)
        assert np.allclose(a.sum(-1), b.sum(-1))


def test_oracle_norm_of_known_rows():
    u, h, x = layer.norm_residual(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), None, 2.0, np.array([[1.0, 1.0]]), None, 0.0)
    r = np.sqrt(12.5)
    assert np.allclose(u, [[3 / r, 8 / r]]) and np.allclose(h, [[1 + 6 / r, 1 + 16 / r]])
    assert np.allclose((x ** 2).mean(-1), 1)


def test_words_that_no_int_holds_are_refused_and_no_call_is_unknown(lib):
    # Arguments travel as 64-bit words: 2^32 + 1 must not become 1.
    cache = qmm.KvCache(4096, 4096, 4096, 4096, 4096, 4096, 1, 1, 64, 16, 4, 32)
    for q_len in (2 ** 32 + 1, -2 ** 32 + 1):
        with pytest.raises(qmm.QmmError, match="q_len"):
            qmm.qmm_attn_cache(cache, 4096, 4096, 1, 4096, 16, 4096, 1, q_len, 1, 1.0, stream=0)
    assert lib.qmm_call_words(4, bytes(23 * 8)) == qmm.QMM_ERR_INVALID_ARGUMENT
    assert lib.qmm_call_words(-1, bytes(23 * 8)) == qmm.QMM_ERR_INVALID_ARGUMENT
    assert lib.qmm_call_words(0, None) == qmm.QMM_ERR_INVALID_ARGUMENT
