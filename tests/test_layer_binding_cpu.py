"""The binding of the layer's operators without a GPU: how a cache is handed over."""
import ctypes

import pytest

import gemm_qmm_gemv_amd as qmm

A16 = 0x10000  # a 16-byte aligned stand-in address; never dereferenced here


def make(**kw):
    a = dict(k=A16, k_scales=A16, k_mins=A16, v=A16, v_scales=A16, v_mins=A16, pages=4, kv_heads=2, head_dim=128, page_size=16,
             bits=4, group_size=64)
    a.update(kw)
    return qmm.KvCache(**a)


def append(cache):
    qmm.qmm_kv_append(cache, A16, A16, A16, True, 512, 256, 256, None, None, 1e-6, A16, 128, False, A16, A16, A16, A16, A16,
                      True, -1, 4, stream=0)


def attend(cache):
    qmm.qmm_attn_cache(cache, A16, A16, 4, A16, 64, A16, 2, 0, 4, 0.1, None, 0, stream=0)


def said(call, cache):
    with pytest.raises(qmm.QmmError) as e:
        call(cache)
    return e.value.status, qmm.qmm_last_error()


# The calls are refused for an argument behind the cache's own checks, or for something of the cache: either way the answer
# tells which struct was read.
@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kw", [{}, dict(head_dim=96), dict(page_size=48), dict(bits=7)])
def test_ways_to_hand_over_a_cache(call, kw):
    cache = make(**kw)
    several = (qmm.KvCache * 2)(make(bits=1), cache)
    want = said(call, cache)
    for way in (ctypes.pointer(cache), ctypes.byref(cache), ctypes.cast(ctypes.addressof(cache), ctypes.POINTER(qmm.KvCache)),
                several[1], ctypes.byref(several[0], ctypes.sizeof(qmm.KvCache)), (qmm.KvCache * 1)(cache)):
        # The pointer object is followed by memory of its own that differs from try to try.
        for _ in range(20):
            assert said(call, way) == want


@pytest.mark.parametrize("call", [append, attend])
def test_no_cache(call):
    for _ in range(50):
        for way in (None, ctypes.POINTER(qmm.KvCache)()):
            assert said(call, way) == (qmm.QMM_ERR_INVALID_ARGUMENT, "NULL cache")


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("other", [A16, 1.0, "cache", ctypes.c_int64(5), ctypes.pointer(ctypes.c_int64(5)),
                                   ctypes.byref(ctypes.c_int64(5)), ctypes.c_void_p(A16)])
def test_other_objects_are_no_cache(call, other):
    with pytest.raises(TypeError):
        call(other)
