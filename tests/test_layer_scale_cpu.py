"""Scales that fp32 cannot carry through the attention kernels are refused before any device is touched."""
import pytest

import gemm_qmm_gemv_amd as qmm

A16 = 0x10000  # a 16-byte aligned stand-in address; never dereferenced here


def cache(scale):
    c = qmm.KvCache(A16, A16, A16, A16, A16, A16, 4, 2, 128, 16, 4, 64)
    qmm.qmm_attn_cache(c, A16, A16, 4, A16, 64, A16, 0, 1, 4, scale, None, 0, stream=0)


def prompt(scale):
    qmm.qmm_attn_prompt(A16, A16, A16, A16, A16, 0, 2, 4, 2, 64, 256, 128, 128, 256, scale, stream=0)


@pytest.mark.parametrize("call", [cache, prompt])
@pytest.mark.parametrize("scale,want", [
    (3e38, qmm.QMM_ERR_UNSUPPORTED), (-3e38, qmm.QMM_ERR_UNSUPPORTED), (2.0 ** 65, qmm.QMM_ERR_UNSUPPORTED),
    (-2.0 ** 65, qmm.QMM_ERR_UNSUPPORTED), (1e39, qmm.QMM_ERR_INVALID_ARGUMENT), (2.0 ** 64, qmm.QMM_OK), (-2.0 ** 64, qmm.QMM_OK),
    (0.0, qmm.QMM_OK), (1e-45, qmm.QMM_OK),
])
def test_scales(call, scale, want):
    # (No sequence and no token: a call that is not refused has nothing to do.)
    try:
        call(scale)
        got = qmm.QMM_OK
    except qmm.QmmError as e:
        got = e.status
    assert got == want
