"""Attention at the largest scales that are taken: the key of the largest product takes all the weight."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import DeviceCache, dev, empty_cache, held
from tests.test_gpu_layer_attn_prompt import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** 64, -2.0 ** 64])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt(scale, d):
    # Products are small whole numbers, different for every key.
    rng = np.random.default_rng([101, d])
    t = 90
    q, k = np.zeros((t, 2, d), np.float16), np.zeros((t, 1, d), np.float16)
    q[:, :, 3] = 1
    k[:, 0, 3] = rng.permutation(t) - t // 2
    v = rng.standard_normal((t, 1, d)).astype(np.float16)
    announce("prompt, scale", scale, d)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), [0, t], scale, out)
    for i in range(t):
        s = k[:i + 1, 0, 3] * np.sign(scale)
        assert np.array_equal(got[i], np.broadcast_to(v[s.argmax()], (2, d))), i


@pytest.mark.parametrize("scale", [2.0 ** 64, -2.0 ** 64])
@pytest.mark.parametrize("bits,d", [(4, 64), (8, 128), (16, 128)])
def test_cache(scale, bits, d):
    rng = np.random.default_rng([102, bits, d])
    n, page = 13, 16
    host = empty_cache(rng, 1, 1, d, page, bits, 32)
    if bits == 16:
        rows = host["k"].view(np.float16)
        rows[:] = 0
        rows[0, 0, :n, 3] = rng.permutation(n) - n // 2
    else:
        codes = np.zeros((page, d), np.int64)
        codes[:n, 3] = rng.permutation(n)
        host["k"][0, 0] = layer.pack_rows(codes, bits)
        host["ks"][:], host["km"][:] = 1, 0
    cache = DeviceCache(host, 1, 1, d, page, bits, 32)
    q = np.zeros((1, 2, d), np.float16)
    q[:, :, 3] = 1
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    announce("cache, scale", scale, bits, d)
    qmm.qmm_attn_cache(cache.handle, dev(q), dev(np.zeros((1, 1), np.int32)), 1, dev(np.array([n], np.int32)), n, out, 1, 1, 2, scale)
    torch.cuda.synchronize()
    ks, vs = (held(host, s, bits, 32)[0, 0, :n] for s in "kv")
    want = vs[(ks[:, 3] * np.sign(scale)).argmax()]
    # fp16(scale * code + min), rounded once.
    assert np.abs(out.cpu().numpy()[0] - want).max() <= 2.0 ** -11 * np.abs(want).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [300, 3000, 30000])
def test_prompt_with_large_queries_and_keys(size, d):
    # Scores of 1e6 to 1e12, a multiple of `size` each: the differences leave one key, or equal ones (their mean).
    rng = np.random.default_rng([103, size, d])
    t, heads = 300, 32
    q, k = (rng.integers(-1, 2, size=(t, h, d)).astype(np.float16) for h in (heads, 1))
    k *= np.float16(size)
    q[:, ::2] *= np.float16(size)
    v = rng.standard_normal((t, 1, d)).astype(np.float16)
    announce("prompt, large scores", size, d)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), [0, t], 1.0, out)
    assert np.isfinite(got).all()
    for i in sorted(set(int(x) for x in rng.integers(0, t, 25)) | {0, t - 1}):
        # Scores are whole multiples of a unit: `size` in odd heads, its square in even ones.  Partial sums are below d units;
        # as fp32 they are exact if the unit's odd part times d is below 2^24, so the weights are those of the equal keys at
        # the top (the rest is e^-300 or less) and the output is rounded once.
        for h in range(heads):
            unit = size ** 2 if h % 2 == 0 else size
            odd = unit // (unit & -unit)
            o, a, _, _ = layer.attend(q[i, h:h + 1], k[:i + 1, 0], v[:i + 1, 0], [i + 1], 1.0)
            slack = 2.0 ** -11 * 1.01 * np.abs(o[0]) + 2.0 ** -18 * a[0] + 2.0 ** -25
            if odd * d < 2 ** 24:
                assert (np.abs(got[i, h] - o[0]) <= slack).all(), (i, h)
            else:
                # A score is off by up to d roundings of 2^-24 times sum |q k|, below d units: d^2 2^-24 units, far below one.
                # Keys that are not at the top stay without weight; which of the equal ones at the top share it is open.
                s = k[:i + 1, 0].astype(np.float64) @ q[i, h].astype(np.float64)
                top = v[:i + 1, 0][s == s.max()].astype(np.float64)
                slack = 2.0 ** -10 * np.abs(top).max(0) + 2.0 ** -25
                assert (got[i, h] >= top.min(0) - slack).all() and (got[i, h] <= top.max(0) + slack).all(), (i, h)
