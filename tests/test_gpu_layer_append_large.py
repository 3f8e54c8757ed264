"""qmm_kv_append with values beyond fp16: what the cache holds of them, and what attention over it gives."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import E16, DeviceCache, check, dev, empty_cache, held

pytestmark = pytest.mark.gpu

D, PAGE, GROUP = 64, 16, 32


def stored(bits, k, v, cached=True):
    """Rows k, v [tokens][64] in a cache of one head, and what the call returned of them."""
    n = len(k)
    cache = DeviceCache(empty_cache(np.random.default_rng(1), 1, 1, D, PAGE, bits, GROUP), 1, 1, D, PAGE, bits, GROUP)
    outs = [torch.zeros((n, 1, D), dtype=torch.float16, device="cuda") for _ in range(3)]
    kd, vd = dev(k.astype(np.float32)), dev(v.astype(np.float32))
    qmm.qmm_kv_append(cache.handle, kd, kd, vd, False, D, D, D, None, None, 0.0, None, 0, False, None, dev(np.arange(n)),
                      *outs, cached, n, 1)
    torch.cuda.synchronize()
    return cache, outs


def group_of(low, high):
    return np.linspace(low, high, GROUP)


# Groups whose lowest value is beyond fp16 in either direction, with a spread of a scale in range.
LOST = [(70000, 70010), (-70010, -70000), (-1e5, 0), (-1e5, 1e5), (65520, 65530), (3e5, 3e5)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("low,high", LOST)
def test_a_group_whose_lowest_value_is_beyond_fp16_reads_back_as_nan(bits, low, high):
    rng = np.random.default_rng(91)
    x = rng.standard_normal((3, D))
    x[1, GROUP:] = group_of(low, high)
    announce("append beyond fp16", bits, low, high)
    cache, outs = stored(bits, x, x)
    after = cache.host()
    for side, out in (("k", outs[1]), ("v", outs[2])):
        got = held(after, side, bits, GROUP)[0, 0, :3]
        assert np.isnan(got[1, GROUP:]).all() and np.isfinite(got[0]).all() and np.isfinite(got[2]).all()
        assert np.isfinite(got[1, :GROUP]).all()
        o = out.cpu().numpy()[:, 0]
        assert np.isnan(o[1, GROUP:]).all() and np.isfinite(o[0]).all() and np.isfinite(o[1, :GROUP]).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("low,high", LOST)
@pytest.mark.parametrize("side", ["k", "v"])
def test_such_a_group_reaches_the_tokens_that_see_it_and_no_others(bits, low, high, side):
    rng = np.random.default_rng(92)
    rows = {s: rng.standard_normal((6, D)) for s in "kv"}
    rows[side][5, GROUP:] = group_of(low, high)
    announce("attention over a group beyond fp16", bits, low, high, side)
    cache, _ = stored(bits, rows["k"], rows["v"])
    # Queries of one sign: the products with an infinite row would be infinities of one sign.
    q = np.abs(rng.standard_normal((2, 1, D))).astype(np.float16)
    out = torch.zeros((2, 1, D), dtype=torch.float16, device="cuda")
    table, lens = dev(np.zeros((1, 1), np.int32)), dev(np.array([6], np.int32))
    qmm.qmm_attn_cache(cache.handle, dev(q), table, 1, lens, 6, out, 1, 2, 1, 0.125)
    torch.cuda.synchronize()
    got = out.cpu().numpy()[:, 0]
    after = cache.host()
    ks, vs = (held(after, s, bits, GROUP)[0, 0] for s in "kv")
    o = layer.attend(q[:1, 0], ks[:5], vs[:5], [5], 0.125)[0]
    assert np.abs(got[0] - o[0]).max() < 2.0 ** -9 * 5  # values of up to 5, rounded to fp16 twice
    # The second token sees all six rows.
    assert np.isnan(got[1]).all() if side == "k" else not np.isfinite(got[1, GROUP:]).any()


@pytest.mark.parametrize("bits", [4, 8])
def test_a_group_whose_highest_value_alone_is_beyond_fp16_is_held(bits):
    # The scale is in range: keys are used as they are held, values (and rows given back) beyond fp16 are infinities.
    x = np.zeros((2, D))
    x[1, :GROUP] = group_of(0, 1e5)
    announce("append, highest value beyond fp16", bits)
    cache, outs = stored(bits, x, x)
    after = cache.host()
    top = 2.0 ** bits - 1
    step = 1e5 / top
    for side, out in (("k", outs[1]), ("v", outs[2])):
        got = held(after, side, bits, GROUP)[0, 0]
        check(got[1, :GROUP], x[1, :GROUP], 0.5 * step + E16 * 1e5, "held")
        o = out.cpu().numpy()[1, 0, :GROUP].astype(np.float64)
        with np.errstate(over="ignore"):
            want = got[1, :GROUP].astype(np.float16).astype(np.float64)
        assert np.array_equal(o, want) and np.isinf(o).any()
    # As a key: weights of two rows, one of zeros.  Scores of up to 6e4 times the query's 2^-12.
    q = np.full((1, 1, D), 2.0 ** -12, dtype=np.float16)
    out = torch.zeros((1, 1, D), dtype=torch.float16, device="cuda")
    v = DeviceCache(after | {"vs": np.zeros_like(after["vs"]), "vm": np.arange(after["vm"].size, dtype=np.float16).reshape(after["vm"].shape)},
                    1, 1, D, PAGE, bits, GROUP)
    qmm.qmm_attn_cache(v.handle, dev(q), dev(np.zeros((1, 1), np.int32)), 1, dev(np.array([2], np.int32)), 2, out, 1, 1, 1, 0.01)
    torch.cuda.synchronize()
    keys, values = (held(v.host(), s, bits, GROUP)[0, 0] for s in "kv")
    o = layer.attend(q[:, 0], keys[:2], values[:2], [2], 0.01)[0]
    assert np.abs(out.cpu().numpy()[0, 0] - o[0]).max() <= 2.0 ** -9 * np.abs(values[:2]).max()
