"""qmm_attn_cache over rows whose scale and min are finite and whose values leave fp16, against the float64 definition."""
import copy

import numpy as np
import pytest

from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import DeviceCache, check
from tests.test_gpu_layer_attn_cache import expect, run, setup

pytestmark = pytest.mark.gpu

FORMS = [(4, 64, 32), (4, 64, 64), (4, 128, 32), (4, 128, 64), (4, 128, 128), (8, 64, 32), (8, 64, 64), (8, 128, 64), (8, 128, 128)]


def spoiled(seed, bits, d, group, codes_of, scale, low):
    """Fifty rows, three drafts; row 48 (seen by drafts 1 and 2) of kv head 1 has `scale`, `low` and its codes changed."""
    rng = np.random.default_rng([seed, bits, d, group])
    lens, hq, hkv, page = [50], 6, 2, 16
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
    clean = copy.deepcopy(host)
    p, place = table[0, 48 // page], 48 % page
    g = d // group - 1  # the last group
    host["vs"][p, 1, g, place], host["vm"][p, 1, g, place] = scale, low
    codes = layer.unpack_rows(host["v"][p, 1, place], bits)
    codes[g * group:] = codes_of(codes[g * group:])
    host["v"][p, 1, place] = layer.pack_rows(codes, bits)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("values beyond fp16", bits, d, group, float(scale), float(low))
    got = run(DeviceCache(host, pages, hkv, d, page, bits, group), q, table, lens, 50, 3, hq, 0.125)
    ask = lambda h: expect(h, table, lens, q, 3, hq, hkv, d, bits, group, 0.125)
    return got, ask(clean), ask(host), g * group


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("bits,d,group", FORMS)
def test_a_value_beyond_fp16_reaches_only_the_drafts_that_see_it(bits, d, group, sign):
    # The lowest code's value is in range, the highest one's is 100020 (or -100020): one element has it.
    top = 2 ** bits - 1

    def one(c):
        c = c * 0
        c[5] = top
        return c
    got, (o, bound), _, at = spoiled(81, bits, d, group, one, np.float16(sign * 1e5 / top), np.float16(0))
    check(got[0], o[0], bound[0], "the draft that does not see it")
    check(got[1:, :3], o[1:, :3], bound[1:, :3], "the other key head")
    # (Beyond fp16 the value is an infinity: no row that sees it stays finite there.)
    assert not np.isfinite(got[1:, 3:, at + 5]).any()


@pytest.mark.parametrize("bits,d,group", FORMS)
def test_a_range_beyond_fp16_whose_values_are_not_is_exact(bits, d, group):
    # The highest code would leave fp16, but the codes that are there do not: nothing is spoiled.
    top = 2 ** bits - 1
    most = int(60000 / (1e5 / top))
    got, _, (o, bound), at = spoiled(82, bits, d, group, lambda c: np.minimum(c, most), np.float16(1e5 / top), np.float16(0))
    check(got, o, bound, "large values")
    assert np.abs(got[1:, 3:, at:]).max() > 100


def test_every_row_beyond_fp16_behind_the_last_one():
    # A recycled page: what lies behind the sequence leaves fp16 with finite scales and mins.
    for bits, d, group in ((4, 64, 32), (8, 128, 64)):
        rng = np.random.default_rng([83, bits])
        lens, hq, hkv, page = [21, 9], 4, 2, 16
        host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
        clean = copy.deepcopy(host)
        for i, n in enumerate(lens):
            for t in range(n, -(-n // page) * page):
                host["vs"][table[i, t // page], :, :, t % page] = np.float16(60000)
                host["vm"][table[i, t // page], :, :, t % page] = np.float16(60000)
        q = rng.standard_normal((2, hq, d)).astype(np.float16)
        announce("values beyond fp16 behind the last row", bits)
        got = run(DeviceCache(host, pages, hkv, d, page, bits, group), q, table, lens, 21, 1, hq, 0.125)
        o, bound = expect(clean, table, lens, q, 1, hq, hkv, d, bits, group, 0.125)
        check(got, o, bound, "rows behind the last one")
