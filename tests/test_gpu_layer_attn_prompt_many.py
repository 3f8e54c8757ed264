"""qmm_attn_prompt on grids that half fill and that fill the device (work-groups of 64 and of 128 rows), against the
float64 definition."""
import numpy as np
import pytest
import torch

from tests.gpu_util import announce
from tests.layer_util import check, dev
from tests.test_gpu_layer_attn_prompt import call, compare, expect, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("behind", [0, 1100])
@pytest.mark.parametrize("d", [64, 128])
def test_non_finite_values_reach_only_the_rows_that_see_them(d, behind):
    # Rows on both sides of each spoiled key, in its tile of keys and far from it; sequences that begin inside a tile.
    rng = np.random.default_rng([41, d])
    lens = [700, 3, 0, 997, behind]
    offsets = [0, 700, 703, 703, 1700, 1700 + behind]
    hq, hkv, t = 32, 4, 1700 + behind
    q, k, v = inputs(rng, t, hq, hkv, d)
    v[333, 0, 3] = np.nan     # rows 333..699, heads 0..7
    v[701, 1, 7] = np.inf     # rows 701 and 702, heads 8..15
    k[1201, 2, 0] = np.nan    # rows 1201..1699, heads 16..23
    v[703, 3, d - 1] = -np.inf  # all of the last sequence, heads 24..31
    announce("non-finite prompt", lens, d)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out)
    spoiled = np.zeros((t, hq), dtype=bool)
    spoiled[333:700, :8] = spoiled[701:703, 8:16] = spoiled[1201:1700, 16:24] = spoiled[703:1700, 24:] = True
    assert np.array_equal(np.isfinite(got).all(-1), ~spoiled)
    k[1201, 2, 0] = v[333, 0, 3] = v[701, 1, 7] = v[703, 3, d - 1] = 0
    rows = sorted({0, 31, 320, 331, 332, 333, 351, 640, 699, 700, 701, 702, 703, 704, 767, 1152, 1199, 1200, 1201, 1215, 1699}
                  | set(int(x) for x in rng.integers(0, t, 12)))
    o, b = expect(q, k, v, offsets, d ** -0.5, rows)
    for r in rows:
        seen = ~spoiled[r]
        check(got[r][seen], o[r][seen], b[r][seen], "row %d" % r)


@pytest.mark.parametrize("hq", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences(d, hq):
    rng = np.random.default_rng([42, d])
    lens = [int(x) for x in rng.integers(0, 60, size=110)]
    lens[50] = 400
    offsets = np.concatenate([[0], np.cumsum(lens)])
    t = int(offsets[-1])
    q, k, v = inputs(rng, t, hq, 2, d)
    announce("many short prompts", len(lens), t, d)
    rows = set(int(x) for x in rng.integers(0, t, 150)) | set(int(x) for x in offsets[:-1] if x < t)
    o, b = expect(q, k, v, offsets, d ** -0.5, rows)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    got = call(dev(q), dev(k), dev(v), offsets, d ** -0.5, out)
    assert np.isfinite(got).all()
    compare(got, o, b, "many short prompts")
