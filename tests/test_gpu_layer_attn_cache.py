"""qmm_attn_cache against the float64 definition."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import DeviceCache, attention_bound, check, dev, empty_cache, held

pytestmark = pytest.mark.gpu


def setup(rng, lens, page, hkv, d, bits, group, spoil=False):
    """A cache whose pages are handed out at random, the table and the host arrays.  `spoil`: whatever lies behind a
    sequence's rows is NaN (scales, mins, fp16 values) or garbage (codes)."""
    width = max(1, -(-max(lens) // page))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = rng.permutation(pages)
    host = empty_cache(rng, pages, hkv, d, page, bits, group)
    bad = empty_cache(rng, pages, hkv, d, page, bits, group, garbage=True)
    table = np.full((len(lens), width + 1), -7, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    if spoil:
        keep = np.zeros((pages, page), dtype=bool)
        for i, n in enumerate(lens):
            for t in range(n):
                keep[table[i, t // page], t % page] = True
        for side in "kv":
            if bits == 16:
                a = host[side].view(np.float16)
                np.swapaxes(a, 1, 2)[~keep] = np.nan
            else:
                for arr in (side + "s", side + "m"):
                    np.moveaxis(host[arr], 3, 1)[~keep] = np.moveaxis(bad[arr], 3, 1)[~keep]
    return host, table, pages


def expect(host, table, lens, q, q_len, hq, hkv, d, bits, group, scale):
    k, v = held(host, "k", bits, group), held(host, "v", bits, group)
    n = len(lens)
    o, bound = np.zeros((n * q_len, hq, d)), np.zeros((n * q_len, hq, d))
    for i, length in enumerate(lens):
        ks, vs = layer.sequence_rows(k, table[i], length), layer.sequence_rows(v, table[i], length)
        limits = [length - q_len + 1 + j for j in range(q_len)]
        rows = slice(i * q_len, (i + 1) * q_len)
        for h in range(hq):
            j = h // (hq // hkv)
            vj = np.nan_to_num(vs[:, j]) if length else vs[:, j]
            r = layer.attend(q[rows, h], ks[:, j], vj, limits, scale)
            o[rows, h] = r[0]
            vmax = np.abs(vj).max() if length else 0.0
            bound[rows, h] = attention_bound(*r, length, vmax, d, bits != 16, bits == 16)
    return o, bound


def scratch(size):
    """A workspace: counters zero, the rest anything."""
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:qmm.QMM_ATTN_COUNTER_BYTES] = 0
    return ws


def run(cache, q, table, lens, max_len, q_len, hq, scale, workspace="full"):
    n = len(lens)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    need = qmm.qmm_attn_cache_workspace_bytes(cache.handle, n, q_len, hq, max_len)
    size = {"full": need, "none": 0, "half": need // 2}[workspace]
    ws = scratch(size) if size else None
    qd, td, ld = dev(q), dev(table), dev(np.asarray(lens, dtype=np.int32))
    qmm.qmm_attn_cache(cache.handle, qd, td, table.shape[1], ld, max_len, out, n, q_len, hq, scale, ws, size)
    torch.cuda.synchronize()
    if ws is not None:
        assert not ws[:qmm.QMM_ATTN_COUNTER_BYTES].any()
    return out.cpu().numpy()


CASES = [
    # lens, q_len, hq, hkv, d, bits, group, page
    ([1], 1, 8, 8, 128, 4, 64, 16),
    ([0, 1, 2, 31, 32, 33], 1, 16, 8, 128, 4, 64, 16),
    ([700, 5, 0, 129], 1, 32, 8, 64, 4, 32, 32),
    ([1500], 1, 16, 8, 128, 4, 64, 64),
    ([63, 64, 65, 127, 128, 129, 200], 1, 10, 5, 64, 4, 64, 64),
    ([300, 17], 1, 7, 1, 128, 4, 128, 128),
    ([300, 17], 1, 8, 2, 128, 4, 32, 16),
    ([400, 1, 260], 1, 16, 2, 128, 8, 64, 32),
    ([90, 512], 1, 4, 4, 64, 8, 32, 16),
    ([513, 30], 1, 8, 1, 64, 8, 64, 64),
    ([200], 1, 8, 4, 128, 8, 32, 64),
    ([333, 0, 4], 1, 32, 4, 128, 8, 128, 64),
    ([333, 2, 96], 1, 16, 4, 128, 16, 64, 16),
    ([100, 1000], 1, 9, 3, 64, 16, 64, 256),
    ([40, 3, 0, 1], 4, 8, 2, 128, 4, 64, 16),       # fewer rows than drafts: the first see nothing
    ([513, 7], 5, 32, 4, 64, 8, 32, 16),             # 40 query rows: three row tiles
    ([200, 18], 17, 4, 4, 64, 16, 64, 32),
    ([70], 1, 40, 2, 128, 4, 64, 16),                # 20 heads to a key head: two row tiles
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join([str(len(c[0])), str(max(c[0]))] + [str(x) for x in c[1:]]))
@pytest.mark.parametrize("spoil", [False, True])
def test_against_float64(c, spoil):
    lens, q_len, hq, hkv, d, bits, group, page = c
    announce("cache attention", c, spoil)
    rng = np.random.default_rng([len(lens), max(lens), q_len, hq, d, bits])
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group, spoil)
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((len(lens) * q_len, hq, d)).astype(np.float16)
    o, bound = expect(host, table, lens, q, q_len, hq, hkv, d, bits, group, d ** -0.5)
    got = run(cache, q, table, lens, max(max(lens), 1), q_len, hq, d ** -0.5)
    check(got, o, bound, "cache attention %s" % (c,))
    for i, n in enumerate(lens):
        for j in range(q_len):
            if n - q_len + 1 + j <= 0:
                assert (got[i * q_len + j] == 0).all()


@pytest.mark.parametrize("workspace", ["full", "half", "none"])
@pytest.mark.parametrize("bits", [4, 16])
def test_splits_with_more_and_less_workspace(workspace, bits):
    # Long enough to be split; a larger max_kv_len than any sequence has.
    rng = np.random.default_rng([21, bits])
    lens, hq, hkv, d, group, page = [2900, 5, 1111], 8, 2, 128, 64, 64
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group, True)
    table = np.concatenate([table, np.full((3, 40), -1, np.int32)], axis=1)
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("splits", workspace, bits)
    o, bound = expect(host, table, lens, q, 1, hq, hkv, d, bits, group, 0.2)
    got = run(cache, q, table, lens, 5000, 1, hq, 0.2, workspace)
    check(got, o, bound, "splits, %s workspace" % workspace)


def test_large_scores_shifted_keys_and_equal_keys():
    # Scores of some hundreds (one row takes all the weight), keys far from
    # zero (their mean cancels in the softmax), and equal keys (plain mean).
    rng = np.random.default_rng(22)
    lens, hq, hkv, d, bits, group, page = [400, 400, 400], 4, 2, 128, 4, 64, 16
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
    own = [table[i, :25] for i in range(3)]
    host["km"][own[1]] += np.float16(30)
    host["ks"][own[2]] = 0
    host["km"][own[2]] = 1
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("large scores")
    for scale in (4.0, d ** -0.5, 0.0, -0.3):
        o, bound = expect(host, table, lens, q, 1, hq, hkv, d, bits, group, scale)
        check(run(cache, q, table, lens, 400, 1, hq, scale), o, bound, "scale %g" % scale)


def test_tiny_and_large_values():
    # Values of 1e-4 and of 1e3: outputs follow, relative to their own size.
    rng = np.random.default_rng(23)
    lens, hq, hkv, d, page = [150, 150], 4, 2, 64, 16
    for bits, group in ((4, 32), (8, 64)):
        host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
        for i, f in ((0, 1e-2), (1, 2e2)):
            p = table[i, :10]
            host["vs"][p] = (host["vs"][p].astype(np.float64) * f).astype(np.float16)
            host["vm"][p] = (host["vm"][p].astype(np.float64) * f).astype(np.float16)
        cache = DeviceCache(host, pages, hkv, d, page, bits, group)
        q = rng.standard_normal((2, hq, d)).astype(np.float16)
        announce("tiny and large values", bits)
        o, bound = expect(host, table, lens, q, 1, hq, hkv, d, bits, group, d ** -0.5)
        check(run(cache, q, table, lens, 150, 1, hq, d ** -0.5), o, bound, "values, %d bits" % bits)


@pytest.mark.parametrize("bits", [4, 16])
def test_non_finite_drafts_reach_only_the_rows_that_see_them(bits):
    rng = np.random.default_rng([24, bits])
    lens, q_len, hq, hkv, d, group, page = [50], 3, 4, 2, 64, 32, 16
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
    t = 48  # seen by drafts 1 and 2, not by 0
    p = table[0, t // page]
    if bits == 16:
        host["v"].view(np.float16)[p, :, t % page, 5] = np.inf
    else:
        host["vm"][p, :, 0, t % page] = np.inf
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("non-finite drafts", bits)
    got = run(cache, q, table, lens, 50, q_len, hq, 0.125)
    o, bound = expect(host, table, [50], q, q_len, hq, hkv, d, bits, group, 0.125)
    check(got[0], o[0], bound[0], "the draft that does not see it")
    assert not np.isfinite(got[1:, :, :32]).all(-1).any()


def test_page_entries_out_of_range_give_nan_and_read_nothing():
    rng = np.random.default_rng(25)
    lens, hq, hkv, d, bits, group, page = [40, 40, 40], 4, 2, 64, 4, 32, 16
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
    table[0, 1] = pages
    table[2, 2] = -1
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("bad pages")
    got = run(cache, q, table, lens, 40, 1, hq, 0.125)
    assert np.isnan(got[0]).all() and np.isnan(got[2]).all()
    o, bound = expect(host, table[1:2], [40], q[1:2], 1, hq, hkv, d, bits, group, 0.125)
    check(got[1:2], o, bound, "the sequence between")


def test_lengths_outside_the_range_are_clamped():
    rng = np.random.default_rng(26)
    lens, hq, hkv, d, bits, group, page = [48, 48], 4, 2, 64, 4, 32, 16
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group)
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((2, hq, d)).astype(np.float16)
    announce("clamped lengths")
    got = run(cache, q, table, [-5, 1000], 48, 1, hq, 0.125)
    assert (got[0] == 0).all()
    o, bound = expect(host, table[1:], [48], q[1:], 1, hq, hkv, d, bits, group, 0.125)
    check(got[1:], o, bound, "clamped to max_kv_len")


def test_nothing_to_see():
    rng = np.random.default_rng(27)
    host, table, pages = setup(rng, [16], 16, 2, 64, 4, 32)
    cache = DeviceCache(host, pages, 2, 64, 16, 4, 32)
    q = rng.standard_normal((3, 4, 64)).astype(np.float16)
    announce("all empty")
    got = run(cache, q, np.zeros((3, 1), np.int32), [0, 0, 0], 0, 1, 4, 0.125)
    assert (got == 0).all()


def test_same_bits_every_time_graphs_and_streams():
    # Two graphs and a stream of their own share inputs; each has a workspace.
    rng = np.random.default_rng(28)
    lens, hq, hkv, d, bits, group, page = [3000, 40, 1777], 8, 4, 128, 4, 64, 64
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group, True)
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((3, hq, d)).astype(np.float16)
    announce("replays")
    want = run(cache, q, table, lens, 3000, 1, hq, 0.1)
    need = qmm.qmm_attn_cache_workspace_bytes(cache.handle, 3, 1, hq, 3000)
    assert need > 0
    qd, td, ld = dev(q), dev(table), dev(np.asarray(lens, dtype=np.int32))

    def call(out, ws, stream=None):
        qmm.qmm_attn_cache(cache.handle, qd, td, table.shape[1], ld, 3000, out, 3, 1, hq, 0.1, ws, need, stream=stream)
    outs = [torch.empty((3, hq, d), dtype=torch.float16, device="cuda") for _ in range(2)]
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o, ws)  # graphs that run one after the other may share a workspace
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(4):
        for o in outs:
            o.zero_()
        ws[qmm.QMM_ATTN_COUNTER_BYTES:] = 0xFF
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        other, ws2 = torch.zeros_like(outs[0]), torch.zeros_like(ws)
        side.wait_stream(torch.cuda.current_stream())
        call(other, ws2, side)
        torch.cuda.synchronize()
        for o in outs + [other]:
            assert np.array_equal(o.cpu().numpy(), want)
