"""qmm_attn_cache at the ends of its ranges, against the float64 definition: many sequences, long runs of one work-group,
one page for everything, many drafts, graphs that share a workspace."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce
from tests.layer_util import DeviceCache, check, dev
from tests.test_gpu_layer_attn_cache import expect, run, scratch, setup

pytestmark = pytest.mark.gpu


def compare(seed, lens, q_len, hq, hkv, d, bits, group, page, workspace="full", max_len=None):
    announce("cache attention", len(lens), max(lens), q_len, hq, hkv, d, bits, group, page, workspace)
    rng = np.random.default_rng(seed)
    host, table, pages = setup(rng, lens, page, hkv, d, bits, group, True)
    cache = DeviceCache(host, pages, hkv, d, page, bits, group)
    q = rng.standard_normal((len(lens) * q_len, hq, d)).astype(np.float16)
    o, bound = expect(host, table, lens, q, q_len, hq, hkv, d, bits, group, d ** -0.5)
    got = run(cache, q, table, lens, max_len or max(lens), q_len, hq, d ** -0.5, workspace)
    check(got, o, bound, "cache attention of %d sequences" % len(lens))
    return got


@pytest.mark.parametrize("n", [63, 64, 65, 300])
def test_many_sequences_share_the_device(n):
    # From 65 on the lengths no longer fit one wave's lanes.  Every fifth sequence is empty, the last ones too.
    rng = np.random.default_rng([61, n])
    lens = [0 if i % 5 == 0 or i > n - 3 else int(rng.integers(1, 500)) for i in range(n)]
    got = compare([62, n], lens, 1, 4, 2, 64, 4, 32, 16)
    for i, length in enumerate(lens):
        if length == 0:
            assert (got[i] == 0).all()


@pytest.mark.parametrize("d,bits,group", [(64, 8, 64), (128, 16, 64)])
def test_more_units_than_shares(d, bits, group):
    # Every unit is one run of one work-group.
    rng = np.random.default_rng([63, d])
    lens = [int(x) for x in rng.integers(0, 40, size=1100)]
    lens[7] = 300
    compare([64, d], lens, 1, 8, 8, d, bits, group, 16)


@pytest.mark.parametrize("workspace", ["none", "full"])
@pytest.mark.parametrize("d,bits,group", [(128, 4, 64), (128, 8, 32), (128, 16, 64), (64, 4, 32), (64, 8, 64)])
def test_long_runs(d, bits, group, workspace):
    # Without a workspace one work-group goes over all of a sequence: more steps than table entries held at a time, with
    # lengths on both sides of where they are read again (4096 rows).
    compare([65, d, bits], [9003, 4096, 4097, 4095], 1, 4, 2, d, bits, group, 64, workspace)


def test_one_page_for_everything():
    compare([66], [5000], 1, 4, 1, 64, 4, 64, 65536)


def test_as_many_drafts_as_there_can_be():
    compare([67], [400, 100, 256], 256, 4, 2, 64, 4, 32, 32)


def test_two_graphs_and_eager_calls_share_a_workspace():
    announce("cache attention, one workspace")
    rng = np.random.default_rng(68)
    jobs = []
    for lens, hq, hkv, d, bits, group in (([3000, 40, 0], 8, 2, 128, 4, 64), ([700, 1900], 16, 4, 64, 8, 32)):
        host, table, pages = setup(rng, lens, 16, hkv, d, bits, group)
        cache = DeviceCache(host, pages, hkv, d, 16, bits, group)
        q = dev(rng.standard_normal((len(lens), hq, d)).astype(np.float16))
        need = qmm.qmm_attn_cache_workspace_bytes(cache.handle, len(lens), 1, hq, max(lens))
        jobs.append((cache, q, dev(table), dev(np.asarray(lens, np.int32)), max(lens), hq, torch.empty_like(q), need))
    ws = scratch(max(j[-1] for j in jobs))

    def call(job):
        cache, q, table, lens, most, hq, out, _ = job
        qmm.qmm_attn_cache(cache.handle, q, table, table.stride(0), lens, most, out, q.shape[0], 1, hq, 0.1, ws, ws.numel())

    want = []
    for job in jobs:
        call(job)
        torch.cuda.synchronize()
        want.append(job[6].clone())
    graphs = []
    for job in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(job)
            call(job)
        graphs.append(g)
    for turn in range(6):
        for job in jobs:
            job[6].zero_()
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        if turn % 3 == 0:
            call(jobs[turn % 2])
        torch.cuda.synchronize()
        for job, w in zip(jobs, want):
            assert torch.equal(job[6], w)
    assert not ws[:qmm.QMM_ATTN_COUNTER_BYTES].any()
