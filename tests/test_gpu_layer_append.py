"""qmm_kv_append against the float64 definition: rotated queries, stored rows, untouched slots."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16, DeviceCache, check, dev, empty_cache, held

pytestmark = pytest.mark.gpu

EPS = 1e-6


def case(rng, tokens, hq, hkv, d, bits, group, page, in16, fused, qknorm, rot, inter, far, pad):
    dt = np.float16 if in16 else np.float32
    if fused:
        qkv = rng.standard_normal((tokens, (hq + 2 * hkv) * d + 16)).astype(dt)
        parts = (qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d])
        whole = dev(qkv)
        dparts = (whole[:, :hq * d], whole[:, hq * d:(hq + hkv) * d], whole[:, (hq + hkv) * d:(hq + 2 * hkv) * d])
    else:
        parts = tuple(rng.standard_normal((tokens, h * d)).astype(dt) for h in (hq, hkv, hkv))
        dparts = tuple(dev(p) for p in parts)
    norms = tuple((1 + 0.1 * rng.standard_normal(d)).astype(np.float32) if qknorm else None for _ in range(2))
    inv = (1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32) if rot else None
    positions = rng.integers(0, far + 1, size=tokens).astype(np.int32)
    pages = (tokens + page - 1) // page + 2
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if pad:
        slots[rng.permutation(tokens)[:pad]] = -1
    return parts, dparts, norms, inv, positions, slots, pages


def definition(parts, norms, inv, positions, hq, hkv, d, rot, inter):
    """float64 rows, and how far fp32 may be from them: a norm's 32 roundings or so, a rotation of two products and a
    sum whose sine and cosine are right to 4 steps."""
    q, k, v = (p.astype(np.float64).reshape(len(p), -1, d) for p in parts)
    if norms[0] is not None:
        q, k = layer.rms_norm(q, norms[0], EPS), layer.rms_norm(k, norms[1], EPS)
    rows, errs = [], []
    for x, turned in ((q, True), (k, True), (v, False)):
        y = layer.rotate(x, positions, inv, rot, inter) if turned and rot else x
        size = np.abs(x)
        if turned and rot:
            size = size + layer.rotate(size, np.zeros_like(positions), inv, rot, inter)
            size = np.maximum(size, np.max(np.abs(x), axis=-1, keepdims=True))
        rows.append(y)
        errs.append((0.0 if not turned else 48.0) * E32 * size)
    return rows, errs


def run(cache, dparts, in16, norms, inv, rot, inter, positions, slots, hq, hkv, d, cached, kv_out=True):
    tokens = dparts[0].shape[0]
    outs = [torch.full((tokens, h, d), float("nan"), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    if not kv_out:
        outs[1] = outs[2] = None
    n = [None if x is None else dev(x) for x in norms]
    q, k, v = dparts
    qmm.qmm_kv_append(cache.handle, q, k, v, in16, q.stride(0), k.stride(0), v.stride(0), n[0], n[1], EPS,
                      None if inv is None else dev(inv), rot, inter, dev(positions), None if slots is None else dev(slots),
                      outs[0], outs[1], outs[2], cached, tokens, hq)
    torch.cuda.synchronize()
    return outs


CASES = [
    # tokens hq hkv d bits group page in16 fused qknorm rot inter far pad
    (1, 16, 8, 128, 4, 64, 16, False, False, True, 128, False, 131071, 0),
    (8, 16, 8, 128, 4, 128, 64, True, True, False, 128, False, 100000, 1),
    (33, 32, 8, 64, 4, 32, 16, True, True, False, 64, False, 4000, 5),
    (17, 7, 1, 64, 4, 64, 32, False, False, False, 32, False, 2000, 0),
    (100, 8, 4, 128, 4, 32, 16, False, True, True, 64, True, 131071, 3),
    (21, 4, 2, 128, 8, 64, 64, True, False, True, 128, True, 2 ** 31 - 1, 2),
    (40, 10, 5, 64, 8, 32, 16, False, False, False, 16, False, 10, 0),
    (700, 4, 4, 64, 8, 64, 128, False, True, False, 48, False, 9000, 11),
    (19, 32, 4, 128, 16, 64, 16, False, False, True, 64, True, 30000, 2),
    (600, 3, 1, 64, 16, 64, 64, True, True, False, 0, False, 0, 9),
    (5, 0, 2, 128, 8, 128, 16, True, False, False, 128, False, 50, 0),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(int(x)) for x in c))
@pytest.mark.parametrize("cached", [True, False])
def test_against_float64(c, cached):
    tokens, hq, hkv, d, bits, group, page, in16, fused, qknorm, rot, inter, far, pad = c
    announce("append", c, cached)
    rng = np.random.default_rng([tokens, hq, d, bits])
    parts, dparts, norms, inv, positions, slots, pages = case(rng, *c)
    before = empty_cache(rng, pages, hkv, d, page, bits, group)
    cache = DeviceCache(before, pages, hkv, d, page, bits, group)
    outs = run(cache, dparts, in16, norms, inv, rot, inter, positions, slots, hq, hkv, d, cached)
    after = cache.host()
    (q, k, v), (eq, ek, ev) = definition(parts, norms, inv, positions, hq, hkv, d, rot, inter)
    if hq:
        check(outs[0].cpu().numpy(), q, eq + E16 * np.abs(q) * 1.01 + TINY16, "q_out")
    stored = np.flatnonzero(slots >= 0)
    at, place = slots[stored] // page, slots[stored] % page
    for side, x, e, out in (("k", k, ek, outs[1]), ("v", v, ev, outs[2])):
        out = out.cpu().numpy().astype(np.float64)
        if not cached or bits == 16:
            check(out, x, e + E16 * np.abs(x) * 1.01 + TINY16, side + "_out")
        if bits == 16:
            rows = after[side].view(np.float16)[at, :, place].astype(np.float64)
            assert np.array_equal(rows, out[stored])
        else:
            top = 2.0 ** bits - 1
            codes = layer.unpack_rows(after[side], bits)[at, :, place].reshape(len(stored), hkv, -1, group)
            s = after[side + "s"][at, :, :, place].astype(np.float64)
            m = after[side + "m"][at, :, :, place].astype(np.float64)
            g = x[stored].reshape(codes.shape)
            eg = np.broadcast_to(e, x.shape)[stored].reshape(codes.shape)
            lo, hi, em = g.min(-1), g.max(-1), eg.max(-1)
            check(m, lo, em + E16 * np.abs(lo) * 1.01 + TINY16, side + " mins")
            check(s, (hi - lo) / top, 2 * em / top + E16 * (hi - lo) / top * 1.01 + TINY16, side + " scales")
            # With the scale and min that were stored, every code is the
            # nearest; a value next to the border of two may take either.
            z = (g - m[..., None]) / s[..., None]
            near = eg / s[..., None] + 2.0 ** -20 * (1 + np.abs(z))
            best = np.clip(np.round(z), 0, top)
            border = np.abs(z - np.floor(z) - 0.5) <= near
            assert ((codes == best) | (border & (np.abs(codes - z) <= 0.5 + near))).all(), side + " codes"
            assert border.mean() < 0.01
            values = (codes * s[..., None] + m[..., None]).reshape(len(stored), hkv, d)
            if cached:
                check(out[stored], values, E16 * np.abs(values) * 1.01 + TINY16, side + "_out as held")
        # Slots that were not named keep their bytes.
        free = np.ones((pages, page), dtype=bool)
        free[at, place] = False
        assert np.array_equal(np.swapaxes(after[side], 1, 2)[free], np.swapaxes(before[side], 1, 2)[free])
        if bits != 16:
            for arr in (side + "s", side + "m"):
                assert np.array_equal(np.moveaxis(after[arr], 3, 1)[free], np.moveaxis(before[arr], 3, 1)[free])


def test_padding_out_of_range_slots_and_no_kv_out():
    # Every token is padding or points behind the cache: nothing is stored,
    # queries come out all the same.
    rng = np.random.default_rng(11)
    c = (9, 4, 2, 64, 4, 32, 16, False, False, False, 64, False, 100, 0)
    parts, dparts, norms, inv, positions, slots, pages = case(rng, *c)
    before = empty_cache(rng, pages, 2, 64, 16, 4, 32)
    cache = DeviceCache(before, pages, 2, 64, 16, 4, 32)
    slots[:] = [-1, pages * 16, -2 ** 62, 2 ** 62, pages * 16 + 5, -16, -1, 2 ** 40, -1]
    announce("append, no slot in range")
    outs = run(cache, dparts, False, norms, inv, 64, False, positions, slots, 4, 2, 64, True, kv_out=False)
    after = cache.host()
    for k in before:
        assert np.array_equal(before[k], after[k])
    (q, _, _), (eq, _, _) = definition(parts, norms, inv, positions, 4, 2, 64, 64, False)
    check(outs[0].cpu().numpy(), q, eq + E16 * np.abs(q) * 1.01 + TINY16, "q_out")


def test_without_slots_nothing_is_stored():
    rng = np.random.default_rng(12)
    c = (9, 4, 2, 64, 8, 64, 16, False, False, False, 64, False, 100, 0)
    parts, dparts, norms, inv, positions, _, pages = case(rng, *c)
    cache = DeviceCache({k: None for k in ("k", "ks", "km", "v", "vs", "vm")}, 0, 2, 64, 16, 8, 64)
    outs = run(cache, dparts, False, norms, inv, 64, False, positions, None, 4, 2, 64, False)
    (q, k, v), (eq, ek, ev) = definition(parts, norms, inv, positions, 4, 2, 64, 64, False)
    for o, x, e, w in zip(outs, (q, k, v), (eq, ek, ev), "qkv"):
        check(o.cpu().numpy(), x, e + E16 * np.abs(x) * 1.01 + TINY16, w)


def test_constant_groups_and_non_finite_values():
    # A constant group has scale 0 and codes 0 and reads back as its value; a
    # group with a NaN or an infinity reads back as NaN and spoils no other.
    d, page = 64, 16
    k = np.full((3, d), 1.5, dtype=np.float32)
    v = np.random.default_rng(13).standard_normal((3, d)).astype(np.float32)
    v[1, 40] = np.nan
    v[2, 3] = np.inf
    cache = DeviceCache(empty_cache(np.random.default_rng(1), 1, 1, d, page, 4, 32), 1, 1, d, page, 4, 32)
    announce("append, constant and non-finite groups")
    run(cache, (dev(k), dev(k), dev(v)), False, (None, None), None, 0, False, np.zeros(3, np.int32), np.arange(3), 1, 1, d, True)
    after = cache.host()
    assert (after["ks"][0, 0, :, :3] == 0).all() and (after["k"][0, 0, :3] == 0).all()
    assert (held(after, "k", 4, 32)[0, 0, :3] == 1.5).all()
    got = held(after, "v", 4, 32)[0, 0, :3]
    assert np.isfinite(got[0]).all() and np.isfinite(got[1, :32]).all() and np.isnan(got[1, 32:]).all()
    assert np.isnan(got[2, :32]).all() and np.isfinite(got[2, 32:]).all()


def test_a_cache_beyond_32_bit_offsets():
    # 5 GiB of fp16 keys: the last page lies past 2^32 bytes.
    d, page, hkv = 128, 64, 8
    pages = 5 * 2 ** 30 // (page * hkv * d * 2)
    announce("append past 4 GiB", pages)
    k = torch.zeros((pages, hkv, page, d), dtype=torch.float16, device="cuda")
    v = torch.zeros((pages, hkv, page, d), dtype=torch.float16, device="cuda")
    handle = qmm.KvCache(k, None, None, v, None, None, pages, hkv, d, page, 16, 64)
    rng = np.random.default_rng(14)
    src = [dev(rng.standard_normal((2, hkv * d)).astype(np.float16)) for _ in range(3)]
    slots = torch.tensor([pages * page - 1, (pages - 1) * page], device="cuda")
    q_out = torch.empty((2, hkv, d), dtype=torch.float16, device="cuda")
    qmm.qmm_kv_append(handle, *src, True, hkv * d, hkv * d, hkv * d, None, None, EPS, None, 0, False, None, slots, q_out, None, None,
                      False, 2, hkv)
    torch.cuda.synchronize()
    assert torch.equal(k[-1, :, -1], src[1].view(2, hkv, d)[0]) and torch.equal(v[-1, :, 0], src[2].view(2, hkv, d)[1])
    # Attention over those rows reads them back.
    q = dev(rng.standard_normal((1, hkv, d)).astype(np.float16))
    out = torch.empty_like(q)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1], dtype=torch.int32, device="cuda")
    qmm.qmm_attn_cache(handle, q, table, 1, lens, 64, out, 1, 1, hkv, d ** -0.5)
    torch.cuda.synchronize()
    assert torch.equal(out[0], src[2].view(2, hkv, d)[1])


def test_graph_replays():
    rng = np.random.default_rng(15)
    c = (12, 8, 4, 128, 4, 64, 16, False, False, True, 128, False, 4000, 1)
    parts, dparts, norms, inv, positions, slots, pages = case(rng, *c)
    before = empty_cache(rng, pages, 4, 128, 16, 4, 64)
    cache = DeviceCache(before, pages, 4, 128, 16, 4, 64)
    outs = run(cache, dparts, False, norms, inv, 128, False, positions, slots, 8, 4, 128, True)
    want = {k: t.clone() for k, t in cache.t.items()}
    q0 = outs[0].clone()
    q, k, v = dparts
    args = (dev(norms[0]), dev(norms[1]), EPS, dev(inv), 128, False, dev(positions), dev(slots))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_kv_append(cache.handle, q, k, v, False, q.stride(0), k.stride(0), v.stride(0), *args, outs[0], outs[1], outs[2],
                          True, 12, 8)
    for _ in range(3):
        for name, t in cache.t.items():
            t.copy_(dev(before[name]))
        outs[0].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], q0)
        for name, t in cache.t.items():
            assert torch.equal(t, want[name])
