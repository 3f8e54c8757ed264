"""qmm_moe_route against the definition in 64 bits: experts and rows have to be equal, weights within their roundings."""
import math

import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import E32, dev

pytestmark = pytest.mark.gpu

UNTOUCHED = -77


def weight_bound(logits, ids, weights, kind, per_lane):
    """A weight is exp(l - top) over a sum of such, or 1 / (1 + exp(-l)) over a sum: the difference is rounded once
    (|l - top| E32 in the exponential), the exponential itself is good to 4 E32, a sum of n terms adds at most one rounding
    for each of a lane's terms and six over the lanes, the quotient and the scale one each.  What the sum's terms lose to
    the difference is at most E32 times the sum of p |l - top|, the entropy, below ln n.  Below fp32's normal range the
    step is 2^-149."""
    l = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    t = np.take_along_axis(l, np.maximum(ids, 0), 1)
    if kind == "softmax":
        top = l.max(1, keepdims=True)
        far = np.where(np.isfinite(top) & np.isfinite(t), np.where(np.isfinite(top), top, 0) - np.where(np.isfinite(t), t, 0), 0)
    else:
        far = np.where(np.isfinite(t), np.abs(t), 0)
    n = l.shape[1]
    return np.abs(weights) * E32 * (far + far.max(1, keepdims=True) + math.log(n) + 2 * 8 + per_lane + 6 + 4) + 2.0 ** -140


def call(logits, bias=None, kind="softmax", groups=1, top_groups=1, best=1, top_k=2, renorm=True, scale=1.0, keep=None,
         group=True, stream=None, pad_stride=0):
    tokens, experts = logits.shape
    wide = torch.full((tokens, experts + pad_stride), 1000.0, dtype=logits.dtype, device="cuda")
    wide[:, :experts] = logits
    out = {"ids": torch.full((tokens, top_k), UNTOUCHED, dtype=torch.int32, device="cuda"),
           "weights": torch.full((tokens, top_k), float(UNTOUCHED), device="cuda"),
           "pair_row": torch.full((tokens, top_k), UNTOUCHED, dtype=torch.int32, device="cuda"),
           "offsets": torch.full((experts + 1,), UNTOUCHED, dtype=torch.int32, device="cuda"),
           "pair_token": torch.full((tokens * top_k,), UNTOUCHED, dtype=torch.int32, device="cuda"),
           "pair_weight": torch.full((tokens * top_k,), float(UNTOUCHED), device="cuda")}
    need = qmm.qmm_moe_route_workspace_bytes(tokens, experts, top_k)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")  # it may hold anything
    qmm.qmm_moe_route(wide, wide.dtype == torch.float16, wide.stride(0), bias, kind == "sigmoid", groups, top_groups, best, top_k, renorm,
                      scale, keep, out["ids"], out["weights"], out["pair_row"], out["offsets"] if group else None, out["pair_token"],
                      out["pair_weight"], ws, need, tokens, experts, stream=stream)
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    return out


def verify(logits, out, bias=None, kind="softmax", groups=1, top_groups=1, best=1, top_k=2, renorm=True, scale=1.0, keep=None, group=True):
    l = logits.float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    k = None if keep is None else keep.cpu().numpy()
    ids, weights, pair_row, offsets, token, weight = moe.route(l, kind, b, groups, top_groups, best, top_k, renorm, scale, k)
    got = {n: t.cpu().numpy() for n, t in out.items()}
    assert np.array_equal(got["ids"], ids)
    bound = weight_bound(l, ids, weights, kind, 16)
    assert np.array_equal(np.isnan(got["weights"]), np.isnan(weights))
    ok = ~np.isnan(weights)
    err = np.abs(got["weights"].astype(np.float64) - weights)
    assert (err[ok] <= bound[ok]).all(), (err[ok] / np.maximum(bound[ok], 1e-300)).max()
    if not group:
        for n in ("pair_row", "offsets", "pair_token", "pair_weight"):
            assert (got[n] == UNTOUCHED).all()
        return
    rows = offsets[-1]
    assert np.array_equal(got["offsets"], offsets)
    assert np.array_equal(got["pair_row"], pair_row)
    assert np.array_equal(got["pair_token"][:rows], token) and (got["pair_token"][rows:] == UNTOUCHED).all()
    # The same numbers as in `weights`, bit for bit.
    at = pair_row[pair_row >= 0]
    assert np.array_equal(got["pair_weight"][at].view(np.int32), got["weights"][pair_row >= 0].view(np.int32))
    assert (got["pair_weight"][rows:] == UNTOUCHED).all()


def run(logits, what, **kw):
    announce("route", what, tuple(logits.shape), {k: v for k, v in kw.items() if not torch.is_tensor(v)})
    extra = {k: kw.pop(k) for k in ("pad_stride",) if k in kw}
    verify(logits, call(logits, **kw, **extra), **kw)


def normal(rng, *shape, dtype=torch.float32):
    return dev(rng.standard_normal(shape).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("tokens", [1, 2, 15, 17, 63, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("experts,top_k", [(8, 2), (60, 4), (128, 8), (256, 8)])
def test_sizes(tokens, experts, top_k):
    rng = np.random.default_rng(tokens * 1000 + experts)
    run(normal(rng, tokens, experts), "sizes", top_k=top_k)


@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 1), (3, 3), (16, 16), (17, 17), (31, 5), (64, 64), (65, 2), (129, 12), (255, 33),
                                           (257, 10), (384, 8), (512, 10), (513, 3), (1000, 22), (1024, 64)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_experts(experts, top_k, kind):
    rng = np.random.default_rng(experts)
    for tokens in (5, 70):
        run(normal(rng, tokens, experts), "experts", top_k=top_k, kind=kind, renorm=False, scale=2.5)
        run(normal(rng, tokens, experts), "experts, bias", top_k=top_k, kind=kind, bias=0.2 * normal(rng, experts))


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(256, 8, 4, 8), (64, 4, 1, 4), (60, 15, 3, 12), (160, 8, 3, 6), (96, 32, 5, 8),
                                                             (128, 64, 64, 8), (12, 6, 2, 4), (512, 16, 4, 10), (1024, 8, 8, 9), (77, 7, 2, 20)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(experts, groups, top_groups, top_k, best, kind, biased):
    rng = np.random.default_rng(experts + groups)
    run(normal(rng, 67, experts), "groups", groups=groups, top_groups=top_groups, best=best, top_k=top_k, kind=kind,
        bias=0.3 * normal(rng, experts) if biased else None)


@pytest.mark.parametrize("experts,stride", [(128, 0), (128, 4), (128, 3), (60, 1), (61, 0), (256, 8), (384, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_rows_apart_and_types(experts, stride, dtype):
    rng = np.random.default_rng(experts + stride)
    run(normal(rng, 66, experts, dtype=dtype), "strides", top_k=6, pad_stride=stride, renorm=False)
    run(normal(rng, 66, experts, dtype=dtype), "strides", top_k=6, pad_stride=stride, kind="sigmoid", bias=normal(rng, experts))


@pytest.mark.parametrize("tokens", [3, 64, 200])
@pytest.mark.parametrize("biased", [False, True])
def test_padding(tokens, biased):
    rng = np.random.default_rng(tokens)
    for keep in (rng.random(tokens) < 0.6, np.zeros(tokens), np.arange(tokens) < tokens - 2):
        run(normal(rng, tokens, 40), "padding", top_k=5, keep=dev(np.asarray(keep, dtype=np.uint8)),
            bias=normal(rng, 40) if biased else None)


@pytest.mark.parametrize("experts", [60, 128, 300])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_equal_scores_go_to_the_lower_index(experts, groups, kind):
    rng = np.random.default_rng(experts)
    l = dev(rng.integers(-2, 2, (70, experts)).astype(np.float32))
    l[3] = 0.0
    l[4, ::2] = -0.0  # equal to 0
    l[4, 1::2] = 0.0
    for best in (1, 2):
        run(l, "ties", top_k=8, groups=groups, top_groups=max(1, groups // 2), kind=kind, best=best)
        run(l, "ties, bias", top_k=8, groups=groups, top_groups=max(1, groups // 2), kind=kind, best=best,
            bias=dev(np.zeros(experts, dtype=np.float32)))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_scores_next_to_each_other(kind):
    # Neighbouring fp32 logits, and, with a bias, sums that 32 bits cannot tell apart.
    rng = np.random.default_rng(5)
    base = rng.standard_normal((40, 1)).astype(np.float32) * 3
    steps = rng.integers(-6, 7, (40, 128)).astype(np.float32)
    l = (base + steps * np.spacing(np.abs(base))).astype(np.float32)
    run(dev(l), "neighbours", top_k=8, kind=kind)
    run(dev(l), "neighbours, bias", top_k=8, kind=kind, bias=dev(np.full(128, 0.5, dtype=np.float32)))
    far = dev((rng.standard_normal((40, 128)) * 3 + 40).astype(np.float32))  # sigmoid is 1 in fp32
    run(far, "saturated", top_k=8, kind=kind)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_infinite_and_nan_scores(renorm, kind, groups, biased):
    rng = np.random.default_rng(8)
    l = rng.standard_normal((24, 32)).astype(np.float32)
    l[0] = -np.inf
    l[1, 5:] = -np.inf
    l[2, :] = -np.inf
    l[2, 17] = 0.5
    l[3] = np.finfo(np.float32).min
    l[4, 7] = np.finfo(np.float32).max
    l[5, 9] = np.inf
    l[6, [3, 20]] = np.inf
    l[7, 11] = np.nan
    l[8] = np.nan
    l[9, ::2] = np.nan
    l[10] = -200 - 5 * np.arange(32)  # scores below fp32, for sigmoid
    l[11] = 200 + 5 * np.arange(32)
    bias = None
    if biased:
        bias = 0.1 * rng.standard_normal(32).astype(np.float32)
        bias[[2, 30]] = [np.nan, -np.inf]
        bias = dev(bias)
    for best in (1, 2):
        run(dev(l), "masked", top_k=6, kind=kind, groups=groups, top_groups=max(1, groups // 2), best=best, renorm=renorm, bias=bias)


def test_without_groups_and_without_tokens():
    rng = np.random.default_rng(2)
    run(normal(rng, 100, 64), "not grouped", top_k=4, group=False)
    run(normal(rng, 9, 64), "not grouped", top_k=4, group=False)
    announce("route without tokens")
    out = call(normal(rng, 0, 64), top_k=4)
    assert (out["offsets"] == 0).all()
    out = call(normal(rng, 0, 300), top_k=4)
    assert (out["offsets"] == 0).all()
    out = call(normal(rng, 0, 64), top_k=4, group=False)
    assert (out["offsets"] == UNTOUCHED).all()


@pytest.mark.parametrize("tokens", [16, 17, 48, 49, 64, 255, 256, 257, 2047, 2049])
@pytest.mark.parametrize("experts,grouped", [(64, False), (128, False), (256, True)])
def test_where_the_launch_changes(tokens, experts, grouped):
    rng = np.random.default_rng(7 * tokens + experts)
    how = dict(kind="sigmoid", groups=8, top_groups=4, best=2, bias=0.1 * normal(rng, experts)) if grouped else {}
    run(normal(rng, tokens, experts), "launches", top_k=8, **how)


@pytest.mark.parametrize("tokens", [1023, 1025, 4097, 8193])
@pytest.mark.parametrize("how", ["best", "groups", "pairs", "biased"])
def test_long_batches_of_256_experts(tokens, how):
    rng = np.random.default_rng(tokens)
    more = {"best": {}, "groups": dict(groups=8, top_groups=3), "pairs": dict(groups=16, top_groups=4, best=2),
            "biased": dict(kind="sigmoid", bias=0.1 * normal(rng, 250))}[how]
    run(normal(rng, tokens, 250 if how in ("best", "biased") else 256), how, top_k=6, keep=dev(np.asarray(rng.random(tokens) < 0.9, dtype=np.uint8)), **more)


@pytest.mark.parametrize("tokens,experts", [(5000, 128), (4096, 100), (4097, 384), (9001, 8), (16384, 40), (16385, 129), (70001, 20), (262145, 16)])
def test_many_tokens(tokens, experts):
    # Against the oracle for a sample's choices, and the grouping whole.
    rng = np.random.default_rng(tokens)
    logits = normal(rng, tokens, experts)
    announce("route many", tokens, experts)
    out = call(logits, top_k=4)
    got = {n: t.cpu().numpy() for n, t in out.items()}
    l = logits.cpu().numpy()
    want = np.argsort(-l, axis=1, kind="stable")[:, :4]
    assert np.array_equal(got["ids"], want)
    flat = want.ravel()
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(got["offsets"], np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=experts))]))
    assert np.array_equal(got["pair_token"], order // 4)
    back = np.empty_like(order)
    back[order] = np.arange(order.size)
    assert np.array_equal(got["pair_row"].ravel(), back)
    assert np.array_equal(got["pair_weight"], got["weights"].ravel()[order])


def test_one_expert_takes_all():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((333, 16)).astype(np.float32)
    l[:, 11] += 50
    run(dev(l), "popular", top_k=1)
    run(dev(l), "popular", top_k=2)
