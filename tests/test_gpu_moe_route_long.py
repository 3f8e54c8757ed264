"""qmm_moe_route for long batches, where sixteen lanes share a token and four tokens a wave: every kind of choice, against the
definition in 64 bits for all tokens at once, and that against the oracle's loops."""
import numpy as np
import pytest
import torch

from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import dev
from tests.test_gpu_moe_route import UNTOUCHED, call, weight_bound

pytestmark = pytest.mark.gpu


def definition(l, kind, bias, groups, top_groups, best, top_k, renorm, scale, keep):
    """(ids, weights) of finite logits [tokens][experts], in float64; stable sorts, so equals stay in the order of their indices."""
    tokens, experts = l.shape
    l = l.astype(np.float64)
    if kind == "sigmoid":
        e = np.exp(-np.abs(l))
        s = np.where(l >= 0, 1 / (1 + e), e / (1 + e))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    c = s if bias is None else s + bias.astype(np.float64)
    rank = l if bias is None else c
    if groups > 1:
        mark = rank.reshape(tokens, groups, -1).max(2) if best == 1 else np.sort(c.reshape(tokens, groups, -1), 2)[:, :, -2:].sum(2)
        stay = np.zeros((tokens, groups), dtype=bool)
        np.put_along_axis(stay, np.argsort(-mark, 1, kind="stable")[:, :top_groups], True, 1)
        rank = np.where(np.repeat(stay, experts // groups, 1), rank, -np.inf)
    ids = np.argsort(-rank, 1, kind="stable")[:, :top_k]
    w = np.take_along_axis(s, ids, 1)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    w = w * scale
    if keep is not None:
        ids, w = np.where(keep[:, None] != 0, ids, -1), np.where(keep[:, None] != 0, w, 0)
    return ids, w


def run(logits, top_k, kind="softmax", bias=None, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, keep=None, pad_stride=0):
    how = dict(kind=kind, bias=bias, groups=groups, top_groups=top_groups, best=best, top_k=top_k, renorm=renorm, scale=scale, keep=keep)
    announce("route long", tuple(logits.shape), {k: v for k, v in how.items() if not torch.is_tensor(v)})
    out = {n: t.cpu().numpy() for n, t in call(logits, **how, pad_stride=pad_stride).items()}
    l, b, k = (None if t is None else t.float().cpu().numpy() for t in (logits, bias, keep))
    ids, weights = definition(l, kind, b, groups, top_groups, best, top_k, renorm, scale, k)
    few = moe.route(l[:40], kind, b, groups, top_groups, best, top_k, renorm, scale, None if k is None else k[:40])
    assert np.array_equal(ids[:40], few[0]) and np.allclose(weights[:40], few[1], rtol=1e-13, atol=0)
    assert np.array_equal(out["ids"], ids)
    bound = weight_bound(l, ids, weights, kind, 16)
    err = np.abs(out["weights"] - weights)
    assert (err <= bound).all(), (err / bound).max()
    # The grouping: pairs sorted by expert, within an expert by token.
    flat = np.where(ids < 0, l.shape[1], ids).ravel()
    order = np.argsort(flat, kind="stable")
    rows = int((ids >= 0).sum())
    back = np.full(flat.size, -1)
    back[order[:rows]] = np.arange(rows)
    assert np.array_equal(out["offsets"], np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=l.shape[1] + 1)[:-1])]))
    assert np.array_equal(out["pair_row"].ravel(), back)
    assert np.array_equal(out["pair_token"][:rows], order[:rows] // top_k) and (out["pair_token"][rows:] == UNTOUCHED).all()
    assert np.array_equal(out["pair_weight"][:rows], out["weights"].ravel()[order[:rows]]) and (out["pair_weight"][rows:] == UNTOUCHED).all()


def mixed(rng, tokens, experts, sums=False):
    """Normal logits, and among them tokens of equal and of neighbouring ones, which leave the choice open in fp32.  (Sums of
    two: near ones, as those of neighbours may be equal but for the last bit of 64.)"""
    l = rng.standard_normal((tokens, experts)).astype(np.float32)
    kinds = rng.integers(0, 8, tokens)
    l[kinds == 0] = rng.integers(-2, 2, ((kinds == 0).sum(), experts))
    base = 2 * rng.standard_normal(((kinds == 1).sum(), 1)).astype(np.float32)
    if sums:
        l[kinds == 1] = base + (1e-5 * rng.standard_normal((len(base), experts))).astype(np.float32)
    else:
        l[kinds == 1] = base + rng.integers(-6, 7, (len(base), experts)).astype(np.float32) * np.spacing(np.abs(base))
    return l


HOW = {
    "logits": dict(),
    "logits in groups": dict(groups=4, top_groups=2),
    "pairs": dict(groups=4, top_groups=2, best=2),
    "biased": dict(bias=0.1),
    "biased in groups": dict(bias=0.3, groups=4, top_groups=2),
    "biased pairs": dict(bias=0.3, groups=4, top_groups=2, best=2),
    "no bias but zeros": dict(bias=0.0),
}


@pytest.mark.parametrize("experts", [8, 40, 60, 64, 100, 128])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_choices(experts, how, kind):
    rng = np.random.default_rng(experts + len(how))
    more = dict(HOW[how])
    if "bias" in more:
        more["bias"] = dev((more["bias"] * rng.standard_normal(experts)).astype(np.float32))
    tokens = 4097 + int(rng.integers(0, 1000))
    keep = dev((rng.random(tokens) < 0.9).astype(np.uint8)) if experts % 8 == 4 else None
    run(dev(mixed(rng, tokens, experts, how == "pairs")), 4, kind=kind, keep=keep, renorm=experts != 64, scale=2.5 if experts == 64 else 1.0,
        pad_stride=3 if experts == 100 else 0, **more)


# Groups that are a part of a lane's experts, one lane's, those of 2, 4 and 8 lanes, and others; up to 16 groups and choices.
@pytest.mark.parametrize("experts,groups", [(64, 16), (64, 8), (64, 4), (64, 2), (32, 16), (60, 15), (48, 16), (128, 16), (128, 8), (128, 4),
                                            (128, 2), (112, 7), (96, 16), (120, 5)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(experts, groups, best, biased):
    rng = np.random.default_rng(experts + groups)
    top_groups = (groups + 1) // 2
    run(dev(mixed(rng, 4100, experts, best == 2)), min(16, experts // groups * top_groups), kind="sigmoid" if groups % 2 == 0 else "softmax", groups=groups,
        top_groups=top_groups, best=best, bias=dev((0.2 * rng.standard_normal(experts)).astype(np.float32)) if biased else None)


@pytest.mark.parametrize("experts", [64, 128, 200, 256])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_fp16_scores(experts, kind, renorm):
    rng = np.random.default_rng(experts)
    l = dev(mixed(rng, 6000, experts)).half()
    run(l, 6, kind=kind, renorm=renorm)
    run(l, 6, kind=kind, renorm=renorm, bias=dev((0.1 * rng.standard_normal(experts)).astype(np.float32)))
