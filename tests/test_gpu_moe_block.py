"""A mixture of experts' feed-forward block through the library: router product, routing, quantized rows, gate and up, down,
gather onto the residual stream; eagerly, captured and replayed with other tokens, on two streams at once.  Every operator's
result is compared with its definition on the inputs that it had in the run."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
import oracle
from gemm_qmm_gemv_amd import inputs, tensors
from oracle import moe_block as moe
from tests.gpu_util import announce, assert_within
from tests.layer_util import E32, dev
from tests.test_gpu_gemm_i8 import check, gated_bound, plain_bound
from tests.test_gpu_moe_route import weight_bound

pytestmark = pytest.mark.gpu

HIDDEN, INTER, EXPERTS, TOP_K = 256, 160, 24, 4


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.float16 else t.cpu().numpy()


class Block:
    """Weights quantized by the library itself, a router in packed codes, the workspace of one stream."""

    def __init__(self, seed, tokens, sigmoid):
        rng = np.random.default_rng(seed)
        self.sigmoid, self.tokens = sigmoid, tokens
        self.router = tensors.upload_matrix(inputs.quantized_matrix(EXPERTS, HIDDEN, 8, 64, key=(seed, 1)))
        self.bias = dev(0.05 * rng.standard_normal(EXPERTS).astype(np.float32)) if sigmoid else None

        def stack(n, k):
            codes, scales = tensors.quantize_rows(dev((rng.standard_normal((EXPERTS * n, k)) / np.sqrt(k)).astype(np.float32)))
            return codes.view(EXPERTS, n, k), scales.view(EXPERTS, n)

        self.gate, self.up, self.down = stack(INTER, HIDDEN), stack(INTER, HIDDEN), stack(HIDDEN, INTER)
        self.workspace = tensors.route_workspace(tokens, EXPERTS, TOP_K)
        self.products = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def run(self, h, x, keep=None, notes=None):
        """h [tokens, HIDDEN] fp32, updated in place by the block of x (fp16)."""
        note = (lambda *a: notes.append(a)) if notes is not None else (lambda *a: None)
        logits = tensors.gemm(self.router, x, workspace=self.products)
        r = tensors.moe_route(logits, TOP_K, self.bias, self.sigmoid, 4, 2, 2 if self.sigmoid else 1, True, 1.5, keep, workspace=self.workspace)
        note("route", logits, keep, r)
        codes, scales = tensors.quantize_rows(x)
        note("quantize", x, codes, scales)
        act = tensors.moe_swiglu_i8(*self.gate, *self.up, codes, scales, r.pair_token, r.offsets)
        note("swiglu", codes, scales, r, act)
        # Rows that no expert covers hold anything.
        rows = torch.arange(act.shape[0], device="cuda")[:, None] < r.offsets[-1]
        act = torch.where(rows, act, 0)
        codes, scales = tensors.quantize_rows(act)
        note("quantize", act, codes, scales)
        y = tensors.moe_i8(*self.down, codes, scales, None, r.offsets)
        note("down", codes, scales, r, y)
        before = h.clone()
        tensors.moe_gather(y, r.pair_row, r.weights, h, h)
        note("gather", y, r, before, h.clone())
        return h

    def verify(self, notes):
        for kind, *args in notes:
            if kind == "route":
                logits, keep, r = args
                ids, w, pair_row, offsets, token, weight = moe.route(
                    host(logits), "sigmoid" if self.sigmoid else "softmax", None if self.bias is None else host(self.bias), 4, 2,
                    2 if self.sigmoid else 1, TOP_K, True, 1.5, None if keep is None else host(keep))
                assert np.array_equal(host(r.ids), ids) and np.array_equal(host(r.pair_row), pair_row)
                assert np.array_equal(host(r.offsets), offsets) and np.array_equal(host(r.pair_token)[:offsets[-1]], token)
                # (The router's logits lie up to 100 apart here, which the derived bound counts.)
                kind = "sigmoid" if self.sigmoid else "softmax"
                assert (np.abs(host(r.weights) - w) <= weight_bound(host(logits), ids, w, kind, 16)).all()
            elif kind == "quantize":
                x, codes, scales = args
                want, unit = moe.quantize_rows(host(x))
                assert np.array_equal(host(codes), want) and np.array_equal(host(scales), unit)
            elif kind == "gather":
                y, r, before, h = args
                want, mag = moe.gather(host(y), host(r.pair_row), host(r.weights), host(before))
                assert (np.abs(host(h) - want) <= (TOP_K + 2) * E32 * mag).all()
            else:
                codes, scales, r, got = args
                off = host(r.offsets)
                pairs = [self.gate, self.up] if kind == "swiglu" else [self.down]
                rows = host(r.pair_token).copy() if kind == "swiglu" else None
                if rows is not None:
                    rows[off[-1]:] = 0
                res = [moe.moe_product_i8(host(w), host(s), host(codes), host(scales), rows, off, got.shape[0]) for w, s in pairs]
                g, covered = res[0]
                if kind == "down":
                    check(host(got), g, plain_bound(g, False), covered, kind)
                else:
                    act = moe.silu(g) * res[1][0]
                    check(host(got), act, gated_bound(g, res[1][0], act, True), covered, kind)


def data(seed, tokens):
    rng = np.random.default_rng(seed)
    return dev(rng.standard_normal((tokens, HIDDEN)).astype(np.float32)), dev(rng.standard_normal((tokens, HIDDEN)).astype(np.float16))


@pytest.mark.parametrize("tokens", [1, 5, 70, 300])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_block(tokens, sigmoid):
    announce("moe block", tokens, sigmoid)
    b = Block(3, tokens, sigmoid)
    h, x = data(tokens, tokens)
    notes = []
    b.run(h, x, notes=notes)
    b.verify(notes)


@pytest.mark.parametrize("tokens", [12, 90])
def test_captured_and_replayed_with_other_tokens_and_padding(tokens):
    announce("moe block captured", tokens)
    b = Block(5, tokens, True)
    steps = [data(20 + s, tokens) for s in range(4)]
    keeps = [dev((np.arange(tokens) < tokens - s).astype(np.uint8)) for s in (0, 3, tokens, 1)]
    want = [b.run(h.clone(), x, keep).clone() for (h, x), keep in zip(steps, keeps)]
    assert torch.equal(want[2], steps[2][0])  # nothing but padding
    for (h, x), keep, w in zip(steps, keeps, want):
        assert torch.equal(w[keep == 0], h[keep == 0])
    h, x, keep = steps[0][0].clone(), steps[0][1].clone(), keeps[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(h, x, keep)
    for i in (0, 1, 2, 3, 1, 0):
        h.copy_(steps[i][0])
        x.copy_(steps[i][1])
        keep.copy_(keeps[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want[i])


def test_two_blocks_on_two_streams_at_once():
    announce("two moe blocks on two streams")
    blocks = [Block(7, 64, False), Block(8, 200, True)]
    steps = [[data(30 + 10 * i + s, b.tokens) for s in range(5)] for i, b in enumerate(blocks)]
    want = [[b.run(h.clone(), x).clone() for h, x in mine] for b, mine in zip(blocks, steps)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[], []]
    for s in range(5):
        for i, (b, st) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(st):
                h, x = steps[i][s]
                got[i].append(b.run(h.clone(), x))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_calls_on_another_stream_than_the_current_one():
    announce("moe operators on another stream")
    b = Block(9, 40, False)
    h, x = data(50, 40)
    logits = torch.randn(40, EXPERTS, device="cuda")
    codes, scales = tensors.quantize_rows(x)
    r = tensors.moe_route(logits, TOP_K, workspace=b.workspace)
    act = tensors.moe_swiglu_i8(*b.gate, *b.up, codes, scales, r.pair_token, r.offsets)
    y = tensors.moe_i8(*b.down, *tensors.quantize_rows(act), None, r.offsets)
    out = tensors.moe_gather(y, r.pair_row, r.weights, h)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    c2, s2 = tensors.quantize_rows(x, stream=st)
    r2 = tensors.moe_route(logits, TOP_K, workspace=b.workspace, stream=st)
    a2 = tensors.moe_swiglu_i8(*b.gate, *b.up, c2, s2, r2.pair_token, r2.offsets, stream=st)
    y2 = tensors.moe_i8(*b.down, *tensors.quantize_rows(a2, stream=st), None, r2.offsets, stream=st)
    o2 = tensors.moe_gather(y2, r2.pair_row, r2.weights, h, stream=st)
    st.synchronize()
    for u, v in ((codes, c2), (scales, s2), (r.ids, r2.ids), (r.pair_row, r2.pair_row), (act, a2), (y, y2), (out, o2)):
        assert torch.equal(u, v)
    with pytest.raises(AssertionError):
        tensors.moe_route(logits, TOP_K, stream=st)  # the workspace would be the current stream's
    with pytest.raises(ValueError):
        tensors.moe_gather(y.cpu(), r.pair_row, r.weights)


def test_routing_feeds_the_packed_experts():
    # The rows that routing groups are what the products of packed weights take.
    announce("routing and packed experts")
    rng = np.random.default_rng(11)
    tokens, n, k = 30, 96, 128
    mats = [inputs.quantized_matrix(n, k, 4, 64, key=(11, e)) for e in range(8)]
    stack = dict(n_experts=8, n=n, k=k, bits=4, group=64, **{f: dev(np.stack([m[f] for m in mats])) for f in ("w", "scales", "mins")})
    x = rng.standard_normal((tokens, k)).astype(np.float16)
    r = tensors.moe_route(dev(rng.standard_normal((tokens, 8)).astype(np.float32)), 2)
    y = tensors.moe(stack, dev(x), r.pair_token, r.offsets, 2 * tokens)
    out = tensors.moe_gather(y, r.pair_row, r.weights)
    combined = torch.zeros((tokens, n), device="cuda")
    tensors.moe_combine(stack, dev(x), r.pair_token, r.offsets, r.pair_token, r.pair_weight, 2 * tokens, combined)
    ids, w = host(r.ids), host(r.weights)
    ref, mag = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        for e, f in zip(ids[t], w[t]):
            m = mats[e]
            a, b = oracle.qmm(m["w"], m["scales"], m["mins"], x[t:t + 1], n, k, 4, 64)
            ref[t] += f * a[0]
            mag[t] += abs(f) * b[0]
    assert_within(host(out), ref, mag, "gather")
    assert_within(host(combined), ref, mag, "combine")
