"""qmm_moe_route's grouping for hundreds of thousands of tokens: the rows that its experts make, and what a token costs there."""
import statistics

import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

UNTOUCHED = -77


class Call:
    def __init__(self, tokens, experts, top_k, padded=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(tokens + experts)
        # Popular experts, too.
        self.logits = torch.randn((tokens, experts), device="cuda", dtype=torch.float16, generator=g)
        self.logits += torch.randn(experts, device="cuda", generator=g).half()
        self.keep = (torch.rand(tokens, device="cuda", generator=g) < 0.8).to(torch.uint8) if padded else None
        self.ids, self.pair_row = (torch.full((tokens, top_k), UNTOUCHED, dtype=torch.int32, device="cuda") for _ in range(2))
        self.weights = torch.full((tokens, top_k), float(UNTOUCHED), device="cuda")
        self.offsets = torch.full((experts + 1,), UNTOUCHED, dtype=torch.int32, device="cuda")
        self.token = torch.full((tokens * top_k,), UNTOUCHED, dtype=torch.int32, device="cuda")
        self.weight = torch.full((tokens * top_k,), float(UNTOUCHED), device="cuda")
        self.need = qmm.qmm_moe_route_workspace_bytes(tokens, experts, top_k)
        self.ws = torch.full((self.need + 16,), 255, dtype=torch.uint8, device="cuda")

    def __call__(self):
        (tokens, top_k), experts = self.ids.shape, self.logits.shape[1]
        qmm.qmm_moe_route(self.logits, True, experts, None, False, 1, 1, 1, top_k, True, 1.0, self.keep, self.ids, self.weights, self.pair_row,
                          self.offsets, self.token, self.weight, self.ws, self.need, tokens, experts)


# Sums of 64 work-groups added up by every one that places, and running ones made of them; a last chunk of one work-group, of 64.
@pytest.mark.parametrize("tokens,experts", [(16385, 1024), (20481, 1000), (65536, 128), (65537, 128), (131073, 64), (262144, 17), (270337, 300),
                                            ((1 << 20) + 77, 64), ((1 << 24) - 1, 8)])
@pytest.mark.parametrize("padded", [False, True])
def test_rows(tokens, experts, padded):
    top_k = 3
    announce("route grouping", tokens, experts, "padded" if padded else "")
    c = Call(tokens, experts, top_k, padded)
    c()
    torch.cuda.synchronize()
    assert (c.ws[c.need:] == 255).all()
    # The choice itself is compared elsewhere: here a token's choices are of the highest logits, in their order.
    l = c.logits.float()
    top = l.topk(top_k, 1).values
    there = torch.ones(tokens, dtype=torch.bool, device="cuda") if c.keep is None else c.keep.bool()
    assert torch.equal(l.gather(1, c.ids.clamp(min=0).long())[there], top[there]) and (c.ids[~there] == -1).all()
    flat = c.ids.flatten().long()
    flat = torch.where(flat < 0, experts, flat)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=experts + 1)[:experts]
    rows = int(counts.sum())
    assert c.offsets[0] == 0 and torch.equal(c.offsets[1:].long(), counts.cumsum(0))
    row = torch.full_like(flat, -1)
    row[order[:rows]] = torch.arange(rows, device="cuda")
    assert torch.equal(c.pair_row.flatten().long(), row)
    assert torch.equal(c.token[:rows].long(), order[:rows] // top_k) and (c.token[rows:] == UNTOUCHED).all()
    assert torch.equal(c.weight[:rows], c.weights.flatten()[order[:rows]]) and (c.weight[rows:] == UNTOUCHED).all()


def test_four_times_the_tokens_take_four_times_as_long():
    # Not sixteen times, as they would if every work-group added up what all others counted.
    took = []
    for tokens in (1 << 20, 1 << 22):
        announce("route, time", tokens)
        c = Call(tokens, 1024, 2)
        got = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            c()
            b.record()
            b.synchronize()
            got.append(a.elapsed_time(b))
        took.append(statistics.median(got))
        print("[time] %d tokens: %.2f ms" % (tokens, took[-1]), flush=True)
        del c
    assert took[1] < 6 * took[0], took


def test_captured_and_replayed():
    # The sums are made running ones in place: each replay starts from its own.
    announce("route grouping, captured")
    a, b = Call(70001, 128, 3, True), Call(70001, 128, 3, True)
    a()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        b()
    stream.synchronize()
    with torch.cuda.graph(graph):
        qmm.qmm_moe_route(b.logits, True, 128, None, False, 1, 1, 1, 3, True, 1.0, b.keep, b.ids, b.weights, b.pair_row, b.offsets, b.token,
                          b.weight, b.ws, b.need, 70001, 128, stream=torch.cuda.current_stream().cuda_stream)
    for i in range(4):
        for c in (a, b):
            c.logits.copy_(c.logits.flip(0))
        a()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ids", "weights", "pair_row", "offsets"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (i, n)
        rows = int(a.offsets[-1])
        assert torch.equal(a.token[:rows], b.token[:rows]) and torch.equal(a.weight[:rows], b.weight[:rows])
