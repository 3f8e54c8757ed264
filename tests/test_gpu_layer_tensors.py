"""The torch-side calls of the layer's operators against the float64 definitions."""
import numpy as np
import pytest
import torch

from gemm_qmm_gemv_amd import tensors
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import check, dev
from tests.test_gpu_layer_norm import EPS, bounds, case

pytestmark = pytest.mark.gpu


def test_one_gate_row_for_several_rows():
    rng = np.random.default_rng(71)
    rows, n = 7, 192
    y, pw, g, res, pre = case(rng, rows, n, True, True, "shared")
    u, h, x = layer.norm_residual(y, pw, g, 0.5, res, pre, EPS)
    eh, ex = bounds(u, h, x, 0.5, pre)
    # Whatever lies behind the gate is no part of it.
    buf = torch.full((rows, n), float("nan"), device="cuda")
    buf[0] = dev(g)[0]
    for gate in (buf[:1], buf[0], buf[:1].expand(rows, n)):
        announce("one gate row", tuple(gate.shape))
        hd, xd = tensors.norm_residual(dev(y), dev(res), dev(pre), EPS, dev(pw), gate, 0.5)
        check(hd.cpu().numpy(), h, eh, "h")
        check(xd.cpu().numpy(), x, ex, "x")


def prompt_call(n, stream):
    q, k, v = (torch.randn(n, h, 64, device="cuda", dtype=torch.float16) for h in (4, 2, 2))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    return tensors.attn_prompt(q, k, v, off), lambda: (tensors.attn_prompt(q, k, v, off, stream=stream),)


def norm_call(n, stream):
    y, res = (torch.randn(n, 256, device="cuda") for _ in range(2))
    return tensors.norm_residual(y, res, None)[1], lambda: tensors.norm_residual(y, res, None, stream=stream)[::-1]


def append_call(n, stream):
    cache = tensors.kv_cache(n // 16 + 1, 2, 64, 16, 4, 32)
    q, k, v = (torch.randn(n, h * 64, device="cuda", dtype=torch.float16) for h in (4, 2, 2))
    slots = torch.arange(n, device="cuda")
    go = lambda s: tensors.kv_append(cache, q, k, v, None, slots, prompt_rows=True, stream=s)
    return go(None)[0], lambda: go(stream)


def cache_call(n, stream):
    cache = tensors.kv_cache(4, 2, 64, 16, 4, 32)
    q = torch.randn(n, 4, 64, device="cuda", dtype=torch.float16)
    table, lens = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.full((n,), 9, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    return (tensors.attn_cache(cache, q, table, lens, 16, workspace=ws),
            lambda: (tensors.attn_cache(cache, q, table, lens, 16, workspace=ws, stream=stream),))


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("make", [norm_call, append_call, cache_call, prompt_call])
def test_outputs_of_another_stream_are_no_memory_that_this_one_still_reads(make, handle):
    announce("outputs on another stream", make.__name__, handle)
    n = 2000
    side = torch.cuda.Stream()
    want, call = make(n, side.cuda_stream if handle else side)
    marks = [torch.full((n, 256), 5.0, dtype=torch.float16, device="cuda") for _ in range(6)]
    marks += [torch.full((n, 256), 5.0, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    # This stream is busy for some milliseconds and then reads blocks that have been given back meanwhile.
    torch.cuda._sleep(20_000_000)
    copies = [m.clone() for m in marks]
    del marks
    got = call()
    side.synchronize()
    torch.cuda.synchronize()
    assert all((c == 5).all() for c in copies)
    assert torch.equal(got[0].view_as(want), want)


def test_outputs_of_the_current_stream_and_of_the_default_one():
    announce("outputs on the current stream")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want, call = norm_call(50, side)
        assert torch.equal(call()[0], want)
    side.synchronize()
    want, call = prompt_call(300, torch.cuda.default_stream().cuda_stream)
    with torch.cuda.stream(side):
        got = call()[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
