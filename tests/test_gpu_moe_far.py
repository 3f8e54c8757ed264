"""The expert block's operators where elements lie beyond 32 bits, and where outputs and rows go past the caches."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from oracle import moe_block as moe
from tests.gpu_util import announce
from tests.layer_util import E16, E32, TINY16, check, dev

pytestmark = pytest.mark.gpu


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    return torch.randint(-128, 128, shape, device="cuda", dtype=torch.int8, generator=g)


def close(y, x, xs, w, ws, f16):
    """The sums are exact in float64; conversion and two scales round once each, an fp16 output once more."""
    want = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()[None, :]
    bound = 3.01 * E32 * want.abs() + (E16 * 1.01 * want.abs() + TINY16 if f16 else 0) + 1e-40
    return ((y.double() - want).abs() <= bound).all()


# Tiles and few rows, outputs of more than 2^31 elements.
@pytest.mark.parametrize("m,n,k", [(66000, 33000, 32), (40, 54000000, 32)])
def test_product_of_many_outputs(m, n, k):
    announce("gemm_i8 far", m, n, k)
    g = generator(m)
    w, x = codes(g, n, k), codes(g, m, k)
    ws, xs = torch.rand(n, device="cuda", generator=g) * 1e-3, torch.rand(m, device="cuda", generator=g)
    y = torch.full((m * n + 8,), 77.0, dtype=torch.float16, device="cuda")
    qmm.qmm_gemm_i8(w, ws, x, xs, y, True, m, n, k)
    torch.cuda.synchronize()
    assert (y[m * n:] == 77).all()
    y = y[:m * n].view(m, n)
    for a, b in ((0, min(m, 300)), (m // 2, m // 2 + min(m // 2, 300)), (m - min(m, 300), m)):
        for c, d in ((0, 3000), (n // 2, n // 2 + 3000), (n - 3000, n)):
            assert close(y[a:b, c:d], x[a:b], xs[a:b], w[c:d], ws[c:d], True), (a, c)


# Outputs of 192 MiB and more, whole and ragged rows, of both types.
@pytest.mark.parametrize("m,n,f16", [(8192, 8192, False), (12300, 8200, True), (7000, 7203, False)])
def test_products_past_the_caches(m, n, f16):
    announce("gemm_i8 past the caches", m, n, f16)
    g, k = generator(n), 160
    assert m * n * (2 if f16 else 4) >= 192 << 20
    w, x = codes(g, n, k), codes(g, m, k)
    ws, xs = torch.rand(n, device="cuda", generator=g) * 1e-4, torch.rand(m, device="cuda", generator=g)
    y = torch.full((m + 1, n), 77.0, dtype=torch.float16 if f16 else torch.float32, device="cuda")
    qmm.qmm_gemm_i8(w, ws, x, xs, y, f16, m, n, k)
    z = y.float() + 1  # read by the next kernel
    torch.cuda.synchronize()
    assert (y[m] == 77).all() and torch.equal(z, y.float() + 1)
    assert close(y[:m], x, xs, w, ws, f16)


def test_experts_past_the_caches():
    announce("moe_i8 past the caches")
    g, experts, n, k = generator(3), 24, 2048, 96
    counts = np.random.default_rng(3).integers(900, 1500, experts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    p = int(offsets[-1])
    assert p * n * 4 >= 192 << 20
    w, x = codes(g, experts, n, k), codes(g, p, k)
    ws, xs = torch.rand((experts, n), device="cuda", generator=g) * 1e-4, torch.rand(p, device="cuda", generator=g)
    y = torch.full((p + 1, n), 77.0, device="cuda")
    qmm.qmm_moe_gemm_i8(w, ws, x, xs, None, p, dev(offsets.astype(np.int32)), y, False, p, experts, n, k)
    torch.cuda.synchronize()
    assert (y[p] == 77).all()
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        assert close(y[a:b], x[a:b], xs[a:b], w[e], ws[e], False), e


@pytest.mark.parametrize("tokens,top_k,n,dtype", [(6600, 8, 2048, torch.float16), (3300, 8, 2052, torch.float32), (9000, 3, 4096, torch.float16)])
def test_gather_past_the_caches(tokens, top_k, n, dtype):
    announce("gather past the caches", tokens, top_k, n, dtype)
    g = generator(tokens)
    assert tokens * top_k * n * (2 if dtype == torch.float16 else 4) >= 192 << 20
    rows = torch.randn((tokens * top_k, n), device="cuda", generator=g).to(dtype)
    at = torch.randperm(tokens * top_k, device="cuda", generator=g).int().view(tokens, top_k)
    at[5, 0], at[7, top_k - 1] = -1, at[8, 0]
    weights, residual = torch.rand((tokens, top_k), device="cuda", generator=g), torch.randn((tokens, n), device="cuda", generator=g)
    y = torch.empty_like(residual)
    qmm.qmm_moe_gather(rows, dtype == torch.float16, at, weights, residual, y, tokens, top_k, tokens * top_k, n)
    want, mag = residual.double(), residual.double().abs()
    for j in range(top_k):
        f = torch.where(at[:, j] < 0, 0.0, weights[:, j]).double()[:, None]
        part = f * rows[at[:, j].clamp(min=0).long()].double()
        want, mag = want + part, mag + part.abs()
    assert ((y.double() - want).abs() <= (top_k + 2) * E32 * mag + 1e-40).all()


def test_gather_of_far_rows():
    p, n, tokens, top_k = 1100000, 2048, 50, 4
    announce("gather far", p, n)
    g = generator(1)
    rows = torch.zeros((p, n), dtype=torch.float16, device="cuda")
    at = torch.randint(p - 5000, p, (tokens, top_k), device="cuda", dtype=torch.int32, generator=g)
    rows[p - 5000:] = torch.randn((5000, n), device="cuda", generator=g).half()
    weights = torch.rand((tokens, top_k), device="cuda", generator=g)
    y = torch.empty((tokens, n), device="cuda")
    qmm.qmm_moe_gather(rows, True, at, weights, None, y, tokens, top_k, p, n)
    near = rows[p - 5000:].cpu().numpy()
    want, mag = moe.gather(near, at.cpu().numpy() - (p - 5000), weights.cpu().numpy(), None)
    check(y.cpu().numpy(), want, (top_k + 2) * E32 * mag + 1e-40, "gather far")


@pytest.mark.parametrize("rows,k,stride", [(40, 64, 60000001), (70000, 32768, 32768)])
def test_quantize_far_rows(rows, k, stride):
    announce("quantize far", rows, k, stride)
    g = generator(rows)
    x = torch.zeros(rows * stride, dtype=torch.float16, device="cuda").view(rows, stride)
    at = sorted({0, 1, rows // 2, rows - 2, rows - 1})
    for r in at:
        x[r, :k] = torch.randn(k, device="cuda", generator=g).half()
    c = torch.full((rows + 1, k), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), 99.0, device="cuda")
    qmm.qmm_quantize_rows(x, True, stride, c, s, rows, k)
    torch.cuda.synchronize()
    assert (c[rows] == 99).all() and s[rows] == 99
    want, unit = moe.quantize_rows(x[at, :k].float().cpu().numpy())
    assert np.array_equal(c[at].cpu().numpy().astype(np.int64), want) and np.array_equal(s[at].cpu().numpy(), unit)


@pytest.mark.parametrize("tokens,experts,stride", [(80, 128, 30000000), (5000, 60, 500000)])
def test_route_far_rows(tokens, experts, stride):
    announce("route far", tokens, experts, stride)
    g = generator(tokens)
    l = torch.zeros(tokens * stride, dtype=torch.float16, device="cuda").view(tokens, stride)
    l[:, :experts] = torch.randn((tokens, experts), device="cuda", generator=g).half()
    near = l[:, :experts].contiguous()
    got = []
    for logits, apart in ((l, stride), (near, experts)):
        out = [torch.full((tokens, 6), -9, dtype=torch.int32, device="cuda"), torch.full((tokens, 6), -9.0, device="cuda"),
               torch.full((tokens, 6), -9, dtype=torch.int32, device="cuda"), torch.full((experts + 1,), -9, dtype=torch.int32, device="cuda"),
               torch.full((tokens * 6,), -9, dtype=torch.int32, device="cuda"), torch.full((tokens * 6,), -9.0, device="cuda")]
        need = qmm.qmm_moe_route_workspace_bytes(tokens, experts, 6)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        qmm.qmm_moe_route(logits, True, apart, None, False, 1, 1, 1, 6, True, 1.0, None, *out, ws, need, tokens, experts)
        got.append([t.cpu().numpy() for t in out])
    assert all(np.array_equal(a, b) for a, b in zip(*got))
    ids = moe.route(near.float().cpu().numpy(), "softmax", None, 1, 1, 1, 6, True, 1.0)[0]
    assert np.array_equal(got[0][0], ids)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("counts", [(1, 0, 3), (2, 40, 300)])
def test_stacks_past_four_gib(glu, counts):
    n, k, experts = 60000, 32768, 3
    announce("moe_i8 far stacks", counts, "glu" if glu else "")
    g = generator(sum(counts))
    offsets = np.concatenate([[0], np.cumsum(counts)])
    p = int(offsets[-1])
    w, x = codes(g, experts, n, k), codes(g, p, k)
    u = w.flip(1) if glu else None
    ws, us = (torch.rand((experts, n), device="cuda", generator=g) * 1e-6 for _ in range(2))
    xs = torch.rand(p, device="cuda", generator=g)
    y = torch.full((p + 1, n), 77.0, device="cuda")
    off = dev(offsets.astype(np.int32))
    if glu:
        qmm.qmm_moe_swiglu_i8(w, ws, u, us, x, xs, None, p, off, y, False, p, experts, n, k)
    else:
        qmm.qmm_moe_gemm_i8(w, ws, x, xs, None, p, off, y, False, p, experts, n, k)
    torch.cuda.synchronize()
    assert (y[p] == 77).all()
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        for c in (0, n // 2, n - 700):
            part = slice(c, c + 700)
            if not glu:
                assert close(y[a:b, part], x[a:b], xs[a:b], w[e, part], ws[e, part], False), (e, c)
                continue
            v, t = ((x[a:b].double() @ m[e, part].double().T) * xs[a:b].double()[:, None] * s[e, part].double() for m, s in ((w, ws), (u, us)))
            h = v * torch.sigmoid(v) * t
            # As for the smaller ones: silu's slope, its exponential, quotient and products.
            bound = E32 * h.abs() * (3 * (1 + v.abs()) + 11) + 1e-35 * t.abs() + 1e-40
            assert ((y[a:b, part].double() - h).abs() <= bound).all(), (e, c)
