"""A small decoder through the products and the layer's operators together: packed prompts into a paged cache, single
tokens and drafts over it, eagerly, in a captured step and on two streams at once.  Every operator's result is compared
with the float64 definition on the inputs that it had in the run."""
import numpy as np
import pytest
import torch

import gemm_qmm_gemv_amd as qmm
from gemm_qmm_gemv_amd import inputs, tensors
from oracle import layer
from tests.gpu_util import announce
from tests.layer_util import E16, TINY16, attention_bound, check, dev, held
from tests.test_gpu_layer_append import definition
from tests.test_gpu_layer_attn_prompt import compare
from tests.test_gpu_layer_attn_prompt import expect as expect_prompt
from tests.test_gpu_layer_norm import bounds

pytestmark = pytest.mark.gpu

HIDDEN, FFN, HQ, HKV, D, PAGE, LAYERS, EPS = 512, 1024, 8, 2, 64, 16, 2, 1e-6
LENS = [37, 1, 20]
STEPS, DRAFTS = 4, 3


def half(a):
    return a.cpu().numpy()


class Decoder:
    """Weights, one cache per layer, the page table and the workspaces of one stream."""

    def __init__(self, bits, seed):
        rng = np.random.default_rng([seed, bits])
        self.bits, self.group = bits, 32
        mat = lambda n, k, *key: tensors.upload_matrix(inputs.quantized_matrix(n, k, 4, 64, key=(seed, *key)))
        one = lambda n: dev((1 + 0.1 * rng.standard_normal(n)).astype(np.float32))
        self.layers = [dict(qkv=mat((HQ + 2 * HKV) * D, HIDDEN, i, 0), o=mat(HIDDEN, HQ * D, i, 1), gate=mat(FFN, HIDDEN, i, 2),
                            up=mat(FFN, HIDDEN, i, 3), down=mat(HIDDEN, FFN, i, 4), pre=one(HIDDEN), mid=one(HIDDEN),
                            post=one(HIDDEN), qn=one(D), kn=one(D)) for i in range(LAYERS)]
        self.last = one(HIDDEN)
        self.inv = dev((1e4 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
        self.max_len = max(LENS) + STEPS + DRAFTS
        width = -(-self.max_len // PAGE)
        self.table = dev(rng.permutation(len(LENS) * width + 2)[:len(LENS) * width].reshape(len(LENS), width).astype(np.int32))
        self.caches = [tensors.kv_cache(len(LENS) * width + 2, HKV, D, PAGE, bits, self.group) for _ in range(LAYERS)]
        self.products = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
        self.scratch = tensors.attn_workspace(self.caches[0], len(LENS), DRAFTS, HQ, self.max_len)

    def product(self, w, x, **kw):
        need = qmm.qmm_gemm_workspace_bytes(x.shape[0], w["n"], w["k"], w["bits"], w["group"])
        assert need <= self.products.numel()
        return tensors.gemm(w, x, workspace=self.products, **kw)

    def run(self, h, positions, slots, attend, notes=None):
        """h [tokens][HIDDEN] fp32, updated in place; `attend`: layer, q, k, v -> attention's output."""
        note = (lambda *a: notes.append(tuple(t.clone() if torch.is_tensor(t) else t for t in a))) if notes is not None \
            else (lambda *a: None)
        _, x = tensors.norm_residual(None, h, self.layers[0]["pre"], EPS)
        note("norm", None, None, h, self.layers[0]["pre"], h, x)
        for i, w in enumerate(self.layers):
            rows = self.product(w["qkv"], x, out_fp16=True)
            q, k, v = rows[:, :HQ * D], rows[:, HQ * D:(HQ + HKV) * D], rows[:, (HQ + HKV) * D:]
            got = tensors.kv_append(self.caches[i], q, k, v, positions, slots, self.inv, False, w["qn"], w["kn"], EPS,
                                    prompt_rows=True, cached_values=True)
            note("append", i, rows, w["qn"], w["kn"], positions, slots, *got)
            a = attend(i, *got)
            note("attention", i, *got, a)
            y = self.product(w["o"], a.view(a.shape[0], -1))
            before = h.clone()
            _, x = tensors.norm_residual(y, h, w["mid"], EPS, post=w["post"], h=h)
            note("norm", y, w["post"], before, w["mid"], h, x)
            act = (torch.nn.functional.silu(self.product(w["gate"], x)) * self.product(w["up"], x)).half()
            y = self.product(w["down"], act)
            pre = self.layers[i + 1]["pre"] if i + 1 < LAYERS else self.last
            before = h.clone()
            _, x = tensors.norm_residual(y, h, pre, EPS, h=h)
            note("norm", y, None, before, pre, h, x)
        return x

    def slots(self, seqs, positions):
        page = self.table[seqs, (positions // PAGE).long()].long()
        return page * PAGE + positions % PAGE

    def prompt(self, h, notes=None):
        offsets = dev(np.concatenate([[0], np.cumsum(LENS)]).astype(np.int32))
        seqs = dev(np.repeat(np.arange(len(LENS)), LENS))
        positions = dev(np.concatenate([np.arange(n) for n in LENS]).astype(np.int32))
        return self.run(h, positions, self.slots(seqs, positions), lambda i, q, k, v: tensors.attn_prompt(q, k, v, offsets), notes)

    def over_cache(self, h, positions, slots, lens, q_len=1, notes=None):
        return self.run(h, positions, slots,
                        lambda i, q, k, v: tensors.attn_cache(self.caches[i], q, self.table, lens, self.max_len, q_len=q_len,
                                                              workspace=self.scratch), notes)

    def state(self):
        return [t for c in self.caches for t in c.keep if t is not None]

    def host(self, i):
        names = ("k", "ks", "km", "v", "vs", "vm")
        return {n: None if t is None else (half(t).view(np.uint32) if n in "kv" else half(t))
                for n, t in zip(names, self.caches[i].keep)}


def inputs_of(dec, lens, q_len, rng):
    """Embeddings, positions, slots and lengths of q_len new tokens behind `lens` rows."""
    seqs = torch.arange(len(LENS), device="cuda").repeat_interleave(q_len)
    positions = (dev(np.asarray(lens, np.int32)).repeat_interleave(q_len)
                 + torch.arange(q_len, device="cuda", dtype=torch.int32).repeat(len(LENS)))
    h = dev(rng.standard_normal((len(LENS) * q_len, HIDDEN)).astype(np.float32))
    return h, positions, dec.slots(seqs, positions), dev(np.asarray(lens, np.int32) + q_len)


def verify(dec, notes, lens=None, q_len=1):
    """Each noted step against its definition (lens: cached rows, None: the packed prompts)."""
    for n, note in enumerate(notes):
        kind, args = note[0], note[1:]
        what = "%s (step %d)" % (kind, n)
        if kind == "norm":
            y, post, before, pre, h, x = (None if t is None else half(t) for t in args)
            u, rh, rx = layer.norm_residual(y, post, None, 1.0, before, pre, EPS)
            eh, ex = bounds(u, rh, rx, 1.0, pre)
            check(h, rh, eh, what + " h")
            check(x, rx, ex, what + " x")
        elif kind == "append":
            i, rows, qn, kn, positions, slots, q, k, v = args
            rows, positions, slots = half(rows), half(positions), half(slots)
            parts = (rows[:, :HQ * D], rows[:, HQ * D:(HQ + HKV) * D], rows[:, (HQ + HKV) * D:])
            ref, err = definition(parts, (half(qn), half(kn)), half(dec.inv), positions, HQ, HKV, D, D, False)
            check(half(q), ref[0], err[0] + E16 * np.abs(ref[0]) * 1.01 + TINY16, what + " q")
            host = dec.host(i)
            at, place = slots // PAGE, slots % PAGE
            for side, r, e, out in (("k", ref[1], err[1], k), ("v", ref[2], err[2], v)):
                stored = held(host, side, dec.bits, dec.group)[at, :, place]
                if dec.bits == 16:
                    bound = e + E16 * np.abs(r) * 1.01 + TINY16
                else:
                    # Half a step, and where a code was cut off at its ends what the fp16 scale and min are off by.
                    g = r.reshape(*r.shape[:2], -1, dec.group)
                    s = host[side + "s"][at, :, :, place].astype(np.float64)
                    span, low = g.max(-1) - g.min(-1), np.abs(g.min(-1))
                    per = 0.5 * s * (1 + 2.0 ** -10) + 1.01 * E16 * (span + low) + 2.0 ** dec.bits * TINY16
                    bound = 2 * np.max(np.broadcast_to(e, r.shape)) + np.repeat(per, dec.group, axis=-1)
                check(stored, r, bound, what + " stored " + side)
                check(half(out), stored, E16 * np.abs(stored) * 1.01 + TINY16, what + " " + side + "_out")
        elif lens is None:
            i, q, k, v, a = args
            o, b = expect_prompt(half(q), half(k), half(v), [0] + list(np.cumsum(LENS)), D ** -0.5)
            compare(half(a), o, b, what)
        else:
            i, q, _, _, a = args
            host, table = dec.host(i), half(dec.table)
            keys, values = held(host, "k", dec.bits, dec.group), held(host, "v", dec.bits, dec.group)
            q, got = half(q), half(a)
            for s, length in enumerate(lens):
                ks, vs = layer.sequence_rows(keys, table[s], length), layer.sequence_rows(values, table[s], length)
                limits = [length - q_len + 1 + j for j in range(q_len)]
                rows = slice(s * q_len, (s + 1) * q_len)
                for h in range(HQ):
                    vj = vs[:, h // (HQ // HKV)]
                    r = layer.attend(q[rows, h], ks[:, h // (HQ // HKV)], vj, limits, D ** -0.5)
                    b = attention_bound(*r, length, np.abs(vj).max(), D, dec.bits != 16, dec.bits == 16)
                    check(got[rows, h], r[0], b, what)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_prompts_then_tokens_then_drafts(bits):
    announce("a decoder's prompts, tokens and drafts", bits)
    rng = np.random.default_rng([31, bits])
    dec = Decoder(bits, 5)
    notes = []
    dec.prompt(dev(rng.standard_normal((sum(LENS), HIDDEN)).astype(np.float32)), notes)
    verify(dec, notes)
    lens = list(LENS)
    for _ in range(STEPS):
        notes = []
        h, positions, slots, now = inputs_of(dec, lens, 1, rng)
        dec.over_cache(h, positions, slots, now, notes=notes)
        lens = [n + 1 for n in lens]
    verify(dec, notes, lens)
    notes = []
    h, positions, slots, now = inputs_of(dec, lens, DRAFTS, rng)
    dec.over_cache(h, positions, slots, now, DRAFTS, notes)
    verify(dec, notes, [n + DRAFTS for n in lens], DRAFTS)


def test_a_captured_step_replays_as_eager_steps():
    announce("a captured decode step")
    rng = np.random.default_rng(32)
    dec = Decoder(4, 6)
    dec.prompt(dev(rng.standard_normal((sum(LENS), HIDDEN)).astype(np.float32)))
    kept = [t.clone() for t in dec.state()]
    steps = [inputs_of(dec, [n + s for n in LENS], 1, rng) for s in range(STEPS)]
    want = []
    for h, positions, slots, now in steps:
        h = h.clone()
        x = dec.over_cache(h, positions, slots, now)
        want.append((h, x.clone()))
    after = [t.clone() for t in dec.state()]
    for t, k in zip(dec.state(), kept):
        t.copy_(k)
    at = [t.clone() for t in steps[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = dec.over_cache(*at)
    for step, (h_want, x_want) in zip(steps, want):
        for t, s in zip(at, step):
            t.copy_(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(at[0], h_want) and torch.equal(x, x_want)
    for t, k in zip(dec.state(), after):
        assert torch.equal(t, k)


def test_two_decoders_on_two_streams_at_once():
    announce("two decoders on two streams")
    want, got, decs, data = [], [], [], []
    for seed in (7, 8):
        rng = np.random.default_rng(seed)
        dec = Decoder(4, seed)
        start = dev(rng.standard_normal((sum(LENS), HIDDEN)).astype(np.float32))
        steps = [inputs_of(dec, [n + s for n in LENS], 1, rng) for s in range(STEPS)]
        decs.append(dec)
        data.append((start, steps))
        dec.prompt(start.clone())
        for h, *rest in steps:
            h = h.clone()
            dec.over_cache(h, *rest)
        want.append(h)
    for dec in decs:
        for t in dec.state():
            t.zero_()
    streams = [torch.cuda.Stream() for _ in decs]
    torch.cuda.synchronize()
    for dec, s, (start, _) in zip(decs, streams, data):
        with torch.cuda.stream(s):
            dec.prompt(start.clone())
    for step in range(STEPS):
        for n, (dec, s, (_, steps)) in enumerate(zip(decs, streams, data)):
            with torch.cuda.stream(s):
                h, *rest = steps[step]
                h = h.clone()
                dec.over_cache(h, *rest)
                got = got[:n] + [h] + got[n + 1:]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
