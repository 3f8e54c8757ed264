"""The attention half of a decoder layer: what it costs next to the quantized products.

Four operators stand between a layer's projections:

  norm    h = residual + scale * gate * rmsnorm(y); x = fp16(rmsnorm(h)): the fp32 output of one product becomes the
          residual stream and the fp16 input of the next
  append  q, k, v of new tokens: optional per-head norm, position rotation, q to fp16, k and v into a paged cache that
          holds them in 4 or 8 bits (affine groups, as the weights) or in fp16
  cache   attention of the newest tokens of many sequences over that paged cache
  prompt  causal attention over whole prompts, packed behind each other, with grouped heads

``run`` computes them in plain torch operations (32 bits, one rounding at the end), or through the library where
``own`` is set.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 1e6


def listed():
    return [
        # One token of a 1024-wide model: the residual add was fused in the projection, only the norm is left.  Latency.
        dict(name="norm_one_token", op="norm", rows=1, n=1024, y16=False, y=False, post=False, gate="none"),
        # A decode batch of a 2048-wide model with norms on both sides of the block and a gate vector; an odd batch.
        dict(name="norm_batch_sandwich", op="norm", rows=37, n=2048, y16=False, y=True, post=True, gate="shared"),
        # A long prefill of a wide model: fp16 block output, both norms, a gate of its own for every token.
        dict(name="norm_prefill", op="norm", rows=8192, n=4096, y16=True, y=True, post=True, gate="rows"),
        # A decode batch of an 0.6B-class model with per-head norms: one new token for each of 8 far sequences, 4 bits.
        dict(name="append_decode", op="append", tokens=8, seqs=8, hq=16, hkv=8, d=128, bits=4, group=64, page=64, in16=False,
             fused=False, qknorm=True, rot=128, inter=False, far=131072, pad=0),
        # The prompt of a 1B-class model: 64-wide heads from one fused q|k|v product in fp16, some padding tokens, 4 bits.
        dict(name="append_prompt", op="append", tokens=4096, seqs=3, hq=32, hkv=8, d=64, bits=4, group=32, page=16, in16=True,
             fused=True, qknorm=False, rot=64, inter=False, far=0, pad=5),
        # A wide prefill batch into an fp16 cache, interleaved rotation of half of each head.
        dict(name="append_prefill_fp16_cache", op="append", tokens=8192, seqs=5, hq=32, hkv=4, d=128, bits=16, group=64, page=64,
             in16=False, fused=False, qknorm=True, rot=64, inter=True, far=32768, pad=0),
        # One conversation of middling length on an 0.6B-class model: one workgroup's worth of rows, split over the length.
        dict(name="cache_one_sequence", op="cache", seqs=1, lo=1500, hi=1500, q_len=1, hq=16, hkv=8, d=128, bits=4, group=64, page=64),
        # A batch of ragged conversations on 64-wide heads, an empty one and one of a single token among them.
        dict(name="cache_ragged_batch", op="cache", seqs=17, lo=0, hi=5000, q_len=1, hq=32, hkv=8, d=64, bits=4, group=32, page=16),
        # Four drafted tokens a sequence, verified together over an 8-bit cache.
        dict(name="cache_drafts_8bit", op="cache", seqs=8, lo=1000, hi=9000, q_len=4, hq=32, hkv=4, d=128, bits=8, group=128, page=64),
        # A full serving batch with long histories: the largest, bound by memory.
        dict(name="cache_long_batch", op="cache", seqs=64, lo=4000, hi=16384, q_len=1, hq=32, hkv=4, d=128, bits=4, group=64, page=64),
        # Ragged short prompts packed together, 64-wide heads, a few rows behind the last one.
        dict(name="prompt_packed", op="prompt", seqs=9, lo=1, hi=700, hq=32, hkv=8, d=64, tail=3),
        # One long prompt, 128-wide heads, eight query heads to a key head: the largest, bound by the matrix cores.
        dict(name="prompt_long", op="prompt", seqs=1, lo=8192, hi=8192, hq=32, hkv=4, d=128, tail=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(8, 8), (16, 8), (32, 8), (32, 4), (16, 2), (10, 5), (7, 1)]


def draw(rng):
    op = rng.choice(["norm", "append", "cache", "prompt"])
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice([64, 128])
    bits = rng.choice([4, 4, 8, 16])
    group = rng.choice([32, 64] if d == 64 else [32, 64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        n = rng.choice([1024, 2048, 4096, 2880, 1001, 8192, 5120])
        return dict(op=op, rows=_log(rng, 1, 7200 * 4096 // max(n, 4096)), n=n, y16=rng.random() < 0.5, y=rng.random() < 0.8,
                    post=rng.random() < 0.5, gate=rng.choice(["none", "shared", "rows"]))
    if op == "append":
        tokens = _log(rng, 1, 6000)
        return dict(op=op, tokens=tokens, seqs=tokens if rng.random() < 0.4 else rng.randint(1, min(tokens, 9)), hq=hq, hkv=hkv, d=d,
                    bits=bits, group=group, page=page, in16=rng.random() < 0.5, fused=rng.random() < 0.5, qknorm=rng.random() < 0.5,
                    rot=rng.choice([d, d, d // 2]), inter=rng.random() < 0.3, far=rng.choice([0, 4096, 131072]),
                    pad=rng.choice([0, 0, min(3, tokens - 1)]))
    if op == "cache":
        q_len = rng.choice([1, 1, 1, 2, 5])
        seqs = _log(rng, 1, 48)
        hi = min(_log(rng, 16, 8000 if q_len == 1 else 4000), int(3.3e8 / (seqs * 2 * hkv * _held_row(d, bits, group))))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, hi // 2, hi]), hi=hi, q_len=q_len, hq=hq, hkv=hkv, d=d, bits=bits, group=group, page=page)
    hi = _log(rng, 2, 4000)
    return dict(op=op, seqs=rng.randint(1, max(1, min(8, 5000 // hi))), lo=rng.choice([1, hi // 2 + 1]), hi=hi, hq=hq, hkv=hkv, d=d,
                tail=rng.choice([0, 0, 7]))


def _held_row(d, bits, group):
    """Bytes that one row of the cache takes: the values, and where they are codes a scale and a min per group."""
    return 2 * d if bits == 16 else d * bits // 8 + 4 * (d // group)


def _lengths(case):
    """The sequences' lengths, from the case alone: the shortest first, the rest spread over the range."""
    if case["seqs"] == 1:
        return [case["hi"]]
    rng = random.Random(case["seqs"] * 1000003 + case["hi"])
    more = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"] - 2)]
    return [case["lo"], case["lo"] + 1 if case["lo"] == 0 else case["hi"]] + more


# ---------------------------------------------------------------- inputs


def _cache_arrays(case, pages, gen):
    """A paged cache: packed rows [pages][kv heads][page][words], fp16 scales and mins [pages][kv heads][groups][page]."""
    hkv, d, bits, group, page = (case[k] for k in ("hkv", "d", "bits", "group", "page"))
    out = {}
    for side in "kv":
        if bits == 16:
            rows = torch.randn((pages, hkv, page, d), device=DEV, generator=gen, dtype=torch.float16)
            out[side] = rows.view(torch.int32)
            out[side + "s"] = out[side + "m"] = None
            continue
        out[side] = torch.randint(-2 ** 31, 2 ** 31, (pages, hkv, page, d * bits // 32), device=DEV, generator=gen, dtype=torch.int64).to(torch.int32)
        # What rows of N(0, 1) values are held as: a range of about five over all codes, and its lower end.
        shape = (pages, hkv, d // group, page)
        span = 4.6 + 0.5 * torch.randn(shape, device=DEV, generator=gen)
        out[side + "s"] = (span / (2 ** bits - 1)).half()
        out[side + "m"] = (-0.5 * span + 0.2 * torch.randn(shape, device=DEV, generator=gen)).half()
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    op = case["op"]
    s = {"case": case}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, device=DEV, generator=gen).to(dtype)

    if op == "norm":
        rows, n = case["rows"], case["n"]
        s["y"] = normal(rows, n, dtype=torch.float16 if case["y16"] else torch.float32) if case["y"] else None
        s["post"] = 1 + 0.1 * normal(n) if case["y"] and case["post"] else None
        s["gate"] = None
        if case["y"] and case["gate"] != "none":
            s["gate"] = torch.sigmoid(normal(1 if case["gate"] == "shared" else rows, n))
        s["residual"] = 3 * normal(rows, n)
        s["pre"] = 1 + 0.1 * normal(n)
        s["scale"] = 0.7
        s["h"] = torch.empty((rows, n), device=DEV)
        s["x"] = torch.empty((rows, n), device=DEV, dtype=torch.float16)
        return s

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "append":
        tokens, seqs, page = case["tokens"], case["seqs"], case["page"]
        dt = torch.float16 if case["in16"] else torch.float32
        if case["fused"]:
            qkv = normal(tokens, (hq + 2 * hkv) * d, dtype=dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
        else:
            s["q"], s["k"], s["v"] = normal(tokens, hq * d, dtype=dt), normal(tokens, hkv * d, dtype=dt), normal(tokens, hkv * d, dtype=dt)
        s["q_norm"] = 1 + 0.1 * normal(d) if case["qknorm"] else None
        s["k_norm"] = 1 + 0.1 * normal(d) if case["qknorm"] else None
        rot = case["rot"]
        s["inv_freq"] = (THETA ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).float()
        # Tokens of a sequence behind each other, each sequence at a position of its own and in pages of its own.
        cut = [tokens * i // seqs for i in range(seqs + 1)]
        need = [(cut[i + 1] - cut[i] + 2 * page - 2) // page for i in range(seqs)]
        pages = sum(need) + 3
        free = list(range(pages))
        rng.shuffle(free)
        positions, slots = [], []
        for i in range(seqs):
            start = rng.randrange(case["far"]) if case["far"] else 0
            mine = [free.pop() for _ in range(need[i])]
            for t in range(cut[i + 1] - cut[i]):
                at = start % page + t
                positions.append(start + t)
                slots.append(mine[at // page] * page + at % page)
        slots[tokens - case["pad"]:] = [-1] * case["pad"]
        s["positions"] = torch.tensor(positions, dtype=torch.int32, device=DEV)
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device=DEV)
        s["cache"] = _cache_arrays(case, pages, gen)
        s["q_out"] = torch.empty((tokens, hq, d), device=DEV, dtype=torch.float16)
        s["k_out"] = torch.empty((tokens, hkv, d), device=DEV, dtype=torch.float16)
        s["v_out"] = torch.empty((tokens, hkv, d), device=DEV, dtype=torch.float16)
    elif op == "cache":
        lens, page, q_len = _lengths(case), case["page"], case["q_len"]
        width = -(-max(max(lens), 1) // page)
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 2
        free = list(range(pages))
        rng.shuffle(free)
        table = [[free.pop() for _ in range(k)] + [-1] * (width - k) for k in need]
        s["table"] = torch.tensor(table, dtype=torch.int32, device=DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["max_len"] = max(lens)
        s["cache"] = _cache_arrays(case, pages, gen)
        s["q"] = normal(len(lens) * q_len, hq, d, dtype=torch.float16)
        s["out"] = torch.zeros((len(lens) * q_len, hq, d), device=DEV, dtype=torch.float16)
    else:
        offsets = [0]
        for x in _lengths(case):
            offsets.append(offsets[-1] + x)
        tokens = offsets[-1] + case["tail"]
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        s["q"] = normal(tokens, hq, d, dtype=torch.float16)
        s["k"] = normal(tokens, hkv, d, dtype=torch.float16)
        s["v"] = normal(tokens, hkv, d, dtype=torch.float16)
        s["out"] = torch.zeros((tokens, hq, d), device=DEV, dtype=torch.float16)
    if own and op in ("append", "cache"):
        import gemm_qmm_gemv_amd as qmm

        c = s["cache"]
        s["handle"] = qmm.KvCache(c["k"], c["ks"], c["km"], c["v"], c["vs"], c["vm"], c["k"].shape[0], hkv, d, case["page"], case["bits"], case["group"])
    if own and op == "cache":
        import gemm_qmm_gemv_amd as qmm

        need = qmm.qmm_attn_cache_workspace_bytes(s["handle"], len(lens), q_len, hq, s["max_len"])
        s["workspace"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- the library's calls


def _own(s):
    import gemm_qmm_gemv_amd as qmm

    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, gate = s["y"], s["gate"]
        qmm.qmm_norm_residual(y, case["y16"], case["n"], s["post"], gate, 0 if gate is None or gate.shape[0] < case["rows"] else case["n"],
                              s["scale"], s["residual"], s["h"] if y is not None else None, s["pre"], s["x"], case["rows"], case["n"], EPS)
        return {"h": s["h"], "x": s["x"]} if y is not None else {"x": s["x"]}
    if op == "append":
        q, k, v = s["q"], s["k"], s["v"]
        qmm.qmm_kv_append(s["handle"], q, k, v, case["in16"], q.stride(0), k.stride(0), v.stride(0), s["q_norm"], s["k_norm"], EPS,
                          s["inv_freq"], case["rot"], case["inter"], s["positions"], s["slots"], s["q_out"], s["k_out"], s["v_out"], True,
                          case["tokens"], case["hq"])
        return _appended(s)
    if op == "cache":
        table = s["table"]
        qmm.qmm_attn_cache(s["handle"], s["q"], table, table.shape[1], s["lens"], s["max_len"], s["out"], table.shape[0], case["q_len"],
                           case["hq"], case["d"] ** -0.5, s["workspace"], s["workspace"].numel())
        return s["out"]
    q, k, v = s["q"], s["k"], s["v"]
    qmm.qmm_attn_prompt(q, k, v, s["offsets"], s["out"], q.shape[0], s["offsets"].shape[0] - 1, case["hq"], case["hkv"], case["d"],
                        q.stride(0), k.stride(0), v.stride(0), s["out"].stride(0), case["d"] ** -0.5)
    return s["out"]


def _appended(s):
    """What an append leaves behind: fp16 queries, the keys and values that the cache stands for, its scales and mins (fp16: the rows)."""
    c = s["cache"]
    out = {k: s[k] for k in ("q_out", "k_out", "v_out")}
    if s["case"]["bits"] == 16:
        return out | {k: c[k].view(torch.float16) for k in "kv"}
    return out | {k: c[k] for k in ("ks", "km", "vs", "vm")}


# ---------------------------------------------------------------- the plain forms


def _rms(x, w):
    r = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return r if w is None else r * w


def _rotate(x, cos, sin, rot, inter):
    a, rest = x[..., :rot], x[..., rot:]
    if inter:
        lo, hi = a[..., 0::2], a[..., 1::2]
        return torch.cat([torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2), rest], -1)
    lo, hi = a[..., :rot // 2], a[..., rot // 2:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, rest], -1)


def _quantize(x, bits, group):
    """(codes, fp16 scales, fp16 mins, the fp16 values they stand for) of rows in groups along the last axis."""
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.half()
    sc = ((hi - lo) / (2 ** bits - 1)).half()
    mf, sf = m.to(x.dtype).unsqueeze(-1), sc.to(x.dtype).unsqueeze(-1)
    codes = torch.where(sf > 0, torch.round((g - mf) / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(g)).clamp(0, 2 ** bits - 1)
    return codes.flatten(-2), sc, m, (codes * sf + mf).flatten(-2).half()


def _pack(codes, bits):
    per = 32 // bits
    c = codes.to(torch.int64).unflatten(-1, (-1, per))
    w = (c << (bits * torch.arange(per, device=c.device))).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _unpack(words, bits):
    shifts = bits * torch.arange(32 // bits, device=words.device, dtype=torch.int32)
    return ((words.unsqueeze(-1) >> shifts) & (2 ** bits - 1)).flatten(-2)


def _plain_norm(s):
    case = s["case"]
    h = s["residual"]
    if s["y"] is not None:
        u = s["y"].float()
        if s["post"] is not None:
            u = _rms(u, s["post"])
        if s["gate"] is not None:
            u = u * s["gate"]
        h = h + s["scale"] * u
    x = _rms(h, s["pre"]).half()
    return {"h": h, "x": x} if case["y"] else {"x": x}


def _plain_append(s):
    case, c = s["case"], s["cache"]
    hq, hkv, d, bits, page = case["hq"], case["hkv"], case["d"], case["bits"], case["page"]
    ang = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q, k, v = s["q"].float().unflatten(-1, (hq, d)), s["k"].float().unflatten(-1, (hkv, d)), s["v"].float().unflatten(-1, (hkv, d))
    if case["qknorm"]:
        q, k = _rms(q, s["q_norm"]), _rms(k, s["k_norm"])
    q, k = (_rotate(x, cos, sin, case["rot"], case["inter"]) for x in (q, k))
    s["q_out"] = q.half()
    keep = s["slots"] >= 0
    at, off = (s["slots"][keep] // page)[:, None], (s["slots"][keep] % page)[:, None]
    head = torch.arange(hkv, device=DEV)
    for side, x in (("k", k), ("v", v)):
        if bits == 16:
            s[side + "_out"] = x.half()
            c[side].view(torch.float16)[at, head, off] = x.half()[keep]
            continue
        codes, sc, m, values = _quantize(x, bits, case["group"])
        s[side + "_out"] = values
        c[side][at, head, off] = _pack(codes, bits)[keep]
        grp = torch.arange(d // case["group"], device=DEV)
        c[side + "s"][at[..., None], head[:, None], grp, off[..., None]] = sc[keep]
        c[side + "m"][at[..., None], head[:, None], grp, off[..., None]] = m[keep]
    return _appended(s)


def _rows(s, side):
    """fp32 rows [sequences][kv heads][positions][d] of one side of the cache, through the page table."""
    case, c = s["case"], s["cache"]
    at = s["table"].clamp(min=0).long()
    w = c[side][at].transpose(1, 2).flatten(2, 3)
    if case["bits"] == 16:
        return w.view(torch.float16).float()
    codes = _unpack(w, case["bits"]).float().unflatten(-1, (-1, case["group"]))
    sc, m = (c[side + x][at].permute(0, 2, 1, 4, 3).flatten(2, 3).float().unsqueeze(-1) for x in "sm")
    return codes.mul_(sc).add_(m).flatten(-2)


def _softmax_rows(scores, visible):
    """exp and its sum over the visible places; a row that sees nothing sums to zero and stays zero."""
    scores = scores.masked_fill(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e, e.sum(-1, keepdim=True)


def _plain_cache(s):
    case = s["case"]
    hq, hkv, d, q_len = case["hq"], case["hkv"], case["d"], case["q_len"]
    n, g = s["table"].shape[0], hq // hkv
    k, v = _rows(s, "k"), _rows(s, "v")
    at = torch.arange(k.shape[2], device=DEV)
    q = s["q"].float().view(n, q_len, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, q_len * g, d)
    sees = s["lens"][:, None] - q_len + 1 + torch.arange(q_len, device=DEV)
    visible = (at < sees[..., None]).repeat_interleave(g, 1)[:, None]
    v = v * (at < s["lens"][:, None])[:, None, :, None]
    e, total = _softmax_rows(torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, visible)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(n, hkv, q_len, g, d).permute(0, 2, 1, 3, 4).reshape(n * q_len, hq, d).half()


def _plain_prompt(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    tokens, g = s["q"].shape[0], hq // hkv
    at = torch.arange(tokens, device=DEV, dtype=torch.int32)
    mine = torch.searchsorted(s["offsets"], at, right=True)
    covered = at < s["offsets"][-1]
    visible = (mine[:, None] == mine) & (at[:, None] >= at) & covered[:, None]
    q = s["q"].float().view(tokens, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * tokens, d)
    k, v = s["k"].float().transpose(0, 1), s["v"].float().transpose(0, 1)
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(hkv, g, tokens, tokens)
    e, total = _softmax_rows(scores, visible)
    o = torch.matmul(e.view(hkv, g * tokens, tokens), v).view(hkv, g, tokens, d) / torch.where(total > 0, total, torch.ones_like(total))
    return torch.where(covered[:, None, None], o.permute(2, 0, 1, 3).reshape(tokens, hq, d).half(), s["out"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "append": _plain_append, "cache": _plain_cache, "prompt": _plain_prompt}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "norm":
        rows, n = case["rows"], case["n"]
        b = rows * n * (4 + 2) + 4 * n
        f = rows * n * 4
        if case["y"]:
            b += rows * n * ((2 if case["y16"] else 4) + 4)
            f += rows * n * 3
            if case["post"]:
                b, f = b + 4 * n, f + rows * n * 4
            if case["gate"] != "none":
                b, f = b + 4 * n * (rows if case["gate"] == "rows" else 1), f + rows * n
        return {"bytes": b, "flops": f}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "append":
        t, size = case["tokens"], 2 if case["in16"] else 4
        kept = t - case["pad"]
        row = _held_row(d, case["bits"], case["group"])
        b = t * (hq + 2 * hkv) * d * (size + 2) + kept * 2 * hkv * row + 12 * t
        return {"bytes": b, "flops": t * (hq + 2 * hkv) * d * 8}
    if op == "cache":
        lens, q_len = _lengths(case), case["q_len"]
        row = _held_row(d, case["bits"], case["group"])
        b = sum(lens) * 2 * hkv * row + 2 * len(lens) * q_len * hq * d * 2
        pairs = sum(max(0, x - q_len + 1 + i) for x in lens for i in range(q_len))
        return {"bytes": b, "flops": pairs * hq * d * 4}
    lens = _lengths(case)
    return {"bytes": sum(lens) * (2 * hq + 2 * hkv) * d * 2, "flops": sum(x * (x + 1) // 2 for x in lens) * hq * d * 4}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_attend(q, k, v, first):
    """Row i of q [rows][heads][d] sees the first ``first + i`` rows of k and v [positions][kv heads][d]."""
    rows, hq, d = q.shape
    out = torch.zeros_like(q)
    g = hq // k.shape[1]
    span = 2048
    for b in range(0, rows, span):
        e = min(rows, b + span)
        n = max(0, min(k.shape[0], first + e - 1))
        if n == 0:
            continue
        dark = torch.arange(n, device=q.device)[None, :] >= (first + torch.arange(b, e, device=q.device))[:, None]
        for h in range(hq):
            w = (q[b:e, h] @ k[:n, h // g].T) / math.sqrt(d)
            w = torch.softmax(w.masked_fill(dark, -math.inf), -1)
            w = w.masked_fill(dark, 0.0)
            out[b:e, h] = w @ v[:n, h // g]
    return out


def _exact_held(x, bits, group):
    """(values, scales, mins) that rows of x are held as: scale and min rounded to fp16, codes to whole numbers."""
    if bits == 16:
        return x, None, None
    top = 2.0 ** bits - 1
    parts = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    low = parts.min(-1).values
    step = ((parts.max(-1).values - low) / top).to(torch.float16).double()
    low = low.to(torch.float16).double()
    codes = torch.round((parts - low[..., None]) / step[..., None]).nan_to_num(0.0).clamp(0.0, top)
    return (low[..., None] + codes * step[..., None]).reshape(x.shape), step, low


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        def unit(x):
            return x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / case["n"] + EPS)
        h = s["residual"].double()
        if case["y"]:
            u = s["y"].double()
            if s["post"] is not None:
                u = unit(u) * s["post"].double()
            if s["gate"] is not None:
                u = u * s["gate"].double()
            h = h + s["scale"] * u
        x = unit(h) * s["pre"].double()
        return {"h": h, "x": x} if case["y"] else {"x": x}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "append":
        t, rot, page, group, bits = case["tokens"], case["rot"], case["page"], case["group"], case["bits"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["positions"].double()[:, None, None] * s["inv_freq"].double())

        def place(x, heads, weight, turned):
            x = x.double().reshape(t, heads, d)
            if weight is not None and turned:
                x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / d + EPS) * weight.double()
            if not turned:
                return x
            x = x.clone()
            one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * turn
            x[..., one], x[..., two] = z.real, z.imag
            return x
        out = {"q_out": place(s["q"], hq, s["q_norm"], True)}
        state = {}
        for side in "kv":
            held, step, low = _exact_held(place(s[side], hkv, s["k_norm"], side == "k"), bits, group)
            out[side + "_out"] = held
            kept = [(i, x) for i, x in enumerate(s["slots"].tolist()) if x >= 0]
            i = torch.tensor([a for a, _ in kept], dtype=torch.int64, device=DEV)
            x = torch.tensor([b for _, b in kept], dtype=torch.int64, device=DEV)
            if bits == 16:
                arrays = {side: (s["cache"][side].view(torch.float16).double(), held)}
                for name, (a, new) in arrays.items():
                    a.transpose(1, 2)[x // page, x % page] = new[i]
                    state[name] = a
            else:
                for name, new in ((side + "s", step), (side + "m", low)):
                    a = s["cache"][name].double()
                    a.permute(0, 3, 1, 2)[x // page, x % page] = new[i]
                    state[name] = a
        return out | state
    if op == "cache":
        page, bits, group, q_len = case["page"], case["bits"], case["group"], case["q_len"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for i, n in enumerate(_lengths(case)):
            if n == 0:
                continue
            at = s["table"][i, :-(-n // page)].long()
            sides = []
            for side in "kv":
                w = s["cache"][side][at]
                if bits == 16:
                    x = w.view(torch.float16).double()
                else:
                    raw = w.contiguous().view(torch.uint8)
                    codes = raw if bits == 8 else torch.stack([raw % 16, raw // 16], -1).flatten(-2)
                    step, low = (s["cache"][side + e][at].double().transpose(-1, -2).repeat_interleave(group, -1) for e in "sm")
                    x = codes.double() * step + low
                sides.append(x.transpose(1, 2).reshape(-1, hkv, d)[:n])
            out[i * q_len:(i + 1) * q_len] = _exact_attend(s["q"][i * q_len:(i + 1) * q_len].double(), sides[0], sides[1], n - q_len + 1)
        return out
    out = s["out"].double()
    ends = s["offsets"].tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        out[a:b] = _exact_attend(s["q"][a:b].double(), s["k"][a:b].double(), s["v"][a:b].double(), 1)
    return out
