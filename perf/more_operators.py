"""A mixture-of-experts block around 8-bit integer products: what it costs next to the products of packed weights.

Four operators:

  route    a token's scores for the experts to its few experts, their weights, and the rows grouped by expert that the
           experts' products take: softmax or sigmoid scores, a bias that only the choice sees, experts in groups
  product  rows to 8-bit codes with a scale for each token, times 8-bit weights with a scale for each channel
  experts  the same over rows grouped by expert: gate and up products with silu(gate) * up on top, or a plain product
  gather   the experts' rows back to their tokens, times the weights, onto the residual stream

``run`` computes them in plain torch operations (32 bits, one rounding at the end; 64 bits where a choice or a code
hangs on the last of them), or through the library where ``own`` is set.  ``exact`` computes the same from the
definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One token of a model with 128 experts: the least there is to decide.  Latency.
        dict(name="route_one_token", op="route", tokens=1, experts=128, top_k=8, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=True, scale=1.0, f16=False, pad=0),
        # A decode batch of a model whose experts stand in groups, balanced by a bias.
        dict(name="route_batch_groups", op="route", tokens=37, experts=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             best=2, renorm=True, scale=2.5, f16=False, pad=0),
        # A middling batch padded to its captured size, an odd number of experts, fp16 scores, weights as they are.
        dict(name="route_padded", op="route", tokens=515, experts=60, top_k=4, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=False, scale=1.0, f16=True, pad=35),
        # A long prefill of the model of the first case.
        dict(name="route_prefill", op="route", tokens=16384, experts=128, top_k=8, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=True, scale=1.0, f16=False, pad=0),
        # One token through a projection of a small model: latency, then the bytes of the weights.
        dict(name="product_one_token", op="product", m=1, n=2048, k=1024, x16=True, y16=False),
        # An odd decode batch through the up projection of a 1B-class model: bound by the weights' bytes.
        dict(name="product_batch", op="product", m=37, n=8192, k=2048, x16=False, y16=False),
        # A long prefill through gate and up as one matrix: bound by the matrix cores.
        dict(name="product_prefill", op="product", m=8192, n=16384, k=2048, x16=True, y16=True),
        # A decode batch of 16 tokens through the experts' gate and up: most of the experts' weights for a row or two each.
        dict(name="experts_decode", op="experts", glu=True, tokens=16, experts=128, top_k=8, n=768, k=2048, x16=True, y16=True),
        # A prefill through the same.
        dict(name="experts_prefill", op="experts", glu=True, tokens=4096, experts=128, top_k=8, n=768, k=2048, x16=True, y16=True),
        # Its down projection: a row of its own for every token and expert.
        dict(name="experts_prefill_down", op="experts", glu=False, tokens=4096, experts=128, top_k=8, n=2048, k=768, x16=True, y16=False),
        # The decode batch's rows back to their tokens: latency.
        dict(name="gather_decode", op="gather", tokens=16, top_k=8, n=2048, f16=False, residual=True, pad=0),
        # A prefill's: bound by memory.
        dict(name="gather_prefill", op="gather", tokens=8192, top_k=8, n=2048, f16=True, residual=True, pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "product", "experts", "gather"])
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        groups = rng.choice([1, 1, 4, 8] if experts % 8 == 0 and experts >= 64 else [1])
        top_groups = groups if groups == 1 else rng.randint(2, groups)
        top_k = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts // groups * top_groups])
        tokens = _log(rng, 1, 16384 * 128 // max(experts, 128))
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, top_groups=top_groups, best=rng.choice([1, 2]), renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    f16=rng.random() < 0.3, pad=rng.choice([0, 0, min(tokens - 1, 5)]))
    if op == "product":
        n, k = rng.choice([512, 768, 1000, 1024, 2048, 4099, 8192, 16384]), rng.choice([512, 768, 1024, 1056, 2048, 4096, 8192])
        return dict(op=op, m=_log(rng, 1, min(8192, 8192 * 16384 * 2048 // (2 * n * k))), n=n, k=k, x16=rng.random() < 0.6, y16=rng.random() < 0.5)
    if op == "experts":
        experts = rng.choice([8, 16, 60, 128])
        top_k = rng.choice([1, 2, 4, 8])
        glu = rng.random() < 0.6
        n, k = rng.choice([(768, 2048), (1408, 2048), (512, 1024), (2048, 768), (1001, 1056)])
        return dict(op=op, glu=glu, tokens=_log(rng, 1, 4096 * 768 * 2048 // max(n * k, 768 * 2048)), experts=experts, top_k=top_k, n=n, k=k,
                    x16=rng.random() < 0.6, y16=rng.random() < 0.6)
    n = rng.choice([1001, 1024, 2048, 2880, 4096])
    tokens = _log(rng, 1, 8192 * 2048 // max(n, 2048) // 2)
    return dict(op=op, tokens=tokens, top_k=rng.choice([1, 2, 4, 6, 8]), n=n, f16=rng.random() < 0.5, residual=rng.random() < 0.6,
                pad=rng.choice([0, 0, min(tokens - 1, 5)]))


# ---------------------------------------------------------------- inputs


def _grouped(ids, experts):
    """Rows grouped by expert, within an expert by token, of the experts `ids` [tokens][top_k] (-1: none):
    (offsets, each row's token, each row's place in `ids`), int64."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets, order // ids.shape[1], order


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, device=DEV, generator=gen).to(dtype)

    def codes(*shape):
        # Normal weights whose largest of a channel, 3.5 deviations away, is 127.
        out = torch.empty(shape, dtype=torch.int8, device=DEV)
        for part in out.view(-1, shape[-1]).split(1 << 16):
            part.copy_(normal(*part.shape).mul_(36).round_().clamp_(-127, 127))
        return out

    def keep(tokens, pad):
        mask = torch.ones(tokens, dtype=torch.uint8, device=DEV)
        mask[tokens - pad:] = 0
        return mask if pad else None

    if op == "route":
        tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
        # Scores with a few popular experts.
        s["logits"] = (1.2 * normal(tokens, experts) + 0.5 * normal(experts)).to(torch.float16 if case["f16"] else torch.float32)
        s["bias"] = 0.1 * normal(experts) if case["bias"] else None
        s["keep"] = keep(tokens, case["pad"])
        s["ids"] = torch.full((tokens, top_k), -1, dtype=torch.int32, device=DEV)
        s["weights"] = torch.zeros((tokens, top_k), device=DEV)
        s["pair_row"] = torch.full((tokens, top_k), -1, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
        s["pair_token"] = torch.zeros(tokens * top_k, dtype=torch.int32, device=DEV)
        s["pair_weight"] = torch.zeros(tokens * top_k, device=DEV)
        if own:
            import gemm_qmm_gemv_amd as qmm

            s["workspace"] = torch.empty(max(16, qmm.qmm_moe_route_workspace_bytes(tokens, experts, top_k)), dtype=torch.uint8, device=DEV)
        return s
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = normal(m, k, dtype=torch.float16 if case["x16"] else torch.float32)
        s["w"], s["ws"] = codes(n, k), (1 + 0.2 * torch.rand(n, device=DEV, generator=gen)) * 1e-3
        rows, width = m, n
    elif op == "experts":
        tokens, experts, top_k, n, k = (case[x] for x in ("tokens", "experts", "top_k", "n", "k"))
        ids = torch.topk(normal(tokens, experts) + 0.5 * normal(experts), top_k, dim=1).indices.int()
        offsets, token, _ = _grouped(ids, experts)
        rows, width = tokens * top_k, n
        s["offsets"], s["rows_of"] = offsets.int(), token.int() if case["glu"] else None
        s["ends"] = offsets.tolist()  # what the plain form cuts its rows by
        m = tokens if case["glu"] else rows
        s["x"] = normal(m, k, dtype=torch.float16 if case["x16"] else torch.float32)
        for name in ("w", "w2") if case["glu"] else ("w",):
            s[name], s[name + "s"] = codes(experts, n, k), (1 + 0.2 * torch.rand((experts, n), device=DEV, generator=gen)) * 1e-3
    else:
        tokens, top_k, n = case["tokens"], case["top_k"], case["n"]
        kept = tokens - case["pad"]
        s["rows"] = normal(tokens * top_k, n, dtype=torch.float16 if case["f16"] else torch.float32)
        # Where a grouping by random experts puts the pairs; the padding has none.
        place = torch.argsort(torch.rand(kept * top_k, device=DEV, generator=gen)).int().view(kept, top_k)
        s["pair_row"] = torch.full((tokens, top_k), -1, dtype=torch.int32, device=DEV)
        s["pair_row"][:kept] = place
        s["weights"] = torch.softmax(normal(tokens, top_k), 1)
        s["residual"] = 3 * normal(tokens, n) if case["residual"] else None
        s["y"] = torch.empty((tokens, n), device=DEV)
        return s
    s["codes"] = torch.empty((m, k), dtype=torch.int8, device=DEV)
    s["xs"] = torch.empty(m, device=DEV)
    s["y"] = torch.empty((rows, width), dtype=torch.float16 if case["y16"] else torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- the library's calls


def _own(s):
    import gemm_qmm_gemv_amd as qmm

    case = s["case"]
    op = case["op"]
    if op == "route":
        logits, ws = s["logits"], s["workspace"]
        qmm.qmm_moe_route(logits, case["f16"], logits.stride(0), s["bias"], case["score"] == "sigmoid", case["groups"], case["top_groups"],
                          case["best"], case["top_k"], case["renorm"], case["scale"], s["keep"], s["ids"], s["weights"], s["pair_row"],
                          s["offsets"], s["pair_token"], s["pair_weight"], ws, ws.numel(), case["tokens"], case["experts"])
        return {k: s[k] for k in ("ids", "weights", "pair_row", "offsets", "pair_token", "pair_weight")}
    if op == "gather":
        qmm.qmm_moe_gather(s["rows"], case["f16"], s["pair_row"], s["weights"], s["residual"], s["y"], case["tokens"], case["top_k"],
                           s["rows"].shape[0], case["n"])
        return s["y"]
    x = s["x"]
    m, k = x.shape
    qmm.qmm_quantize_rows(x, case["x16"], x.stride(0), s["codes"], s["xs"], m, k)
    if op == "product":
        qmm.qmm_gemm_i8(s["w"], s["ws"], s["codes"], s["xs"], s["y"], case["y16"], m, case["n"], k)
        return s["y"]
    rows = s["y"].shape[0]
    if case["glu"]:
        qmm.qmm_moe_swiglu_i8(s["w"], s["ws"], s["w2"], s["w2s"], s["codes"], s["xs"], s["rows_of"], m, s["offsets"], s["y"], case["y16"],
                              rows, case["experts"], case["n"], k)
    else:
        qmm.qmm_moe_gemm_i8(s["w"], s["ws"], s["codes"], s["xs"], s["rows_of"], m, s["offsets"], s["y"], case["y16"], rows, case["experts"],
                            case["n"], k)
    return s["y"]


# ---------------------------------------------------------------- the plain forms


def _plain_route(s):
    case = s["case"]
    tokens, experts, top_k, groups = case["tokens"], case["experts"], case["top_k"], case["groups"]
    l = s["logits"].double()  # a choice hangs on the last bits
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1)
    choice = p if s["bias"] is None else p + s["bias"]
    if s["bias"] is None:
        # The scores' order is the logits', which never run together.
        order = l
    else:
        order = choice
    if groups > 1:
        per = (order if case["best"] == 1 else choice).view(tokens, groups, -1)
        top = torch.sort(per, -1, descending=True).values[..., :case["best"]].sum(-1)
        best = torch.sort(top, dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        inside = torch.zeros((tokens, groups), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        order = order.masked_fill(~inside.repeat_interleave(experts // groups, 1), -math.inf)
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :top_k]
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w, ids = (w * case["scale"]).float(), ids.int()
    if s["keep"] is not None:
        off = s["keep"][:, None] == 0
        w, ids = w.masked_fill(off, 0.0), ids.masked_fill(off, -1)
    offsets, token, pair = _grouped(ids, experts)
    # Rows behind the last expert's stay as they were.
    row = torch.arange(tokens * top_k, device=DEV)
    used = row < offsets[-1]
    pair_row = torch.empty_like(row)
    pair_row[pair] = torch.where(used, row, -1)
    return {"ids": ids, "weights": w, "pair_row": pair_row.int().view(tokens, top_k), "offsets": offsets.int(),
            "pair_token": torch.where(used, token.int(), s["pair_token"]), "pair_weight": torch.where(used, w.flatten()[pair], s["pair_weight"])}


def _codes(x):
    """Codes (as fp32 numbers) and the scale of each row: the quotient in 64 bits, where next to a border 32 decide wrongly."""
    x = x.double()
    scale = (x.abs().amax(-1, keepdim=True) / 127).float()
    q = torch.round(x / torch.where(scale > 0, scale, 1.0).double())
    return q.float(), scale


def _plain_experts(s):
    case = s["case"]
    q, scale = _codes(s["x"])
    if s["rows_of"] is not None:
        at = s["rows_of"].long()
        q, scale = q[at], scale[at]
    y = torch.empty_like(s["y"])
    for e, (a, b) in enumerate(zip(s["ends"][:-1], s["ends"][1:])):
        if a == b:
            continue
        u = torch.matmul(q[a:b], s["w"][e].float().T) * scale[a:b] * s["ws"][e]
        if case["glu"]:
            u = u * torch.sigmoid(u) * (torch.matmul(q[a:b], s["w2"][e].float().T) * scale[a:b] * s["w2s"][e])
        y[a:b] = u
    return y


def _plain_gather(s):
    at = s["pair_row"].long()
    w = torch.where(at < 0, 0.0, s["weights"])
    y = (s["rows"].float()[at.clamp(min=0)] * w[..., None]).sum(1)
    return y if s["residual"] is None else s["residual"] + y


def run(state):
    if own:
        return _own(state)
    op, case = state["case"]["op"], state["case"]
    if op == "product":
        q, scale = _codes(state["x"])
        return (torch.matmul(q, state["w"].float().T) * scale * state["ws"]).to(torch.float16 if case["y16"] else torch.float32)
    return {"route": _plain_route, "experts": _plain_experts, "gather": _plain_gather}[op](state)


# ---------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        kept = t - case["pad"]
        return {"bytes": kept * e * (2 if case["f16"] else 4) + t * k * 12 + kept * k * 8 + 4 * (e + 1), "flops": kept * e * (4 + k)}
    if op == "gather":
        t, k, n = case["tokens"], case["top_k"], case["n"]
        kept = t - case["pad"]
        return {"bytes": kept * k * n * (2 if case["f16"] else 4) + t * n * (8 if case["residual"] else 4) + t * k * 8, "flops": 2 * kept * k * n}
    n, k = case["n"], case["k"]
    xb, yb = 2 if case["x16"] else 4, 2 if case["y16"] else 4
    if op == "product":
        m = case["m"]
        return {"bytes": m * k * xb + n * k + 4 * n + m * n * yb, "flops": 2 * m * n * k}
    rows = case["tokens"] * case["top_k"]
    mats = 2 if case["glu"] else 1
    # Experts that a row is likely to meet: what has to be read of the weights.
    hit = case["experts"] * (1 - (1 - case["top_k"] / case["experts"]) ** case["tokens"])
    x = (case["tokens"] if case["glu"] else rows) * k * xb
    return {"bytes": int(x + hit * mats * (n * k + 4 * n) + rows * n * yb), "flops": 2 * rows * n * k * mats}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_route(s):
    case = s["case"]
    tokens, experts, top_k, groups = case["tokens"], case["experts"], case["top_k"], case["groups"]
    l = s["logits"].double()
    p = 1 / (1 + torch.exp(-l)) if case["score"] == "sigmoid" else torch.exp(l) / torch.exp(l).sum(1, keepdim=True)
    biased = s["bias"] is not None
    c = p + s["bias"].double() if biased else p
    rank = c if biased else l
    each = experts // groups
    allowed = torch.zeros((tokens, experts), dtype=torch.bool, device=DEV)
    scores = []
    for g in range(groups):
        part = (rank if case["best"] == 1 else c)[:, g * each:(g + 1) * each]
        scores.append(part.topk(min(case["best"], each), 1).values.sum(1))
    left = torch.stack(scores, 1)
    row = torch.arange(tokens, device=DEV)
    for _ in range(case["top_groups"]):
        g = (left == left.max(1, keepdim=True).values).byte().argmax(1)  # the first of equals
        left[row, g] = -math.inf
        for j in range(each):
            allowed[row, g * each + j] = True
    left = rank.masked_fill(~allowed, -math.inf)
    ids, weights = [], []
    for _ in range(top_k):
        e = (left == left.max(1, keepdim=True).values).byte().argmax(1)
        left[row, e] = -math.inf
        ids.append(e)
        weights.append(p[row, e])
    ids, weights = torch.stack(ids, 1), torch.stack(weights, 1)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = weights * case["scale"]
    kept = tokens - case["pad"]
    ids[kept:], weights[kept:] = -1, 0
    chosen = ids.tolist()
    host = weights.tolist()
    lists = [[] for _ in range(experts)]
    for t in range(kept):
        for j, e in enumerate(chosen[t]):
            lists[e].append((t, j))
    offsets, token, weight = [0], s["pair_token"].tolist(), s["pair_weight"].double().tolist()
    pair_row = [[-1] * top_k for _ in range(tokens)]
    for mine in lists:
        for i, (t, j) in enumerate(mine):
            at = offsets[-1] + i
            token[at], weight[at], pair_row[t][j] = t, host[t][j], at
        offsets.append(offsets[-1] + len(mine))

    def whole(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    return {"ids": ids.int(), "weights": weights, "pair_row": whole(pair_row), "offsets": whole(offsets), "pair_token": whole(token),
            "pair_weight": torch.tensor(weight, dtype=torch.float64, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "gather":
        y = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device=DEV)
        if s["residual"] is not None:
            y += s["residual"]
        kept = case["tokens"] - case["pad"]
        for j in range(case["top_k"]):
            y[:kept] += s["weights"][:kept, j, None].double() * s["rows"].index_select(0, s["pair_row"][:kept, j]).double()
        return y
    # A scale is held in 32 bits; the codes are whole numbers from there on.
    x = s["x"].double()
    unit = (x.abs().max(1).values / 127.0).float().double().unsqueeze(1)
    held = (x / unit).round() * unit
    if op == "product":
        w = s["w"].double() * s["ws"].double().unsqueeze(1)
        return held @ w.t()
    if s["rows_of"] is not None:
        held = held.index_select(0, s["rows_of"])
    out = []
    for e in range(case["experts"]):
        rows = held[s["ends"][e]:s["ends"][e + 1]]
        y = rows @ (s["w"][e].double() * s["ws"][e].double().unsqueeze(1)).t()
        if case["glu"]:
            y = y / (1 + torch.exp(-y)) * (rows @ (s["w2"][e].double() * s["w2s"][e].double().unsqueeze(1)).t())
        out.append(y)
    return torch.cat(out)
