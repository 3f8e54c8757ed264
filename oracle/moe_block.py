"""CPU oracle of a mixture of experts' feed-forward block: routing, 8-bit
integer products and the gather of the experts' rows.  Plain definitions in
numpy float64 and whole numbers, one loop per thing that the definition names;
test infrastructure only, and no code shared with the library.
"""
from __future__ import annotations

import math

import numpy as np


def sigmoid(v):
    v = float(v)
    return 1.0 / (1.0 + math.exp(-v)) if v >= 0 else math.exp(v) / (1.0 + math.exp(v))


def scores(row, kind):
    """Scores of one token's logits (float64), NaN logits placed as -inf."""
    l = [-math.inf if math.isnan(v) else float(v) for v in row]
    if kind == "sigmoid":
        return [0.0 if v == -math.inf else 1.0 if v == math.inf else sigmoid(v) for v in l]
    top = max(l)
    if top == -math.inf:
        return [0.0] * len(l)
    e = [1.0 if v == top else math.exp(v - top) if top < math.inf else 0.0 for v in l]
    return [v / math.fsum(e) for v in e]


def route_token(row, kind, bias, n_groups, top_groups, group_best, top_k, renormalize, scale):
    """(experts, weights) of one token."""
    n = len(row)
    l = [-math.inf if math.isnan(v) else float(v) for v in row]
    s = scores(row, kind)
    c = s if bias is None else [a + float(b) for a, b in zip(s, bias)]
    c = [-math.inf if math.isnan(v) else v for v in c]
    rank = l if bias is None else c  # the same order, and nothing runs together
    each = n // n_groups
    if n_groups > 1:
        marks = []
        for g in range(n_groups):
            mine = range(g * each, (g + 1) * each)
            if group_best == 1:
                marks.append(max(rank[e] for e in mine))
            else:
                two = sorted((c[e] for e in mine), reverse=True)[:2]
                total = two[0] + two[1]
                marks.append(-math.inf if math.isnan(total) else total)
        stay = sorted(range(n_groups), key=lambda g: (-marks[g], g))[:top_groups]
    else:
        stay = [0]
    left = [e for e in range(n) if e // each in stay]
    ids = sorted(left, key=lambda e: (-rank[e], e))[:top_k]
    w = [s[e] for e in ids]
    if renormalize:
        if kind == "sigmoid":
            # Ratios, also where the scores themselves vanish.
            top = max(l[e] for e in ids)
            shift = min(top, 0.0)
            if top == -math.inf:
                w = [0.0] * top_k
            else:
                w = [0.0 if l[e] == -math.inf else math.exp(l[e] - shift) / (1.0 + math.exp(l[e])) if l[e] <= 0 else s[e]
                     for e in ids]
        else:
            top = max(l[e] for e in ids)
            w = [0.0 if l[e] == -math.inf else 1.0 if l[e] == top else math.exp(l[e] - top) for e in ids]
        total = math.fsum(w)
        w = [v / total if total > 0 else 0.0 for v in w]
    bad = any(math.isnan(v) for v in row) or (kind == "softmax" and max(l) == math.inf)
    return ids, [math.nan if bad else v * scale for v in w]


def route(logits, kind, bias, n_groups, top_groups, group_best, top_k, renormalize, scale, keep=None):
    """(ids, weights, pair_row, offsets, pair_token, pair_weight); pair arrays as long as there are rows."""
    tokens, n = logits.shape
    ids = np.full((tokens, top_k), -1, dtype=np.int64)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        if keep is not None and not keep[t]:
            continue
        ids[t], weights[t] = route_token(logits[t], kind, bias, n_groups, top_groups, group_best, top_k, renormalize, scale)
    offsets, token, weight = [0], [], []
    pair_row = np.full((tokens, top_k), -1, dtype=np.int64)
    for e in range(n):
        for t, j in zip(*np.nonzero(ids == e)):
            pair_row[t, j] = len(token)
            token.append(int(t))
            weight.append(weights[t, j])
        offsets.append(len(token))
    return ids, weights, pair_row, np.array(offsets), np.array(token, dtype=np.int64), np.array(weight)


def quantize_rows(x):
    """(codes int64, scales float32): the scale is held in 32 bits, the quotient taken in 64."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.int64)
    out = np.zeros(x.shape[0], dtype=np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            out[r] = np.nan
            continue
        out[r] = np.float32(np.abs(row).max() / 127.0)
        if out[r] > 0:
            codes[r] = np.clip(np.rint(row / float(out[r])), -127, 127)
    return codes, out


def product_i8(w, ws, x, xs):
    """float64 [rows][n]: exact whole-number sums times the scales."""
    sums = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T  # below 2^53: exact
    return sums * np.asarray(xs, dtype=np.float64)[:, None] * np.asarray(ws, dtype=np.float64)[None, :]


def moe_product_i8(w, ws, x, xs, x_rows, offsets, p_rows):
    """float64 [p_rows][n]; rows of no expert are None in the second result's mask."""
    n = w.shape[1]
    y, covered = np.zeros((p_rows, n)), np.zeros(p_rows, dtype=bool)
    for e in range(len(offsets) - 1):
        for p in range(max(0, offsets[e]), min(p_rows, offsets[e + 1])):
            r = p if x_rows is None else int(x_rows[p])
            covered[p] = True
            y[p] = product_i8(w[e], ws[e], x[r:r + 1], xs[r:r + 1])[0] if 0 <= r < len(x) else np.nan
    return y, covered


def silu(v):
    return np.array([a * sigmoid(a) for a in np.ravel(v)]).reshape(np.shape(v))


def gather(rows, pair_row, weights, residual):
    """(y, sum of magnitudes) in float64."""
    tokens, n = len(pair_row), rows.shape[1]
    y, a = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        for r, w in zip(pair_row[t], weights[t]):
            if 0 <= r < len(rows):
                y[t] += float(w) * rows[r].astype(np.float64)
                a[t] += abs(float(w)) * np.abs(rows[r].astype(np.float64))
        if residual is not None:
            y[t] += residual[t]
            a[t] += np.abs(residual[t])
    return y, a
