"""fp64 oracle of the routed half of the layer: routing to experts, the 8-bit block-scaled
product and the routed experts' SwiGLU (numpy; shares no code with the library).

The 8-bit form follows the format's definition: the scale a / 448, the factor
448 (1 / a) and the scaled value are fp32 numbers, and the stored value is the nearest e4m3 value, ties
to even.  Everything after that is fp64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = 448.0
TINY = 1e-30


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (3 mantissa bits, smallest exponent -6, largest value 448)."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    r = np.round(v / step) * step  # numpy rounds halves to even
    return np.clip(r, -TOP, TOP)


def quantize(x: np.ndarray, block_rows: int = 1):
    """e4m3 values (as fp64) and fp32 scales of x [rows, cols]."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    q = np.zeros((rows, cols))
    s = np.zeros((blocks(rows) if block_rows == BLOCK else rows, blocks(cols)), np.float32)
    for i in range(s.shape[0]):
        r = slice(i * block_rows, (i + 1) * block_rows)
        for b in range(s.shape[1]):
            c = slice(b * BLOCK, (b + 1) * BLOCK)
            a = np.maximum(np.abs(x[r, c]).max(), np.float32(TINY))
            s[i, b] = a / np.float32(TOP)
            q[r, c] = e4m3_round(x[r, c] * (np.float32(TOP) * (np.float32(1.0) / a)))
    return q, s


def dequantize(q: np.ndarray, s: np.ndarray, block_rows: int = 1) -> np.ndarray:
    full = np.repeat(np.repeat(np.asarray(s, np.float64), block_rows, 0), BLOCK, 1)
    return q * full[:q.shape[0], :q.shape[1]]


def linear(x64: np.ndarray, w64: np.ndarray):
    """x w^T and, per output, the sum of the absolute products."""
    return x64 @ w64.T, np.abs(x64) @ np.abs(w64).T


def route_choice(logits, score="sigmoid", bias=None):
    """Scores and choice values (fp64); NaN choices become -inf."""
    v = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-v))
            c = s
        else:
            m = v.max(axis=1, keepdims=True)
            p = np.exp(v - np.where(np.isneginf(m), 0.0, m))
            t = p.sum(axis=1, keepdims=True)
            s = np.where(t == 0, 0.0, p / np.where(t == 0, 1.0, t))
            c = v if bias is None else s
    if bias is not None:
        c = c + np.asarray(bias, np.float64)
    return s, np.where(np.isnan(c), -np.inf, c)


def _best(row, k):
    """Indices of the k largest, largest first, ties to the lower index."""
    return sorted(range(len(row)), key=lambda i: (-row[i], i))[:k]


def route(logits, topk, score="sigmoid", bias=None, groups=1, top_groups=None, group_top=1, renormalize=True,
          scale=1.0):
    """ids [T, topk] and weights [T, topk], one row at a time."""
    s, c = route_choice(logits, score, bias)
    T, E = s.shape
    per = E // groups
    top_groups = groups if top_groups is None else top_groups
    ids = np.zeros((T, topk), np.int64)
    w = np.zeros((T, topk))
    for t in range(T):
        rank = [sum(sorted(c[t, g * per:(g + 1) * per], reverse=True)[:group_top]) for g in range(groups)]
        stay = set(_best(rank, top_groups)) if groups > 1 else {0}
        open_ = [e for e in range(E) if e // per in stay]
        order = _best([c[t, e] for e in open_], topk)
        ids[t] = [open_[i] for i in order]
        w[t] = s[t, ids[t]]
        if renormalize:
            total = w[t].sum()
            w[t] = 0.0 if total == 0 else w[t] / total
    return ids, w * scale


def experts(x64, ids, weights, w_gate_up64, w_down64, first_expert=0):
    """Output [T, H] from dequantised x [T, H] and weights [E, 2I, H], [E, H, I]; also, per
    output, the sum of absolute products behind it, how far the output moves when one h value
    of each pair rounds to the neighbouring e4m3 value, and the sum of its pairs' magnitudes."""
    T, H = x64.shape
    E, _, I = w_down64.shape
    out, size, flip, parts = (np.zeros((T, H)) for _ in range(4))
    for t in range(T):
        for j, e in enumerate(np.asarray(ids[t], np.int64) - first_expert):
            if not 0 <= e < E:
                continue
            gu = w_gate_up64[e] @ x64[t]
            g, u = gu[:I], gu[I:]
            h = g / (1.0 + np.exp(-g)) * u
            q, s = quantize(h[None, :].astype(np.float32))
            h = dequantize(q, s)[0]
            w = abs(float(weights[t, j]))
            y = float(weights[t, j]) * (w_down64[e] @ h)
            out[t] += y
            parts[t] += np.abs(y)
            size[t] += w * (np.abs(w_down64[e]) @ np.abs(h))
            step = np.maximum(np.abs(h) / 8.0, np.repeat(s[0].astype(np.float64), BLOCK)[:I] * 2.0 ** -9)
            flip[t] += w * (np.abs(w_down64[e]) * step).max(axis=1)
    return out, size, flip, parts
