"""Float64 definitions of the operators around the experts: residual addition with root-mean-
square norm, expert selection (softmax / sigmoid scores, choice bias, groups), products with
4-bit weights and group scales, and the SwiGLU expert on such weights.

Selection is a plain loop over tokens and groups; the products are numpy float64 products of the
dequantised weights, an expert at a time.
"""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ residual addition and norm
def add_rmsnorm(x, residual, gamma, eps: float):
    """(s, y, row_scale): s = x + residual, y = s / sqrt(mean(s^2) + eps) * gamma, row_scale =
    max |y| / 448 per row (1 for a zero row)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    top = np.max(np.abs(y), axis=1)
    return s, y, np.where(top > 0, top / 448.0, 1.0)


# ------------------------------------------------------------------ expert selection
def scores(l, sigmoid: bool):
    """Scores of one token's logits; -inf and NaN logits are out (score 0), +inf is the largest float."""
    l = [(-math.inf if (v != v) else min(float(v), 3.4028234663852886e38)) for v in l]
    if sigmoid:
        return l, [0.0 if v == -math.inf else (1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0) for v in l]
    top = max(l)
    if top == -math.inf:
        return l, [0.0] * len(l)
    e = [math.exp(v - top) if v - top > -745 else 0.0 for v in l]
    total = math.fsum(e)
    return l, [v / total for v in e]


def select_token(l, bias, k: int, *, sigmoid: bool, n_groups: int, topk_groups: int, group_best: int,
                 renormalise: bool, weight_scale: float):
    """(idx, w, choices) of one token: k experts in descending order of the choice, ties to the lower index;
    -1 and 0 where none is left."""
    E = len(l)
    l, s = scores(l, sigmoid)
    c = []
    for e in range(E):
        v = s[e] + (float(bias[e]) if bias is not None else 0.0)
        c.append(-math.inf if l[e] == -math.inf or v != v else v)
    live = [e for e in range(E) if c[e] > -math.inf]
    S = E // n_groups
    if topk_groups < n_groups:
        worth = {}
        # one expert's score and no bias: the order of the logits, as below
        of = l if bias is None and group_best == 1 else c
        for g in range(n_groups):
            mine = sorted((of[e] for e in live if e // S == g), reverse=True)[:group_best]
            if mine:
                worth[g] = sum(mine)
        stay = sorted(worth, key=lambda g: (-worth[g], g))[:topk_groups]
        live = [e for e in live if e // S in stay]
    # without a bias the order of the scores is the order of the logits
    chosen = sorted(live, key=lambda e: (-(c[e] if bias is not None else l[e]), e))[:k]
    w = [s[e] for e in chosen]
    if renormalise and chosen:
        if sigmoid:  # log sigmoid, so that ratios of tiny scores keep their value
            ls = [-math.log1p(math.exp(-l[e])) if l[e] > -30 else l[e] for e in chosen]
            m = max(ls)
            w = [math.exp(v - m) for v in ls]
        else:
            m = max(l[e] for e in chosen)
            w = [math.exp(l[e] - m) if l[e] - m > -745 else 0.0 for e in chosen]
        total = math.fsum(w)
        w = [v / total for v in w]
    miss = k - len(chosen)
    return chosen + [-1] * miss, [v * weight_scale for v in w] + [0.0] * miss, c


def select_experts(logits, bias, k: int, **routing):
    """idx [T][k] int32 and w [T][k] float64 for logits [T][E]."""
    got = [select_token(row, bias, k, **routing)[:2] for row in np.asarray(logits, np.float64).tolist()]
    T = len(got)
    return (np.array([g[0] for g in got], np.int32).reshape(T, k), np.array([g[1] for g in got], np.float64).reshape(T, k))


# ------------------------------------------------------------------ 4-bit weights
def w4_pack(q):
    """Codes q [..., K] in 0..15 -> bytes [..., K/2], the even element in the low four bits."""
    q = np.asarray(q, np.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def w4_dequant(codes, scale, zero, group: int):
    """Weights [..., K] float64 of packed codes [..., K/2]."""
    codes = np.asarray(codes, np.uint8)
    q = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.float64)
    q[..., 0::2] = codes & 15
    q[..., 1::2] = codes >> 4
    z = 8.0 if zero is None else np.repeat((np.asarray(zero) & 15).astype(np.float64), group, axis=-1)
    return (q - z) * np.repeat(np.asarray(scale, np.float64), group, axis=-1)


def w4_rows(x, weights, counts):
    """(y, a): y = x W_e^T for rows grouped by expert, a = the sums of |x| |W| (for error bounds);
    weights(e) -> [N][K] float64."""
    x = np.asarray(x, np.float64)
    y, a, at = [], [], 0
    for e, m in enumerate(counts):
        if m == 0:
            continue
        w = weights(e)
        y.append(x[at:at + m] @ w.T)
        a.append(np.abs(x[at:at + m]) @ np.abs(w).T)
        at += m
    return np.concatenate(y), np.concatenate(a)


def swiglu(gate_up):
    """silu(gate) * up for rows [gate | up]."""
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def w4_expert_rows(x, w13, w2, counts):
    """Y = swiglu(x W13_e^T) W2_e^T for rows grouped by expert."""
    return w4_rows(swiglu(w4_rows(x, w13, counts)[0]), w2, counts)[0]
