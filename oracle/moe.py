"""CPU reference of the operators around a mixture-of-experts block, in
float64 and written from their definitions: the layer on block-scaled FP4 /
FP8 experts, the routing, and the norm between blocks.  Each comes with a
bound on what FP32 arithmetic in any order may add, for the comparison.

TEST INFRASTRUCTURE ONLY (see the package docstring).

u = 2^-24 is the largest relative error of one FP32 rounding.  A sum of n
products in FP32, in any order, is off by at most about n u sum |terms| (the
standard bound, to first order), and every bound below is made of that, of the
derivative of what follows, and of a few u for each further operation.

Pins (tests/test_oracle_moe.py): the layer against plain Python loops over
exact fractions of the weights, special cases that a matmul of the library's
oracle gives, the routing against a brute-force sort, the norm against
``math.fsum``.  No function here is "parity unpinned".
"""

import math

import numpy as np

from .codecs import E2M1_TABLE, E4M3FN_TABLE

U = 2.0 ** -24


def expert_matrix(w, scale, scale_2, block_size, fp8):
    """One expert's weights [N, K] in float64: codes times block scales (times scale_2)."""
    if fp8:
        v = np.asarray(E4M3FN_TABLE, np.float64)[w]
        s = scale.astype(np.float64)
    else:
        v = np.empty((w.shape[0], 2 * w.shape[1]))
        table = np.asarray(E2M1_TABLE, np.float64)
        v[:, 0::2] = table[w & 15]
        v[:, 1::2] = table[w >> 4]
        s = np.asarray(E4M3FN_TABLE, np.float64)[scale] * float(scale_2)
    return v * np.repeat(s, block_size, axis=1)[:, : v.shape[1]]


def activation(kind, g):
    """act(g), and a bound on the slope |act'|."""
    with np.errstate(over="ignore"):
        if kind == "silu":
            return g / (1.0 + np.exp(-g)), 1.1
        z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        return 0.5 * g * (1.0 + np.tanh(z)), 1.13


def moe(A, ids, weights, w13, s13, g13, w2, s2, g2, block_size, act, fp8):
    """(Y, tol): float64 [M, K], and how far an FP32 result may be off before
    its final rounding.  A float64 [M, K]; g13 / g2 None for FP8."""
    M, K = A.shape
    E, I = w13.shape[0], w13.shape[1] // 2  # noqa: E741
    Y, tol = np.zeros((M, K)), np.zeros((M, K))
    for e in range(E):
        use = ids == e
        rows = np.nonzero(use.any(axis=1))[0]
        if not rows.size or I == 0:
            continue
        W13 = expert_matrix(w13[e], s13[e], None if fp8 else g13[e], block_size, fp8)
        W2 = expert_matrix(w2[e], s2[e], None if fp8 else g2[e], block_size, fp8)
        x = A[rows]
        dots = x @ W13.T
        # FP32 sums of K terms, a scale or two applied to parts of them
        d_dots = (K + 4) * U * (np.abs(x) @ np.abs(W13).T)
        g, up = dots[:, :I], dots[:, I:]
        a, slope = activation(act, g)
        h = a * up
        # the exponential's argument is off by 4 u |z| at most; the division and
        # products by a few u; h is handed on with 16 significand bits (2^-17)
        arg = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
        bend = np.where(arg < 100, arg, 0.0)  # beyond, the factor is 0 or 1 whatever the last bits are
        d_h = slope * d_dots[:, :I] * np.abs(up) + np.abs(a) * d_dots[:, I:] + np.abs(h) * ((12 + 4 * bend) * U + 2.0 ** -17)
        d_h = d_h + d_dots[:, :I] * d_dots[:, I:] * slope
        y = h @ W2.T
        d_y = d_h @ np.abs(W2).T + (I + 6) * U * (np.abs(h) @ np.abs(W2).T)
        for j in range(ids.shape[1]):
            on = use[rows, j]
            w = weights[rows, j].astype(np.float64)[:, None]
            Y[rows[on]] += (w * y)[on]
            tol[rows[on]] += (np.abs(w) * (d_y + (ids.shape[1] + 2) * U * np.abs(y)))[on]
    return Y, tol


def route(logits, topk, score="softmax", select_bias=None, renormalize=True, scale=1.0):
    """(ids, weights, rel): the choice, float64 weights, and the relative error that FP32 weights may have."""
    M, E = logits.shape
    x = logits.astype(np.float64)
    ids = np.full((M, topk), -1, np.int32)
    weights = np.zeros((M, topk))
    spread = 0.0
    for m in range(M):
        on = [e for e in range(E) if x[m, e] > -math.inf]  # false for NaN too
        if not on:
            continue
        top = max(x[m, e] for e in on)
        if score == "softmax":
            s = {e: 1.0 if x[m, e] == top else math.exp(x[m, e] - top) if x[m, e] - top > -700 else 0.0 for e in on}
            total = math.fsum(s.values())
            s = {e: v / total for e, v in s.items()}
        else:
            s = {e: 1.0 / (1.0 + math.exp(-x[m, e])) if x[m, e] > -700 else 0.0 for e in on}
        key = {e: x[m, e] if select_bias is None else s[e] + float(select_bias[e]) for e in on}
        order = sorted((e for e in on if key[e] > -math.inf), key=lambda e: (-key[e], e))[:topk]
        ids[m, : len(order)] = order
        w = np.array([s[e] for e in order])
        if renormalize and len(order):
            total = math.fsum(w)
            w = w / total if total > 0 else w * 0
        weights[m, : len(order)] = w * scale
        if order:
            # (below a top of +inf every score is exactly 0 or a share)
            below = abs(top) if score == "softmax" and math.isfinite(top) else 0.0
            reach = [abs(x[m, e]) + below for e in order if math.isfinite(x[m, e])]
            spread = max([spread] + reach)
    # an FP32 exponential's argument is off by u of the operands, the sums by
    # u per term, a handful of operations
    return ids, weights, (2 * spread + E + 12) * U


def block_norm(x, residual=None, pre=None, post=None, gate=None, scale=1.0, eps=1e-6, offset=0.0):
    """(r, y, tol_r, tol_y) in float64, the bounds before the final rounding."""
    K = x.shape[1]
    scale, eps, offset = (float(np.float32(v)) for v in (scale, eps, offset))

    def inv(v):
        return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)

    sum_rel = (K + 6) / 2 * U + 4 * U  # a positive sum of K terms, halved by the root; division, root, product
    b, b_rel = x, 0.0
    if post is not None:
        b = x * inv(x) * (offset + post)
        b_rel = sum_rel + 3 * U
    t = b * (scale if gate is None else scale * gate)
    r = t if residual is None else residual + t
    tol_r = np.abs(t) * (b_rel + 2 * U) + np.abs(r) * U
    if pre is None:
        return r, None, tol_r, None
    i = inv(r)
    y = r * i * (offset + pre)
    # r's own error moves y directly and through the norm
    through = (np.abs(r) * tol_r).mean(axis=1, keepdims=True) * i * i
    tol_y = np.abs(i * (offset + pre)) * tol_r + np.abs(y) * (sum_rel + 3 * U + through)
    return r, y, tol_r, tol_y
