"""Pins of oracle/moe.py (CPU)."""

import itertools
import math
from fractions import Fraction

import numpy as np
import pytest

from moe_cases import make_moe, moe_want
from oracle import codecs
from oracle import moe as om


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_against_exact_loops(fp8):
    """Dots as exact fractions, element by element; only the activation is float64."""
    c = make_moe(fp8, 2, 6, 4, 3, 2, "bf16", 5, block_size=4, masked=0.2)
    Y, tol = moe_want(c)

    def weight(w, s, g, e, n, k):
        if fp8:
            return Fraction(codecs.e4m3fn_value(int(w[e, n, k]))) * Fraction(float(s[e, n, k // 4]))
        code = (int(w[e, n, k // 2]) >> (4 * (k % 2))) & 15
        return Fraction(codecs.e2m1_value(code)) * Fraction(codecs.e4m3fn_value(int(s[e, n, k // 4]))) * Fraction(float(g[e]))

    for m, n in itertools.product(range(2), range(6)):
        total = 0.0
        for j in range(2):
            e = int(c["ids"][m, j])
            if e < 0:
                continue
            acc = 0.0
            for i in range(4):
                dot = [float(sum(Fraction(float(c["A64"][m, k])) * weight(c["w13"], c["s13"], c["g13"], e, r, k) for k in range(6)))
                       for r in (i, 4 + i)]
                acc += dot[0] / (1 + math.exp(-dot[0])) * dot[1] * float(weight(c["w2"], c["s2"], c["g2"], e, n, i))
            total += float(c["weights"][m, j]) * acc
        assert abs(total - Y[m, n]) <= 1e-12 * (1 + abs(total))
        assert tol[m, n] < 1e-3 * (1 + np.abs(Y).max())


def test_masked_and_repeated_choices():
    c = make_moe(False, 3, 32, 32, 4, 3, "bf16", 6)
    c["ids"][:] = [[-1, 7, -5], [2, 2, 2], [1, -1, 4]]
    Y, _ = moe_want(c)
    assert not Y[0].any()  # nothing but ids outside [0, E)
    one = dict(c, ids=c["ids"][1:2, :1], weights=c["weights"][1:2].sum(1, keepdims=True), A64=c["A64"][1:2])
    assert np.allclose(moe_want(one)[0][0], Y[1], rtol=1e-6)  # the float32 sum of the weights


def test_activations():
    g = np.array([-1000.0, -3.0, 0.0, 2.0, 50.0])
    silu, _ = om.activation("silu", g)
    assert silu[0] == 0 and silu[2] == 0 and silu[4] == pytest.approx(50) and silu[3] == pytest.approx(1.7615941559557649)
    gelu, _ = om.activation("gelu", g)
    assert gelu[0] == 0 and gelu[4] == 50 and gelu[3] == pytest.approx(1.9545976940877752)


@pytest.mark.parametrize("score,bias", itertools.product(("softmax", "sigmoid"), (False, True)))
def test_route_against_a_brute_force_sort(score, bias):
    rng = np.random.default_rng(8)
    x = np.round(rng.standard_normal((20, 9)) * 4) / 4  # many ties
    b = np.round(rng.standard_normal(9) * 4).astype(np.float32) / 8 if bias else None
    ids, w, rel = om.route(x, 4, score, b, renormalize=False, scale=2.0)
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x))
    for m in range(20):
        key = x[m] if b is None else p[m] + b
        # rounding noise of the two formulas must not part equal keys
        want = sorted(range(9), key=lambda e: (-round(key[e], 12), e))[:4]
        assert list(ids[m]) == want
        assert np.allclose(w[m], 2 * p[m][want], rtol=1e-12)
    again = om.route(x, 4, score, b, renormalize=True, scale=2.0)[1]
    assert np.allclose(again.sum(1), 2.0) and rel < 1e-5


def test_route_masks():
    x = np.array([[-math.inf, math.nan, 1.0, -math.inf], [-math.inf] * 4, [math.inf, 0.0, math.inf, -1.0],
                  [-3e38, -3e38, -3e38, -3e38]])
    ids, w, _ = om.route(x, 3, "softmax")
    assert ids.tolist() == [[2, -1, -1], [-1, -1, -1], [0, 2, 1], [0, 1, 2]]
    assert np.allclose(w, [[1, 0, 0], [0, 0, 0], [0.5, 0.5, 0], [1 / 3] * 3])


def test_block_norm_against_fsum():
    rng = np.random.default_rng(9)
    x, res, gate = (rng.standard_normal((3, 37)) for _ in range(3))
    pre, post = rng.standard_normal(37), rng.standard_normal(37)
    r, y, tol_r, tol_y = om.block_norm(x, res, pre, post, gate, 0.5, 1e-6, 1.0)
    eps = float(np.float32(1e-6))
    for m in range(3):
        inv = 1 / math.sqrt(math.fsum(v * v for v in x[m]) / 37 + eps)
        want = [res[m, k] + 0.5 * gate[m, k] * x[m, k] * inv * (1 + post[k]) for k in range(37)]
        assert np.allclose(r[m], want, rtol=1e-13, atol=1e-14)
        inv = 1 / math.sqrt(math.fsum(v * v for v in want) / 37 + eps)
        assert np.allclose(y[m], [want[k] * inv * (1 + pre[k]) for k in range(37)], rtol=1e-12, atol=1e-14)
    # an FP32 evaluation stays inside the bounds, and the bounds stay small
    f = np.float32
    b = x.astype(f) / np.sqrt((x.astype(f) ** 2).mean(1, keepdims=True, dtype=f) + f(1e-6)) * (f(1) + post.astype(f))
    assert (tol_r < 1e-4).all() and (tol_y < 1e-4).all() and b.dtype == f


def test_block_norm_parts():
    x = np.array([[3.0, -4.0]])
    r, y, *_ = om.block_norm(x, None, None, None, None, 2.0)
    assert y is None and r.tolist() == [[6.0, -8.0]]
    r, y, *_ = om.block_norm(x, None, np.array([1.0, 2.0]), eps=0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]])


def test_renormalised_weights_of_small_scores():
    """sigmoid(x) is exp(x) to 1e-40 that far below 0, so the quotients are a softmax of the chosen logits."""
    x = np.array([[-200.0, -201.0, -203.5, -200.0], [-600.0, -601.0, -640.0, -700.5]])
    ids, w, _ = om.route(x, 3, "sigmoid")
    assert ids.tolist() == [[0, 3, 1], [0, 1, 2]]
    for m, z in enumerate(([0, 0, -1], [0, -1, -40])):
        total = math.fsum(math.exp(v) for v in z)
        assert np.allclose(w[m], [math.exp(v) / total for v in z], rtol=1e-12)
    bias = np.array([-10.0, 1, 1, 2], np.float32)
    ids, w, _ = om.route(np.array([[0.0, -120, -121, -119], [0, -760, -770, -800]]), 2, "softmax", bias)
    assert ids.tolist() == [[3, 1]] * 2
    assert np.allclose(w[0], [1 / (1 + math.exp(-1)), 1 / (1 + math.e)], rtol=1e-12) and (w[1] == 0).all()


@pytest.mark.parametrize("K", [37, 1000, 5120])
def test_block_norm_bounds_hold_an_fp32_evaluation(K):
    """r and y computed step by step in FP32 from FP32 inputs stay inside the bounds, sums in two orders."""
    f = np.float32
    rng = np.random.default_rng(K)
    x, res, gate = (rng.standard_normal((4, K)).astype(f) for _ in range(3))
    pre, post = (rng.standard_normal(K).astype(f) for _ in range(2))

    def norm(v, w, total):
        inv = f(1) / np.sqrt(total(v * v) * f(1.0 / K) + f(1e-6))
        return v * (inv * (f(0.5) + w))

    def one_by_one(v):
        return np.cumsum(v, axis=1, dtype=f)[:, -1:]

    def pairs(v):
        return v.sum(axis=1, keepdims=True, dtype=f)

    for has_post, has_gate, has_res in itertools.product((False, True), repeat=3):
        r64, y64, tol_r, tol_y = om.block_norm(
            x.astype(np.float64), res.astype(np.float64) if has_res else None, pre.astype(np.float64),
            post.astype(np.float64) if has_post else None, gate.astype(np.float64) if has_gate else None, 0.22, 1e-6, 0.5)
        for total in (one_by_one, pairs):
            b = norm(x, post, total) if has_post else x
            t = (f(0.22) * gate if has_gate else f(0.22)) * b
            r = res + t if has_res else t
            y = norm(r, pre, total)
            assert r.dtype == f and y.dtype == f
            assert (np.abs(r - r64) <= tol_r).all() and (np.abs(y - y64) <= tol_y).all()
        # and they are no wider than FP32 needs
        assert (tol_r <= 2e-3 * (np.abs(r64) + np.abs(x) + 1)).all() and (tol_y <= 4e-3 * (np.abs(y64) + 1)).all()
