"""Pins of the oracle between the projections of an attention block (CPU)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from attention_cases import batch, cache, filled, rounded
from oracle import attention as oa


def test_codes_against_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2, 20000), oa.TABLE[:127], -oa.TABLE[:127],
                        (oa.GRID[1:] + oa.GRID[:-1]) / 2, [0.0, -0.0, 448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oa.encode(x.astype(np.float64)), want)
    assert (oa.encode(np.array([np.inf, -np.inf, np.nan])) == 127).all()


def test_powers():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e8m0fnu).double().numpy()
    assert np.array_equal(oa.power(b)[:255], want[:255]) and np.isnan(oa.power(b)[255]) and np.isnan(want[255])
    for top, e in ((0.0, -126), (448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (65504.0, 8), (2.0 ** -140, -126)):
        assert oa.exponent_byte(top) == e + 127


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_one_of_the_plane(interleaved):
    rng = np.random.default_rng(1)
    x, D, R = rng.standard_normal((5, 3, 24)), 24, 16
    angle = rng.uniform(-3, 3, (9, R // 2))
    pos = np.array([8, 0, 3, 9, -1])
    y, _ = oa.norm_rope(x, None, np.cos(angle), np.sin(angle), pos, interleaved)
    for m in range(3):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            z = (x[m, :, a] + 1j * x[m, :, b]) * np.exp(1j * angle[pos[m], i])
            assert np.allclose(y[m, :, a] + 1j * y[m, :, b], z, atol=1e-14)
    assert np.isnan(y[3:, :, :R]).all() and np.array_equal(y[:, :, R:], x[:, :, R:])


def test_norm_against_fsum():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((2, 2, 7)), rng.standard_normal(7)
    y, _ = oa.norm_rope(x, w, offset=1.0, eps=0.5)
    for m in range(2):
        for h in range(2):
            r = math.sqrt(math.fsum(v * v for v in x[m, h]) / 7 + 0.5)
            assert np.allclose(y[m, h], [v / r * (1 + u) for v, u in zip(x[m, h], w)], rtol=1e-14)


def test_append_at_once_and_token_by_token():
    """With the largest value first in each page, the exponent does not move afterwards."""
    rng = np.random.default_rng(3)
    page, H, D = 16, 2, 8
    starts, lens, table, pages = batch(rng, [0, 5], [40, 20], page)
    x = rounded(rng, (60, H, D), "bf16")
    at = oa.places(starts, lens, table, page, pages, 60)
    for m, (b, t, p) in enumerate(at):
        x[m] = np.clip(x[m], -3, 3)
        if t % page == 0 or (b == 1 and t == 5):
            x[m, :, 0] = 3.5
    codes, _, scale, _ = cache(rng, pages, H, page, D, nan_slots=False)
    scale[:] = 100
    once = oa.append(x, codes, scale, starts, lens, table, page)
    step = (codes, scale)
    for i in range(40):
        n = [1, 1 if i < 20 else 0]
        rows = [i] + ([40 + i] if i < 20 else [])
        now = np.array([i + 1, 5 + min(i + 1, 20)], np.int32)
        step = oa.append(x[rows], *step, np.concatenate([[0], np.cumsum(n)]), now, table, page)
    assert np.array_equal(once[0], step[0]) and np.array_equal(once[1], step[1])
    # what is stored is within half a step of the value
    for m, (b, t, p) in enumerate(at):
        y = oa.TABLE[once[0][p, :, t % page]] * oa.power(once[1][p])[:, None]
        assert (np.abs(y - x[m]) <= np.maximum(np.abs(x[m]) * 2.0 ** -4, 2.0 ** -10 * oa.power(once[1][p])[:, None])).all()


def test_append_leaves_what_is_not_its_own():
    rng = np.random.default_rng(4)
    starts, lens, table, pages = batch(rng, [3], [2], 16)
    codes, _, scale, _ = cache(rng, pages, 1, 16, 8)
    scale[:] = 254
    x = rounded(rng, (4, 1, 8), "bf16")  # two rows behind the last sequence
    got, s = oa.append(x, codes, scale, starts, lens, table, 16)
    changed = np.argwhere((got != codes).any(axis=-1))
    assert {(int(p), int(t)) for p, _, t in changed} <= {(int(table[0, 0]), 3), (int(table[0, 0]), 4)}
    table[0, 0] = pages  # no such page
    got, s = oa.append(x, codes, scale, starts, lens, table, 16)
    assert np.array_equal(got, codes) and np.array_equal(s, scale)


def test_attention_against_fractions():
    """Two tokens with equal scores, then plain loops."""
    page, D = 4, 2
    k = np.zeros((1, 1, page, D), np.uint8)
    v = np.zeros((1, 1, D, page), np.uint8)
    v[0, 0, :, 0], v[0, 0, :, 1] = oa.encode([1.0, -2.0]), oa.encode([3.0, 7.0])
    ks = vs = np.full((1, 1), 128, np.uint8)
    Y, L, _, _ = oa.attention(np.ones((1, 1, D)), k, v, ks, vs, None, [2], np.zeros((1, 1), np.int32), 1.0)
    want = [float(Fraction(1 + 3, 2) * 2), float(Fraction(-2 + 7, 2) * 2)]
    assert np.allclose(Y[0, 0], want, rtol=1e-15) and abs(L[0, 0] - math.log(2)) < 1e-15


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0), (False, 5)])
def test_attention_against_loops(causal, window):
    rng = np.random.default_rng(5)
    page, H, G, D = 4, 2, 3, 8
    starts, lens, table, pages = batch(rng, [0, 6, 0], [5, 3, 1], page)
    table[1, 0] = -1  # an absent page
    c = filled(rng, starts, lens, table, page, pages, H, D)
    q = rounded(rng, (10, H * G, D), "bf16")
    Y, L, _, _ = oa.attention(q, *c, starts, lens, table, 0.3, causal, window)
    k, v, ks, vs = c
    assert np.isnan(Y[9]).all()
    for m, place in enumerate(oa.places(starts, lens, table, page, pages, 10)):
        if place is None:
            continue
        b, p, _ = place
        on = [t for t in range(lens[b]) if (t <= p or not causal) and (window == 0 or t > p - window) and table[b, t // page] >= 0]
        for h in range(H * G):
            s, rows = [], []
            for t in on:
                i = table[b, t // page]
                s.append(float(np.float32(0.3)) * sum(q[m, h, d] * oa.TABLE[k[i, h // G, t % page, d]] for d in range(D)) * oa.power(ks[i, h // G]))
                rows.append([oa.TABLE[v[i, h // G, d, t % page]] * oa.power(vs[i, h // G]) for d in range(D)])
            e = [math.exp(x) for x in s]
            want = [math.fsum(w * r[d] for w, r in zip(e, rows)) / math.fsum(e) for d in range(D)] if on else [0.0] * D
            assert np.allclose(Y[m, h], want, rtol=1e-6, atol=1e-12)
            assert np.isclose(L[m, h], math.log(math.fsum(e)), rtol=1e-6) if on else L[m, h] == -math.inf
