"""CPU reference of the operators between the projections of an attention
block, in float64 and written from their definitions: norm and rotation of
heads, the append to the paged 8-bit cache, and attention over it.  Each comes
with a bound on what FP32 arithmetic in any order may add, for the comparison.

TEST INFRASTRUCTURE ONLY (see the package docstring).

u = 2^-24 is the largest relative error of one FP32 rounding; a sum of n
products in any order is off by at most about n u sum |terms|.

Pins (tests/test_oracle_attention.py): the codes against torch's own
conversion, the append token by token against all tokens at once where the
scale does not move, attention against exact fractions, plain softmax loops and
lists of tokens that no page holds.  No function here is "parity unpinned".
"""

import math

import numpy as np

from .codecs import E4M3FN_TABLE

U = 2.0 ** -24
TABLE = np.asarray(E4M3FN_TABLE, np.float64)
GRID = TABLE[:127]  # the finite values from 0 up, code by code


def power(byte):
    """E8M0 bytes as values."""
    b = np.asarray(byte).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.where(b == 255, 0, b - 127)))


def encode(x):
    """E4M3 codes of float64 values within +-448, ties to the even code; NaN codes for others."""
    x = np.asarray(x, np.float64)
    mag = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(GRID, mag, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = mag - GRID[lo], GRID[hi] - mag
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 127)
    return code.astype(np.uint8)


def exponent_byte(top):
    """The byte of the smallest 2^e >= 2^-126 with top <= 448 * 2^e."""
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e + 127


def norm_rope(x, weight=None, cos=None, sin=None, positions=None, interleaved=False, offset=0.0, eps=1e-6):
    """(y, tol) of x [M, H, D] float64; cos, sin [rows, R / 2], positions [M]."""
    M, _, D = x.shape
    offset, eps = float(np.float32(offset)), float(np.float32(eps))
    rel = 0.0
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps) * (offset + weight)
        rel = ((D + 6) / 2 + 8) * U  # a sum of D squares, halved by the root; mean, root, division, products
    if cos is None:
        return y, np.abs(y) * (rel + U)
    y = y.copy()
    tol = np.abs(y) * (rel + U)
    half = cos.shape[1]
    a_at = np.arange(half) * 2 if interleaved else np.arange(half)
    b_at = a_at + (1 if interleaved else half)
    for m in range(M):
        p = m if positions is None else int(positions[m])
        a, b = y[m][:, a_at], y[m][:, b_at]
        if 0 <= p < cos.shape[0]:
            c, s = cos[p].astype(np.float64), sin[p].astype(np.float64)
        else:
            c = s = np.full(half, np.nan)
        y[m][:, a_at], y[m][:, b_at] = a * c - b * s, b * c + a * s
        tol[m][:, a_at] = (np.abs(a * c) + np.abs(b * s)) * (rel + 4 * U)
        tol[m][:, b_at] = (np.abs(b * c) + np.abs(a * s)) * (rel + 4 * U)
    return y, tol


def spans(starts, lens):
    """(first row, rows, length) of each sequence."""
    B = len(lens)
    at = list(range(B + 1)) if starts is None else [int(v) for v in starts]
    return [(at[b], at[b + 1] - at[b], int(lens[b])) for b in range(B)]


def places(starts, lens, table, page, num_pages, M):
    """For each row: (sequence, position, page id or -1); None for rows of no sequence."""
    out = [None] * M
    for b, (row, n, length) in enumerate(spans(starts, lens)):
        for i in range(n):
            t = length - n + i
            inside = 0 <= t < table.shape[1] * page
            p = int(table[b, t // page]) if inside else -1
            out[row + i] = (b, t, p if 0 <= p < num_pages else -1)
    return out


def append(x, codes, scale, starts, lens, table, page):
    """What a cache holds afterwards: (codes, scale) of tokens-by-values pages
    [P, H, page, D] (v's are transposed by the caller), for x [M, H, D] float64."""
    codes, scale = codes.copy(), scale.copy()
    H = x.shape[1]
    at = places(starts, lens, table, page, codes.shape[0], x.shape[0])
    groups = {}
    for m, place in enumerate(at):
        if place is not None and place[2] >= 0:
            groups.setdefault(place[2], []).append((place[1] % page, m))
    for p, tokens in groups.items():
        first = min(slot for slot, _ in tokens)
        for h in range(H):
            new = np.stack([x[m, h] for _, m in tokens])
            finite = np.abs(new[np.isfinite(new)])
            byte = exponent_byte(float(finite.max()) if finite.size else 0.0)
            before = int(scale[p, h])
            if first > 0:
                byte = max(byte, before)
                if byte != before:
                    old = TABLE[codes[p, h, :first]] * 2.0 ** (before - byte)
                    codes[p, h, :first] = encode(old)
            scale[p, h] = byte
            for slot, m in tokens:
                codes[p, h, slot] = encode(x[m, h] * 2.0 ** (127 - byte)) if byte != 255 else 127
    return codes, scale


def attention(q, kc, vc, ks, vs, starts, lens, table, scale, causal=True, window=0, dtype="bf16"):
    """(Y, lse, tol, tol_lse) in float64 for q [M, Hq, D]; the cache as the
    library has it (v [P, H, D, page]).  NaN rows of Y and lse: of no sequence.
    tol is the bound before the final rounding; where a token is attended whose
    score or value is not finite, Y is what IEEE arithmetic makes of it."""
    M, Hq, D = q.shape
    P, Hk, page, _ = kc.shape
    G = Hq // Hk
    scale = float(np.float32(scale))
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    Y, L = np.full((M, Hq, D), np.nan), np.full((M, Hq), np.nan)
    tol, tol_l = np.zeros((M, Hq, D)), np.zeros((M, Hq))
    for b, (row, n, length) in enumerate(spans(starts, lens)):
        if n <= 0:
            continue
        room = min(max(length, 0), table.shape[1] * page)
        t = np.arange(room)
        ids = table[b, t // page].astype(np.int64)
        here = (ids >= 0) & (ids < P)
        t, ids = t[here], ids[here]
        pos = (length - n + np.arange(n))[:, None]
        seen = np.ones((n, len(t)), bool)
        if causal:
            seen &= t[None] <= pos
        if window > 0:
            seen &= t[None] > pos - window
        for hk in range(Hk):
            k = TABLE[kc[ids, hk, t % page]] * power(ks[ids, hk])[:, None]
            v = TABLE[vc[ids, hk, :, t % page]] * power(vs[ids, hk])[:, None]
            for h in range(hk * G, (hk + 1) * G):
                x = q[row:row + n, h]
                with np.errstate(invalid="ignore", over="ignore"):
                    s, size = x @ k.T * scale, np.abs(x) @ np.abs(k).T * abs(scale)
                for i in range(n):
                    on = np.nonzero(seen[i])[0]
                    m = row + i
                    if not on.size:
                        Y[m, h], L[m, h] = 0.0, -math.inf
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        si, vi = s[i, on], v[on]
                        top = si.max()
                        e = np.exp(si - top)
                        w = e / e.sum()
                        Y[m, h] = w @ vi
                        L[m, h] = top + math.log(e.sum())
                        # a score: a sum of D products, its factors, and the exponential's argument
                        err = (D + 6) * U * size[i, on] + 6 * U * (np.abs(si) + abs(top)) + 4 * U
                        sums = (on.size + 16) * U
                        av = np.abs(vi)
                        tol[m, h] = (w * (err + half + sums)) @ av + np.abs(Y[m, h]) * (w @ err + sums)
                        if dtype == "fp16":  # numerators from 2^-33 up, values in steps of 2^-24
                            tol[m, h] += on.size * 2.0 ** -33 * av.max(axis=0) + 2.0 ** -24
                        tol_l[m, h] = w @ err + sums + 2 * U * (abs(top) + abs(L[m, h]))
    return Y, L, tol, tol_l
