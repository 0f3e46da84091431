"""Attention at the ends of the numbers' range, on the GPU, through every kernel
that takes the case: against the float64 oracle."""

import numpy as np
import pytest

from attention_cases import batch, filled, rounded
from gpu_helpers import require_gpu
from oracle import attention as oa
from test_gpu_attention import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# held before, new, page, Hq, Hk, D, window
ENDLESS = [
    ([0], [1], 16, 1, 1, 64, 0),                  # one token attended
    ([900, 3], [1, 1], 16, 5, 1, 128, 0),
    ([3000, 0, 40], [2, 1, 3], 16, 8, 2, 128, 0),  # joined from several shares
    ([9000, 100], [1, 1], 64, 40, 8, 64, 0),
    ([200, 3, 70], [2, 4, 3], 32, 28, 4, 64, 30),
    ([70], [150], 16, 3, 1, 128, 64),
    ([5000], [40], 16, 8, 1, 64, 0),              # joined from several parts
    ([33, 0], [2, 30], 10, 2, 1, 48, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", ENDLESS, ids=lambda c: f"{max(c[0])}+{max(c[1])}-{c[3]}/{c[4]}x{c[5]}-w{c[6]}")
def test_rows_whose_every_score_is_minus_infinity(case, dtype):
    """An infinity in a query whose keys all have the other sign there: 0 / 0, and not the zeros of a row without a token."""
    held, new, page, Hq, Hk, D, window = case
    rng = np.random.default_rng(70 + D)
    starts, lens, table, pages = batch(rng, held + [20], new + [1], page)
    table[-1] = -1  # a sequence without a page: its rows attend nothing, whatever their queries hold
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    parts[0][..., 5] = 0x38  # 1
    q = rounded(rng, (int(starts[-1]), Hq, D), dtype, 1.5)
    hit = [(int(s), 0) for s in starts[:-1]] + [(int(starts[1]) - 1, Hq - 1)]
    for m, h in hit:
        q[m, h, 5] = -np.inf
    Y, L, _, _ = oa.attention(q, *parts, starts, lens, table, 1.0, True, window)
    lone = int(starts[-2])
    assert all(np.isnan(Y[m, h]).all() and np.isnan(L[m, h]) for m, h in hit if m != lone)
    assert (Y[lone] == 0).all() and np.isnan(Y).any(-1).sum() == len({x for x in hit if x[0] != lone})
    check(q, parts, starts, lens, table, dtype, scale=1.0, window=window)


# held before, new, page, Hq, Hk, D
FAR = [
    ([900, 3], [1, 1], 16, 5, 1, 128),
    ([3000, 0, 40], [2, 1, 3], 16, 8, 2, 128),
    ([500, 20], [5, 4], 32, 8, 2, 128),   # 20 rows of a key head
    ([200, 3, 70], [2, 4, 3], 32, 28, 4, 64),
    ([70], [150], 16, 3, 1, 128),
    ([5000], [40], 16, 8, 1, 64),         # joined from several parts
    ([33, 0], [2, 30], 10, 2, 1, 48),
]


@pytest.mark.parametrize("case", FAR, ids=lambda c: f"{max(c[0])}+{max(c[1])}-{c[3]}/{c[4]}x{c[5]}")
def test_queries_near_the_end_of_bf16_and_small_keys(case):
    """q times the codes passes FP32, q times the keys does not; rows of ordinary queries stand beside."""
    held, new, page, Hq, Hk, D = case
    rng = np.random.default_rng(71 + D)
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    parts[2][:] = rng.integers(1, 4, parts[2].shape)
    M = int(starts[-1])
    q = rounded(rng, (M, Hq, D), "bf16", 1.2)
    up = rng.integers(104, 126, (M, Hq, 1))
    up[rng.random((M, Hq, 1)) < 0.3] = 0
    up[0, 0], up[-1, -1] = 125, 104
    q = q * 2.0 ** up
    assert np.abs(q).max() * 448 * 16 > np.finfo(np.float32).max > np.abs(q).max()
    Y, L, _, _ = oa.attention(q, *parts, starts, lens, table, 0.125)
    assert np.isfinite(Y).all() and np.isfinite(L).all()
    check(q, parts, starts, lens, table, "bf16", scale=0.125)
    check(q, parts, starts, lens, table, "bf16", scale=-0.125)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (24, 6)])
def test_keys_of_zero_under_the_largest_scale(D, page, n):
    """2^127 times the call's own scale passes FP32; times a key of 0 it is 0."""
    rng = np.random.default_rng(72)
    starts, lens, table, pages = batch(rng, [100, 20], [n, n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    for b in range(2):
        parts[2][table[b, 1]] = 254
        parts[0][table[b, 1]] = 0
    q = rounded(rng, (2 * n, 3, D), "bf16", 0.1)
    check(q, parts, starts, lens, table, "bf16", scale=3.0)
