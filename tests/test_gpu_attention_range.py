"""Attention at the ends of the numbers' range, on the GPU, through every kernel
that takes the case: against the float64 oracle."""

import numpy as np
import pytest

import fp8_weight_only_fp4w_amd as fw
from attention_cases import batch, filled, on_gpu, rounded, to_cache, within
from gpu_helpers import require_gpu
from oracle import attention as oa
from test_gpu_attention import check, paths

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


# held before, new, page, Hq, Hk, D
LARGE = [
    ([0], [1], 16, 2, 1, 64),
    ([40, 3], [1, 1], 16, 5, 1, 128),
    ([30, 9], [20, 7], 16, 4, 2, 64),
    ([8], [40], 32, 20, 2, 128),
    ([20, 5], [4, 2], 10, 2, 1, 48),
]


@pytest.mark.parametrize("byte", [245, 246, 247, 250, 254])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{max(c[0])}+{max(c[1])}-{c[3]}/{c[4]}x{c[5]}")
def test_values_near_the_end_of_bf16(case, byte):
    """Pages of BF16 values with a scale of up to 2^127: an appended value above 1.75 * 2^127 leads to 2^120."""
    held, new, page, Hq, Hk, D = case
    rng = np.random.default_rng(73 + D)
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    last = 0.5 * 2.0 ** 127  # half the end: sums in FP32 stay below it
    for b in range(len(lens)):
        p = table[b, 0]
        v = rng.choice([0.0, 2.0 ** -9, 2.0 ** -6, 3.0, 104.0], (Hk, D))
        parts[1][p] = oa.encode(rng.choice([0.0, 2.0 ** -9, -(2.0 ** -9)], (Hk, D, page)))
        parts[1][p, :, :, 0] = oa.encode(np.minimum(v, last / 2.0 ** (byte - 127)))  # one large token
        parts[3][p] = byte
    q = rounded(rng, (int(starts[-1]), Hq, D), "bf16")
    Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 0.05)
    assert np.isfinite(Y).all() and np.isfinite(tol).all() and np.abs(Y).max() > 2.0 ** 110
    check(q, parts, starts, lens, table, "bf16", scale=0.05)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
@pytest.mark.parametrize("byte,code,below", [(136, 0x78, 0x01), (150, 0xF8, 0x00), (170, 0x01, 0x00), (254, 0x31, 0x80)])
def test_values_that_fp16_does_not_hold(byte, code, below, D, page, n):
    """In the decode and prompt kernels, stored values of 2^17 and more count as NaN each for itself: rows that do not
    attend them and the values beside them stay as they are."""
    dtype = "fp16"
    rng = np.random.default_rng(75)
    starts, lens, table, pages = batch(rng, [3, 20], [n, n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    t = 3 + n // 2
    p, slot = table[0, t // page], t % page
    parts[1][p] = 0
    parts[1][p, 0, 1, slot] = below
    parts[3][p] = byte
    want = [x.copy() for x in parts]
    want[1][p, 0, 2, slot] = 0x7F
    parts[1][p, 0, 2, slot] = code
    q = rounded(rng, (2 * n, 4, D), dtype)
    Y, _, tol, _ = oa.attention(q, *want, starts, lens, table, 0.05, dtype=dtype)
    assert np.isnan(Y[n // 2: n, :, 2]).all() and np.isnan(Y).sum() == 4 * (n - n // 2)  # the token's own row and those behind it
    c, g, ids, st, ln = to_cache(parts), on_gpu(q, dtype), on_gpu(table), on_gpu(starts), on_gpu(lens)
    for path in paths(D, page, 4 * n):
        if path == fw.PATH_ATTN_GENERIC:
            continue
        got = fw.fp8w_attention(g, c, ids, ln, starts=st, max_new=n, scale=0.05, path=path)
        within(got, Y, tol, dtype, f"path {fw.fp4w_path_name(path)}")


@pytest.mark.parametrize("byte", [222, 223, 240, 246, 247])
@pytest.mark.parametrize("D,page,n", [(64, 16, 2), (128, 64, 40), (64, 32, 130), (40, 8, 3)])
def test_a_growing_score_with_a_large_value(D, page, n, byte):
    """A token behind several tiles that scores 2^6 times the ones before, and whose values reach 2^126."""
    rng = np.random.default_rng(74)
    starts, lens, table, pages = batch(rng, [300], [n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    parts[0][:] = oa.encode(rng.choice([0.0, 0.125, -0.125], parts[0].shape))
    parts[2][:], parts[3][:] = 127, 127
    t = 200
    p = table[0, t // page]
    parts[0][p, 0, t % page] = oa.encode(np.full(D, 4.0))
    parts[1][p] = oa.encode(rng.choice([0.0, 2.0 ** -9, -(2.0 ** -9)], (1, D, page)))
    parts[1][p, 0, :, t % page] = oa.encode(np.minimum(rng.uniform(100, 400, D), 2.0 ** (126 + 127 - byte)))
    parts[3][p] = byte
    q = np.ones((n, 2, D))
    Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 1.0 / D)
    assert np.isfinite(Y).all() and np.isfinite(tol).all()
    check(q, parts, starts, lens, table, "bf16", scale=1.0 / D)


@pytest.mark.parametrize("held,n,page,D", [(400, 1, 16, 64), (5000, 3, 16, 128), (400, 60, 16, 128), (6000, 50, 64, 64), (300, 2, 6, 40)])
def test_sums_of_values_near_the_end_of_bf16(held, n, page, D):
    """Values near 2^128, and stored ones above: their sum is not FP32's, their average is."""
    rng = np.random.default_rng(76)
    starts, lens, table, pages = batch(rng, [held], [n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    q = rounded(rng, (n, 2, D), "bf16")
    parts[3][:] = 247
    for codes in (np.where(rng.random((1, 1, D, 1)) < 0.5, 0x77, 0xF6),             # 240 and -224
                  np.where(rng.random(parts[1].shape) < 0.45, 0x7E, 0x00)):         # 448 now and then
        parts[1][:] = codes
        Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 0.01)
        assert (np.abs(Y) > 2.0 ** 126).all() and (np.abs(Y) < 2.0 ** 128).all()
        check(q, parts, starts, lens, table, "bf16", scale=0.01)


@pytest.mark.parametrize("lo,hi", [(24, 27), (14, 30)])
@pytest.mark.parametrize("held,n,page,D", [(100, 1, 16, 64), (3000, 2, 16, 128), (100, 60, 16, 128), (90, 2, 6, 40)])
def test_smallest_values(held, n, page, D, lo, hi):
    """Page scales down to 2^-113, of FP32's smallest numbers times 2^13: right to the steps of 2^-109 that values are held in."""
    rng = np.random.default_rng(77)
    starts, lens, table, pages = batch(rng, [held], [n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    parts[3][:] = rng.integers(lo, hi, parts[3].shape)
    q = rounded(rng, (n, 4, D), "bf16")
    Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 0.05)
    assert np.abs(Y).max() > 2.0 ** -106
    c, g, ids, st, ln = to_cache(parts), on_gpu(q, "bf16"), on_gpu(table), on_gpu(starts), on_gpu(lens)
    for path in paths(D, page, 4 * n):
        got = fw.fp8w_attention(g, c, ids, ln, starts=st, max_new=n, scale=0.05, path=path)
        within(got, Y, tol + 2.0 ** -109, "bf16", f"path {fw.fp4w_path_name(path)}")


@pytest.mark.parametrize("held,n,page,D", [(900, 1, 16, 64), (3000, 2, 16, 128), (100, 60, 16, 128), (500, 40, 64, 64), (90, 2, 6, 40)])
def test_pages_of_zeros(held, n, page, D):
    """As the append leaves them: codes of 0 of either sign under the smallest scale, beside pages of ordinary and of the
    smallest values."""
    rng = np.random.default_rng(78)
    starts, lens, table, pages = batch(rng, [held], [n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    kind = rng.integers(0, 4, pages)
    parts[1][kind == 0] = rng.choice([0x00, 0x80], parts[1][kind == 0].shape)
    parts[3][kind == 0], parts[3][kind == 1] = 1, 20
    q = rounded(rng, (n, 4, D), "bf16")
    check(q, parts, starts, lens, table, "bf16", scale=0.05)
    parts[1][:], parts[3][:] = 0, 1
    check(q, parts, starts, lens, table, "bf16", scale=0.05)
