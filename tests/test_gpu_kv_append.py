"""The append to the paged 8-bit cache on the GPU, against the float64 oracle:
codes and scales as they are stored, and every slot that is nobody's left
alone."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from attention_cases import TORCH_DT, batch, cache, on_gpu, rounded, to_cache, within
from gpu_helpers import require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def by_token(v):
    return v.transpose(0, 1, 3, 2)  # [P, H, D, page] -> [P, H, page, D]


def same_codes(a, b):
    """Equal, any NaN code like any other."""
    return ((a == b) | (((a & 127) == 127) & ((b & 127) == 127))).all()


def check_codes(got, scale, x, tol, before, scale_before, starts, lens, table, page, what):
    """Stored pages against x +- tol (float64): every code between those of
    x - tol and x + tol, every scale one that such values give."""
    lo = oa.append(np.sign(x) * np.maximum(np.abs(x) - tol, 0), before, scale_before, starts, lens, table, page)
    hi = oa.append(np.sign(x) * (np.abs(x) + tol), before, scale_before, starts, lens, table, page)
    assert ((scale == lo[1]) | (scale == hi[1])).all(), f"{what}: scales"
    same = (lo[1] == hi[1])[:, :, None, None]
    low, high = np.minimum(lo[0] & 127, hi[0] & 127), np.maximum(lo[0] & 127, hi[0] & 127)
    sign = (lo[0] & 128) == (got & 128)
    ok = ((got & 127) >= low) & ((got & 127) <= high) & (sign | ((got & 127) == 0))
    ok |= ((lo[0] & 127) == 127) & ((got & 127) == 127)
    bad = ~ok & same
    assert not bad.any(), f"{what}: {int(bad.sum())} codes, first {np.argwhere(bad)[:3].tolist()}"


# held before, new, page, Hq, Hk, D, R (None: no norm and rotation)
CASES = [
    ([700], [1], 64, 40, 8, 128, 128),
    ([0], [1], 16, 5, 1, 64, 64),
    ([0, 15, 16, 17, 31], [1, 1, 1, 1, 1], 16, 4, 2, 128, 64),
    ([3, 0, 20], [40, 0, 1], 16, 0, 2, 64, None),
    ([0, 10, 63], [64, 200, 130], 64, 2, 2, 128, None),
    ([5, 127], [300, 2], 128, 4, 1, 128, 128),
    ([0, 0, 7], [1, 33, 90], 32, 0, 3, 256, None),
    ([12], [500], 16, 8, 8, 16, 16),
    # pages and heads that no vector holds
    ([2, 9], [11, 3], 5, 2, 1, 64, 64),
    ([0, 4], [20, 1], 1, 0, 2, 32, None),
    ([6, 0], [30, 9], 24, 3, 1, 80, 40),
    ([100], [300], 256, 0, 1, 128, None),
    ([1], [20], 16, 0, 2, 1, None),
    ([50] * 150, [1] * 150, 16, 0, 1, 64, None),
    ([0] * 90, [2] * 90, 16, 1, 1, 64, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}seq-{c[2]}-{c[4]}x{c[5]}-{sum(c[1])}")
def test_against_oracle(case, dtype):
    held, new, page, Hq, Hk, D, R = case
    rng = np.random.default_rng(sum(held) * 7 + page)
    M, spare_rows = sum(new), 3 if set(new) != {1} else 0
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = cache(rng, pages, Hk, page, D)
    if len(held) % 2:  # pages of large values, whose exponent stays
        parts[2][:], parts[3][:] = 135, 136
    k = rounded(rng, (M + spare_rows, Hk, D), dtype, 3.0) * 2.0 ** rng.integers(-6, 3, (M + spare_rows, 1, 1))
    v = rounded(rng, (M + spare_rows, Hk, D), dtype, 3.0)
    q = rounded(rng, (M + spare_rows, Hq, D), dtype)
    wq = wk = cos = sin = None
    if R:
        wq, wk = rounded(rng, D, dtype), rounded(rng, D, dtype)
        a = rng.uniform(-3, 3, (int(lens.max()) + 1, R // 2))
        cos, sin = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    gpu = lambda x, t=None: None if x is None else on_gpu(x, t)  # noqa: E731
    for use_starts in (True, False) if set(new) == {1} else (True,):
        c = to_cache(parts)
        out = fw.fp8w_kv_append(on_gpu(k, dtype), on_gpu(v, dtype), c, on_gpu(table), on_gpu(lens),
                                starts=on_gpu(starts) if use_starts else None, q=on_gpu(q, dtype) if Hq else None,
                                q_weight=gpu(wq, dtype) if Hq else None, k_weight=gpu(wk, dtype), cos=gpu(cos), sin=gpu(sin),
                                weight_offset=1.0 if R else 0.0, eps=1e-5)
        pos = [-1] * (M + spare_rows)
        for m, place in enumerate(oa.places(starts, lens, table, page, pages, M + spare_rows)):
            if place:
                pos[m] = place[1]
        kx, tol = oa.norm_rope(k, wk, cos, sin, pos, False, 1.0, 1e-5) if R else (k, 0 * k)
        kx, tol = np.nan_to_num(kx), np.nan_to_num(tol)  # rows of no sequence
        got = [t.cpu().numpy() for t in c]
        check_codes(got[0], got[2], kx, tol, parts[0], parts[2], starts, lens, table, page, "k")
        want = oa.append(v, by_token(parts[1]), parts[3], starts, lens, table, page)
        assert same_codes(by_token(got[1]), want[0])
        assert np.array_equal(got[3], want[1])
        if not R:
            want = oa.append(k, parts[0], parts[2], starts, lens, table, page)
            assert same_codes(got[0], want[0]) and np.array_equal(got[2], want[1])
        if Hq:
            want, tol = oa.norm_rope(q[:M], wq, cos, sin, pos, False, 1.0, 1e-5)
            within(out[:M], want, tol, dtype, "q")
        else:
            assert out is None


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (5, 64), (16, 24)])
def test_token_by_token_then_growing_scales(page, D):
    """A page filled one token at a time, each larger than the ones before: the earlier codes follow."""
    rng = np.random.default_rng(11)
    n = 2 * page + 3
    starts, lens, table, pages = batch(rng, [0], [n], page)
    x = rounded(rng, (n, 2, D), "bf16") * 2.0 ** (np.arange(n) % page * 0.75).round()[:, None, None]
    parts = cache(rng, pages, 2, page, D)
    c, want = to_cache(parts), (parts[0], parts[2])
    g = on_gpu(x, "bf16")
    for i in range(n):
        fw.fp8w_kv_append(g[i:i + 1], g[i:i + 1], c, on_gpu(table), torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
        want = oa.append(x[i:i + 1], *want, None, [i + 1], table, page)
    got = [t.cpu().numpy() for t in c]
    for codes, scale in ((got[0], got[2]), (by_token(got[1]), got[3])):
        for t in range(n):
            p = table[0, t // page]
            assert np.array_equal(codes[p, :, t % page], want[0][p, :, t % page]), t
            assert np.array_equal(scale[p], want[1][p])


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (7, 48)])
def test_special_values_and_zeros(page, D):
    """Infinities and NaN become NaN codes and leave the page's scale alone; a page of zeros has the smallest."""
    rng = np.random.default_rng(12)
    starts, lens, table, pages = batch(rng, [0, 0, 2], [4, 3, 2], page)
    x = rounded(rng, (9, 1, D), "fp16")
    x[1, 0, 3], x[2, 0, 5], x[3, 0, 7] = np.inf, -np.inf, np.nan
    x[4:7] = 0.0
    x[7, 0, 0] = 65504.0
    x[8] = 2.0 ** -24
    parts = cache(rng, pages, 1, page, D)
    c = to_cache(parts)
    fw.fp8w_kv_append(on_gpu(x, "fp16"), on_gpu(x, "fp16"), c, on_gpu(table), on_gpu(lens), starts=on_gpu(starts))
    want = oa.append(x, parts[0], parts[2], starts, lens, table, page)
    want_v = oa.append(x, by_token(parts[1]), parts[3], starts, lens, table, page)
    for codes, scale, w in ((c.k.cpu().numpy(), c.k_scale.cpu().numpy(), want), (by_token(c.v.cpu().numpy()), c.v_scale.cpu().numpy(), want_v)):
        assert np.array_equal(scale, w[1])
        assert same_codes(codes, w[0])
    assert int(c.k_scale[table[1, 0], 0]) == 1


@pytest.mark.parametrize("page,D", [(16, 64), (5, 24)])
def test_absent_pages_and_rows_of_no_sequence(page, D):
    rng = np.random.default_rng(13)
    starts, lens, table, pages = batch(rng, [0, 3, 1], [2 * page, page, 2], page, extra_columns=0)
    table[0, 1], table[2, 0] = -1, pages  # no such pages
    lens[1] = 40 * page                   # far more tokens than the table has pages for: its new ones are behind it
    M = int(starts[-1])
    x = rounded(rng, (M + 2, 2, D), "bf16")
    q = on_gpu(rounded(rng, (M + 2, 3, D), "bf16"), "bf16")
    parts = cache(rng, pages, 2, page, D)
    c = to_cache(parts)
    q_out = torch.full_like(q, 9.0)
    fw.fp8w_kv_append(on_gpu(x, "bf16"), on_gpu(x, "bf16"), c, on_gpu(table), on_gpu(lens), starts=on_gpu(starts), q=q, q_out=q_out)
    want = oa.append(x, parts[0], parts[2], starts, lens, table, page)
    assert same_codes(c.k.cpu().numpy(), want[0])
    assert np.array_equal(c.k_scale.cpu().numpy(), want[1])
    assert torch.equal(q_out[:M], q[:M]) and (q_out[M:] == 9).all()
    # more new rows than tokens: the rows before the first token are absent
    parts = cache(rng, 4, 2, page, D)
    c = to_cache(parts)
    one = np.array([[2]], np.int32)
    fw.fp8w_kv_append(on_gpu(x[:4], "bf16"), on_gpu(x[:4], "bf16"), c, on_gpu(one), torch.tensor([3], dtype=torch.int32, device="cuda"),
                      starts=torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    want = oa.append(x[:4], parts[0], parts[2], [0, 4], [3], one, page)
    assert same_codes(c.k.cpu().numpy(), want[0])
    # no pages at all, and nothing to append
    for args in ((on_gpu(x[:1], "bf16"), fw.fp8w_kv_cache(0, 2, page, D), torch.zeros(1, 1, dtype=torch.int32, device="cuda")),
                 (on_gpu(x[:1], "bf16"), c, torch.zeros(1, 0, dtype=torch.int32, device="cuda")),
                 (on_gpu(x[:0], "bf16"), c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"))):
        y, cc, t = args
        before = cc.k.clone()
        fw.fp8w_kv_append(y, y, cc, t, torch.ones(t.shape[0], dtype=torch.int32, device="cuda"))
        assert torch.equal(cc.k, before)


def test_given_positions_and_strided_projection():
    """k and v as parts of one row with q, q written over itself, and positions that are not the places."""
    rng = np.random.default_rng(14)
    Hq, Hk, D, page = 6, 2, 128, 16
    starts, lens, table, pages = batch(rng, [4, 0], [20, 3], page)
    row = rounded(rng, (23, (Hq + 2 * Hk) * D), "bf16")
    g = on_gpu(row, "bf16")
    q, k, v = g[:, : Hq * D].unflatten(1, (Hq, D)), g[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D)), g[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    a = rng.uniform(-3, 3, (40, D // 2))
    cos, sin = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    pos = rng.integers(0, 40, 23).astype(np.int32)
    parts = cache(rng, pages, Hk, page, D)
    c = to_cache(parts)
    out = fw.fp8w_kv_append(k, v, c, on_gpu(table), on_gpu(lens), starts=on_gpu(starts), q=q, cos=on_gpu(cos), sin=on_gpu(sin),
                            positions=on_gpu(pos), q_out=q)
    x = row.reshape(23, -1, D)
    want, tol = oa.norm_rope(x[:, :Hq], None, cos, sin, pos)
    within(out, want, tol, "bf16", "q")
    kx, tol = oa.norm_rope(x[:, Hq: Hq + Hk], None, cos, sin, pos)
    check_codes(c.k.cpu().numpy(), c.k_scale.cpu().numpy(), kx, tol, parts[0], parts[2], starts, lens, table, page, "k")
    assert torch.equal(g[:, Hq * D:].cpu(), on_gpu(row, "bf16")[:, Hq * D:].cpu())


def test_replayed_graph_appends_again():
    rng = np.random.default_rng(15)
    starts, lens, table, pages = batch(rng, [9, 30], [1, 1], 16)
    x = on_gpu(rounded(rng, (2, 2, 64), "bf16"), "bf16")
    t, n = on_gpu(table), on_gpu(lens)
    c = fw.fp8w_kv_cache(pages, 2, 16, 64)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        fw.fp8w_kv_append(x, x, c, t, n)
    for i in range(3):
        x.copy_(on_gpu(rounded(rng, (2, 2, 64), "bf16", 1 + i), "bf16"))
        n.add_(1)
        want = fw.KVCache(*(p.clone() for p in c))
        fw.fp8w_kv_append(x, x, want, t, n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c, want))
