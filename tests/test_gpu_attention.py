"""Attention over the paged 8-bit cache on the GPU, against the float64 oracle,
through every kernel that takes the case."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from attention_cases import batch, cache, filled, on_gpu, rounded, to_cache, within
from gpu_helpers import require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def paths(D, page, rows):
    """The kernels that take heads of D, pages of `page` tokens and `rows` rows of a sequence and key head."""
    got = [fw.PATH_AUTO, fw.PATH_ATTN_GENERIC]
    if D in (64, 128) and page % 16 == 0:
        got += [fw.PATH_ATTN_PROMPT] + ([fw.PATH_ATTN_DECODE] if rows <= 64 else [])
    return got


def check(q, parts, starts, lens, table, dtype, scale=None, causal=True, window=0, which=None, use_starts=True, max_new=None):
    """Every path against the oracle; rows of no sequence left alone."""
    M, Hq, D = q.shape
    Hk, page = parts[0].shape[1:3]
    new = np.diff(starts)
    if scale is None:
        scale = D ** -0.5
    Y, L, tol, tol_l = oa.attention(q, *parts, starts, lens, table, scale, causal, window, dtype)
    behind = int(starts[-1])
    c, g, n = to_cache(parts), on_gpu(q, dtype), on_gpu(lens)
    # the decode kernel has a form of its own for tables with room for up to 1024 tokens
    wide = np.pad(table, ((0, 0), (0, -(-1040 // page))), constant_values=-1)
    st = on_gpu(starts) if use_starts else None
    got = []
    for path in which or paths(D, page, int(new.max(initial=0)) * Hq // Hk):
        out = torch.full_like(g, 9.0)
        lse = torch.full((M, Hq), 9.0, device="cuda")
        t = on_gpu(wide if path == fw.PATH_ATTN_DECODE else table)
        fw.fp8w_attention(g, c, t, n, starts=st, max_new=int(new.max(initial=0)) if max_new is None else max_new, scale=scale,
                          causal=causal, window=window, out=out, lse=lse, path=path)
        torch.cuda.synchronize()
        what = f"path {fw.fp4w_path_name(path)}"
        within(out[:behind], Y[:behind], tol[:behind], dtype, what)
        assert (out[behind:] == 9).all() and (lse[behind:] == 9).all(), what
        l, want = lse[:behind].double().cpu().numpy(), L[:behind]
        fine = np.isfinite(want)
        assert np.array_equal(np.isnan(l), np.isnan(want)) and np.array_equal(l[np.isinf(want)], want[np.isinf(want)]), what
        assert (np.abs(l[fine] - want[fine]) <= tol_l[:behind][fine] + 2.0 ** -24 * np.abs(want[fine])).all(), what
        got.append(out)
    return got


# held before, new, page, Hq, Hk, D, window
CASES = [
    ([0], [1], 16, 1, 1, 64, 0),
    ([900], [1], 64, 40, 8, 128, 0),
    ([0, 1, 15, 16, 62, 63, 64, 65, 127], [1] * 9, 16, 5, 1, 128, 0),
    ([300, 0, 5], [1, 1, 1], 16, 16, 1, 64, 0),
    ([1000, 10], [1, 1], 32, 34, 2, 64, 0),        # 17 rows of a key head
    ([130, 7], [1, 1], 16, 64, 1, 128, 0),         # 64 rows
    ([200, 3, 70], [2, 4, 3], 32, 28, 4, 64, 0),
    ([513, 64], [5, 3], 128, 6, 2, 128, 0),
    ([40, 3], [4, 2], 16, 16, 2, 128, 20),         # 32 rows
    ([60, 0, 200], [5, 7, 2], 16, 16, 2, 128, 0),  # 56 rows
    ([700, 3], [3, 3], 64, 22, 1, 64, 0),          # 66 rows: too many
    ([400, 100], [1, 2], 16, 8, 2, 128, 50),
    ([5000], [1], 16, 4, 4, 128, 0),
    ([4100, 3], [1, 1], 64, 7, 1, 64, 1000),
    ([0, 30], [70, 41], 16, 4, 2, 64, 0),          # prompts
    ([0], [257], 64, 5, 1, 128, 0),
    ([100, 0, 5], [33, 1, 64], 32, 8, 8, 128, 0),
    ([70], [150], 16, 3, 1, 128, 64),
    ([2000], [20], 16, 12, 2, 64, 0),
    ([300], [200], 128, 2, 2, 64, 1),
    ([17, 0, 90], [9, 0, 1], 16, 2, 1, 128, 0),    # a sequence without new tokens
    # heads and pages that no tile holds
    ([40, 3], [1, 5], 7, 4, 2, 64, 0),
    ([33], [2], 16, 3, 1, 80, 0),
    ([20], [3], 1, 2, 2, 16, 5),
    ([300], [1], 16, 2, 1, 256, 0),
    ([10], [2], 24, 2, 2, 1024, 0),
    ([9], [4], 16, 1, 1, 1, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}seq-{max(c[0])}+{max(c[1])}-p{c[2]}-{c[3]}/{c[4]}x{c[5]}-w{c[6]}")
def test_against_oracle(case, dtype):
    held, new, page, Hq, Hk, D, window = case
    rng = np.random.default_rng(sum(held) * 31 + D + page)
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    spare = 0 if set(new) == {1} else 2
    q = rounded(rng, (sum(new) + spare, Hq, D), dtype, 1.5)
    check(q, parts, starts, lens, table, dtype, window=window, use_starts=set(new) != {1})


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (48, 10)])
def test_not_causal(D, page):
    rng = np.random.default_rng(21)
    starts, lens, table, pages = batch(rng, [90, 0, 3], [7, 20, 1], page)
    parts = filled(rng, starts, lens, table, page, pages, 2, D)
    q = rounded(rng, (28, 4, D), "bf16")
    check(q, parts, starts, lens, table, "bf16", causal=False)
    check(q, parts, starts, lens, table, "bf16", causal=False, window=9, scale=-0.2)


@pytest.mark.parametrize("D,page,Hq", [(128, 16, 6), (128, 16, 10), (128, 32, 24), (64, 32, 6), (40, 8, 6)])
def test_rows_without_a_token(D, page, Hq):
    """Sequences that hold nothing, pages that are absent in the middle or throughout, more new rows than tokens."""
    rng = np.random.default_rng(22)
    starts, lens, table, pages = batch(rng, [0, 200, 40, 0, 300], [3, 2, 4, 5, 1], page)
    lens[0] = 0                       # three rows at positions -3 .. -1
    table[1, 1:-2] = -1
    table[2, :] = pages + 5
    lens[3] = 2                       # five rows, two tokens
    lens[4] = 2 ** 31 - 1             # more than the table has pages for; the row is behind them all
    parts = filled(rng, starts, np.minimum(lens, 400), table, page, pages, 2, D)
    q = rounded(rng, (15, Hq, D), "bf16")
    check(q, parts, starts, lens, table, "bf16")
    check(q, parts, starts, lens, table, "bf16", window=2)
    # the batch without any page, and without any token
    y = fw.fp8w_attention(on_gpu(q[:2], "bf16"), fw.fp8w_kv_cache(0, 2, page, D), torch.zeros(2, 3, dtype=torch.int32, device="cuda"),
                          torch.full((2,), 9, dtype=torch.int32, device="cuda"))
    assert (y == 0).all()
    y = fw.fp8w_attention(on_gpu(q[:2], "bf16"), to_cache(parts), torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                          torch.full((2,), 9, dtype=torch.int32, device="cuda"))
    assert (y == 0).all()
    assert fw.fp8w_attention(on_gpu(q[:0], "bf16"), to_cache(parts), on_gpu(table[:0]), on_gpu(lens[:0])).shape == (0, Hq, D)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 3, 8, 14, 40])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (24, 6)])
def test_nan_and_infinity_where_they_are_masked(D, page, n, dtype):
    """A later token's NaN value or key, or a NaN scale of a page before the window, does not reach a row that does not
    attend it; a row that does has NaN in the values concerned."""
    rng = np.random.default_rng(23)
    held = 5 * page + 3
    starts, lens, table, pages = batch(rng, [held, 2], [n, n], page)
    parts = filled(rng, starts, lens, table, page, pages, 1, D)
    k, v, ks, vs = parts
    last = held + n - 1
    v[table[0, last // page], 0, D // 2, last % page] = 0x7F     # the last token's value: NaN in one place
    if n > 2:
        t = held + 1
        v[table[0, t // page], 0, 1, t % page] = 0xFF
        k[table[0, t // page], 0, t % page, 3] = 0x7F            # and a key
    ks[table[0, 0], 0], vs[table[0, 1], 0] = 255, 255            # pages that only a call without a window attends
    q = rounded(rng, (2 * n, 4, D), dtype)
    for window in (2 * page, n + 1, 0):
        Y = oa.attention(q, *parts, starts, lens, table, 1.0, True, window)[0]
        assert np.isnan(Y).any() and not np.isnan(Y[n:]).any()
        if n > 1 and 0 < window <= held - 2 * page:  # the first row attends neither of those pages, nor a later token
            assert not np.isnan(Y[0]).any()
        check(q, parts, starts, lens, table, dtype, scale=1.0, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 50])
def test_scales_at_both_ends(n, dtype):
    """Page scales from 2^-127 up, scores of some hundreds either way, and one token that outweighs all."""
    rng = np.random.default_rng(24)
    D, page = 64, 16
    starts, lens, table, pages = batch(rng, [200, 20], [n, n], page)
    parts = filled(rng, starts, lens, table, page, pages, 2, D)
    parts[2][:] = rng.integers(112, 128, parts[2].shape)
    parts[3][:] = rng.integers(100, 128, parts[3].shape) if dtype == "bf16" else rng.integers(112, 128, parts[3].shape)
    parts[2][0], parts[3][1] = 0, 0
    q = rounded(rng, (2 * n, 4, D), dtype, 4.0)
    check(q, parts, starts, lens, table, dtype, scale=0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_infinite_queries_and_zero_scale(n):
    rng = np.random.default_rng(25)
    starts, lens, table, pages = batch(rng, [60], [n], 16)
    parts = filled(rng, starts, lens, table, 16, pages, 1, 64)
    q = rounded(rng, (n, 2, 64), "bf16")
    check(q, parts, starts, lens, table, "bf16", scale=0.0)
    q[0, 0, 5], q[-1, 1, 6] = np.nan, np.inf
    c = to_cache(parts)
    for path in paths(64, 16, 2 * n):
        y = fw.fp8w_attention(on_gpu(q, "bf16"), c, on_gpu(table), on_gpu(lens), starts=on_gpu(starts), max_new=n, path=path)
        bad = torch.isnan(y).all(-1).cpu().numpy()
        assert bad[0, 0] and bad[-1, 1] and bad.sum() == 2, path


def test_tokens_behind_max_new_are_left():
    rng = np.random.default_rng(26)
    starts, lens, table, pages = batch(rng, [30, 30], [6, 2], 16)
    parts = filled(rng, starts, lens, table, 16, pages, 2, 64)
    q = rounded(rng, (8, 4, 64), "bf16")
    Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 0.125)
    c = to_cache(parts)
    for path in paths(64, 16, 6):
        out = torch.full((8, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        fw.fp8w_attention(on_gpu(q, "bf16"), c, on_gpu(table), on_gpu(lens), starts=on_gpu(starts), max_new=3, out=out, path=path)
        on = [0, 1, 2, 6, 7]
        within(out[on], Y[on], tol[on], "bf16")
        assert (out[3:6] == 9).all()


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (3, 3)])
def test_many_sequences(Hq, Hk):
    """More sequences than a workgroup has threads, of lengths from nothing to some hundreds."""
    rng = np.random.default_rng(27)
    B = 1300
    held = (rng.integers(0, 2, B) * rng.integers(0, 60, B)).tolist()
    held[700] = 900
    new = rng.integers(0, 3, B).tolist()
    starts, lens, table, pages = batch(rng, held, new, 16)
    parts = cache(rng, pages, Hk, 16, 64, nan_slots=False)
    q = rounded(rng, (sum(new) + 3, Hq, 64), "bf16")
    check(q, parts, starts, lens, table, "bf16")


@pytest.mark.parametrize("path", [fw.PATH_ATTN_DECODE, fw.PATH_ATTN_PROMPT, fw.PATH_ATTN_GENERIC])
def test_same_bits_again_and_for_a_dirty_workspace(path):
    rng = np.random.default_rng(28)
    starts, lens, table, pages = batch(rng, [3000, 50, 1200], [2, 1, 2], 16)
    parts = cache(rng, pages, 2, 16, 128, nan_slots=False)
    q = on_gpu(rounded(rng, (5, 8, 128), "bf16"), "bf16")
    c, t, n, s = to_cache(parts), on_gpu(table), on_gpu(lens), on_gpu(starts)
    size = fw.fp8w_attention_workspace(5, 8, 2, 128, 3, 2)
    want = None
    for fill in (0, 255, 127):
        work = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        y = fw.fp8w_attention(q, c, t, n, starts=s, max_new=2, workspace=work[:size], path=path)
        assert (work[size:] == fill).all()
        want = y if want is None else want
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    if size:
        with pytest.raises(fw.FP4WError):
            fw.fp8w_attention(q, c, t, n, starts=s, max_new=2, workspace=work[:size - 1], path=path)


def test_strided_query_and_unaligned_parts():
    """q as a part of a projection's row, and a cache and a query that no vector load takes."""
    rng = np.random.default_rng(29)
    starts, lens, table, pages = batch(rng, [100], [3], 16)
    parts = filled(rng, starts, lens, table, 16, pages, 2, 64)
    q = rounded(rng, (3, 4, 64), "bf16")
    Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 0.125)
    t, n, s = on_gpu(table), on_gpu(lens), on_gpu(starts)
    for pad in (0, 8, 1):
        row = torch.zeros(3, 8 * 64 + pad, dtype=torch.bfloat16, device="cuda")
        view = row[:, pad: pad + 256].unflatten(1, (4, 64))
        view.copy_(on_gpu(q, "bf16"))
        within(fw.fp8w_attention(view, to_cache(parts), t, n, starts=s, max_new=3), Y, tol, "bf16", f"pad {pad}")
    c = to_cache(parts)
    moved = []
    for p in c[:2]:
        flat = torch.zeros(p.numel() + 1, dtype=torch.uint8, device="cuda")
        flat[1:].copy_(p.flatten())
        moved.append(flat[1:].view(p.shape))
    odd = fw.KVCache(*moved, *c[2:])
    within(fw.fp8w_attention(on_gpu(q, "bf16"), odd, t, n, starts=s, max_new=3), Y, tol, "bf16", "unaligned cache")
    with pytest.raises(fw.FP4WError):
        fw.fp8w_attention(on_gpu(q, "bf16"), odd, t, n, starts=s, max_new=3, path=fw.PATH_ATTN_DECODE)


def test_two_streams_at_once():
    rng = np.random.default_rng(30)
    calls = []
    for i in range(2):
        starts, lens, table, pages = batch(rng, [700 + 900 * i, 40], [1, 1], 16)
        parts = filled(rng, starts, lens, table, 16, pages, 2, 128)
        q = rounded(rng, (2, 10, 128), "bf16")
        calls.append((on_gpu(q, "bf16"), to_cache(parts), on_gpu(table), on_gpu(lens)))
    want = [fw.fp8w_attention(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(fw.fp8w_attention(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_follows_growing_sequences():
    """One captured call serves every length that the page table has room for."""
    rng = np.random.default_rng(31)
    starts, lens, table, pages = batch(rng, [2000, 1500], [1, 1], 16)
    parts = cache(rng, pages, 2, 16, 64, nan_slots=False)
    c, t, n = to_cache(parts), on_gpu(table), on_gpu(lens)
    q = on_gpu(rounded(rng, (2, 8, 64), "bf16"), "bf16")
    out = torch.empty_like(q)
    work = torch.empty(fw.fp8w_attention_workspace(2, 8, 2, 64, 2, 1), dtype=torch.uint8, device="cuda")
    fw.fp8w_attention(q, c, t, n, out=out, workspace=work)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        fw.fp8w_attention(q, c, t, n, out=out, workspace=work)
    for length in ((1, 1), (17, 900), (2001, 3), (0, 1501), (2001, 1501)):
        n.copy_(torch.tensor(length, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fw.fp8w_attention(q, c, t, n)), length
