"""The operators between the projections of an attention block where counts are
large: prompts with more row tiles than the GPU has places, and caches past
2^32 bytes."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from attention_cases import STEP, TINY, batch, cache, on_gpu, to_cache
from gpu_helpers import require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu
U = oa.U


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def dense(q, parts, lens, starts, table, window, half):
    """(Y, tol) in float64 on the GPU, sequence by sequence; tol as in the oracle's attention()."""
    codes, page, (M, Hq, D) = on_gpu(oa.TABLE), parts[0].shape[2], q.shape
    k, v = (codes[on_gpu(parts[i]).long()] * on_gpu(oa.power(parts[i + 2]))[:, :, None, None] for i in (0, 1))
    G = Hq // k.shape[1]
    Y, tol = torch.zeros(M, Hq, D, dtype=torch.float64, device="cuda"), torch.zeros(M, Hq, D, dtype=torch.float64, device="cuda")
    scale = float(np.float32(D ** -0.5))
    for b, n in enumerate(lens.tolist()):
        ids = on_gpu(table[b, :-(-n // page)]).long()
        kb = k[ids].transpose(1, 2).reshape(-1, k.shape[1], D)[:n]
        vb = v[ids].permute(0, 3, 1, 2).reshape(-1, k.shape[1], D)[:n]
        rows = slice(int(starts[b]), int(starts[b + 1]))
        new = int(starts[b + 1] - starts[b])
        pos = torch.arange(n - new, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        on = (t <= pos) & ((t > pos - window) if window else True)
        for h in range(Hq):
            x, kh, vh = q[rows, h], kb[:, h // G].contiguous(), vb[:, h // G].contiguous()
            s, size = x @ kh.t() * scale, x.abs() @ kh.abs().t() * scale
            s = s.masked_fill(~on, -torch.inf)
            top = s.amax(1, keepdim=True)
            w = torch.softmax(s, 1)
            y = w @ vh
            err = (D + 6) * U * size + 6 * U * (s.masked_fill(~on, 0.0).abs() + top.abs()) + 4 * U
            sums = (on.sum(1, keepdim=True) + 16) * U
            Y[rows, h] = y
            tol[rows, h] = (w * (err + half + sums)) @ vh.abs() + y.abs() * ((w * err).sum(1, keepdim=True) + sums)
            if half == 2.0 ** -11:  # numerators from 2^-33 up, values in steps of 2^-24
                tol[rows, h] += n * 2.0 ** -33 * vh.abs().amax(0) + 2.0 ** -24
    return Y, tol


@pytest.mark.parametrize("Hq,Hk,D,page,window,dtype", [(64, 8, 128, 64, 0, "bf16"), (56, 8, 64, 16, 300, "fp16"), (40, 8, 128, 16, 700, "fp16"),
                                                     (64, 16, 64, 128, 0, "bf16")])
def test_prompts_that_fill_the_gpu(Hq, Hk, D, page, window, dtype):
    rng = np.random.default_rng(60)
    new = [1100, 1, 903]
    starts, lens, table, pages = batch(rng, [0, 700, 130], new, page)
    parts = cache(rng, pages, Hk, page, D, nan_slots=False)
    q = on_gpu(rng.standard_normal((sum(new), Hq, D)).astype(np.float32), dtype)
    Y, tol = dense(q.double(), parts, lens, starts, table, window, STEP[dtype])
    for path in (fw.PATH_AUTO, fw.PATH_ATTN_GENERIC):
        got = fw.fp8w_attention(q, to_cache(parts), on_gpu(table), on_gpu(lens), starts=on_gpu(starts), max_new=1100, window=window, path=path)
        far = (got.double() - Y).abs() - (tol + STEP[dtype] * (Y.abs() + tol) + TINY[dtype])
        assert not (far > 0).any(), f"path {path}: {int((far > 0).sum())} outside, worst by {far.max().item():.3g}"


def test_many_drafted_rows_over_long_sequences():
    """64 rows of a key head, cut into many shares."""
    rng = np.random.default_rng(61)
    for Hq, Hk, D, new, dtype in ((32, 4, 128, [8, 3, 0, 7], "bf16"), (33, 1, 128, [1, 1, 1, 1], "fp16"), (40, 8, 128, [5, 5, 2, 4], "fp16"), (24, 2, 64, [5, 1, 4, 2], "bf16")):
        starts, lens, table, pages = batch(rng, [9000, 20000, 5, 63], new, 16)
        parts = cache(rng, pages, Hk, 16, D, nan_slots=False)
        q = on_gpu(rng.standard_normal((sum(new), Hq, D)).astype(np.float32), dtype)
        for window in (0, 6000):
            Y, tol = dense(q.double(), parts, lens, starts, table, window, STEP[dtype])
            for path in (fw.PATH_AUTO, fw.PATH_ATTN_DECODE, fw.PATH_ATTN_PROMPT):
                got = fw.fp8w_attention(q, to_cache(parts), on_gpu(table), on_gpu(lens), starts=on_gpu(starts), max_new=max(new), window=window,
                                        path=path)
                far = (got.double() - Y).abs() - (tol + STEP[dtype] * (Y.abs() + tol) + TINY[dtype])
                assert not (far > 0).any(), f"{Hq} heads, path {path}: {int((far > 0).sum())} outside, worst by {far.max().item():.3g}"


@pytest.mark.parametrize("D,page,pages", [(128, 64, 66000), (128, 24, 176000)])
def test_pages_past_32_bit_offsets(D, page, pages):
    """A call on pages at the end of a large cache does what it does on the same pages of a small one."""
    Hq, Hk, new = 8, 8, [40, 3]
    assert pages * page * D * Hk > 1 << 32
    rng = np.random.default_rng(62)
    starts, lens, table, few = batch(rng, [100, 17], new, page)
    far = np.where(table >= 0, pages - few + table, -1).astype(np.int32)
    small, large = fw.fp8w_kv_cache(few, Hk, page, D), fw.fp8w_kv_cache(pages, Hk, page, D)
    for s, g, p in zip(small, large, cache(rng, few, Hk, page, D, nan_slots=False)):
        s.copy_(on_gpu(p))
        g[-few:].copy_(s)
    q, k, v = (on_gpu(rng.standard_normal((sum(new), 8, D)).astype(np.float32), "bf16") for _ in range(3))
    st, n = on_gpu(starts), on_gpu(lens)
    got = []
    for c, t in ((small, on_gpu(table)), (large, on_gpu(far))):
        fw.fp8w_kv_append(k, v, c, t, n, starts=st)
        got.append([x[-few:].clone() for x in c])
        rows = on_gpu(np.array([39, 42]))
        one = [fw.fp8w_attention(q[rows], c, t, n)]  # one new token each
        for path in [fw.PATH_AUTO, fw.PATH_ATTN_GENERIC] + ([fw.PATH_ATTN_DECODE] if page % 16 == 0 else []):
            one.append(fw.fp8w_attention(q, c, t, n, starts=st, max_new=40, path=path))
        got[-1] += [x.view(torch.int16) for x in one]
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][4].abs().max() > 0 and not torch.equal(got[0][0], got[0][1].transpose(2, 3))
