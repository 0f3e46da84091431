"""Inputs of the tests between the projections of an attention block: batches
over a paged cache, on the host, and their way to the device."""

import numpy as np
import torch

import fp8_weight_only_fp4w_amd as fw
from oracle import attention as oa

TORCH_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step, relative
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half a step of the subnormals


def rounded(rng, shape, dtype, scale=1.0):
    """Normal values that dtype holds, as float64."""
    x = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TORCH_DT[dtype])
    return x.double().numpy()


def on_gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(TORCH_DT[dtype]) if dtype else t).to("cuda")


def batch(rng, held, new, page, spare=2, extra_columns=1):
    """(starts, lens, table, pages) of sequences that hold `held` tokens before
    `new` ones, on shuffled pages."""
    lens = [h + n for h, n in zip(held, new)]
    each = [-(-t // page) for t in lens]
    pages = sum(each) + spare
    ids = rng.permutation(pages)
    table = np.full((len(lens), max(each, default=0) + extra_columns), -1, np.int32)
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = ids[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return starts, np.array(lens, np.int32), table, pages


def cache(rng, pages, heads, page, D, nan_slots=True):
    """(k, v, k_scale, v_scale): every code in every slot, NaN codes too unless
    told otherwise, and scales around one."""
    k = rng.integers(0, 256, (pages, heads, page, D), dtype=np.uint8)
    v = rng.integers(0, 256, (pages, heads, D, page), dtype=np.uint8)
    if not nan_slots:
        for c in (k, v):
            c[(c & 127) == 127] = 5
    ks = rng.integers(117, 122, (pages, heads), dtype=np.uint8)
    vs = rng.integers(119, 124, (pages, heads), dtype=np.uint8)
    return k, v, ks, vs


def filled(rng, starts, lens, table, page, pages, heads, D):
    """A cache whose held tokens are ordinary values, with NaN codes and every
    other code in the slots that hold none."""
    k, v, ks, vs = cache(rng, pages, heads, page, D)
    for b, length in enumerate(lens):
        for t in range(min(int(length), table.shape[1] * page)):
            p = table[b, t // page]
            if 0 <= p < pages:
                k[p, :, t % page] = oa.encode(np.clip(rng.standard_normal((heads, D)) * 60, -448, 448))
                v[p, :, :, t % page] = oa.encode(np.clip(rng.standard_normal((heads, D)) * 60, -448, 448))
    return k, v, ks, vs


def to_cache(parts):
    return fw.KVCache(*(on_gpu(p) for p in parts))


def within(got, want, tol, dtype, what=""):
    """got (a tensor) against want +- tol, rounded to dtype: NaN where want is NaN."""
    g = got.double().cpu().numpy()
    assert g.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN at other places, first {np.argwhere(np.isnan(g) != nan)[:3].tolist()}"
    inf = np.isinf(want)
    assert np.array_equal(g[inf], want[inf]), f"{what}: infinities differ"
    on = ~(nan | inf)
    err = np.abs(g[on] - want[on])
    far = err - (tol[on] + STEP[dtype] * (np.abs(want[on]) + tol[on]) + TINY[dtype])
    assert not (far > 0).any(), f"{what}: {int((far > 0).sum())} of {far.size} outside, worst by {far.max():.3g} at {want[on][far.argmax()]:.6g} (tol {tol[on][far.argmax()]:.3g}, err {err[far.argmax()]:.3g})"
