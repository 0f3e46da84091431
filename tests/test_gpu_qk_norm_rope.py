"""Norms of query and key heads with the rotation, on the GPU, against the
float64 oracle; and the same values in and out of strided projections."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from attention_cases import TORCH_DT, on_gpu, rounded, within
from gpu_helpers import require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def tables(rng, rows, R):
    a = rng.uniform(-3.2, 3.2, (rows, R // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# M, Hq, Hk, D, R, norm of q, norm of k, interleaved, offset
CASES = [
    (1, 40, 8, 128, 128, True, True, False, 0.0),
    (1, 1, 0, 64, 64, False, False, False, 0.0),
    (7, 5, 1, 64, 32, True, False, True, 1.0),
    (300, 14, 2, 64, 64, False, True, False, 0.0),
    (33, 8, 8, 128, 64, True, True, True, 0.0),
    (5, 4, 4, 256, 256, True, True, False, 0.0),
    (9, 3, 2, 512, 0, True, True, False, 1.0),
    (4, 2, 1, 1024, 1024, True, True, False, 0.0),
    (11, 3, 3, 16, 16, True, True, False, 0.0),
    (6, 2, 2, 32, 16, True, True, False, 0.0),
    # head sizes and rotated parts that no vector holds
    (5, 3, 2, 80, 80, True, True, False, 0.0),
    (4, 3, 1, 96, 24, True, True, True, 0.0),
    (3, 2, 1, 1, 0, True, True, False, 0.0),
    (3, 2, 1, 2, 2, False, True, True, 0.0),
    (2, 2, 2, 127, 126, True, True, False, 0.0),
    (3, 1, 1, 128, 2, False, False, False, 0.0),
    (5000, 3, 1, 64, 64, True, True, False, 0.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_against_oracle(case, dtype):
    M, Hq, Hk, D, R, nq, nk, interleaved, offset = case
    rng = np.random.default_rng(M * 1000 + D)
    q, k = rounded(rng, (M, Hq, D), dtype, 1.5), rounded(rng, (M, Hk, D), dtype, 1.5)
    wq = rounded(rng, D, dtype) if nq else None
    wk = rounded(rng, D, dtype) if nk else None
    cos, sin = tables(rng, 50, R) if R else (None, None)
    pos = rng.integers(0, 50, M).astype(np.int32)
    gpu = lambda x: None if x is None else on_gpu(x)  # noqa: E731
    args = dict(q_weight=None if wq is None else on_gpu(wq, dtype), k_weight=None if wk is None or not Hk else on_gpu(wk, dtype),
                cos=gpu(cos), sin=gpu(sin), positions=on_gpu(pos), interleaved=interleaved, weight_offset=offset, eps=1e-5)
    gq, gk = on_gpu(q, dtype), on_gpu(k, dtype) if Hk else None
    yq, yk = fw.fp4w_qk_norm_rope(gq, gk, **args)
    want, tol = oa.norm_rope(q, wq, cos, sin, pos, interleaved, offset, 1e-5)
    within(yq, want, tol, dtype, "q")
    if Hk:
        want, tol = oa.norm_rope(k, wk, cos, sin, pos, interleaved, offset, 1e-5)
        within(yk, want, tol, dtype, "k")
    # in place, and as parts of one projection's rows: the same bits where both are in 16-byte pieces
    for pad in (0, 8, 3):
        width = (Hq + 2 * Hk) * D + pad
        flat = torch.full((M * width + pad,), 7.0, dtype=TORCH_DT[dtype], device="cuda")
        rows = flat[pad:].view(M, width)
        vq = rows[:, : Hq * D].unflatten(1, (Hq, D))
        vk = rows[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
        vq.copy_(gq)
        if Hk:
            vk.copy_(gk)
        a, b = fw.fp4w_qk_norm_rope(vq, vk, q_out=vq, k_out=vk, **args)
        assert a is vq and b is vk
        for got, same, x, w in ((a, yq, q, wq), (b, yk, k, wk))[: 2 if Hk else 1]:
            if pad == 3:
                want, tol = oa.norm_rope(x, w, cos, sin, pos, interleaved, offset, 1e-5)
                within(got.contiguous(), want, tol, dtype, "unaligned")
            else:
                assert torch.equal(got.contiguous().view(torch.int16), same.view(torch.int16)), pad
        assert (rows[:, (Hq + Hk) * D:] == 7).all()  # what lies between is left alone


@pytest.mark.parametrize("D", [64, 80])
def test_positions(D):
    """None counts from 0; a position outside the tables makes the rotated values NaN and no others."""
    rng = np.random.default_rng(3)
    x = rounded(rng, (6, 2, D), "bf16")
    cos, sin = tables(rng, 6, 32)
    q = on_gpu(x, "bf16")
    y, none = fw.fp4w_qk_norm_rope(q, cos=on_gpu(cos), sin=on_gpu(sin))
    assert none is None
    want, tol = oa.norm_rope(x, None, cos, sin)
    within(y, want, tol, "bf16")
    pos = np.array([5, 6, -1, 2 ** 31 - 1, -2 ** 31, 0], np.int32)
    y, _ = fw.fp4w_qk_norm_rope(q, cos=on_gpu(cos), sin=on_gpu(sin), positions=on_gpu(pos))
    want, tol = oa.norm_rope(x, None, cos, sin, pos)
    assert np.isnan(want[1:5, :, :32]).all()
    within(y, want, tol, "bf16")


@pytest.mark.parametrize("D", [128, 96])
def test_special_values_stay_in_their_heads(D):
    rng = np.random.default_rng(4)
    x = rounded(rng, (4, 3, D), "bf16")
    x[1, 1, 5], x[2, 0, 7], x[3, 2, :] = np.nan, np.inf, 0.0
    w = rounded(rng, D, "bf16")
    y, _ = fw.fp4w_qk_norm_rope(on_gpu(x, "bf16"), q_weight=on_gpu(w, "bf16"))
    bad = torch.isnan(y).any(-1).cpu().numpy()
    assert bad[1, 1] and bad[2, 0] and bad.sum() == 2 and (y[3, 2] == 0).all()


def test_empty():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = fw.fp4w_qk_norm_rope(q)
    assert y.shape == q.shape
    y, k = fw.fp4w_qk_norm_rope(torch.ones(3, 2, 64, dtype=torch.float16, device="cuda"), torch.empty(3, 0, 64, dtype=torch.float16, device="cuda"))
    assert (y == 1).all() and k.shape == (3, 0, 64)


def test_another_stream_and_graph():
    rng = np.random.default_rng(5)
    x = rounded(rng, (20, 6, 128), "bf16")
    w = rounded(rng, 128, "bf16")
    cos, sin = tables(rng, 20, 128)
    q, gw, gc, gs = on_gpu(x, "bf16"), on_gpu(w, "bf16"), on_gpu(cos), on_gpu(sin)
    out = torch.empty_like(q)
    want, _ = fw.fp4w_qk_norm_rope(q, q_weight=gw, cos=gc, sin=gs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fw.fp4w_qk_norm_rope(q, q_weight=gw, cos=gc, sin=gs, q_out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
