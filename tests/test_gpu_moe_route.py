"""fp4w_moe_route on the GPU: ids equal to the oracle's, weights within its bound."""

import itertools
import math

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from gpu_helpers import require_gpu
from moe_cases import rounded
from oracle import moe as om

pytestmark = pytest.mark.gpu

SIZES = [(1, 128, 8), (1, 1, 1), (3, 8, 8), (7, 60, 4), (5, 64, 1), (130, 65, 6), (4, 129, 8), (33, 256, 8), (2, 257, 3),
         (3, 512, 16), (2, 1000, 64), (2, 1024, 10), (4, 5, 7)]


def check(x64, t, topk, score, bias, renormalize, scale, exact_w=True):
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = fw.fp4w_moe_route(t.cuda(), topk, score, b, renormalize, scale)
    want_ids, want_w, rel = om.route(x64, topk, score, bias, renormalize, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().double().numpy()
    # 2^-149 and below: where an FP32 exponential runs out
    assert (np.abs(got - want_w) <= rel * np.abs(want_w) + 1e-37).all()


@pytest.mark.parametrize("score,bias,renormalize", itertools.product(("softmax", "sigmoid"), (False, True), (False, True)))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_oracle(size, score, bias, renormalize):
    require_gpu()
    M, E, topk = size
    rng = np.random.default_rng(M + 7 * E)
    b = rng.uniform(-0.2, 0.2, E).astype(np.float32) if bias else None
    for dtype in ("fp32", "bf16", "fp16"):
        x64, t = rounded(2 * rng.standard_normal((M, E)), dtype)
        check(x64, t, topk, score, b, renormalize, 2.5)


@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lowest_index(bias):
    require_gpu()
    rng = np.random.default_rng(4)
    x64, t = rounded(np.round(rng.standard_normal((64, 200))), "bf16")  # few distinct values
    x64[:8] = 1.0
    t[:8] = 1.0
    b = np.round(rng.standard_normal(200)).astype(np.float32) if bias else None
    for topk in (1, 8, 64):
        check(x64, t, topk, "sigmoid", b, True, 1.0)
    z = torch.tensor([[-0.0, 0.0, -0.0, 0.0]])
    assert fw.fp4w_moe_route(z.cuda(), 4)[0].tolist() == [[0, 1, 2, 3]]  # the two zeros are one value


@pytest.mark.parametrize("score,bias", itertools.product(("softmax", "sigmoid"), (False, True)))
def test_masks(score, bias):
    """-inf and NaN are never chosen; rows that leave too few, or none; the type's lowest value is a value; +inf."""
    require_gpu()
    low = float(np.finfo(np.float32).min)
    x = np.random.default_rng(5).standard_normal((8, 70)).astype(np.float32)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, ::2] = math.nan
    x[3, 1::4] = -math.inf
    x[4] = low
    x[5, :66] = low
    if score == "softmax":
        x[6, [3, 50]] = math.inf
    x[7, 5:] = -math.inf
    b = np.linspace(-0.5, 0.5, 70).astype(np.float32) if bias else None
    with np.errstate(all="ignore"):
        for renormalize in (False, True):
            check(x.astype(np.float64), torch.from_numpy(x), 8, score, b, renormalize, 1.0)
    ids, w = fw.fp4w_moe_route(torch.from_numpy(x[:3]).cuda(), 4, score, None)
    assert ids.tolist() == [[-1] * 4, [-1] * 4, [0, -1, -1, -1]]
    assert w.tolist() == [[0] * 4, [0] * 4, [1, 0, 0, 0]]


def test_masks_by_the_bias_and_low_precision_types():
    require_gpu()
    x = torch.zeros(2, 6, dtype=torch.float16)
    x[1] = torch.finfo(torch.float16).min
    b = torch.tensor([0.0, -math.inf, math.nan, 0.0, 0.0, -math.inf]).cuda()
    ids, w = fw.fp4w_moe_route(x.cuda(), 5, "softmax", b)
    assert ids.tolist() == [[0, 3, 4, -1, -1]] * 2
    assert torch.allclose(w.cpu(), torch.tensor([[1 / 3, 1 / 3, 1 / 3, 0, 0]] * 2))
    # a sigmoid that underflows to zero everywhere
    ids, w = fw.fp4w_moe_route(torch.full((1, 4), -200.0).cuda(), 2, "sigmoid")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]


def test_shapes_outputs_stream_and_graph():
    require_gpu()
    x = torch.randn(2, 5, 40, device="cuda")
    ids, w = fw.fp4w_moe_route(x, 3)
    assert ids.shape == w.shape == (2, 5, 3)
    for shape, k in (((0, 8), 2), ((3, 8), 0)):
        ids, w = fw.fp4w_moe_route(torch.zeros(shape, device="cuda"), k)
        assert ids.shape == (shape[0], k)
    ids, w = fw.fp4w_moe_route(torch.zeros(3, 0, device="cuda"), 2)  # no experts at all
    assert (ids == -1).all() and (w == 0).all()
    # nothing behind the last row is written
    ids = torch.full((12, 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((12, 3), 7.0, device="cuda")
    fw.fp4w_moe_route(x.view(10, 40), 3, ids=ids[:10], weights=w[:10])
    assert (ids[10:] == 77).all() and (w[10:] == 7).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = fw.fp4w_moe_route(x.view(10, 40), 3)
    s.synchronize()
    assert torch.equal(a[0], ids[:10]) and torch.equal(a[1], w[:10])
    y = x.view(10, 40).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.fp4w_moe_route(y, 3, ids=ids[:10], weights=w[:10])
    for k in range(3):
        y.copy_(torch.roll(x.view(10, 40), k + 1, 1))
        g.replay()
        torch.cuda.synchronize()
        a = fw.fp4w_moe_route(y, 3)
        assert torch.equal(a[0], ids[:10]) and torch.equal(a[1], w[:10])


def test_a_prompt_of_rows():
    require_gpu()
    x = torch.randn(20000, 256, device="cuda").to(torch.bfloat16)
    ids, w = fw.fp4w_moe_route(x, 8)
    want = x.float().sort(dim=-1, descending=True, stable=True).indices[:, :8].int()
    assert torch.equal(ids, want)
    p = x.double().gather(1, want.long()).softmax(-1)
    assert ((w.double() - p).abs() <= p * 60 * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_scores_below_the_range_of_fp32(renormalize, dtype):
    """Renormalised weights are ordinary numbers however small the chosen scores; a score that is 0 in FP64 weighs 0."""
    require_gpu()

    def check_rows(x64, t, *args):  # a row at a time: the bound grows with the largest logit
        for m in range(len(x64)):
            check(x64[m:m + 1], t[m:m + 1], *args)

    x = [[-103, -104, -105, -130], [-100, -101, -120, -99], [-200, -200, -200, -200], [-600, -601, -602, -640],
         [-87, -88, -89, -90], [3, -104, -105, -200], [0, -0.5, 0.25, -1], [-690, -760, -2000, -6e4], [-2000, -2001, -2002, -6e4]]
    x64, t = rounded(np.array(x), dtype)
    for topk in (1, 2, 3, 6):
        check_rows(x64, t, topk, "sigmoid", None, renormalize, 2.5)
        check_rows(x64, t, topk, "sigmoid", np.array([0.5, -0.5, 0.25, 2], np.float32), renormalize, 1.0)
    # a bias that chooses experts far below the top
    x = [[0, -120, -121, -119], [0, -88, -95, -104], [7, -600, -601, -640], [-200, -500, -501, -490], [0, -760, -2000, -6e4],
         [50, -60, -61, 49]]
    x64, t = rounded(np.array(x), dtype)
    for topk in (1, 2, 3, 4):
        for score in ("softmax", "sigmoid"):
            check_rows(x64, t, topk, score, np.array([-10, 1, 1, 2], np.float32), renormalize, 1.0)
    rng = np.random.default_rng(9)
    x64, t = rounded(2 * rng.standard_normal((30, 300)) - 150, dtype)
    x64[:, 7] = 0  # the top, which the bias keeps out
    t[:, 7] = 0
    b = rng.uniform(0.5, 1.0, 300).astype(np.float32)
    b[7] = -10
    for score in ("softmax", "sigmoid"):
        check_rows(x64, t, 8, score, b, renormalize, 1.0)


def test_masks_by_the_bias_against_the_oracle():
    """Masked by its key alone, an expert is never chosen but has its share of the softmax: the bias is for the choice."""
    require_gpu()
    x64, t = rounded(np.random.default_rng(10).standard_normal((5, 6)), "fp16")
    x64[4] = t[4] = float(np.finfo(np.float16).min)
    b = np.array([0, -math.inf, math.nan, 0, 0, -math.inf], np.float32)
    for score, renormalize in itertools.product(("softmax", "sigmoid"), (False, True)):
        check(x64, t, 5, score, b, renormalize, 1.0)
    ids, w = fw.fp4w_moe_route(t.cuda(), 5, "softmax", torch.from_numpy(b).cuda(), False)
    p = torch.from_numpy(x64).softmax(-1)
    assert (w[:, :3].cpu().double().sum(1) < 0.9).all()
    assert torch.allclose(w[:, :3].cpu().double(), p.gather(1, ids[:, :3].cpu().long()), rtol=1e-5)
    assert (ids[:, 3:] == -1).all() and (w[:, 3:] == 0).all()


@pytest.mark.parametrize("bias", [False, True])
def test_more_rows_than_waves(bias):
    """A wave per row: rows past the 4 x 2^20 of a launch are a wave's second."""
    require_gpu()
    M, E = (4 << 20) + 13, 3
    x = torch.empty(M, E, device="cuda").normal_()
    b = np.array([0.1, -0.2, 0.15], np.float32) if bias else None
    ids, w = fw.fp4w_moe_route(x, 2, "sigmoid", None if b is None else torch.from_numpy(b).cuda())
    for s in (slice(0, 13), slice(M - 40, M)):
        want_ids, want_w, rel = om.route(x[s].double().cpu().numpy(), 2, "sigmoid", b)
        assert np.array_equal(ids[s].cpu().numpy(), want_ids)
        assert (np.abs(w[s].cpu().double().numpy() - want_w) <= rel * want_w).all()
