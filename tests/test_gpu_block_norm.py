"""fp4w_block_norm on the GPU against the oracle's float64 and its bound."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from gpu_helpers import require_gpu
from moe_cases import TORCH, assert_within, rounded
from oracle import moe as om

pytestmark = pytest.mark.gpu

# M, K, post, pre, gate rows (0, 1 or M), residual, offset: every length class
# of the kernel (one wave per row, a workgroup per row with 1 .. 16 values or
# chunks per thread, rows longer than the registers hold) and both widths
CASES = [
    (1, 1, True, True, 1, True, 0.0),
    (3, 8, True, True, 0, True, 1.0),
    (5, 63, False, True, 5, True, 0.0),
    (6, 64, True, False, 1, False, 0.0),
    (9, 512, True, True, 9, True, 0.0),
    (4, 520, False, True, 0, True, 0.0),
    (2, 1000, True, True, 2, True, 1.0),
    (3, 1001, True, True, 1, True, 0.0),
    (2, 2049, True, True, 2, True, 1.0),
    (1, 5120, True, True, 0, True, 0.0),
    (300, 5120, False, True, 1, True, 0.0),
    (2, 4099, True, True, 0, False, 0.0),
    (2, 9000, True, True, 2, True, 0.0),
    (2, 16384, True, True, 1, True, 0.0),
    (2, 20000, False, True, 0, True, 0.0),
    (2, 20001, True, True, 2, True, 1.0),
    (1, 40008, True, True, 1, True, 0.0),
    (7, 128, False, False, 7, True, 0.0),
]


def make(M, K, post, pre, gate, residual, offset, dtype, seed):
    rng = np.random.default_rng(seed)
    c = {"x": rounded(rng.standard_normal((M, K)), dtype)}
    if residual:
        c["residual"] = rounded(4 * rng.standard_normal((M, K)), dtype)
    if pre:
        c["pre"] = rounded(1 - offset + 0.3 * rng.standard_normal(K), dtype)
    if post:
        c["post"] = rounded(1 - offset + 0.3 * rng.standard_normal(K), dtype)
    if gate:
        c["gate"] = rounded(rng.uniform(-1, 1, (M, K) if gate == M and M > 1 else K), dtype)
    return c


def call(c, offset, scale=0.5, **kw):
    d = {k: v[1].cuda() for k, v in c.items()}
    d.update({k: v for k, v in kw.pop("use", {}).items()})
    return fw.fp4w_block_norm(d["x"], d.get("residual"), d.get("pre"), d.get("post"), d.get("gate"), scale, 1e-5, offset,
                              **kw)


def want(c, offset, scale=0.5):
    f = {k: v[0] for k, v in c.items()}
    return om.block_norm(f["x"], f.get("residual"), f.get("pre"), f.get("post"), f.get("gate"), scale, 1e-5, offset)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_against_oracle(case, dtype):
    require_gpu()
    M, K, post, pre, gate, residual, offset = case
    c = make(M, K, post, pre, gate, residual, offset, dtype, seed=M + K)
    r, y = call(c, offset)
    wr, wy, tr, ty = want(c, offset)
    assert_within(r, wr, tr, dtype, "residual_out")
    if pre:
        assert_within(y, wy, ty, dtype, "y")
    else:
        assert y is None


@pytest.mark.parametrize("K", [64, 1000, 1001, 20001])
def test_in_place_and_one_output(K):
    require_gpu()
    c = make(5, K, True, True, 5, True, 0.0, "bf16", 3)
    r, y = call(c, 0.0)
    for first, second in (("x", "residual"), ("residual", "x")):
        d = {k: c[k][1].cuda() for k in ("x", "residual")}
        r2, y2 = call(c, 0.0, use=d, residual_out=d[first], out=d[second])
        assert r2.data_ptr() == d[first].data_ptr() and y2.data_ptr() == d[second].data_ptr()
        assert torch.equal(r2, r) and torch.equal(y2, y)
    none, y3 = call(c, 0.0, write_residual=False)
    assert none is None and torch.equal(y3, y)


def test_unaligned_pointers_and_rows_behind():
    """A slice that starts off 16 bytes gives what an aligned copy gives, and nothing behind the last row is written."""
    require_gpu()
    c = make(3, 256, True, True, 1, True, 0.0, "fp16", 4)
    r, y = call(c, 0.0)
    room = torch.full((5 * 256 + 8,), 7.0, dtype=torch.float16, device="cuda")
    x = room.clone()[3:3 + 3 * 256].view(3, 256).copy_(c["x"][1])
    outs = [room.clone(), room.clone()]
    views = [o[1:1 + 3 * 256].view(3, 256) for o in outs]
    call(c, 0.0, use={"x": x}, residual_out=views[0], out=views[1])
    # the 2-byte path sums a row in another order: both are within the bound
    wr, wy, tr, ty = want(c, 0.0)
    assert_within(views[0], wr, tr, "fp16")
    assert_within(views[1], wy, ty, "fp16")
    assert_within(y, wy, ty, "fp16")
    for o in outs:
        assert (o[0] == 7).all() and (o[1 + 3 * 256:] == 7).all()


def test_zero_rows_infinities_and_nan_stay_in_their_row():
    require_gpu()
    c = make(4, 300, True, True, 0, True, 0.0, "bf16", 5)
    x, res = c["x"][1].clone(), c["residual"][1].clone()
    x[0] = 0
    res[0] = 0
    x[1, 7] = float("nan")
    res[2, 9] = float("inf")
    r, y = call(c, 0.0, use={"x": x.cuda(), "residual": res.cuda()})
    assert (r[0] == 0).all() and (y[0] == 0).all()  # eps keeps a zero row finite
    assert y[1].isnan().all() and r[1].isnan().all()
    assert r[2, 9].isinf() and y[2, 9].isnan() and (y[2, :9] == 0).all()
    wr, wy, tr, ty = want(c, 0.0)
    assert_within(y[3:], wy[3:], ty[3:], "bf16")


def test_many_rows_and_empty():
    require_gpu()
    M = 70000  # more rows than one wave per row leaves workgroups of at once
    x = torch.randn(M, 24, device="cuda").to(torch.bfloat16)
    w = torch.ones(24, dtype=torch.bfloat16, device="cuda")
    _, y = fw.fp4w_block_norm(x, pre_weight=w)
    f = x.double()
    ref = f / (f.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert ((y.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 1e-30).all()
    for shape in ((0, 24), (3, 0)):
        e = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        r, y = fw.fp4w_block_norm(e, pre_weight=torch.empty(shape[1], dtype=torch.bfloat16, device="cuda"))
        assert r.shape == y.shape == shape


def test_leading_dimensions_stream_and_graph():
    require_gpu()
    c = make(6, 1024, True, True, 1, True, 0.0, "bf16", 6)
    d = {k: v[1].cuda() for k, v in c.items()}
    d3 = {k: v.view(2, 3, 1024) if v.dim() == 2 else v for k, v in d.items()}
    eager = call(c, 0.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r, y = fw.fp4w_block_norm(d3["x"], d3["residual"], d["pre"], d["post"], d["gate"], 0.5, 1e-5)
    s.synchronize()
    assert r.shape == (2, 3, 1024) and torch.equal(y.view(6, 1024), eager[1])
    out = [torch.empty_like(d["x"]) for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call({}, 0.0, use=d, residual_out=out[0], out=out[1])
    for k in range(3):
        d["x"].copy_(torch.roll(c["x"][1], k, 0))
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        again = call({}, 0.0, use=d)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1]), k
    assert TORCH["bf16"] == out[0].dtype


@pytest.mark.parametrize("K,post,pre", [(65, True, True), (65, False, True), (65, True, False), (65, False, False), (16385, True, True)])
def test_more_rows_than_workgroups(K, post, pre):
    """Rows past the 2^20 workgroups of a launch: some take a second row, with the sums of the first behind them."""
    require_gpu()
    M = (1 << 20) + 70
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    some = [slice(0, 70), slice(M - 140, M)]  # the rows that a workgroup takes first and second, and some between
    c = {"x": (None, None)}
    w = [rounded(1 + 0.3 * np.random.default_rng(K + i).standard_normal(K), "bf16") for i in range(2)]
    x64 = np.concatenate([x[s].double().cpu().numpy() for s in some])
    if post:
        c["post"] = w[0]
    if pre:
        c["pre"] = w[1]
    d = {k: v[1].cuda() for k, v in c.items() if k != "x"}
    # in place where the rows are long (34 GB): one output
    r, y = fw.fp4w_block_norm(x, None, d.get("pre"), d.get("post"), None, 0.5, 1e-5,
                              **({"out": x, "write_residual": False} if K > 1000 else {}))
    wr, wy, tr, ty = om.block_norm(x64, None, w[1][0] if pre else None, w[0][0] if post else None, None, 0.5, 1e-5)
    for got, want, tol in ((r, wr, tr), (y, wy, ty)):
        if got is not None:
            assert_within(torch.cat([got[s] for s in some]), want, tol, "bf16", f"K {K}")


def test_more_rows_than_waves():
    """A wave per row: rows past 4 x 2^20."""
    require_gpu()
    M = (4 << 20) + 9
    x = torch.empty(M, 8, dtype=torch.bfloat16, device="cuda").normal_()
    pre64, pre = rounded(1 + 0.3 * np.random.default_rng(3).standard_normal(8), "bf16")
    _, y = fw.fp4w_block_norm(x, pre_weight=pre.cuda(), eps=1e-5)
    for s in (slice(0, 9), slice(M - 20, M)):
        _, want, _, tol = om.block_norm(x[s].double().cpu().numpy(), None, pre64, eps=1e-5)
        assert_within(y[s], want, tol, "bf16")


@pytest.mark.parametrize("K,off", [(4095, 0), (4096, 1), (4097, 0), (8193, 0), (16384, 3), (16384, 0), (16392, 0), (32768, 0), (32776, 0)])
def test_rows_at_the_borders_of_the_forms(K, off):
    """Lengths where another form of the kernel begins, aligned and off 16 bytes, apart and in place."""
    require_gpu()
    c = make(3, K, True, True, 3, True, 0.0, "bf16", K)

    def placed(t):
        room = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        return room[off:].view(t.shape).copy_(t)

    x, res = placed(c["x"][1]), placed(c["residual"][1])
    wr, wy, tr, ty = want(c, 0.0)
    r, y = call(c, 0.0, use={"x": x, "residual": res})
    assert_within(r, wr, tr, "bf16", "residual_out")
    assert_within(y, wy, ty, "bf16", "y")
    call(c, 0.0, use={"x": x, "residual": res}, residual_out=res, out=x)
    assert torch.equal(res, r) and torch.equal(x, y)
