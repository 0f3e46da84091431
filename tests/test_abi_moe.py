"""Argument checks of the entry points around a mixture-of-experts block.  No
call here reaches a kernel launch, and none needs a GPU."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from moe_cases import make_moe, moe_call, moe_on

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _vp(x):
    return ctypes.c_void_p(x)


def _norm(x=0x100000, M=4, K=64, post=None, gate=None, gate_rows=1, res=0x200000, pre=0x300000, r=0x400000, y=0x500000,
          dtype=fw.BF16):
    return fw.load_library().fp4w_block_norm(_vp(x), M, K, _vp(post), _vp(gate), gate_rows, 1.0, _vp(res), _vp(pre),
                                             0.0, 1e-6, _vp(r), _vp(y), dtype, None)


def test_block_norm_refusals():
    assert _norm(dtype=fw.F32) == fw.ERR_DTYPE
    assert _norm(M=-1) == fw.ERR_SHAPE
    assert _norm(M=1 << 40, K=1 << 40) == fw.ERR_SHAPE
    assert _norm(gate=0x600000, gate_rows=3) == fw.ERR_SHAPE
    assert _norm(x=None) == fw.ERR_NULL
    assert _norm(r=None, y=None, pre=None) == fw.ERR_NULL
    assert _norm(pre=None) == fw.ERR_NULL            # y without its weight
    assert _norm(y=None) == fw.ERR_NULL              # a weight without y
    assert _norm(r=0x100000 + 8) == fw.ERR_ALIAS     # partly over x
    assert _norm(y=0x200000 - 8) == fw.ERR_ALIAS     # partly over the residual
    assert _norm(y=0x400000) == fw.ERR_ALIAS         # both outputs
    assert _norm(r=0x300000 + 64) == fw.ERR_ALIAS    # over a weight
    assert _norm(gate=0x600000, gate_rows=4, y=0x600000) == fw.ERR_ALIAS
    assert _norm(x=None, M=0) == fw.OK and _norm(x=None, K=0) == fw.OK


def _route(logits=0x100000, M=4, E=16, topk=2, score=0, bias=None, ids=0x200000, w=0x300000, dtype=fw.F32):
    return fw.load_library().fp4w_moe_route(_vp(logits), M, E, topk, score, _vp(bias), 1, 1.0, _vp(ids), _vp(w), dtype,
                                            None)


def test_route_refusals():
    assert _route(dtype=3) == fw.ERR_DTYPE
    assert _route(score=2) == fw.ERR_DTYPE
    assert _route(M=-1) == fw.ERR_SHAPE
    assert _route(E=fw.MOE_MAX_EXPERTS + 1) == fw.ERR_SHAPE
    assert _route(topk=fw.MOE_MAX_TOPK + 1) == fw.ERR_SHAPE
    assert _route(topk=-1) == fw.ERR_SHAPE
    assert _route(M=1 << 58, E=1000) == fw.ERR_SHAPE
    assert _route(logits=None) == fw.ERR_NULL
    assert _route(ids=None) == fw.ERR_NULL
    assert _route(w=None) == fw.ERR_NULL
    assert _route(w=0x200000 + 16) == fw.ERR_ALIAS
    assert _route(ids=0x100000 + 128) == fw.ERR_ALIAS
    assert _route(bias=0x300000) == fw.ERR_ALIAS
    assert _route(logits=None, M=0) == fw.OK
    assert _route(ids=None, w=None, topk=0) == fw.OK


def _fp4(A=0x1000000, M=2, K=64, ids=0x2000000, w=0x2100000, topk=2, w13=0x3000000, s13=0x4000000, g13=0x5000000,
         w2=0x6000000, s2=0x7000000, g2=0x8000000, E=4, I=32, bs=16, act=0, work=0x9000000, bytes=None, Y=0xa000000,  # noqa: E741
         dtype=fw.BF16, path=0):
    lib = fw.load_library()
    if bytes is None:
        bytes = max(0, lib.fp4w_moe_workspace(M, topk, K, I))
    return lib.fp4w_moe_ex(_vp(A), M, K, _vp(ids), _vp(w), topk, _vp(w13), _vp(s13), _vp(g13), _vp(w2), _vp(s2), _vp(g2),
                           E, I, bs, act, _vp(work), bytes, _vp(Y), dtype, None, path)


def _fp8(A=0x1000000, M=2, K=64, ids=0x2000000, w=0x2100000, topk=2, w13=0x3000000, s13=0x4000000, w2=0x6000000,
         s2=0x7000000, E=4, I=32, bs=128, act=0, work=0x9000000, bytes=None, Y=0xa000000, dtype=fw.BF16, path=0):  # noqa: E741
    lib = fw.load_library()
    if bytes is None:
        bytes = max(0, lib.fp4w_moe_workspace(M, topk, K, I))
    return lib.fp8w_moe_ex(_vp(A), M, K, _vp(ids), _vp(w), topk, _vp(w13), _vp(s13), _vp(w2), _vp(s2), E, I, bs, act,
                           _vp(work), bytes, _vp(Y), dtype, None, path)


@pytest.mark.parametrize("f", [_fp4, _fp8])
def test_moe_refusals(f):
    assert f(dtype=fw.F32) == fw.ERR_DTYPE
    assert f(act=2) == fw.ERR_DTYPE
    assert f(bs=0) == fw.ERR_BLOCK
    for bad in (dict(M=-1), dict(K=-2), dict(E=-1), dict(I=-2), dict(topk=-1), dict(E=fw.MOE_MAX_EXPERTS + 1),
                dict(topk=fw.MOE_MAX_TOPK + 1), dict(M=1 << 30), dict(M=1 << 31, topk=0), dict(M=1 << 62),
                dict(K=1 << 42), dict(K=1 << 30, I=1 << 30, E=1024)):
        assert f(**bad) == fw.ERR_SHAPE, bad
    for name in ("A", "ids", "w", "w13", "s13", "w2", "s2", "work", "Y"):
        assert f(**{name: None}) == fw.ERR_NULL, name
    need = fw.fp4w_moe_workspace(2, 2, 64, 32)
    assert f(bytes=need - 1) == fw.ERR_SHAPE
    assert f(work=0x9000002) == fw.ERR_SHAPE
    for name, at in (("Y", 0x1000000 + 16), ("Y", 0x2000000), ("Y", 0x3000000), ("Y", 0x6000000 + 64), ("Y", 0x9000000),
                     ("work", 0x1000000), ("work", 0x4000000), ("work", 0x2100000), ("work", 0x7000000)):
        assert f(**{name: at}) == fw.ERR_ALIAS, (name, hex(at))
    assert f(path=fw.PATH_FP4_GEMV) == fw.ERR_PATH
    assert f(A=None, ids=None, w=None, w13=None, s13=None, w2=None, s2=None, work=None, Y=None, M=0) == fw.OK
    assert f(A=None, Y=None, K=0) == fw.OK


def test_moe_fp4_only_refusals():
    assert _fp4(K=63) == fw.ERR_SHAPE
    assert _fp4(I=31) == fw.ERR_SHAPE
    assert _fp4(g13=None) == fw.ERR_NULL
    assert _fp4(g2=None) == fw.ERR_NULL
    assert _fp4(Y=0x5000000) == fw.ERR_ALIAS
    assert _fp4(path=fw.PATH_MOE_FP8_GENERIC) == fw.ERR_PATH
    assert _fp8(path=fw.PATH_MOE_FP4_GENERIC) == fw.ERR_PATH


def test_workspace_size():
    assert fw.fp4w_moe_workspace(4, 8, 128, 64) >= 4 * 8 * 64 * 4
    assert fw.load_library().fp4w_moe_workspace(-1, 8, 128, 64) == fw.ERR_SHAPE
    with pytest.raises(fw.FP4WError):
        fw.fp4w_moe_workspace(1 << 30, 2, 128, 64)
    # many tokens are worked through in parts: the workspace stays that of one
    assert fw.fp4w_moe_workspace(1 << 29, 2, 128, 64) == fw.fp4w_moe_workspace(2048, 2, 128, 64)
    assert fw.fp4w_moe_workspace(2049, 2, 128, 64) <= fw.fp4w_moe_workspace(2048, 2, 128, 64)


@pytest.mark.parametrize("topk", [1, 2, 3, 5, 8, 63, 64])
@pytest.mark.parametrize("K,I", [(2048, 768), (128, 5120), (7168, 2048)])
def test_a_workspace_serves_every_smaller_call(K, I, topk):  # noqa: E741
    """Whatever the parts that a call's tokens are cut into: the size never falls as M, topk or I grows."""
    size = fw.fp4w_moe_workspace
    most = 4096 // topk
    last = 0
    for M in sorted({*range(0, 40), *(n * most + d for n in (1, 2, 3, 5) for d in (-2, -1, 0, 1, 2, 7)), 100000, 1 << 24}):
        if M < 0:
            continue
        need = size(M, topk, K, I)
        assert need >= last, M
        last = need
        if topk > 1:
            assert size(M, topk - 1, K, I) <= need
        assert size(M, topk, K, max(0, I - 64)) <= need and size(M, topk, K - 64, I) <= need
    # the buffer of a large batch takes a call at which a part is full
    lib = fw.load_library()
    held = lib.fp4w_moe_workspace(most + 1, topk, K, I)
    for M in (most - 1, most):
        assert lib.fp4w_moe_workspace(M, topk, K, I) <= held


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_refuses_what_does_not_fit(fp8):
    c = make_moe(fp8, 2, 64, 32, 4, 2, "bf16", 1)
    good = moe_on(c, "cpu")
    bad = {
        "A": [good["A"].float(), good["A"][:, :62], good["A"].t().contiguous().t()],
        "ids": [good["ids"].long(), good["ids"][:1], good["ids"][:, :1]],
        "weights": [good["weights"].double(), good["weights"][:, :1]],
        "w13": [good["w13"][:, :, :31], good["w13"].float(), good["w13"][:3], good["w13"][0]],
        "s13": [good["s13"][:, :, :0], good["s13"].to(torch.int8)],
        "w2": [good["w2"][:, :63], good["w2"].transpose(1, 2)],
        "s2": [good["s2"][:, :, :0], good["s2"][:3]],
    }
    if not fp8:
        bad["g13"] = [good["g13"][:3], good["g13"].double()]
        bad["g2"] = [good["g2"].reshape(2, 2)]
    for name, values in bad.items():
        for v in values:
            with pytest.raises((ValueError, TypeError)):
                moe_call(fw, c, dict(good, **{name: v}))
    with pytest.raises(ValueError):
        moe_call(fw, c, good, act="relu")
    with pytest.raises(ValueError):
        moe_call(fw, c, good, out=torch.empty(2, 63, dtype=torch.bfloat16))
    with pytest.raises(fw.FP4WError):
        moe_call(fw, dict(c, block_size=0), good)


def test_binding_refuses_norm_and_route_arguments():
    x = torch.zeros(3, 16, dtype=torch.bfloat16)
    w = torch.zeros(16, dtype=torch.bfloat16)
    for kw in (dict(residual=x[:2]), dict(pre_weight=w[:8]), dict(post_weight=w.float()), dict(gate=torch.zeros(3, 1)),
               dict(gate=x.float()), dict(out=x), dict(write_residual=False),
               dict(write_residual=False, pre_weight=w, residual_out=x), dict(residual=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            fw.fp4w_block_norm(x, **kw)
    with pytest.raises(TypeError):
        fw.fp4w_block_norm(x.float())
    logits = torch.zeros(3, 8)
    for kw in (dict(score="max"), dict(select_bias=torch.zeros(7)), dict(ids=torch.zeros(3, 2)),
               dict(weights=torch.zeros(3, 3))):
        with pytest.raises(ValueError):
            fw.fp4w_moe_route(logits, 2, **kw)
    with pytest.raises(TypeError):
        fw.fp4w_moe_route(logits.double(), 2)
    with pytest.raises(ValueError):
        fw.fp4w_moe_route(logits, -1)


def test_binding_refuses_a_column_as_the_row_of_gates():
    """[K, 1] has K values, but they would be one for each row."""
    x = torch.zeros(16, 16, dtype=torch.bfloat16)
    for gate in (torch.zeros(16, 1), torch.zeros(4, 4), torch.zeros(1, 1, 16)):
        with pytest.raises(ValueError, match="gate must be"):
            fw.fp4w_block_norm(x, gate=gate.bfloat16())


@pytest.mark.parametrize("fp8", [False, True])
def test_binding_refuses_tensors_without_dimensions(fp8):
    c = make_moe(fp8, 2, 64, 32, 4, 2, "bf16", 1)
    good = moe_on(c, "cpu")
    for name in ("A", "ids"):
        with pytest.raises(ValueError, match="leading dimensions"):
            moe_call(fw, c, dict(good, **{name: good[name][0, 0]}))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_dispatch_moe_under_asan_ubsan(tmp_path):
    """The validation and dispatch, built with g++ under AddressSanitizer and
    UndefinedBehaviorSanitizer against host stand-ins for the launchers."""
    exe = tmp_path / "moe_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           os.path.join(ROOT, "fp8_weight_only_fp4w_amd", "csrc", "dispatch_moe.cpp"),
           os.path.join(HERE, "host_sanitize", "moe_driver.cpp"), "-o", str(exe)]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
