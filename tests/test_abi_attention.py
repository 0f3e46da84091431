"""Argument checks of the entry points between the projections of an attention
block.  No call here reaches a kernel launch, and none needs a GPU."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import fp8_weight_only_fp4w_amd as fw

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _vp(x):
    return ctypes.c_void_p(x)


G = 1 << 32  # stand-in device addresses, 4 GiB apart


def _rope(q=1 * G, qs=512, Hq=4, k=2 * G, ks=256, Hk=2, M=8, D=128, qw=3 * G, kw=4 * G, cos=5 * G, sin=6 * G, rows=100,
          dims=128, pos=7 * G, qo=8 * G, qos=512, ko=9 * G, kos=256, dtype=fw.BF16):
    return fw.load_library().fp4w_qk_norm_rope(_vp(q), qs, Hq, _vp(k), ks, Hk, M, D, _vp(qw), _vp(kw), 0.0, 1e-6, _vp(cos),
                                               _vp(sin), rows, dims, 0, _vp(pos), _vp(qo), qos, _vp(ko), kos, dtype, None)


def test_qk_norm_rope_refusals():
    assert _rope(dtype=fw.F32) == fw.ERR_DTYPE
    for bad in (dict(M=-1), dict(Hq=-1), dict(D=fw.MAX_HEAD_SIZE + 1), dict(M=1 << 31), dict(sin=None), dict(cos=None),
                dict(dims=3), dict(dims=130), dict(dims=-2), dict(rows=-1), dict(rows=0), dict(qs=511), dict(ks=255), dict(qos=0),
                dict(kos=-256), dict(qs=1 << 61)):
        assert _rope(**bad) == fw.ERR_SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None)):
        assert _rope(**bad) == fw.ERR_NULL, bad
    assert _rope(qo=1 * G, qos=1024) == fw.ERR_ALIAS       # its own input with another stride
    assert _rope(qo=1 * G + 16) == fw.ERR_ALIAS            # partly over its input
    assert _rope(qo=2 * G) == fw.ERR_ALIAS                 # over the other input
    assert _rope(ko=8 * G + 1024) == fw.ERR_ALIAS          # both outputs
    for table in (3, 4, 5, 6, 7):
        assert _rope(ko=table * G) == fw.ERR_ALIAS
    # side by side in one larger row: neither overlaps, unless it reaches into the next
    assert _rope(qs=1024, k=1 * G + 1024, ks=1024, qo=1 * G, qos=1024, ko=1 * G + 1536, kos=1024, q=None) == fw.ERR_NULL
    assert _rope(qs=1024, k=1 * G + 1024, ks=1024, qo=1 * G + 1024, qos=1024) == fw.ERR_ALIAS
    assert _rope(qs=1024, k=1 * G + 1024, ks=1024, ko=1 * G + 1792, kos=1024) == fw.ERR_ALIAS  # wraps into the next q
    assert _rope(M=0, q=None) == fw.OK and _rope(D=0, q=None, cos=None, sin=None) == fw.OK
    assert _rope(Hq=0, Hk=0, q=None) == fw.OK


def _append(k=1 * G, ks=256, v=2 * G, vs=256, M=8, Hk=2, D=128, q=3 * G, qs=512, Hq=4, qw=4 * G, kw=5 * G, cos=6 * G,
            sin=7 * G, rows=100, dims=128, pos=8 * G, qo=9 * G, qos=512, starts=10 * G, B=3, lens=11 * G, table=12 * G,
            columns=4, kc=13 * G, ksc=14 * G, vc=15 * G, vsc=16 * G, pages=20, page=16, dtype=fw.BF16):
    return fw.load_library().fp8w_kv_append(_vp(k), ks, _vp(v), vs, M, Hk, D, _vp(q), qs, Hq, _vp(qw), _vp(kw), 0.0, 1e-6,
                                            _vp(cos), _vp(sin), rows, dims, 0, _vp(pos), _vp(qo), qos, _vp(starts), B,
                                            _vp(lens), _vp(table), columns, _vp(kc), _vp(ksc), _vp(vc), _vp(vsc), pages,
                                            page, dtype, None)


def test_kv_append_refusals():
    assert _append(dtype=3) == fw.ERR_DTYPE
    for bad in (dict(M=-1), dict(Hk=-1), dict(D=fw.MAX_HEAD_SIZE + 1), dict(B=-1), dict(page=0), dict(pages=-1),
                dict(columns=-1), dict(columns=1 << 28), dict(starts=None), dict(ks=100), dict(vs=100), dict(qs=100),
                dict(qos=100), dict(dims=5), dict(rows=0), dict(sin=None), dict(pages=1 << 30, page=1 << 30, columns=1, Hk=1000)):
        assert _append(**bad) == fw.ERR_SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(lens=None), dict(table=None), dict(kc=None),
                dict(ksc=None), dict(vc=None), dict(vsc=None)):
        assert _append(**bad) == fw.ERR_NULL, bad
    for part in ("kc", "ksc", "vc", "vsc"):
        for other in (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12):
            assert _append(**{part: other * G}) == fw.ERR_ALIAS, (part, other)
    assert _append(vc=13 * G + 64) == fw.ERR_ALIAS and _append(vsc=14 * G) == fw.ERR_ALIAS
    for other in (1, 2, 4, 5, 6, 7, 8, 10, 11, 12):
        assert _append(qo=other * G) == fw.ERR_ALIAS, other
    assert _append(qo=3 * G + 2) == fw.ERR_ALIAS
    assert _append(M=0, k=None) == fw.OK and _append(B=0, k=None) == fw.OK
    assert _append(Hq=0, Hk=0, k=None) == fw.OK


def _attn(q=1 * G, qs=512, M=8, Hq=4, Hk=2, D=128, starts=2 * G, B=3, lens=3 * G, table=4 * G, columns=4, most=8, kc=5 * G,
          ksc=6 * G, vc=7 * G, vsc=8 * G, pages=20, page=16, scale=0.1, causal=1, window=0, work=9 * G, held=1 << 30,
          y=10 * G, lse=11 * G, dtype=fw.BF16, path=fw.PATH_AUTO):
    return fw.load_library().fp8w_attention_ex(_vp(q), qs, M, Hq, Hk, D, _vp(starts), B, _vp(lens), _vp(table), columns,
                                               most, _vp(kc), _vp(ksc), _vp(vc), _vp(vsc), pages, page, scale, causal,
                                               window, _vp(work), held, _vp(y), _vp(lse), dtype, None, path)


def test_attention_refusals():
    assert _attn(dtype=fw.F32) == fw.ERR_DTYPE
    for bad in (dict(M=-1), dict(Hq=3), dict(Hk=0), dict(D=fw.MAX_HEAD_SIZE + 1), dict(B=-1), dict(page=0), dict(pages=-1),
                dict(columns=1 << 28), dict(starts=None), dict(qs=511), dict(window=-1), dict(most=-1),
                dict(pages=1 << 30, page=1 << 30, columns=1, Hq=1000, Hk=1000, qs=1 << 20)):
        assert _attn(**bad) == fw.ERR_SHAPE, bad
    for bad in (dict(q=None), dict(y=None), dict(lens=None), dict(table=None), dict(kc=None), dict(ksc=None),
                dict(vc=None), dict(vsc=None)):
        assert _attn(**bad) == fw.ERR_NULL, bad
    for other in range(1, 9):
        assert _attn(y=other * G) == fw.ERR_ALIAS and _attn(lse=other * G) == fw.ERR_ALIAS, other
    assert _attn(lse=10 * G) == fw.ERR_ALIAS
    assert _attn(path=fw.PATH_FP4_GEMV) == fw.ERR_PATH
    assert _attn(M=0, q=None) == fw.OK and _attn(B=0, q=None) == fw.OK and _attn(most=0, q=None) == fw.OK
    assert _attn(Hq=0, Hk=0, q=None) == fw.OK


def test_attention_workspace():
    n = fw.fp8w_attention_workspace
    assert n(0, 8, 2, 128, 0, 0) >= 0
    for bad in ((-1, 8, 2, 128, 1, 1), (1, 7, 2, 128, 1, 1), (1, 8, 0, 128, 1, 1), (1, 8, 2, 2000, 1, 1), (1, 8, 2, 128, -1, 1),
                (1, 8, 2, 128, 1, -1)):
        with pytest.raises(fw.FP4WError):
            n(*bad)
    rng = __import__("random").Random(0)
    for _ in range(400):
        Hk = rng.choice((1, 2, 8))
        big = [rng.randint(1, 5000), Hk * rng.randint(1, 16), Hk, rng.choice((64, 80, 128)), rng.randint(1, 3000), rng.randint(1, 5000)]
        small = list(big)
        for i in (0, 4, 5):
            small[i] = rng.randint(0, big[i])
        assert n(*small) <= n(*big), (small, big)


def test_path_names():
    assert [fw.fp4w_path_name(p) for p in (fw.PATH_ATTN_DECODE, fw.PATH_ATTN_PROMPT, fw.PATH_ATTN_GENERIC)] == [
        "attn_decode", "attn_prompt", "attn_generic"]


# ---------------------------------------------------------------- the binding's own checks

def _inputs(dtype=torch.bfloat16):
    return dict(q=torch.zeros(3, 4, 32, dtype=dtype), k=torch.zeros(3, 2, 32, dtype=dtype), v=torch.zeros(3, 2, 32, dtype=dtype),
                cache=fw.fp8w_kv_cache(6, 2, 16, 32, "cpu"), table=torch.zeros(3, 2, dtype=torch.int32),
                lens=torch.ones(3, dtype=torch.int32))


def test_binding_refuses_the_cpu_and_wrong_tensors():
    d = _inputs()
    q, k, v, c, table, lens = d.values()
    with pytest.raises(ValueError, match="GPU"):
        fw.fp4w_qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="GPU"):
        fw.fp8w_kv_append(k, v, c, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        fw.fp8w_attention(q, c, table, lens)
    for bad in (lambda: fw.fp4w_qk_norm_rope(q[0], k), lambda: fw.fp4w_qk_norm_rope(q, k[:2]),
                lambda: fw.fp4w_qk_norm_rope(q, k, q_weight=torch.zeros(32)), lambda: fw.fp4w_qk_norm_rope(q, k, cos=torch.zeros(9, 4)),
                lambda: fw.fp4w_qk_norm_rope(q, k, cos=torch.zeros(9, 17), sin=torch.zeros(9, 17)),
                lambda: fw.fp4w_qk_norm_rope(q, k, cos=torch.zeros(0, 16), sin=torch.zeros(0, 16)),
                lambda: fw.fp4w_qk_norm_rope(q, k, positions=torch.zeros(3, dtype=torch.int64)),
                lambda: fw.fp4w_qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2)),
                lambda: fw.fp4w_qk_norm_rope(q, k, q_out=torch.zeros_like(k)),
                lambda: fw.fp4w_qk_norm_rope(q, None, k_weight=torch.zeros(32, dtype=torch.bfloat16)),
                lambda: fw.fp8w_kv_append(k, v[:, :1], c, table, lens), lambda: fw.fp8w_kv_append(k, v, c, table[:2], lens),
                lambda: fw.fp8w_kv_append(k, v, c, table, lens.long()),
                lambda: fw.fp8w_kv_append(k, v, c, table, lens, starts=torch.zeros(3, dtype=torch.int32)),
                lambda: fw.fp8w_kv_append(k, v, c, table[:2], lens[:2]),
                lambda: fw.fp8w_kv_append(k, v, c._replace(v=c.k), table, lens),
                lambda: fw.fp8w_kv_append(k, v, c._replace(k_scale=c.k_scale[:, :1]), table, lens),
                lambda: fw.fp8w_kv_append(k, v, c, table, lens, q_out=q),
                lambda: fw.fp8w_attention(q, c, table, lens, window=-1),
                lambda: fw.fp8w_attention(q, c, table, lens, out=q[:, :2]),
                lambda: fw.fp8w_attention(q, c, table, lens, lse=torch.zeros(3)),
                lambda: fw.fp8w_attention(q[:, :, :16], c, table, lens)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fw.fp4w_qk_norm_rope(q.float(), k.float())
    with pytest.raises(TypeError):
        fw.fp8w_attention(q, c._replace(k_scale=c.k_scale.float()), table, lens)
    with pytest.raises(fw.FP4WError):
        fw.fp8w_attention(torch.zeros(3, 3, 32, dtype=torch.bfloat16), c, table, lens)  # three heads over two


def test_cache_is_what_the_header_says():
    c = fw.fp8w_kv_cache(5, 3, 16, 64, "cpu")
    assert c.k.shape == (5, 3, 16, 64) and c.v.shape == (5, 3, 64, 16) and c.k_scale.shape == c.v_scale.shape == (5, 3)
    assert all(t.dtype == torch.uint8 and t.is_contiguous() for t in c)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_dispatch_under_asan_ubsan(tmp_path):
    exe = tmp_path / "attn_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           os.path.join(ROOT, "fp8_weight_only_fp4w_amd", "csrc", "dispatch_attn.cpp"),
           os.path.join(HERE, "host_sanitize", "attn_driver.cpp"), "-o", str(exe)]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
