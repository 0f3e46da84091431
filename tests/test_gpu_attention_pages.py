"""Page sizes that are multiples of 16 and no power of two, or larger than a
workgroup's share, through the fast kernels of the append and of attention;
rotation in neighbouring pairs on the way into the cache; prompts from a
replayed graph."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
import test_gpu_kv_append as append
from attention_cases import batch, cache, filled, on_gpu, rounded, to_cache, within
from gpu_helpers import require_gpu
from oracle import attention as oa
from test_gpu_attention import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# held before, new, Hq, Hk, D, window
CASES = [
    ([900, 0, 47], [1, 1, 1], 10, 2, 128, 0),
    ([2000, 95], [1, 1], 6, 1, 64, 0),
    ([300, 20], [3, 5], 16, 4, 128, 0),
    ([700], [6], 10, 2, 128, 100),        # 30 rows of a key head
    ([0, 130], [150, 70], 4, 2, 64, 0),
    ([95, 5], [200, 33], 6, 2, 128, 60),
    ([3000], [40], 4, 1, 128, 0),         # several parts
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [48, 80, 96, 256])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{max(c[0])}+{max(c[1])}-{c[2]}/{c[3]}x{c[4]}-w{c[5]}")
def test_attention_against_oracle(case, page, dtype):
    held, new, Hq, Hk, D, window = case
    rng = np.random.default_rng(sum(held) + D + page)
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    q = rounded(rng, (sum(new) + 1, Hq, D), dtype, 1.5)
    check(q, parts, starts, lens, table, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", [
    ([700], [1], 48, 40, 8, 128, 128),
    ([0, 47, 48, 49], [1, 1, 1, 1], 48, 4, 2, 64, 64),
    ([3, 0, 20], [140, 0, 1], 48, 0, 2, 64, None),
    ([5, 95, 40], [300, 2, 60], 96, 4, 1, 128, 128),
    ([0, 10], [250, 90], 112, 0, 2, 128, None),
    ([30], [200], 240, 2, 1, 64, 32),
], ids=lambda c: f"{c[2]}-{c[4]}x{c[5]}-{sum(c[1])}")
def test_append_against_oracle(case, dtype):
    append.test_against_oracle(case, dtype)


@pytest.mark.parametrize("new", [[40, 1, 9], [1, 1, 1]])
@pytest.mark.parametrize("page,D,R", [(16, 64, 32), (32, 128, 128), (96, 128, 64), (5, 24, 8)])
def test_append_turns_neighbouring_pairs(page, D, R, new):
    """Keys and queries rotated in pairs (2 i, 2 i + 1) of a part of the head, with norms."""
    rng = np.random.default_rng(90)
    starts, lens, table, pages = batch(rng, [7, 30, 0], new, page)
    M = sum(new)
    q, k, v = rounded(rng, (M, 3, D), "bf16"), rounded(rng, (M, 2, D), "bf16", 3.0), rounded(rng, (M, 2, D), "bf16")
    w = rounded(rng, D, "bf16")
    a = rng.uniform(-3, 3, (60, R // 2))
    cos, sin = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    parts = cache(rng, pages, 2, page, D)
    c = to_cache(parts)
    out = fw.fp8w_kv_append(on_gpu(k, "bf16"), on_gpu(v, "bf16"), c, on_gpu(table), on_gpu(lens),
                            starts=on_gpu(starts) if max(new) > 1 else None, q=on_gpu(q, "bf16"), q_weight=on_gpu(w, "bf16"),
                            k_weight=on_gpu(w, "bf16"), cos=on_gpu(cos), sin=on_gpu(sin), interleaved=True)
    pos = [p[1] for p in oa.places(starts, lens, table, page, pages, M)]
    want, tol = oa.norm_rope(q, w, cos, sin, pos, True)
    within(out, want, tol, "bf16", "q")
    want, tol = oa.norm_rope(k, w, cos, sin, pos, True)
    append.check_codes(c.k.cpu().numpy(), c.k_scale.cpu().numpy(), want, tol, parts[0], parts[2], starts, lens, table, page, "k")
    want = oa.append(v, append.by_token(parts[1]), parts[3], starts, lens, table, page)
    assert append.same_codes(append.by_token(c.v.cpu().numpy()), want[0]) and np.array_equal(c.v_scale.cpu().numpy(), want[1])


@pytest.mark.parametrize("D,page,Hq,Hk", [(128, 32, 10, 2), (64, 16, 4, 1), (40, 8, 3, 1)])
def test_prompts_from_a_replayed_graph(D, page, Hq, Hk):
    """Append and attention of a piece of a prompt, captured once and replayed at other places of the sequences."""
    rng = np.random.default_rng(91)
    new = [50, 30]
    starts, _, table, pages = batch(rng, [4000, 2000], new, page)
    c = fw.fp8w_kv_cache(pages, Hk, page, D)
    for s, p in zip(c, cache(rng, pages, Hk, page, D, nan_slots=False)):
        s.copy_(on_gpu(p))
    t, st = on_gpu(table), on_gpu(starts)
    n = torch.tensor([50, 30], dtype=torch.int32, device="cuda")
    q, k, v = (on_gpu(rounded(rng, (80, H, D), "bf16"), "bf16") for H in (Hq, Hk, Hk))
    out, work = torch.empty_like(q), torch.empty(fw.fp8w_attention_workspace(80, Hq, Hk, D, 2, 50), dtype=torch.uint8, device="cuda")

    def piece(c, out=None, work=None):
        fw.fp8w_kv_append(k, v, c, t, n, starts=st)
        return fw.fp8w_attention(q, c, t, n, starts=st, max_new=50, out=out, workspace=work)

    piece(fw.KVCache(*(x.clone() for x in c)), out, work)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        piece(c, out, work)
    for held in ([0, 0], [3950, 5], [123, 1970], [2000, 0]):
        n.copy_(torch.tensor([h + m for h, m in zip(held, new)], dtype=torch.int32))
        k.copy_(on_gpu(rounded(rng, (80, Hk, D), "bf16"), "bf16"))
        want = fw.KVCache(*(x.clone() for x in c))
        y = piece(want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), y.view(torch.int16)), held
        assert all(torch.equal(a, b) for a, b in zip(c, want)), held
