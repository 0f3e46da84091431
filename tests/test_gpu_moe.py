"""fp4w_moe and fp8w_moe on the GPU against the oracle's float64 and its bound."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from gpu_helpers import require_gpu
from moe_cases import assert_within, make_moe, moe_call, moe_on, moe_want, rounded
from oracle import moe as om

pytestmark = pytest.mark.gpu

FORMATS = [False, True]
GENERIC = {False: fw.PATH_MOE_FP4_GENERIC, True: fw.PATH_MOE_FP8_GENERIC}
STREAM = {False: fw.PATH_MOE_FP4_STREAM, True: fw.PATH_MOE_FP8_STREAM}
ids_of = lambda c: "x".join(map(str, c))  # noqa: E731

# M, K, I, E, topk: sizes that fill tiles, end inside them, one token and
# many, one expert, more choices than experts
SIZES = [
    (1, 128, 128, 4, 2), (1, 64, 64, 1, 1), (1, 2048, 768, 16, 8), (2, 192, 320, 3, 3), (3, 256, 64, 8, 2),
    (5, 320, 192, 8, 6), (4, 1024, 512, 2, 1), (7, 128, 1408, 6, 4), (16, 512, 256, 4, 2), (17, 256, 448, 1, 1),
    (33, 448, 128, 4, 3), (64, 256, 192, 16, 8), (100, 192, 128, 5, 2), (130, 128, 64, 3, 1), (9, 64, 128, 40, 20),
]
# sizes that only the generic kernels take
ODD = [(1, 2, 2, 1, 1, 16), (3, 30, 22, 4, 2, 15), (2, 66, 34, 3, 2, 16), (5, 96, 40, 4, 3, 32), (2, 256, 128, 4, 2, 24)]


def run(c, act="silu", **kw):
    return moe_call(fw, c, moe_on(c), act, **kw)


@pytest.mark.parametrize("path", ["auto", "generic"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("size", SIZES, ids=ids_of)
def test_against_oracle(size, fp8, dtype, path):
    require_gpu()
    M, K, I, E, topk = size  # noqa: E741
    c = make_moe(fp8, M, K, I, E, topk, dtype, seed=M + K + I, masked=0.1 if M > 2 else 0.0)
    act = "gelu" if (M + I) % 3 == 0 else "silu"
    Y = run(c, act, path=GENERIC[fp8] if path == "generic" else fw.PATH_AUTO)
    want, tol = moe_want(c, act)
    assert_within(Y, want, tol, dtype, f"{size}")


# sizes that bring the streaming kernels to the other layouts of LDS: one
# buffer of token rows, weights straight to registers, the second product's sum
# in parts, fewer rows than tokens, and as many assignments and experts as a
# call may have
LAYOUTS = [(6, 4096, 256, 8, 2), (4, 7168, 128, 4, 2), (20, 2880, 192, 2, 1), (40, 128, 2048, 2, 1),
           (70, 192, 2880, 3, 1), (40, 8192, 128, 2, 1), (33, 128, 4160, 2, 1), (2, 16384, 64, 3, 2),
           (512, 64, 64, 1024, 8), (64, 64, 64, 70, 64)]


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("size", LAYOUTS, ids=ids_of)
def test_layouts_of_the_streaming_kernels(size, fp8):
    require_gpu()
    M, K, I, E, topk = size  # noqa: E741
    c = make_moe(fp8, M, K, I, E, topk, "bf16", seed=K + I, masked=0.05)
    want, tol = moe_want(c)
    assert_within(run(c, path=STREAM[fp8]), want, tol, "bf16", f"{size}")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("M", [1, 3])
def test_rows_that_no_lds_holds_take_the_generic_kernels(fp8, M):
    require_gpu()
    c = make_moe(fp8, M, 98304, 64, 2, 2, "bf16", seed=M)
    want, tol = moe_want(c)
    assert_within(run(c), want, tol, "bf16")
    with pytest.raises(fw.FP4WError) as e:
        run(c, path=STREAM[fp8])
    assert e.value.status == fw.ERR_PATH


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_one_token_with_many_choices(fp8):
    """A single token: topk up to 64, masked and repeated choices, rows that do and do not fit beside the ring."""
    require_gpu()
    for K, I, E, topk in ((128, 64, 70, 64), (512, 320, 9, 9), (192, 2048, 12, 8), (256, 1024, 20, 16), (64, 128, 3, 5)):  # noqa: E741
        c = make_moe(fp8, 1, K, I, E, topk, "bf16", seed=K + topk)
        c["ids"][0, topk // 2] = -1
        c["ids"][0, -1] = c["ids"][0, 0]
        want, tol = moe_want(c)
        assert_within(run(c, path=STREAM[fp8]), want, tol, "bf16", f"{(K, I, E, topk)}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("size", ODD, ids=ids_of)
def test_odd_sizes_and_blocks(size, fp8, dtype):
    require_gpu()
    M, K, I, E, topk, bs = size  # noqa: E741
    if fp8:
        K, I = K + 1, I + 1  # noqa: E741
    c = make_moe(fp8, M, K, I, E, topk, dtype, seed=K, block_size=bs)
    want, tol = moe_want(c)
    assert_within(run(c), want, tol, dtype, f"{size}")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_masked_rows_repeated_and_foreign_ids(fp8):
    """Rows without any valid id give zeros; an expert named twice counts twice; ids past E and below 0 are skipped."""
    require_gpu()
    c = make_moe(fp8, 6, 256, 128, 5, 4, "bf16", 11)
    c["ids"][:] = [[-1, -1, -1, -1], [2, 2, 2, 2], [5, 1000, -7, 2 ** 31 - 1], [0, 5, -2 ** 31, 0], [4, 3, 2, 1],
                   [3, -1, 3, 9]]
    want, tol = moe_want(c)
    for path in (fw.PATH_AUTO, GENERIC[fp8]):
        Y = run(c, path=path)
        assert (Y[0] == 0).all() and (Y[2] == 0).all()
        assert_within(Y, want, tol, "bf16")
    c["ids"][:] = -1
    assert (run(c) == 0).all()


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_all_tokens_to_one_expert(fp8):
    require_gpu()
    for M in (16, 17, 40, 100):
        c = make_moe(fp8, M, 256, 192, 6, 2, "fp16", 12 + M)
        c["ids"][:, 0] = 4
        c["ids"][:, 1] = -1
        want, tol = moe_want(c)
        assert_within(run(c), want, tol, "fp16", f"M {M}")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("size", [(520, 128, 64, 16, 8), (4097, 64, 64, 3, 1), (130, 64, 128, 70, 64), (65, 66, 34, 70, 64)],
                         ids=ids_of)
def test_tokens_beyond_one_part(size, fp8):
    """More choices than the kernels sort at once: parts of the tokens, in one workspace, nothing behind the last row."""
    require_gpu()
    M, K, I, E, topk = size  # noqa: E741
    c = make_moe(fp8, M, K, I, E, topk, "bf16", seed=M + E, masked=0.05)
    want, tol = moe_want(c)
    d = moe_on(c)
    Y = torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")
    moe_call(fw, c, d, out=Y[:M])
    assert_within(Y[:M], want, tol, "bf16", f"{size}")
    assert (Y[M:] == 7).all()
    s = slice(M // 2, M // 2 + 9)  # a token's result does not hang on its part
    e = {**d, **{k: d[k][s].contiguous() for k in ("A", "ids", "weights")}}
    near, near_tol = want[s], tol[s]
    assert_within(moe_call(fw, c, e), near, near_tol, "bf16", f"{size}")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_empty(fp8):
    require_gpu()
    for M, K, I, E, topk in ((0, 128, 64, 4, 2), (3, 0, 64, 4, 2), (3, 128, 0, 4, 2), (3, 128, 64, 0, 2), (3, 128, 64, 4, 0)):  # noqa: E741
        c = make_moe(fp8, M, K, I, E, topk, "bf16", 1)
        out = torch.full((M, K), 5.0, dtype=torch.bfloat16, device="cuda")
        run(c, out=out)
        assert (out == 0).all()


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_nan_and_infinity_stay_with_their_token_and_expert(fp8):
    require_gpu()
    c = make_moe(fp8, 5, 192, 192, 4, 1, "bf16", 13)
    c["ids"][:, 0] = [0, 1, 1, 2, 3]
    c["A"][2, 5] = float("nan")
    c["A"][3, 100] = float("inf")
    c["A64"] = c["A"].double().numpy()
    if fp8:
        c["w2"][3, 7, 11] = 0x7F      # one weight: one column of token 4
        bad = [7]
    else:
        c["s2"][3, 7, -1] = 0x7F      # the row's last block
        bad = [7]
    with np.errstate(all="ignore"):
        want, tol = moe_want(c)
    Y = run(c).cpu()
    assert Y[2].isnan().all() and not Y[3].isfinite().any()
    assert [i for i in range(192) if Y[4, i].isnan()] == bad
    keep = [0, 1]
    assert_within(Y[keep], want[keep], tol[keep], "bf16")
    cols = [i for i in range(192) if i not in bad]
    assert_within(Y[4:5, cols], want[4:5, cols], tol[4:5, cols], "bf16")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_large_intermediates_do_not_overflow(fp8):
    """gate * up past the range of FP16 is an intermediate only: the output is finite."""
    require_gpu()
    c = make_moe(fp8, 3, 256, 128, 2, 1, "fp16", 14, spread=300.0)
    c["weights"][:] = 2.0 ** -12
    want, tol = moe_want(c)
    assert np.abs(want).max() < 60000
    h = c["A64"][0] @ om.expert_matrix(c["w13"][c["ids"][0, 0]], c["s13"][c["ids"][0, 0]],
                                       None if fp8 else c["g13"][c["ids"][0, 0]], c["block_size"], fp8).T
    assert np.abs(h[:128] * h[128:]).max() > 65504
    assert_within(run(c), want, tol, "fp16")


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_unaligned_pointers(fp8):
    """Weights, activations and scales that start anywhere, and nothing written outside Y."""
    require_gpu()
    c = make_moe(fp8, 3, 128, 128, 4, 2, "bf16", 15)
    d = moe_on(c)

    def shifted(t, by):
        room = torch.empty(t.numel() + by + 8, dtype=t.dtype, device="cuda")
        return room[by:by + t.numel()].view(t.shape).copy_(t)

    want, tol = moe_want(c)
    for name, by in (("A", 1), ("w13", 1), ("w2", 3), ("s13", 1), ("s2", 1), ("ids", 1), ("weights", 3)):
        Y = moe_call(fw, c, dict(d, **{name: shifted(d[name], by)}))
        assert_within(Y, want, tol, "bf16", name)
    room = torch.full((5 * 128 + 1,), 9.0, dtype=torch.bfloat16, device="cuda")
    moe_call(fw, c, d, out=room[1:1 + 3 * 128].view(3, 128))
    assert_within(room[1:1 + 3 * 128].view(3, 128), want, tol, "bf16")
    assert room[0] == 9 and (room[1 + 3 * 128:] == 9).all()


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_same_bits_again_whatever_the_workspace_held(fp8):
    require_gpu()
    c = make_moe(fp8, 24, 512, 320, 12, 4, "bf16", 16)
    d = moe_on(c)
    need = fw.fp4w_moe_workspace(24, 4, 512, 320)
    first = moe_call(fw, c, d)
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(moe_call(fw, c, d, workspace=ws).view(torch.int16), first.view(torch.int16))
    with pytest.raises(fw.FP4WError):
        moe_call(fw, c, d, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_two_streams_at_once(fp8):
    require_gpu()
    cs = [make_moe(fp8, M, 512, 256, 8, 4, "bf16", 17 + M) for M in (4, 30)]
    ds = [moe_on(c) for c in cs]
    alone = [moe_call(fw, c, d) for c, d in zip(cs, ds)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(moe_call(fw, cs[i], ds[i]))
    torch.cuda.synchronize()
    for a, got in zip(alone, outs):
        assert all(torch.equal(a, y) for y in got)


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_captured_and_replayed_with_other_routings(fp8):
    """A graph that was captured with one routing serves every other: nothing of the ids is kept on the host."""
    require_gpu()
    c = make_moe(fp8, 8, 256, 192, 16, 4, "bf16", 18)
    d = moe_on(c)
    ws = torch.empty(fw.fp4w_moe_workspace(8, 4, 256, 192), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["A"])
    moe_call(fw, c, d, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe_call(fw, c, d, out=out, workspace=ws)
    rng = np.random.default_rng(19)
    for k in range(5):
        c["ids"] = rng.integers(-1, 16, (8, 4)).astype(np.int32) if k != 3 else np.full((8, 4), 5, np.int32)
        d["ids"].copy_(torch.from_numpy(c["ids"]))
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        eager = moe_call(fw, c, d)
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), k
        want, tol = moe_want(c)
        assert_within(out, want, tol, "bf16", f"replay {k}")


def test_float8_views_and_leading_dimensions():
    require_gpu()
    c = make_moe(True, 6, 128, 64, 4, 2, "bf16", 20)
    d = moe_on(c)
    Y = moe_call(fw, c, d)
    e = dict(d, A=d["A"].view(2, 3, 128), ids=d["ids"].view(2, 3, 2), weights=d["weights"].view(2, 3, 2),
             w13=d["w13"].view(torch.float8_e4m3fn), w2=d["w2"].view(torch.float8_e4m3fn))
    assert torch.equal(moe_call(fw, c, e), Y.view(2, 3, 128))


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_a_whole_block(fp8):
    """Norm, router product, routing, layer and closing norm as a decode step chains them, eagerly and replayed."""
    require_gpu()
    M, K, E, topk = 5, 256, 12, 3
    c = make_moe(fp8, M, K, 192, E, topk, "bf16", 21)
    d = moe_on(c)
    rng = np.random.default_rng(22)
    x64, x = rounded(rng.standard_normal((M, K)), "bf16")
    pre64, pre = rounded(1 + 0.1 * rng.standard_normal(K), "bf16")
    post64, post = rounded(1 + 0.1 * rng.standard_normal(K), "bf16")
    router = torch.from_numpy(rng.standard_normal((E, K)) / 16).float().cuda()
    x, pre, post = x.cuda(), pre.cuda(), post.cuda()
    ws = torch.empty(fw.fp4w_moe_workspace(M, topk, K, 192), dtype=torch.uint8, device="cuda")

    def block(x):
        _, a = fw.fp4w_block_norm(x, pre_weight=pre, write_residual=False)
        logits = a.float() @ router.t()
        ids, w = fw.fp4w_moe_route(logits, topk)
        y = moe_call(fw, c, dict(d, A=a, ids=ids, weights=w), workspace=ws)
        r, nxt = fw.fp4w_block_norm(y, residual=x, pre_weight=pre, post_weight=post, scale=0.5)
        return a, logits, ids, w, y, r, nxt

    a, logits, ids, w, y, r, nxt = block(x)
    # each step against the oracle on the step's own inputs
    _, want, _, tol = om.block_norm(x64, None, pre64)
    assert_within(a, want, tol, "bf16", "norm")
    want_ids, want_w, rel = om.route(logits.cpu().double().numpy(), topk)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().double().numpy() - want_w) <= rel * want_w).all()
    c.update(A64=a.cpu().double().numpy(), ids=ids.cpu().numpy(), weights=w.cpu().numpy())
    want, tol = moe_want(c)
    assert_within(y, want, tol, "bf16", "layer")
    wr, wy, tr, ty = om.block_norm(y.cpu().double().numpy(), x64, pre64, post64, None, 0.5)
    assert_within(r, wr, tr, "bf16", "residual")
    assert_within(nxt, wy, ty, "bf16", "next norm")

    xs = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = block(xs)
    for k in range(3):
        xs.copy_(torch.roll(x, k, 0))
        g.replay()
        torch.cuda.synchronize()
        again = block(xs)
        for p, q in zip(kept, again):
            assert torch.equal(p, q), k


@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
def test_a_workspace_of_the_largest_batch_serves_smaller_ones(fp8):
    """513 tokens of 8 choices are two parts, 512 are one, larger than either."""
    require_gpu()
    ws = torch.full((fw.fp4w_moe_workspace(513, 8, 128, 64),), 0xFF, dtype=torch.uint8, device="cuda")
    c = make_moe(fp8, 513, 128, 64, 16, 8, "bf16", seed=31, masked=0.05)
    want, tol = moe_want(c)
    d = moe_on(c)
    for M in (513, 512, 40, 1):
        part = {**d, **{k: d[k][:M].contiguous() for k in ("A", "ids", "weights")}}
        assert_within(moe_call(fw, c, part, workspace=ws), want[:M], tol[:M], "bf16", f"M {M}")


@pytest.mark.parametrize("block_size", [256, 384, 640, 4096])
@pytest.mark.parametrize("size", [(1, 1152, 320, 6, 3), (3, 448, 1408, 4, 2), (17, 2048, 192, 3, 2), (40, 704, 576, 2, 1),
                                  (64, 192, 192, 16, 8)], ids=ids_of)
def test_fp8_blocks_of_several_windows(size, block_size):
    """Scale blocks of 2, 3 and 5 windows, whole and partial, and one block per row, through the streaming kernels."""
    require_gpu()
    M, K, I, E, topk = size  # noqa: E741
    c = make_moe(True, M, K, I, E, topk, "bf16", seed=K + block_size, block_size=block_size, masked=0.1 if M > 1 else 0.0)
    # scales that differ by far: a block's neighbour in its place would show
    for name in ("s13", "s2"):
        c[name] *= 4.0 ** (np.arange(c[name].shape[2]) % 3 - 1).astype(np.float32)
    want, tol = moe_want(c)
    assert_within(run(c, path=STREAM[True]), want, tol, "bf16", f"{size} {block_size}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", FORMATS, ids=["fp4", "fp8"])
@pytest.mark.parametrize("size", [(64, 768, 70, 64), (128, 5120, 9, 8), (192, 8192, 7, 6), (64, 1024, 40, 40)], ids=ids_of)
def test_one_token_whose_choices_do_not_fit_in_lds_together(size, fp8, dtype):
    """The choices' rows of I pass LDS: a single token takes the kernels for several, a pass for each of its choices."""
    require_gpu()
    K, I, E, topk = size  # noqa: E741
    assert topk * 2 * (-(-I // 128) * 256 + 16) > 160 * 1024
    c = make_moe(fp8, 1, K, I, E, topk, dtype, seed=I + topk)
    c["ids"][0, topk // 2] = -1
    c["ids"][0, -1] = c["ids"][0, 1] = c["ids"][0, 0]
    want, tol = moe_want(c)
    assert_within(run(c, path=STREAM[fp8]), want, tol, dtype, f"{size}")
    c["ids"][0] = E - 1
    want, tol = moe_want(c)
    assert_within(run(c, path=STREAM[fp8]), want, tol, dtype, f"{size} one expert")
