"""Seeded inputs and comparisons of the tests around mixture-of-experts
blocks.  Inputs are drawn on the CPU with numpy; only the comparison with the
oracle's bounds is shared by the tests."""

import numpy as np
import torch

import workloads

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rounded(x, dtype):
    """x in float64 after rounding to the type, and the torch tensor."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype])
    return t.double().numpy(), t


def make_moe(fp8, M, K, I, E, topk, dtype, seed, block_size=None, masked=0.0, spread=1.0):  # noqa: E741
    """A layer's inputs: dict of numpy arrays (A in float64 too, as A64)."""
    rng = np.random.default_rng(seed)
    bs = block_size or (128 if fp8 else 16)
    c = {"fp8": fp8, "dtype": dtype, "block_size": bs, "M": M, "K": K, "I": I, "E": E, "topk": topk}
    c["A64"], c["A"] = rounded(rng.standard_normal((M, K)) * spread, dtype)
    ids = np.stack([rng.permutation(max(E, topk))[:topk] for _ in range(M)]) if M else np.zeros((0, topk))
    ids = np.where(rng.random((M, topk)) < masked, -1, ids % max(E, 1))
    c["ids"] = ids.astype(np.int32)
    c["weights"] = rng.uniform(0.05, 1.0, (M, topk)).astype(np.float32)
    cols = lambda n: -(-n // bs)  # noqa: E731
    if fp8:
        c["w13"] = workloads.fp8_weights(rng, E * 2 * I, K).reshape(E, 2 * I, K)
        c["w2"] = workloads.fp8_weights(rng, E * K, I).reshape(E, K, I)
        c["s13"] = (rng.uniform(0.004, 0.012, (E, 2 * I, cols(K))) / np.sqrt(max(K, 1))).astype(np.float32)
        c["s2"] = (rng.uniform(0.004, 0.012, (E, K, cols(I))) / np.sqrt(max(I, 1))).astype(np.float32)
        c["g13"] = c["g2"] = None
    else:
        c["w13"] = rng.integers(0, 256, (E, 2 * I, K // 2), dtype=np.uint8)
        c["w2"] = rng.integers(0, 256, (E, K, I // 2), dtype=np.uint8)
        c["s13"] = workloads.e4m3_scale_bytes(rng, E * 2 * I, cols(K), 0.25, 4.0).reshape(E, 2 * I, cols(K))
        c["s2"] = workloads.e4m3_scale_bytes(rng, E * K, cols(I), 0.25, 4.0).reshape(E, K, cols(I))
        c["g13"] = (rng.uniform(0.08, 0.2, E) / np.sqrt(max(K, 1))).astype(np.float32)
        c["g2"] = (rng.uniform(0.08, 0.2, E) / np.sqrt(max(I, 1))).astype(np.float32)
    return c


def moe_on(c, device="cuda"):
    """The inputs as tensors on the device."""
    d = {}
    for k in ("ids", "weights", "w13", "w2", "s13", "s2", "g13", "g2"):
        d[k] = None if c[k] is None else torch.from_numpy(np.ascontiguousarray(c[k])).to(device)
    d["A"] = c["A"].to(device)
    return d


def moe_call(fw, c, d, act="silu", **kw):
    if c["fp8"]:
        return fw.fp8w_moe(d["A"], d["ids"], d["weights"], d["w13"], d["s13"], d["w2"], d["s2"],
                           block_size=c["block_size"], activation=act, **kw)
    return fw.fp4w_moe(d["A"], d["ids"], d["weights"], d["w13"], d["s13"], d["g13"], d["w2"], d["s2"], d["g2"],
                       block_size=c["block_size"], activation=act, **kw)


def moe_want(c, act="silu"):
    from oracle import moe as om
    return om.moe(c["A64"], c["ids"], c["weights"], c["w13"], c["s13"], c["g13"], c["w2"], c["s2"], c["g2"],
                  c["block_size"], act, c["fp8"])


def assert_within(got, want, tol, dtype, what=""):
    """got (a tensor of the type) lies in [round(want - tol), round(want + tol)]; NaN where want is NaN."""
    assert tuple(got.shape) == want.shape, what
    g = got.detach().cpu().double().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in other places"
    if dtype == "fp32":
        lo, hi = want - tol - np.abs(want) * 2.0 ** -24, want + tol + np.abs(want) * 2.0 ** -24
    else:
        lo, hi = (torch.from_numpy(x).to(TORCH[dtype]).double().numpy() for x in (want - tol, want + tol))
    bad = ~nan & ~((lo <= g) & (g <= hi))
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside, first at {at}: got {g[at]!r}, "
                             f"want {want[at]!r} +- {tol[at]!r}")
