"""A whole attention block as it is used: FP4 qkv projection, norms, rotation
and append in one call, attention over the cache, FP4 output projection and the
norm before the next block; first a prompt, then tokens one by one, then the
same from a replayed graph."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
import workloads
from attention_cases import STEP, on_gpu
from gpu_helpers import require_gpu
from oracle import attention as oa, reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Block:
    """Weights and cache of one block: 4 query heads, 2 key heads of 64, hidden size 256."""

    def __init__(self, page=16, room=8):
        rng = np.random.default_rng(50)
        self.Hq, self.Hk, self.D, self.K = 4, 2, 64, 256
        n = (self.Hq + 2 * self.Hk) * self.D
        self.host = []
        for rows, cols in ((n, self.K), (self.K, self.Hq * self.D)):
            B = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
            s = workloads.e4m3_scale_bytes(rng, rows, cols // 16, 0.25, 4.0)
            self.host.append((B, s, np.float32(0.02)))
        self.dev = [(on_gpu(B), on_gpu(s), torch.tensor([g], device="cuda")) for B, s, g in self.host]
        self.wq, self.wk = (torch.ones(64, dtype=torch.bfloat16, device="cuda") * f for f in (1.0, 0.5))
        self.norm = torch.ones(self.K, dtype=torch.bfloat16, device="cuda")
        angle = np.arange(page * room)[:, None] * 10000.0 ** (-np.arange(32) / 32)
        self.cos, self.sin = on_gpu(np.cos(angle).astype(np.float32)), on_gpu(np.sin(angle).astype(np.float32))
        self.table = torch.from_numpy(rng.permutation(2 * room).reshape(2, room).astype(np.int32)).cuda()
        self.cache = fw.fp8w_kv_cache(2 * room, self.Hk, page, self.D)

    def __call__(self, x, lens, starts=None, most=None, keep=None):
        q_width = self.Hq * self.D
        qkv = fw.fp4w_matmul(x, *self.dev[0])
        heads = qkv.view(x.shape[0], -1, self.D)
        q, k, v = heads.split((self.Hq, self.Hk, self.Hk), 1)
        q = fw.fp8w_kv_append(k, v, self.cache, self.table, lens, starts=starts, q=q, q_weight=self.wq, k_weight=self.wk,
                              cos=self.cos, sin=self.sin)
        a = fw.fp8w_attention(q, self.cache, self.table, lens, starts=starts, max_new=most)
        o = fw.fp4w_matmul(a.view(x.shape[0], q_width), *self.dev[1])
        if keep is not None:
            keep.update(qkv=qkv, q=q, a=a, o=o)
        return fw.fp4w_block_norm(o, residual=x, pre_weight=self.norm)


def test_prompt_then_tokens():
    """Each step against the oracle, on what the steps before it have really produced."""
    block = Block()
    rng = np.random.default_rng(51)
    new, held = [19, 33], [0, 0]
    for step in range(4):
        M = sum(new)
        x = torch.from_numpy(rng.standard_normal((M, block.K)).astype(np.float32)).bfloat16().cuda()
        lens = np.array([h + n for h, n in zip(held, new)], np.int32)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        before = [t.cpu().numpy().copy() for t in block.cache]
        kept = {}
        _, y = block(x, on_gpu(lens), on_gpu(starts) if step == 0 else None, max(new), kept)
        torch.cuda.synchronize()
        table = block.table.cpu().numpy()
        qkv = kept["qkv"].double().cpu().numpy().reshape(M, -1, 64)
        pos = [p[1] for p in oa.places(starts, lens, table, 16, 16, M)]
        cos, sin = block.cos.cpu().numpy(), block.sin.cpu().numpy()
        want, tol = oa.norm_rope(qkv[:, :4], np.ones(64), cos, sin, pos)
        q = kept["q"].double().cpu().numpy()
        assert (np.abs(q - want) <= tol + STEP["bf16"] * (np.abs(want) + tol)).all()
        parts = [t.cpu().numpy() for t in block.cache]
        kx, tol = oa.norm_rope(qkv[:, 4:6], np.full(64, 0.5), cos, sin, pos)
        stored, scale = oa.append(kx, before[0], before[2], starts, lens, table, 16)
        assert np.array_equal(scale, parts[2])
        # codes next to a tie may go either way
        off = np.abs(oa.TABLE[stored] - oa.TABLE[parts[0]]) * oa.power(scale)[:, :, None, None]
        assert (stored != parts[0]).mean() < 1e-4 and (off <= 2.0 ** -3 * np.abs(kx).max()).all()
        stored, scale = oa.append(qkv[:, 6:], before[1].transpose(0, 1, 3, 2), before[3], starts, lens, table, 16)
        assert np.array_equal(stored, parts[1].transpose(0, 1, 3, 2)) and np.array_equal(scale, parts[3])
        Y, _, tol, _ = oa.attention(q, *parts, starts, lens, table, 64 ** -0.5)
        a = kept["a"].double().cpu().numpy()
        assert (np.abs(a - Y) <= tol + STEP["bf16"] * (np.abs(Y) + tol)).all()
        B, s, g = block.host[1]
        bits = kept["a"].reshape(M, -1).cpu().view(torch.int16).numpy().view(np.uint16)
        Yo, S = ref.matmul_fp4_reference(bits, "bf16", B, s, 16, g, None)
        assert ref.check_matmul(kept["o"].cpu().view(torch.int16).numpy().view(np.uint16), "bf16", Yo, S)["ok"]
        assert torch.isfinite(y).all()
        held, new = lens.tolist(), [1, 1]


def test_decode_loop_from_a_graph():
    """Tokens from a replayed graph and from eager calls give the same outputs and caches."""
    rng = np.random.default_rng(52)
    eager, replayed = Block(), Block()
    prompt = torch.from_numpy(rng.standard_normal((40, 256)).astype(np.float32)).bfloat16().cuda()
    first, starts = torch.tensor([25, 15], dtype=torch.int32, device="cuda"), torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    for b in (eager, replayed):
        b(prompt, first, starts, 25)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    lens = first.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        r, y = replayed(x, lens)
    seen = first.clone()
    for step in range(20):
        x.copy_(torch.from_numpy(rng.standard_normal((2, 256)).astype(np.float32)))
        seen += 1
        want = eager(x, seen)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, want[0]) and torch.equal(y, want[1]), step
        assert all(torch.equal(a, b) for a, b in zip(eager.cache, replayed.cache)), step
    assert lens.tolist() == [45, 35]
