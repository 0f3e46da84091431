"""Attention over page tables with room for far more than the sequences hold, as
a server has them: the prompt kernel's parts follow the lengths."""

import numpy as np
import pytest
import torch

import fp8_weight_only_fp4w_amd as fw
from attention_cases import batch, filled, on_gpu, rounded, to_cache, within
from gpu_helpers import require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def run(rng, held, new, page, Hq, Hk, D, window, dtype, room):
    """The prompt kernel over a table with room for `room` tokens, checked; bytes of its workspace that it has written."""
    starts, lens, table, pages = batch(rng, held, new, page)
    parts = filled(rng, starts, lens, table, page, pages, Hk, D)
    q = rounded(rng, (sum(new), Hq, D), dtype, 1.5)
    Y, L, tol, tol_l = oa.attention(q, *parts, starts, lens, table, D ** -0.5, True, window, dtype)
    table = np.pad(table, ((0, 0), (0, room // page - table.shape[1])), constant_values=-1)
    work = torch.full((fw.fp8w_attention_workspace(sum(new), Hq, Hk, D, len(new), max(new)),), 0xAB, dtype=torch.uint8, device="cuda")
    lse = torch.empty(sum(new), Hq, device="cuda")
    got = fw.fp8w_attention(on_gpu(q, dtype), to_cache(parts), on_gpu(table), on_gpu(lens), starts=on_gpu(starts), max_new=max(new),
                            window=window, lse=lse, workspace=work, path=fw.PATH_ATTN_PROMPT)
    within(got, Y, tol, dtype)
    l = lse.double().cpu().numpy()
    assert (np.abs(l - L) <= tol_l + 2.0 ** -24 * np.abs(L)).all()
    return int((work != 0xAB).sum())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("held,new,Hq,Hk,D,window", [([0], [200], 10, 2, 128, 0), ([0, 300, 20], [130, 5, 64], 8, 2, 64, 0), ([5000], [40], 8, 1, 128, 400)])
def test_short_rows_are_not_cut(held, new, Hq, Hk, D, window, dtype):
    """No row has 16 tiles of keys, so none has two parts of 8: nothing goes through the workspace."""
    assert run(np.random.default_rng(80), held, new, 16, Hq, Hk, D, window, dtype, 32768) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("held,new,D,window", [([900, 10, 2600], [150, 40, 1], 128, 0), ([1500, 4000], [33, 20], 64, 0), ([5000], [40], 128, 1500)])
def test_rows_of_unequal_length(held, new, D, window, dtype):
    """Rows with one part, two and many in one call."""
    rng = np.random.default_rng(81)
    assert run(rng, held, new, 16, 4, 1, D, window, dtype, 32768) > 0
    run(rng, held, new, 64, 6, 2, D, window, dtype, 8192)
