"""The top alternatives of rows that hold many NaN: NaN rank above all numbers,
the lowest id first, whatever the row's length, its number of NaN and theirs of
alternatives, and the same on repetition. (NaN logits are what a model that has
diverged gives.)"""
import math

import pytest
import torch

import fsdp_sharded_mixed_gb300 as zs
import loss_reference as ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: zs.ZS_BF16, torch.float32: zs.ZS_FP32}
BF16, FP32 = torch.bfloat16, torch.float32


def _top(rows, R, k):
    """ids and log probabilities of R rows that repeat ``rows`` in turn."""
    n, V = rows.shape
    z = rows.to(DEV)[torch.arange(R, device=DEV) % n]
    ids = torch.full((R, k), -7, dtype=torch.int32, device=DEV)
    top = torch.empty(R, k, dtype=torch.float32, device=DEV)
    zs.zs_token_logprobs(z, CODE[rows.dtype], R, V, V, None, 1.0, top_k=k, top_ids=ids,
                         top_logprobs=top)
    return ids, top


def _check_top(rows, R, k):
    ids, top = _top(rows, R, k)
    want = ref.top(rows.double(), k)
    assert torch.equal(ids.cpu().long(), want[torch.arange(R) % rows.shape[0]])
    again, top2 = _top(rows, R, k)
    assert torch.equal(again, ids)
    assert torch.equal(top.view(torch.int32), top2.view(torch.int32))
    return top


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V,k", [(151936, 20), (151936, 128), (32000, 64), (50257, 40),
                                 (50257, 1), (1000, 128)])
@pytest.mark.parametrize("R", [3, 200])
def test_rows_with_many_nan(R, V, k, dtype):
    """Rows of NaN throughout, and rows with 30, 200 and 5000 of them."""
    g = torch.Generator().manual_seed(V + k)
    rows = (torch.randn(6, V, generator=g) * 2.5).to(dtype)
    rows[0] = math.nan
    for r, n in ((1, 30), (2, 200), (3, 5000)):
        rows[r, torch.randperm(V, generator=g)[:n]] = math.nan
    rows[4, 1::2] = -math.nan                 # either sign, beside infinities
    rows[4, ::2] = math.inf
    rows[5, V // 2:] = math.nan               # the last half, over masked logits
    rows[5, :V // 2] = -math.inf
    top = _check_top(rows, R, k)
    assert bool(torch.isnan(top).all())
