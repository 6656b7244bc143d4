"""The top alternatives where the search for them is not the usual one: rows that
hold many NaN (as of a model that has diverged), which rank above all numbers, the
lowest id first; and rows whose largest elements are more than the first listing
holds. Ids as the reference's, and the same on repetition."""
import math

import numpy as np
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


def _first_listing(row, k, threads):
    """(chunks, elements) that the search first lists of a row in one block of
    `threads`: those that reach a bound which the best chunks of k to 1.25 k + 2
    threads reach, a chunk's place after its value, every thread's own chunks apart."""
    per = 32 // row.element_size()
    body = row.numel() // per
    z = row[:body * per].float().numpy() + np.float32(0)
    bits = z.view(np.uint32).astype(np.uint64)
    ordered = np.where(bits >> 31 == 1, ~bits & 0xFFFFFFFF, bits | 0x80000000).reshape(body, per)
    place = 0xFFFFFFFE - np.arange(body, dtype=np.uint64)   # (the head of the row comes first)
    chunk = (ordered.max(1) << np.uint64(32)) | place
    best = np.zeros(threads, np.uint64)
    np.maximum.at(best, np.arange(body) % threads, chunk)
    bound = 0
    for bit in range(63, -1, -1):
        if per == 16 and 32 <= bit < 48:
            continue
        n = int((best >= np.uint64(bound | 1 << bit)).sum())
        if n >= k:
            bound |= 1 << bit
            if n <= k + k // 4 + 2:
                break
    listed = chunk >= np.uint64(bound)
    element = (ordered[listed] << np.uint64(32)) | place[listed, None]
    return int(listed.sum()), int((element >= np.uint64(bound)).sum())


FOUND = 512                 # chunks that are read again


def _capacity(k):           # elements that are ranked
    return 16 * max(k, 16)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [50257, 151936])
@pytest.mark.parametrize("k", [40, 128])
def test_more_chunks_than_are_listed(k, V, dtype):
    """Hundreds of the largest chunks in 32 threads' shares, over more rows than are
    in flight at once: every row takes the exact search over its table."""
    per = 32 // torch.finfo(dtype).bits * 8
    g = torch.Generator().manual_seed(V)
    rows = torch.randn(3, V, generator=g)
    high = torch.arange(V) // per % 256 < 32
    rows[0, high] += 10.0
    rows[1, high] = 4.0
    rows[2, high] += torch.randint(8, 11, (int(high.sum()),), generator=g)
    rows = rows.to(dtype)
    for row in rows:
        chunks, elements = _first_listing(row, k, 256)
        assert elements > _capacity(k) and (chunks > FOUND or V < 100000)
    _check_top(rows, 1300, k)


@pytest.mark.parametrize("V", [20011, 32000])
def test_more_elements_than_are_listed(V):
    """Constant rows and rows of two values, 128 alternatives: each of the first
    chunks is full of them."""
    rows = torch.zeros(3, V)
    rows[1] = torch.arange(V) // 2 % 2
    rows[2, 1::2] = -math.inf
    rows = rows.to(BF16)
    assert _first_listing(rows[0], 128, 256)[1] > _capacity(128)
    _check_top(rows, 2500, 128)
