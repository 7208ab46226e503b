"""Eviction from caches of more slots than a cluster's registers hold, up to the most tokens
that a call takes."""
import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from sink_testutil import params

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def evict(p, A, budget, K, V, acc, n):
    B, Hk, T, d = K.shape
    Ko, Vo = (torch.full((B, Hk, budget, d), 3.0, dtype=K.dtype, device=K.device) for _ in range(2))
    ao = torch.full((B, Hk, budget), 3.0, device=K.device)
    idx = torch.full((B, Hk, budget), 99, dtype=torch.int32, device=K.device)
    out = torch.zeros(B, dtype=torch.int32, device=K.device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_CACHE_EVICT, T, budget, device=K.device)
    hils.hils_cache_evict(p, A, budget, K, V, acc, n, Ko, Vo, ao, idx, out, workspace=ws)
    torch.cuda.synchronize()
    return Ko, Vo, ao, idx, out


@pytest.mark.parametrize("heavy_from", [0, 2 ** 31 - 4000])
def test_the_most_tokens(cuda_device, heavy_from):
    """2^31 - 1025 slots (their rows one and the same in memory): the count of a thread's slots
    steps past 2^31 behind the last one."""
    T, d, W, A, budget = 2 ** 31 - 1025, 64, 10, 2, 40
    K = torch.randn(1, 1, 1, d, generator=torch.Generator().manual_seed(1)).to(BF).to(cuda_device).expand(1, 1, T, d)
    acc = torch.zeros(1, 1, T, device=cuda_device)
    first, last = max(A, heavy_from), T - W - 1
    heavy = sorted({first, first + 77, last - 1100, last - 1, last})
    for i, j in enumerate(heavy):
        acc[0, 0, j] = 1.0 + i
    n = torch.tensor([T], dtype=torch.int32, device=cuda_device)
    Ko, Vo, ao, idx, out = evict(params(1, 1, 1, d, W, BF), A, budget, K, K, acc, n)
    light = [j for j in range(A, A + budget) if j not in heavy][:budget - A - W - len(heavy)]  # of equal weights, the first
    want = sorted(set(range(A)) | set(light) | set(heavy)) + list(range(T - W, T))
    assert len(want) == budget and idx[0, 0].tolist() == want and out.tolist() == [budget]
    assert torch.equal(Ko[0, 0], K[0, 0, :budget]) and torch.equal(Vo[0, 0], K[0, 0, :budget])
    assert torch.equal(ao[0, 0], acc[0, 0, torch.tensor(want, device=cuda_device)])
