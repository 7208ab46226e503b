"""Eviction from caches of more slots than a cluster's registers hold, up to the most tokens
that a call takes."""
import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from oracle import sink as ref
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


@pytest.mark.parametrize("T,budget,W,A,lens", [(140001, 70000, 64, 4, [140001, 133000]), (200000, 199000, 0, 0, [200000, 199500]),
                                               (300007, 1000, 512, 16, [300007, 131600])])
@pytest.mark.parametrize("spread,dtype,d", [(3.0, BF, 128), (1e-4, F32, 64)])
def test_more_slots_than_the_registers_hold(cuda_device, T, budget, W, A, lens, spread, dtype, d):
    """Two sequences with more than 131072 slots between the sinks and the window: weights over
    many exponents or close together, ties of zeros of both signs, infinities and NaN, on both
    sides of the border between registers and memory."""
    g = torch.Generator(device="cuda").manual_seed(T)
    acc = torch.exp(spread * torch.randn(2, 1, T, generator=g, device="cuda") - 2.0)
    u = torch.rand(acc.shape, generator=g, device="cuda")
    for lo, hi, x in ((0.0, 0.2, 0.0), (0.2, 0.3, -0.0), (0.3, 0.31, float("inf")), (0.31, 0.33, float("nan")), (0.33, 0.36, float("-inf"))):
        acc[(u >= lo) & (u < hi)] = x
    K, V = (torch.randn(2, 1, T, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    Ko, Vo, ao, idx, out = evict(params(2, 1, 1, d, W, dtype), A, budget, K, V, acc, n)
    rows, new = ref.evict(acc, torch.tensor(lens), budget, W, A)
    assert out.tolist() == new == [budget, budget]
    for b in range(2):
        at = torch.tensor(rows[b][0], dtype=torch.long, device=cuda_device)
        assert torch.equal(idx[b, 0].long(), at)
        assert torch.equal(Ko[b, 0], K[b, 0, at]) and torch.equal(Vo[b, 0], V[b, 0, at])
        assert torch.equal(ao[b, 0].view(torch.int32), acc[b, 0, at].view(torch.int32))
