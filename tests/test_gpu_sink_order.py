"""What a call leaves in its workspace is written before it is read, whatever was there: the
float32 backward's D = dO . o, and every part of every call."""
import math

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from oracle import sink as ref
from sink_testutil import grad_bounds, make, params, prefill, status_of, within
from test_gpu_sink_use import Calls

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("B,H,Hk,d,N,W,A", [
    (2, 4, 4, 64, 509, 96, 1),     # a few CTAs: all of the call's kernels fit the GPU side by side
    (1, 2, 1, 128, 70, 70, 0),
    (2, 6, 2, 64, 700, 700, 0),    # several rounds of CTAs
    (1, 8, 8, 128, 900, 200, 3),
])
def test_backward_over_a_used_workspace(cuda_device, B, H, Hk, d, N, W, A):
    """The workspace (D and the partial sums) holds NaN before each call, and L2 other data: a
    read before its write would show."""
    Q, K, V = make(B, H, Hk, N, N, d, F32, 600 + N, cuda_device)
    p = params(B, H, Hk, d, W, F32)
    O, lse = prefill(p, A, Q, K, V)
    g = torch.Generator().manual_seed(2)
    dOs = [torch.randn(Q.shape, generator=g).to(cuda_device) for _ in range(2)]
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_BACKWARD, N, A, device=cuda_device)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    first = [None, None]
    for k in range(12):
        out = [torch.full_like(x, 7.0) for x in (Q, K, V)]
        ws[256:].fill_(255)
        if k % 3 == 0:
            flush.fill_(k)
        hils.hils_sink_prefill_backward(p, A, Q, K, V, O, lse, dOs[k % 2], *out, workspace=ws)
        first[k % 2] = first[k % 2] or out
        assert all(torch.equal(x, y) for x, y in zip(out, first[k % 2])), f"call {k} gives other bits than the first"
    assert status_of(ws) == 0
    see, scale = ref.visible(N, N, W, A), 1 / math.sqrt(d)
    L, lm = ref.attend(Q, K, V, see, scale)[4].max().item(), lse.abs().max().item()
    for dO, got in zip(dOs, first):
        val, mag, es = ref.backward(Q, K, V, O, lse, dO, see, scale)
        for name, x, v, t in zip(("dQ", "dK", "dV"), got, val, grad_bounds(val, mag, es, L, lm, d, N * H // Hk, F32)):
            within(x, v, t, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
@pytest.mark.parametrize("sizes", [dict(), dict(B=2, H=8, Hk=1, d=128, P=3000), dict(B=1, H=6, Hk=2, N=1500, W=600, A=0, budget=700),
                                   dict(B=2, H=14, Hk=2, d=128, N=2100, W=64, A=70, P=5000, budget=1999)])
def test_every_part_of_a_workspace_is_written_before_it_is_read(cuda_device, dtype, sizes):
    """All six calls over workspaces of zeros and over workspaces of NaN: the same bits."""
    c = Calls(cuda_device, dtype, 7, **sizes)
    c.clear()
    c.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in c.outputs()]
    for _ in range(2):
        for w in c.ws:
            w[256:].fill_(255)  # NaN as float32; the status word's block stays
        c.clear()
        c.run()
        torch.cuda.synchronize()
        assert [i for i, (x, y) in enumerate(zip(c.outputs(), want)) if not torch.equal(x, y)] == []
        assert all(status_of(w) == 0 for w in c.ws)
