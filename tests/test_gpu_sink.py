"""Attention with a sliding window and sinks on the GPU: prefill, backward, decode and
accumulated weights against the float64 evaluation."""
import math

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from oracle import sink as ref
from sink_testutil import (check_prefill, forward_bounds, grad_bounds, make, params, prefill, status_of, weight_bound,
                           within)

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# B, H, Hk, d, Lq, N, W, A
SHAPES = [
    (1, 1, 1, 128, 1, 1, 1, 0),
    (1, 1, 1, 64, 1, 1, 0, 0),          # nothing visible: o = 0, lse = -inf
    (2, 2, 1, 128, 5, 5, 0, 2),         # sinks only
    (1, 2, 2, 64, 130, 130, 1, 0),      # each token itself
    (2, 4, 2, 128, 257, 257, 64, 4),
    (1, 3, 1, 64, 300, 300, 100, 1),    # groups of three
    (1, 8, 1, 128, 200, 200, 33, 130),  # sinks past a tile, groups of eight
    (1, 4, 4, 128, 384, 384, 384, 0),   # full causal
    (2, 5, 1, 64, 77, 901, 2000, 3),    # a later piece, window longer than the sequence
    (1, 6, 2, 128, 1, 1300, 500, 5),    # one query of a long sequence
    (3, 2, 2, 64, 65, 1025, 128, 200),
    (1, 14, 2, 128, 513, 700, 90, 7),   # groups of seven
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,Lq,N,W,A", SHAPES)
def test_prefill(cuda_device, B, H, Hk, d, Lq, N, W, A, dtype):
    Q, K, V = make(B, H, Hk, Lq, N, d, dtype, 100 + N, cuda_device)
    p = params(B, H, Hk, d, W, dtype)
    O, lse = prefill(p, A, Q, K, V)
    check_prefill(p, A, Q, K, V, O, lse)


def test_prefill_without_lse_and_with_a_scale(cuda_device):
    Q, K, V = make(1, 4, 2, 150, 150, 128, BF, 5, cuda_device)
    p = params(1, 4, 2, 128, 40, BF, scale=-0.02)
    O, _ = prefill(p, 3, Q, K, V, lse=False)
    check_prefill(p, 3, Q, K, V, O, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_strided_views(cuda_device, dtype):
    """[B, T, H, d] memory seen as [B, H, T, d], for inputs and outputs."""
    Q, K, V = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in make(2, 6, 3, 200, 333, 64, dtype, 8, cuda_device))
    p = params(2, 6, 3, 64, 70, dtype)
    O = torch.empty(2, 200, 6, 64, dtype=dtype, device=cuda_device).transpose(1, 2)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_PREFILL, 200, 2, device=cuda_device)
    hils.hils_sink_prefill(p, 2, Q, K, V, O, None, workspace=ws)
    check_prefill(p, 2, Q, K, V, O, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unseen_slots_may_hold_anything(cuda_device, dtype):
    """Between the sinks and the first window no query looks: NaN there changes nothing."""
    Q, K, V = make(1, 4, 2, 100, 1000, 128, dtype, 9, cuda_device)
    p = params(1, 4, 2, 128, 150, dtype)
    want = prefill(p, 5, Q, K, V)
    K[:, :, 5:751 - 0] = math.nan
    V[:, :, 5:751] = math.inf
    got = prefill(p, 5, Q, K, V)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _backward(p, A, Q, K, V, O, lse, dO):
    out = [torch.full_like(x, 7.0) for x in (Q, K, V)]
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_BACKWARD, Q.shape[2], A, device=Q.device)
    hils.hils_sink_prefill_backward(p, A, Q, K, V, O, lse, dO, *out, workspace=ws)
    torch.cuda.synchronize()
    assert status_of(ws) == 0
    return out


def _check_backward(p, A, Q, K, V, O, lse, dO, got, what=""):
    d, N = Q.shape[3], Q.shape[2]
    see = ref.visible(N, N, p.W, A)
    scale = p.scale or 1 / math.sqrt(d)
    val, mag, es = ref.backward(Q, K, V, O, lse, dO, see, scale)
    L = ref.attend(Q, K, V, see, scale)[4].max().item()
    fin = lse[torch.isfinite(lse)]
    lm = fin.abs().max().item() if fin.numel() else 0.0
    G = p.H // p.Hk
    for name, g, v, t in zip(("dQ", "dK", "dV"), got, val, grad_bounds(val, mag, es, L, lm, d, N * G, p.dtype)):
        within(g, v, t, f"{what} {name}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,N,W,A", [
    (1, 1, 1, 128, 1, 1, 0), (1, 2, 1, 64, 3, 0, 0), (2, 2, 1, 128, 6, 0, 2), (1, 2, 2, 64, 130, 1, 0),
    (2, 4, 2, 128, 257, 64, 4), (1, 3, 1, 64, 300, 100, 1), (1, 8, 1, 128, 200, 33, 130), (1, 4, 4, 128, 384, 384, 0),
    (1, 7, 1, 64, 900, 50, 4), (1, 8, 2, 128, 1100, 300, 140),
])
def test_backward(cuda_device, B, H, Hk, d, N, W, A, dtype):
    Q, K, V = make(B, H, Hk, N, N, d, dtype, 200 + N, cuda_device)
    p = params(B, H, Hk, d, W, dtype)
    O, lse = prefill(p, A, Q, K, V)
    dO = torch.randn(Q.shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(cuda_device)
    got = _backward(p, A, Q, K, V, O, lse, dO)
    _check_backward(p, A, Q, K, V, O, lse, dO, got)
    again = _backward(p, A, Q, K, V, O, lse, dO)
    assert all(torch.equal(x, y) for x, y in zip(got, again)), "equal calls, other bits"


def test_backward_against_differences(cuda_device):
    """Float32 gradients against central differences of the float64 forward."""
    B, H, Hk, d, N, W, A = 1, 4, 2, 64, 90, 20, 3
    Q, K, V = make(B, H, Hk, N, N, d, F32, 77, cuda_device)
    p = params(B, H, Hk, d, W, F32)
    O, lse = prefill(p, A, Q, K, V)
    g = torch.Generator().manual_seed(3)
    dO = torch.randn(Q.shape, generator=g)
    got = _backward(p, A, Q, K, V, O, lse, dO.to(cuda_device))
    see = ref.visible(N, N, W, A)

    def loss(q, k, v):
        return (ref.attend(q, k, v, see, 1 / math.sqrt(d))[0] * dO.double()).sum()

    x = [t.cpu().double() for t in (Q, K, V)]
    h = 1e-5
    for i in range(3):
        u = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        hi, lo = ([t + s * h * u if k == i else t for k, t in enumerate(x)] for s in (1, -1))
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        mine = (got[i].cpu().double() * u).sum()
        # float32 gradients: relative 1e-5 of the terms' size; differences: h^2 and 1e-16 / h
        size = (got[i].cpu().double() * u).abs().sum()
        assert abs(want - mine) <= 1e-5 * size + 1e-8 * size, (i, want, mine)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_strided_views(cuda_device, dtype):
    def far(x):
        return x.transpose(1, 2).contiguous().transpose(1, 2)

    Q, K, V = (far(x) for x in make(2, 6, 3, 210, 210, 64, dtype, 18, cuda_device))
    p = params(2, 6, 3, 64, 70, dtype)
    O, lse = prefill(p, 2, Q, K, V)
    dO = far(torch.randn(Q.shape, generator=torch.Generator().manual_seed(2)).to(dtype).to(cuda_device))
    got = _backward(p, 2, Q, K, V, far(O), lse, dO)
    _check_backward(p, 2, Q, K, V, O, lse, dO, got)


def _weights(p, A, Q, K, lse, acc, out=None):
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_WEIGHTS, K.shape[2], A, device=Q.device)
    hils.hils_sink_weights(p, A, Q, K, lse, acc, out, workspace=ws)
    torch.cuda.synchronize()
    assert status_of(ws) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,Lq,N,W,A", SHAPES)
def test_weights(cuda_device, B, H, Hk, d, Lq, N, W, A, dtype):
    Q, K, V = make(B, H, Hk, Lq, N, d, dtype, 300 + N, cuda_device)
    p = params(B, H, Hk, d, W, dtype)
    _, lse = prefill(p, A, Q, K, V)
    T = N + 9
    acc = torch.rand(B, Hk, T, generator=torch.Generator().manual_seed(4)).to(cuda_device)
    out = torch.full_like(acc, -5.0)
    _weights(p, A, Q, K, lse, acc, out)
    see = ref.visible(Lq, N, W, A)
    scale = 1 / math.sqrt(d)
    add = ref.weights(Q, K, lse, see, scale)
    L = ref.attend(Q, K, V, see, scale)[4].max().item()
    fin = lse[torch.isfinite(lse)]
    lm = fin.abs().max().item() if fin.numel() else 0.0
    want = acc.cpu().double()
    tol = torch.zeros_like(want)
    tol[:, :, :N] = weight_bound(add, L, lm, d, Lq * H // Hk) + 2.0 ** -23 * (want[:, :, :N] + add)
    want[:, :, :N] += add
    seen = torch.zeros(T, dtype=torch.bool)
    seen[:N] = see.any(0)
    want[:, :, ~seen] = -5.0  # slots that no query sees are left as they were
    within(out, want, tol, "acc")
    _weights(p, A, Q, K, lse, acc)  # in place: the same numbers where they are written
    assert torch.equal(acc[:, :, seen.to(cuda_device)], out[:, :, seen.to(cuda_device)])


def _decode(p, A, Q, K, V, lens, acc=None, out=None):
    O = torch.full_like(Q, 7.0)
    lse = torch.full(Q.shape[:2], 7.0, dtype=F32, device=Q.device)
    call = hils.HILS_CALL_SINK_DECODE if acc is None else hils.HILS_CALL_SINK_DECODE_ACC
    ws = hils.alloc_workspace(p, call, K.shape[2], A, device=Q.device)
    hils.hils_sink_decode(p, A, Q, K, V, lens, O, lse, acc=acc, acc_out=out, workspace=ws)
    torch.cuda.synchronize()
    assert status_of(ws) == 0
    return O, lse


def _check_decode(p, A, Q, K, V, lens, O, lse, what=""):
    d, T = Q.shape[3], K.shape[2]
    rO, rl, pr, Om, L = ref.attend(Q, K, V, ref.decode_visible(lens, T, p.W, A), p.scale or 1 / math.sqrt(d))
    tO, tl = forward_bounds(rO, Om, rl, L, d, min(T, p.W + A), p.dtype)
    within(O, rO, tO, f"{what} O")
    within(lse, rl[..., 0], tl[..., 0], f"{what} lse")
    return pr, L


# B, H, Hk, d, T, W, A, lens
DECODES = [
    (1, 1, 1, 128, 1, 1, 0, [1]),
    (2, 2, 2, 64, 5, 0, 0, [5, 0]),                      # nothing visible; an empty cache
    (3, 4, 1, 128, 300, 64, 4, [300, 1, 3]),
    (2, 3, 1, 64, 700, 700, 0, [700, 699]),
    (4, 8, 1, 128, 1000, 100, 70, [1000, 100, 101, 65]),
    (2, 10, 2, 64, 513, 0, 5, [513, 2]),                 # sinks only, groups of five
    (3, 14, 2, 128, 2049, 4000, 9, [2049, -3, 5000]),    # lengths outside the cache count as its ends
    (1, 6, 6, 128, 5000, 5000, 0, [4999]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,T,W,A,lens", DECODES)
def test_decode(cuda_device, B, H, Hk, d, T, W, A, lens, dtype):
    Q, K, V = make(B, H, Hk, 1, T, d, dtype, 400 + T, cuda_device)
    for b, n in enumerate(lens):  # what lies behind a sequence is never part of it
        K[b, :, max(0, n):] = math.nan
        V[b, :, max(0, n):] = math.inf
        lo = max(0, min(n, T) - W)
        K[b, :, min(A, lo):lo] = math.nan
        V[b, :, min(A, lo):lo] = math.nan
    p = params(B, H, Hk, d, W, dtype)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    O, lse = _decode(p, A, Q, K, V, n)
    pr, L = _check_decode(p, A, Q, K, V, n, O, lse)
    acc = torch.rand(B, Hk, T, generator=torch.Generator().manual_seed(6)).to(cuda_device)
    out = torch.full_like(acc, -5.0)
    O2, lse2 = _decode(p, A, Q, K, V, n, acc, out)
    assert torch.equal(O2, O) and torch.equal(lse2, lse), "the accumulated weights change the output"
    add = pr.view(B, Hk, H // Hk, T).sum(2)
    see = ref.decode_visible(n, T, W, A)[:, 0].expand(B, Hk, T)
    want = torch.where(see, acc.cpu().double() + add, torch.full((), -5.0, dtype=torch.float64))
    fin = lse[torch.isfinite(lse)]
    lm = fin.abs().max().item() if fin.numel() else 0.0
    # the weight's own lse has the forward's error beside the logit's
    tol = 2 * weight_bound(add, L.max().item(), lm, d, T) + 2.0 ** -23 * want.abs()
    within(out, want, torch.where(see, tol, torch.zeros_like(tol)), "acc")
    _decode(p, A, Q, K, V, n, acc)
    assert torch.equal(acc[see.to(cuda_device)], out[see.to(cuda_device)])


def test_decode_equals_the_prefill_row(cuda_device):
    """A token decoded over its cache and the same token as the last row of a prompt."""
    Q, K, V = make(1, 8, 2, 400, 400, 128, BF, 41, cuda_device)
    p = params(1, 8, 2, 128, 100, BF)
    O, lse = prefill(p, 4, Q, K, V)
    n = torch.tensor([400], dtype=torch.int32, device=cuda_device)
    o, l = _decode(p, 4, Q[:, :, -1:], K, V, n)
    _check_decode(p, 4, Q[:, :, -1:], K, V, n, o, l)
    assert (lse[..., -1] - l).abs().max() < 1e-4


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,P,T,lens", [
    (1, 1, 1, 128, 0, 3, [2]),                             # no prefix
    (2, 4, 2, 64, 1, 1, [0, 1]),
    (3, 3, 1, 128, 700, 70, [0, 70, 33]),                  # groups of three
    (5, 8, 1, 64, 1029, 20, [20, 0, 1, 7, 19]),
    (33, 4, 1, 128, 600, 40, [(7 * i) % 41 for i in range(33)]),  # more rows than one tile
    (70, 10, 2, 64, 300, 12, [i % 13 for i in range(70)]),        # groups of five, several tiles
    (4, 8, 8, 128, 5000, 300, [300, -1, 400, 0]),
    (2, 2, 2, 128, 64, 0, [0, 0]),                         # prefix only
])
def test_prefix(cuda_device, B, H, Hk, d, P, T, lens, dtype):
    Q, Kp, Vp = make(B, H, Hk, 1, P, d, dtype, 500 + P, cuda_device)
    Kp, Vp = Kp[:1].contiguous(), Vp[:1].contiguous()
    _, Kc, Vc = make(B, H, Hk, 1, T, d, dtype, 501 + P, cuda_device)
    for b, n in enumerate(lens):
        Kc[b, :, max(0, n):] = math.nan
        Vc[b, :, max(0, n):] = math.nan
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    p = params(B, H, Hk, d, 0, dtype)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_PREFIX_DECODE, T, P, device=cuda_device)
    O = torch.full_like(Q, 7.0)
    lse = torch.full((B, H), 7.0, device=cuda_device)
    hils.hils_prefix_decode(p, Q, Kp, Vp, Kc, Vc, n, O, lse, workspace=ws)
    torch.cuda.synchronize()
    assert status_of(ws) == 0
    rO, rl, _, Om, L = ref.prefix(Q, Kp, Vp, Kc, Vc, n, 1 / math.sqrt(d))
    tO, tl = forward_bounds(rO, Om, rl, L, d, P + T, dtype)
    within(O, rO, tO, "O")
    within(lse, rl[..., 0], tl[..., 0], "lse")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hk,d,T,budget,W,A,lens", [
    (1, 1, 128, 1, 1, 0, 0, [1]),
    (2, 2, 64, 40, 0, 0, 0, [40, 0]),               # nothing kept
    (3, 1, 128, 500, 100, 20, 3, [500, 100, 101]),
    (2, 3, 64, 1500, 700, 0, 0, [1500, 702]),
    (2, 2, 128, 5000, 33, 30, 3, [5000, 34]),       # nothing between the sinks and the window
    (2, 2, 64, 3000, 5000, 10, 1, [3000, 7000]),    # a budget beyond the cache
    (2, 1, 128, 9000, 8000, 64, 4, [9000, -1]),
])
def test_evict(cuda_device, B, Hk, d, T, budget, W, A, lens, dtype):
    g = torch.Generator().manual_seed(T)
    K = torch.randn(B, Hk, T, d, generator=g).to(dtype).to(cuda_device)
    V = torch.randn(B, Hk, T, d, generator=g).to(dtype).to(cuda_device)
    acc = torch.randint(0, 40, (B, Hk, T), generator=g).float() / 8  # many ties
    acc[torch.rand(acc.shape, generator=g) < 0.05] = -0.0
    acc[torch.rand(acc.shape, generator=g) < 0.02] = math.nan
    acc[torch.rand(acc.shape, generator=g) < 0.02] = math.inf
    acc[torch.rand(acc.shape, generator=g) < 0.02] = -math.inf
    acc = acc.to(cuda_device)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    p = params(B, Hk, Hk, d, W, dtype)
    Ko, Vo = (torch.full((B, Hk, budget, d), 3.0, dtype=dtype, device=cuda_device) for _ in range(2))
    ao = torch.full((B, Hk, budget), 3.0, device=cuda_device)
    idx = torch.full((B, Hk, budget), 99, dtype=torch.int32, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_CACHE_EVICT, T, budget, device=cuda_device)
    hils.hils_cache_evict(p, A, budget, K, V, acc, n, Ko, Vo, ao, idx, n, workspace=ws)  # lengths in place
    torch.cuda.synchronize()
    rows, new = ref.evict(acc, torch.tensor(lens), budget, W, A)
    assert n.tolist() == new
    for b in range(B):
        for h in range(Hk):
            at = torch.tensor(rows[b][h], dtype=torch.long, device=cuda_device)
            m = len(rows[b][h])
            assert idx[b, h].tolist() == rows[b][h] + [-1] * (budget - m), (b, h)
            assert torch.equal(Ko[b, h, :m], K[b, h, at]) and torch.equal(Vo[b, h, :m], V[b, h, at])
            assert torch.equal(ao[b, h, :m].nan_to_num(nan=-9.0), acc[b, h, at].nan_to_num(nan=-9.0))
            assert (Ko[b, h, m:] == 3.0).all() and (Vo[b, h, m:] == 3.0).all() and (ao[b, h, m:] == 3.0).all()


@pytest.mark.parametrize("T,budget,W,A", [(33, 20, 3, 1), (2048, 700, 30, 4), (2300, 1000, 0, 0), (16384, 5000, 512, 4),
                                          (16500, 16000, 100, 0), (40000, 9000, 64, 4)])
@pytest.mark.parametrize("spread", [1.5, 1e-4])
def test_evict_by_distinct_weights(cuda_device, T, budget, W, A, spread):
    """Weights without ties but for a fifth of zeros, close together or far apart: several
    histograms deep, and (40000) with slots beyond a CTA's registers."""
    B, Hk, d = 2, 2, 64
    g = torch.Generator().manual_seed(T)
    acc = torch.exp(spread * torch.randn(B, Hk, T, generator=g) - 2.0)
    acc[torch.rand(acc.shape, generator=g) < 0.2] = 0.0
    acc = acc.to(cuda_device)
    K = torch.randn(B, Hk, T, d, generator=g).to(BF).to(cuda_device)
    lens = [T, T - T // 9]
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    p = params(B, Hk, Hk, d, W, BF)
    Ko, Vo = (torch.zeros(B, Hk, budget, d, dtype=BF, device=cuda_device) for _ in range(2))
    ao = torch.zeros(B, Hk, budget, device=cuda_device)
    idx = torch.full((B, Hk, budget), -7, dtype=torch.int32, device=cuda_device)
    out = torch.zeros(B, dtype=torch.int32, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_CACHE_EVICT, T, budget, device=cuda_device)
    hils.hils_cache_evict(p, A, budget, K, K, acc, n, Ko, Vo, ao, idx, out, workspace=ws)
    rows, new = ref.evict(acc, torch.tensor(lens), budget, W, A)
    assert out.tolist() == new
    for b in range(B):
        for h in range(Hk):
            m = len(rows[b][h])
            assert idx[b, h].tolist() == rows[b][h] + [-1] * (budget - m), (b, h)
            at = torch.tensor(rows[b][h], dtype=torch.long, device=cuda_device)
            assert torch.equal(Ko[b, h, :m], K[b, h, at]) and torch.equal(ao[b, h, :m], acc[b, h, at])


@pytest.mark.parametrize("T,budget,W,A", [(4000, 1500, 30, 4), (8000, 7000, 100, 1), (16384, 1000, 0, 0), (60000, 9000, 64, 4),
                                          (131072, 30000, 512, 4), (140000, 9000, 64, 4), (150000, 149000, 64, 4)])
@pytest.mark.parametrize("steps", [None, 7])
def test_evict_selects_over_several_ctas(cuda_device, T, budget, W, A, steps):
    """Rows that several CTAs share, with slots behind all their registers (140000, 150000):
    distinct weights, or seven values whose ties begin and end anywhere."""
    g = torch.Generator().manual_seed(T + 1)
    acc = torch.rand(1, 2, T, generator=g)
    if steps is not None:
        acc = torch.floor(acc * steps)
    acc = acc.to(cuda_device)
    K = torch.randn(1, 2, T, 64, generator=g).to(BF).to(cuda_device)
    p = params(1, 2, 2, 64, W, BF)
    n = torch.tensor([T - 3], dtype=torch.int32, device=cuda_device)
    Ko, Vo = (torch.zeros(1, 2, budget, 64, dtype=BF, device=cuda_device) for _ in range(2))
    ao = torch.zeros(1, 2, budget, device=cuda_device)
    idx = torch.full((1, 2, budget), -7, dtype=torch.int32, device=cuda_device)
    out = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_CACHE_EVICT, T, budget, device=cuda_device)
    hils.hils_cache_evict(p, A, budget, K, K, acc, n, Ko, Vo, ao, idx, out, workspace=ws)
    rows, new = ref.evict(acc, torch.tensor([T - 3]), budget, W, A)
    assert out.tolist() == new
    for h in range(2):
        at = torch.tensor(rows[0][h], dtype=torch.long, device=cuda_device)
        assert len(rows[0][h]) == budget and torch.equal(idx[0, h].long(), at)
        assert torch.equal(Ko[0, h], K[0, h, at]) and torch.equal(Vo[0, h], K[0, h, at]) and torch.equal(ao[0, h], acc[0, h, at])


def test_prompt_then_evict_then_decode(cuda_device):
    """The calls as a server makes them: a prompt in two pieces, its weights, the cache cut,
    then tokens decoded on the cut cache with their weights added, and a second cut."""
    B, H, Hk, d, N, W, A, budget = 2, 8, 2, 128, 700, 1000, 4, 256
    Q, K, V = make(B, H, Hk, N, N, d, BF, 61, cuda_device)
    p = params(B, H, Hk, d, W, BF)
    cut = 450
    O1, l1 = prefill(p, A, Q[:, :, :cut], K[:, :, :cut], V[:, :, :cut])
    O2, l2 = prefill(p, A, Q[:, :, cut:], K, V)
    check_prefill(p, A, Q, K, V, torch.cat([O1, O2], 2), torch.cat([l1, l2], 2))
    T = 800
    acc = torch.zeros(B, Hk, T, device=cuda_device)
    _weights(p, A, Q[:, :, :cut], K[:, :, :cut], l1, acc)
    _weights(p, A, Q[:, :, cut:], K, l2, acc)
    total = acc.sum((1, 2)).cpu()
    assert torch.allclose(total, torch.full((B,), float(H * N)), rtol=1e-4)  # every query's weights sum to one
    Kc, Vc = (torch.zeros(B, Hk, T, d, dtype=BF, device=cuda_device) for _ in range(2))
    Kc[:, :, :N], Vc[:, :, :N] = K, V
    n = torch.full((B,), N, dtype=torch.int32, device=cuda_device)
    pe = params(B, H, Hk, d, 32, BF)
    Ko, Vo = (torch.zeros(B, Hk, T, d, dtype=BF, device=cuda_device) for _ in range(2))
    ao = torch.zeros(B, Hk, budget, device=cuda_device)
    idx = torch.empty(B, Hk, budget, dtype=torch.int32, device=cuda_device)

    def evict(k, v, a, lens, ko, vo):
        ws = hils.alloc_workspace(pe, hils.HILS_CALL_CACHE_EVICT, T, budget, device=cuda_device)
        hils.hils_cache_evict(pe, A, budget, k, v, a, lens, ko[:, :, :budget], vo[:, :, :budget], ao, idx, lens, workspace=ws)

    before = acc.clone()
    evict(Kc, Vc, acc, n, Ko, Vo)
    rows, _ = ref.evict(before, torch.tensor([N] * B), budget, 32, A)
    assert idx.tolist() == rows
    acc2 = torch.zeros(B, Hk, T, device=cuda_device)
    acc2[:, :, :budget] = ao
    g = torch.Generator().manual_seed(9)
    for step in range(3):  # append a token, decode it over the whole cut cache
        at = budget + step
        Ko[:, :, at] = torch.randn(B, Hk, d, generator=g).to(BF).to(cuda_device)
        Vo[:, :, at] = torch.randn(B, Hk, d, generator=g).to(BF).to(cuda_device)
        n += 1
        q = torch.randn(B, H, 1, d, generator=g).to(BF).to(cuda_device)
        was = acc2.clone()
        o, l = _decode(p, A, q, Ko, Vo, n, acc2)
        _check_decode(p, A, q, Ko, Vo, n, o, l, f"token {step}")
        assert torch.allclose((acc2 - was).sum((1, 2)).cpu(), torch.full((B,), float(H)), rtol=1e-4)
    was = acc2.clone()
    evict(Ko, Vo, acc2, n, Kc, Vc)
    rows, new = ref.evict(was, torch.tensor([budget + 3] * B), budget, 32, A)
    assert idx.tolist() == rows and n.tolist() == new == [budget] * B
