"""Prefill and shared prefix in bf16 where a row's largest score comes late in its keys, so
that the running softmax has to rescale what it has summed: at a prompt's size by chance,
with logits that grow along the keys, and for single rows. Checked in float64 on the GPU."""
import math

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from sink_testutil import forward_bounds, params, status_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LN2 = math.log(2.0)


def attend64(Q, K, V, see):
    """Q [h, r, d] over K, V [t, d] with see [r, t]: O, lse, sum p |v| and the rows' largest
    sum |q_x k_x| of a logit."""
    scale = 1 / math.sqrt(Q.shape[-1])
    Q, K, V = Q.double(), K.double(), V.double()
    s = (Q @ K.T * scale).masked_fill(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    p = e / torch.where(z > 0, z, torch.ones_like(z))
    L = (Q.abs() @ K.abs().T * scale).masked_fill(~see, 0.0).amax(-1)
    return p @ V, (m + torch.log(z))[..., 0], p @ V.abs(), L


def check(got, lse, O, l, Om, L, d, n, what):
    tO, tl = forward_bounds(O, Om, l, L, d, n, BF)
    over = (got.double() - O).abs() - tO
    assert bool((over <= 0).all()), f"{what}: O off by up to {(got.double() - O).abs().max():.3e} in {int((over > 0).any(-1).sum())} rows"
    assert bool(((lse.double() - l).abs() <= tl).all()), f"{what}: lse"


def check_rows(Q, K, V, O, lse, W, A, what):
    """All rows of a prefill, 512 queries at a time over the keys that they see."""
    B, H, N, d = Q.shape
    G = H // K.shape[1]
    for b in range(B):
        for hk in range(K.shape[1]):
            h = slice(hk * G, hk * G + G)
            for i in range(0, N, 512):
                e = min(N, i + 512)
                t = torch.arange(i, e, device=Q.device)[:, None]
                lo = max(0, i - W + 1)
                j = torch.cat([torch.arange(min(A, lo), device=Q.device), torch.arange(lo, e, device=Q.device)])
                see = (j <= t) & ((j < A) | (j > t - W))
                want = attend64(Q[b, h, i:e], K[b, hk, j], V[b, hk, j], see)
                check(O[b, h, i:e], lse[b, h, i:e], *want, d, min(N, W + A), f"{what} b {b} heads {hk * G}.. rows {i}..")


def run_prefill(Q, K, V, W, A, times=4):
    """The call over and over, each time after other data has filled L2: equal bits."""
    B, H, N, d = Q.shape
    p = params(B, H, K.shape[1], d, W, BF)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_PREFILL, N, A, device=Q.device)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=Q.device)
    first = None
    for k in range(times):
        O, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:3], 7.0, device=Q.device)
        flush.fill_(k)
        hils.hils_sink_prefill(p, A, Q, K, V, O, lse, workspace=ws)
        first = first or (O, lse)
        assert torch.equal(O, first[0]) and torch.equal(lse, first[1]), f"call {k} gives other bits than the first"
    assert status_of(ws) == 0
    return first


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def growing(g, heads, tokens, d, per_tile, u, period=None):
    """Keys along u whose logits with 12 u grow by per_tile (log2 units) each 64 keys, over and
    over if there is a period (in tiles)."""
    j = torch.arange(tokens, device="cuda") / 64.0
    if period is not None:
        j = j % period
    return (j * per_tile * LN2 * math.sqrt(d) / 12.0)[:, None] * u + 0.3 * normal(g, 1, heads, tokens, d)


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("W,A,Hk,d", [(512, 4, 32, 128), (512, 0, 32, 128), (512, 0, 8, 64), (300, 2, 8, 128)])
def test_a_prompt_of_8192(cuda_device, W, A, Hk, d, seed):
    """The sizes of the benchmark's prompt, with and without sinks: a row whose first key tile
    holds only one or two of its keys starts low and rises when it comes to the others."""
    H, N = 32, 8192
    g = torch.Generator(device="cuda").manual_seed(100 * seed + W + A + Hk)
    lean = torch.nn.functional.normalize(normal(g, d), dim=0)
    Q = (normal(g, 1, H, N, d) + 3.0 * lean).to(BF)
    K = normal(g, 1, Hk, N, d)
    K[:, :, :4] += 0.6 * math.sqrt(d) * lean
    K, V = K.to(BF), (normal(g, 1, Hk, N, d) + 0.25 * normal(g, 1, Hk, 1, d)).to(BF)
    O, lse = run_prefill(Q, K, V, W, A)
    check_rows(Q, K, V, O, lse, W, A, "8K")


@pytest.mark.parametrize("seed", range(2))
@pytest.mark.parametrize("per_tile", [3, 6, 12])
@pytest.mark.parametrize("W,A,H,Hk,d", [(512, 0, 8, 8, 128), (512, 4, 8, 2, 128), (1500, 0, 4, 4, 64), (700, 70, 6, 2, 128)])
def test_logits_that_grow_along_the_keys(cuda_device, W, A, H, Hk, d, per_tile, seed):
    B, N = 2, 1500
    g = torch.Generator(device="cuda").manual_seed(seed + 10 * per_tile + W)
    u = torch.nn.functional.normalize(normal(g, d), dim=0)
    Q = (12.0 * u + 0.3 * normal(g, B, H, N, d)).to(BF)
    K = torch.cat([growing(g, Hk, N, d, per_tile, u) for _ in range(B)]).to(BF)
    V = normal(g, B, Hk, N, d).to(BF)
    O, lse = run_prefill(Q, K, V, W, A)
    check_rows(Q, K, V, O, lse, W, A, f"{per_tile} a tile")


@pytest.mark.parametrize("d", [64, 128])
def test_single_rows_that_rise(cuda_device, d):
    """Among rows that never rise, one row of each 256 whose largest score is in the fourth, the
    fifth or the last of the item's key tiles."""
    H, N, W, A = 8, 8192, 512, 0
    g = torch.Generator(device="cuda").manual_seed(d)
    Q, K = 0.2 * normal(g, 1, H, N, d), normal(g, 1, H, N, d)
    for item in range(2, N // 256):
        lo = item * 256 - W + 1  # the item's first key
        for h in range(H):
            t = item * 256 + (37 * item + 91 * h) % 256
            j = (lo + 64 * 3 + 9, lo + 64 * 4 + 30, t - 1)[(item + h) % 3]
            if not t - W < j <= t:
                j = t
            Q[0, h, t] = K[0, h, j] * (20 * LN2 * math.sqrt(d) / float(K[0, h, j].square().sum()))
    Q, K, V = Q.to(BF), K.to(BF), normal(g, 1, H, N, d).to(BF)
    O, lse = run_prefill(Q, K, V, W, A)
    check_rows(Q, K, V, O, lse, W, A, "single rows")


@pytest.mark.parametrize("per_tile", [0, 3, 6, 12])
@pytest.mark.parametrize("B,H,Hk,d,P", [(70, 32, 8, 128, 9000), (3, 24, 8, 128, 20000), (40, 24, 8, 64, 20011)])
def test_a_shared_prefix_that_rises(cuda_device, B, H, Hk, d, P, per_tile):
    """Logits that grow again and again along a prefix that has its own pass."""
    T, G = 40, H // Hk
    g = torch.Generator(device="cuda").manual_seed(P + per_tile)
    u = torch.nn.functional.normalize(normal(g, d), dim=0)
    Q = (12.0 * u + 0.3 * normal(g, B, H, 1, d)).to(BF)
    Kp, Vp = growing(g, Hk, P, d, per_tile, u, period=11).to(BF), normal(g, 1, Hk, P, d).to(BF)
    Kc, Vc = normal(g, B, Hk, T, d).to(BF), normal(g, B, Hk, T, d).to(BF)
    n = torch.arange(B, dtype=torch.int32, device=cuda_device) % (T + 1)
    p = params(B, H, Hk, d, 0, BF)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_PREFIX_DECODE, T, P, device=cuda_device)
    # only the prefix's own pass has waits that can expire: it is the one that is chosen
    O, lse = torch.full_like(Q, 7.0), torch.full((B, H), 7.0, device=cuda_device)
    p.flags = hils.HILS_FLAG_DIAG_EXPIRE_WAITS
    hils.hils_prefix_decode(p, Q, Kp, Vp, Kc, Vc, n, O, lse, workspace=ws)
    assert status_of(ws) == 1, "each sequence reads this prefix by itself"
    p.flags = 0
    hils.hils_workspace_init(ws)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    first = None
    for k in range(4):
        O, lse = torch.full_like(Q, 7.0), torch.full((B, H), 7.0, device=cuda_device)
        flush.fill_(k)
        hils.hils_prefix_decode(p, Q, Kp, Vp, Kc, Vc, n, O, lse, workspace=ws)
        first = first or (O, lse)
        assert torch.equal(O, first[0]) and torch.equal(lse, first[1]), f"call {k} gives other bits than the first"
    assert status_of(ws) == 0
    for b in range(B):
        for hk in range(Hk):
            h, m = slice(hk * G, hk * G + G), int(n[b])
            k, v = torch.cat([Kp[0, hk], Kc[b, hk, :m]]), torch.cat([Vp[0, hk], Vc[b, hk, :m]])
            want = attend64(Q[b, h], k, v, torch.ones(1, P + m, dtype=torch.bool, device=cuda_device))
            check(O[b, h], lse[b, h, None], *want, d, P + T, f"{per_tile} a tile, sequence {b}")
