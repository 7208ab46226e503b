"""Inputs and error bounds shared by the tests of the window-and-sink calls."""
from __future__ import annotations

import math

import torch

import hierarchical_chunk_sparse_b200 as hils
from oracle import sink as ref

# Rounding units: a value rounded once to the type is off by at most this, relative to it.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -23  # one float32 step: sums on tensor cores may truncate


def make(B, H, Hk, Lq, N, d, dtype, seed, device):
    g = torch.Generator().manual_seed(seed)
    lean = torch.nn.functional.normalize(torch.randn(d, generator=g), dim=0)
    Q = torch.randn(B, H, Lq, d, generator=g) + 2.0 * lean
    K = torch.randn(B, Hk, N, d, generator=g)
    K[:, :, :3] += 0.5 * math.sqrt(d) * lean
    V = torch.randn(B, Hk, N, d, generator=g) + 0.3 * torch.randn(B, Hk, 1, d, generator=g)
    return tuple(x.to(dtype).to(device) for x in (Q, K, V))


def within(got, want, tol, what):
    """Elementwise |got - want| <= tol where want is finite; the same infinities elsewhere."""
    got = got.detach().to("cpu").double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: the finite places differ"
    assert torch.equal(got[~fin], want[~fin]), f"{what}: the infinities differ"
    over = ((got - want).abs() - tol.expand_as(want))[fin]
    if over.numel():
        assert over.max() <= 0, f"{what}: off by up to {(got - want).abs()[fin].max():.3e}, {over.max():.3e} over its bound"


def forward_bounds(O, Om, lse, L, d, n, dtype):
    """Bounds of O and lse. A logit's float32 error is at most (d + 4) steps of its sum of
    magnitudes L (plus its scaling); a probability is off by twice that (its own logit and
    its share of the sum), and by the sums over n keys. bf16: each probability is rounded
    as an operand (HALF relative), then the output."""
    e = 2 * (d + 4) * U32 * L + (n + 32) * U32
    u = HALF[dtype]
    p = u if dtype == torch.bfloat16 else 0.0
    tol_o = u * O.abs() + (e + p * (1 + e))[..., None] * Om * (1 + u) if torch.is_tensor(e) else None
    return tol_o, e + 4 * U32 * (1 + lse.abs().nan_to_num(posinf=0.0, neginf=0.0))


def weight_bound(value, L_max, lse_max, d, n):
    """p = exp2(x - l) from a given lse: the logit's error, the rounding of x and l in log2
    units, the exponential's, and a float32 sum of n terms."""
    return value * ((d + 4) * U32 * L_max + 4 * U32 * (L_max + lse_max + 2) + (n + 8) * U32) + 1e-30


def grad_bounds(val, mag, es, L_max, lse_max, d, n, dtype):
    """val, mag, es as oracle.sink.backward's: the operands' rounding (bf16: HALF of each
    |term|), the result's own, the probability's error in every term, the float32 error of
    dO . v - D (es), and sums of n terms."""
    u = HALF[dtype]
    p = u if dtype == torch.bfloat16 else 0.0
    e = (d + 4) * U32 * L_max + 4 * U32 * (L_max + lse_max + 2) + (n + 8) * U32
    return [u * v.abs() + (1 + u) * ((p + e) * m + (2 * d + 16) * U32 * (1 + p) * s) + 1e-30 for v, m, s in zip(val, mag, es)]


def params(B, H, Hk, d, W, dtype, **kw):
    return hils.Params(B=B, H=H, d=d, K=0, W=W, dtype=dtype, H_kv=Hk, **kw)


def status_of(ws):
    return int(ws[:4].view(torch.int32).item())


def prefill(p, A, Q, K, V, lse=True):
    O = torch.full_like(Q, 7.0)
    L = torch.full(Q.shape[:3], 7.0, dtype=torch.float32, device=Q.device) if lse else None
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_PREFILL, Q.shape[2], A, device=Q.device)
    hils.hils_sink_prefill(p, A, Q, K, V, O, L, workspace=ws)
    torch.cuda.synchronize()
    assert status_of(ws) == 0
    return O, L


def check_prefill(p, A, Q, K, V, O, lse, what=""):
    d, N = Q.shape[3], K.shape[2]
    see = ref.visible(Q.shape[2], N, p.W, A)
    rO, rl, _, Om, L = ref.attend(Q, K, V, see, p.scale or 1 / math.sqrt(d))
    tO, tl = forward_bounds(rO, Om, rl, L, d, min(N, p.W + A), p.dtype)
    within(O, rO, tO, f"{what} O")
    if lse is not None:
        within(lse, rl, tl, f"{what} lse")
