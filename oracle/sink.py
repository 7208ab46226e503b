"""Float64 evaluation of the window-and-sink attention, its gradients and accumulated
weights, the shared-prefix decode and the cache eviction (plain torch on the CPU, dense
scores: for small problems).

A query at position t sees V(t) = {j <= t : j < A or j > t - W}; o_t = softmax over V(t) of
scale q_t . k_j times v_j; an empty V(t) gives o = 0, lse = -inf. Beside each result stand
the magnitudes that its rounding error is bounded with (sums of absolute values)."""
from __future__ import annotations

import math

import torch

INF = math.inf


def f64(t):
    return None if t is None else t.detach().to("cpu").double()


def visible(Lq: int, N: int, W: int, A: int) -> torch.Tensor:
    """[Lq, N]: which tokens the Lq newest queries see."""
    t = torch.arange(N - Lq, N)[:, None]
    j = torch.arange(N)[None]
    return (j <= t) & ((j < A) | (j > t - W))


def _group(x, G):
    return x.repeat_interleave(G, 1)


def attend(Q, K, V, see, scale):
    """Q [B,H,Lq,d], K, V [B,Hk,N,d], see broadcastable to [B,H,Lq,N]: O, lse, the
    probabilities p, Om = sum p |v|, and L = the largest scale sum |q_x k_x| of a row."""
    Q, K, V = f64(Q), f64(K), f64(V)
    G = Q.shape[1] // max(1, K.shape[1])
    K, V = _group(K, G), _group(V, G)
    see = see.expand(Q.shape[:3] + (K.shape[2],))
    zero = torch.zeros((), dtype=torch.float64)
    s = torch.where(see, Q @ torch.where(torch.isfinite(K), K, zero).transpose(2, 3) * scale, torch.full((), -INF, dtype=torch.float64))
    m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full(s.shape[:3] + (1,), -INF, dtype=torch.float64)
    e = torch.exp(s - torch.where(m == -INF, zero, m))
    z = e.sum(-1, keepdim=True)
    p = e / torch.where(z > 0, z, zero + 1)
    lse = (torch.log(z) + torch.where(m == -INF, zero, m))[..., 0]
    Vf = torch.where(torch.isfinite(V), V, zero)
    L = torch.where(see, Q.abs() @ torch.where(torch.isfinite(K), K, zero).abs().transpose(2, 3) * abs(scale), zero)
    L = L.amax(-1) if L.shape[-1] else torch.zeros(L.shape[:3], dtype=torch.float64)
    return p @ Vf, lse, p, p @ Vf.abs(), L


def backward(Q, K, V, O, lse, dO, see, scale):
    """dQ, dK, dV from the given O and lse, and their magnitudes: sums of |terms|, and the
    sums with |ds| replaced by scale p (|dO| . |v| + |dO| . |o|)."""
    Q, K, V, O, lse, dO = (f64(x) for x in (Q, K, V, O, lse, dO))
    B, Hk = K.shape[:2]
    G = Q.shape[1] // Hk
    Kg, Vg = _group(K, G), _group(V, G)
    see = see.expand(Q.shape[:3] + (K.shape[2],))
    zero = torch.zeros((), dtype=torch.float64)
    s = Q @ Kg.transpose(2, 3) * scale
    p = torch.where(see & torch.isfinite(lse)[..., None], torch.exp(s - lse[..., None]), zero)
    ds = scale * p * (dO @ Vg.transpose(2, 3) - (dO * O).sum(-1, keepdim=True))
    es = abs(scale) * p * (dO.abs() @ Vg.abs().transpose(2, 3) + (dO * O).abs().sum(-1, keepdim=True))

    def heads(x):
        return x.view(B, Hk, G, *x.shape[2:]).sum(2)

    def all_of(d_s, p_, q, k, do):
        return d_s @ k, heads(d_s.transpose(2, 3) @ q), heads(p_.transpose(2, 3) @ do)

    return all_of(ds, p, Q, Kg, dO), all_of(ds.abs(), p, Q.abs(), Kg.abs(), dO.abs()), \
        all_of(es, p, Q.abs(), Kg.abs(), dO.abs())


def weights(Q, K, lse, see, scale):
    """[B, Hk, N]: each token's weight, summed over the queries and the group's heads."""
    Q, K, lse = f64(Q), f64(K), f64(lse)
    B, Hk = K.shape[:2]
    G = Q.shape[1] // Hk
    s = Q @ _group(K, G).transpose(2, 3) * scale
    see = see.expand(s.shape)
    p = torch.where(see & torch.isfinite(lse)[..., None], torch.exp(s - lse[..., None]), torch.zeros((), dtype=torch.float64))
    return p.sum(2).view(B, Hk, G, -1).sum(2)


def decode_visible(cache_len, T: int, W: int, A: int) -> torch.Tensor:
    """[B, 1, 1, T]: the slots that each sequence's newest token sees."""
    n = cache_len.detach().to("cpu").long().clamp(0, T)[:, None]
    j = torch.arange(T)[None]
    return ((j < n) & ((j < A) | (j >= n - W)))[:, None, None]


def prefix(Q, Kp, Vp, Kc, Vc, cache_len, scale):
    """One query per sequence over the shared prefix and its own cache: as attend()."""
    B, P, T = Q.shape[0], Kp.shape[2], Kc.shape[2]
    see = torch.cat([torch.ones(B, 1, 1, P, dtype=torch.bool), decode_visible(cache_len, T, T, 0)], 3)
    K = torch.cat([f64(Kp).expand(B, -1, -1, -1), f64(Kc)], 2)
    V = torch.cat([f64(Vp).expand(B, -1, -1, -1), f64(Vc)], 2)
    return attend(Q, K, V, see, scale)


def evict(acc, cache_len, budget: int, W: int, A: int):
    """Kept slots per (b, head) in slot order (lists), and the new lengths."""
    acc = acc.detach().to("cpu")
    B, Hk, T = acc.shape
    out, lens = [], []
    for b in range(B):
        n = min(max(int(cache_len[b]), 0), T)
        lens.append(min(n, budget))
        rows = []
        for h in range(Hk):
            if n <= budget:
                rows.append(list(range(n)))
                continue
            a = [-INF if x != x else x for x in acc[b, h].tolist()]
            # NaN below every number, -inf included
            nan = [x != x for x in acc[b, h].tolist()]
            mid = sorted(range(A, n - W), key=lambda t: (nan[t], -a[t], t))[:budget - A - W]
            rows.append(sorted(list(range(A)) + mid + list(range(n - W, n))))
        out.append(rows)
    return out, lens
