"""The float64 evaluation of the window-and-sink calls against loops written from the
definition, and its gradients against differences."""
import math
import random

import pytest
import torch

from oracle import sink as ref


def _seen(t, W, A):
    return [j for j in range(t + 1) if j < A or j > t - W]


@pytest.mark.parametrize("Lq,N,W,A", [(1, 1, 1, 0), (1, 1, 0, 0), (4, 9, 3, 2), (9, 9, 20, 0), (7, 7, 0, 3), (3, 12, 1, 1), (5, 5, 2, 9)])
@pytest.mark.parametrize("G", [1, 3])
def test_attend_by_loops(Lq, N, W, A, G):
    g = torch.Generator().manual_seed(N + 10 * G)
    B, Hk, d, scale = 2, 2, 8, 0.3
    Q = torch.randn(B, Hk * G, Lq, d, generator=g).double()
    K, V = (torch.randn(B, Hk, N, d, generator=g).double() for _ in range(2))
    see = ref.visible(Lq, N, W, A)
    O, lse, p, _, _ = ref.attend(Q, K, V, see, scale)
    for b in range(B):
        for h in range(Hk * G):
            for i in range(Lq):
                js = _seen(N - Lq + i, W, A)
                assert see[i].nonzero()[:, 0].tolist() == js
                e = [math.exp(scale * float(Q[b, h, i] @ K[b, h // G, j])) for j in js]
                if not js:
                    assert lse[b, h, i] == -math.inf and (O[b, h, i] == 0).all()
                    continue
                assert abs(lse[b, h, i] - math.log(sum(e))) < 1e-12
                want = sum(x / sum(e) * V[b, h // G, j] for x, j in zip(e, js))
                assert (O[b, h, i] - want).abs().max() < 1e-12
                assert abs(p[b, h, i].sum() - 1) < 1e-12


def test_gradients_by_differences():
    g = torch.Generator().manual_seed(3)
    B, Hk, G, N, d, W, A, scale = 1, 2, 2, 11, 8, 4, 2, 0.4
    x = [torch.randn(B, Hk * G, N, d, generator=g).double()] + [torch.randn(B, Hk, N, d, generator=g).double() for _ in range(2)]
    dO = torch.randn(x[0].shape, generator=g).double()
    see = ref.visible(N, N, W, A)
    O, lse, _, _, _ = ref.attend(*x, see, scale)
    val, mag, es = ref.backward(*x, O, lse, dO, see, scale)
    for k in range(3):
        u = torch.randn(x[k].shape, generator=g).double()
        hi, lo = ([t + s * 1e-5 * u if i == k else t for i, t in enumerate(x)] for s in (1, -1))
        num = (((ref.attend(*hi, see, scale)[0] - ref.attend(*lo, see, scale)[0]) * dO).sum()) / 2e-5
        assert abs(num - (val[k] * u).sum()) < 1e-8 * (val[k] * u).abs().sum() + 1e-8  # h^2 = 1e-10 and 1e-16 / h
        assert (mag[k] >= val[k].abs() - 1e-12).all() and (es[k] >= 0).all()


def test_weights_and_decode_sets():
    g = torch.Generator().manual_seed(4)
    B, Hk, G, Lq, N, d, W, A, scale = 2, 2, 2, 5, 13, 8, 4, 1, 0.5
    Q = torch.randn(B, Hk * G, Lq, d, generator=g)
    K, V = (torch.randn(B, Hk, N, d, generator=g) for _ in range(2))
    see = ref.visible(Lq, N, W, A)
    _, lse, p, _, _ = ref.attend(Q, K, V, see, scale)
    w = ref.weights(Q, K, lse, see, scale)
    assert (w - p.view(B, Hk, G, Lq, N).sum((2, 3))).abs().max() < 1e-12
    assert abs(w.sum() - B * Hk * G * Lq) < 1e-10
    for n in (0, 1, 5, 13, 20, -2):
        got = ref.decode_visible(torch.tensor([n]), 13, W, A)[0, 0, 0].nonzero()[:, 0].tolist()
        m = min(max(n, 0), 13)
        assert got == ([] if m == 0 else _seen(m - 1, W, A))


def test_evict_by_sorting():
    rng = random.Random(5)
    for _ in range(60):
        T = rng.randint(1, 30)
        n, budget = rng.randint(0, T), rng.randint(0, T)
        A = rng.randint(0, budget)
        W = rng.randint(0, budget - A)
        acc = torch.tensor([[[rng.choice([0.0, -0.0, 1.0, 2.5, math.nan, math.inf, -math.inf]) for _ in range(T)]]])
        rows, lens = ref.evict(acc, torch.tensor([n]), budget, W, A)
        kept = rows[0][0]
        assert lens == [min(n, budget)] and len(kept) == lens[0] and kept == sorted(set(kept)) and all(0 <= j < n for j in kept)
        if n > budget:
            assert set(range(A)) | set(range(n - W, n)) <= set(kept)
            val = [-2.0 if x != x else (-1.0 if x == -math.inf else x) for x in acc[0, 0].tolist()]
            out = [j for j in range(A, n - W) if j not in kept]
            mid = [j for j in kept if A <= j < n - W]
            assert all((val[i], -i) > (val[j], -j) for i in mid for j in out)
