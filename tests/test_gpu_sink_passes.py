"""Paths of the window-and-sink and shared-prefix calls that only some sizes take: the shared
prefix's own pass in bf16, weights whose steps pack several heads, random sizes of the
backward and the weights."""
import math

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
import test_gpu_sink as by_call
from sink_testutil import make, params, status_of
from test_gpu_sink_rises import attend64, check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Prefix:
    """One decode over a shared prefix that has its own pass."""

    def __init__(self, dev, seed, B, H, Hk, d, P, T):
        self.Q, self.Kp, self.Vp = make(1, H, Hk, B, P, d, BF, seed, dev)
        self.Q = self.Q.transpose(0, 2).contiguous()  # [B, H, 1, d]
        _, self.Kc, self.Vc = make(B, H, Hk, 1, T, d, BF, seed + 1, dev)
        lens = [(7 * b + 5 * seed) % (T + 1) for b in range(B)]
        for b, m in enumerate(lens):  # behind a sequence's last slot there is anything
            self.Kc[b, :, m:], self.Vc[b, :, m:] = math.nan, math.inf
        self.n = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.p = params(B, H, Hk, d, 0, BF)
        self.ws = hils.alloc_workspace(self.p, hils.HILS_CALL_PREFIX_DECODE, T, P, device=dev)
        self.O, self.lse = torch.full_like(self.Q, 7.0), torch.full((B, H), 7.0, device=dev)

    def run(self, ws=None, stream=None):
        hils.hils_prefix_decode(self.p, self.Q, self.Kp, self.Vp, self.Kc, self.Vc, self.n, self.O, self.lse,
                                workspace=self.ws if ws is None else ws, stream=stream)

    def clear(self):
        self.O.fill_(5)
        self.lse.fill_(5)

    def same(self, want):
        return torch.equal(self.O, want[0]) and torch.equal(self.lse, want[1])

    def check(self):
        B, Hk, T, d = self.Kc.shape
        G, P = self.Q.shape[1] // Hk, self.Kp.shape[2]
        for b in range(B):
            for hk in range(Hk):
                h, m = slice(hk * G, hk * G + G), int(self.n[b])
                k, v = torch.cat([self.Kp[0, hk], self.Kc[b, hk, :m]]), torch.cat([self.Vp[0, hk], self.Vc[b, hk, :m]])
                see = torch.ones(1, P + m, dtype=torch.bool, device=k.device)
                check(self.O[b, h], self.lse[b, h, None], *attend64(self.Q[b, h], k, v, see), d, P + T, f"sequence {b} head {hk}")


# B, H, Hk, d, P, T
DIRECT = [(90, 14, 2, 128, 1091, 17)]  # just short of a pass of its own
PASSES = [
    (3, 24, 8, 128, 8450, 30),     # groups of three; 33 key ranges, the last without a second one; two keys in the last tile
    (3, 8, 8, 128, 9000, 100),     # one head a group
    (300, 16, 4, 64, 1500, 20),    # ten row tiles of a head, the last one partly filled
    (300, 16, 4, 64, 400, 5),      # the same over one key range
    (320, 64, 8, 128, 700, 10),    # more items than SMs
    (90, 14, 2, 128, 1191, 17),    # groups of seven: rows that no head fills
]


@pytest.mark.parametrize("B,H,Hk,d,P,T", PASSES + DIRECT)
def test_prefix_in_its_own_pass(cuda_device, B, H, Hk, d, P, T):
    c = Prefix(cuda_device, 1, B, H, Hk, d, P, T)
    # only the prefix's own pass has waits that can run out: the status tells that it is the one chosen
    c.p.flags = hils.HILS_FLAG_DIAG_EXPIRE_WAITS
    c.run()
    torch.cuda.synchronize()
    own = (B, H, Hk, d, P, T) in PASSES
    assert status_of(c.ws) == own, f"{'each sequence reads' if own else 'a pass of its own over'} this prefix"
    c.p.flags = 0
    hils.hils_workspace_init(c.ws)
    c.clear()
    c.run()
    torch.cuda.synchronize()
    assert status_of(c.ws) == 0
    c.check()


def test_prefix_on_streams_and_in_graphs(cuda_device):
    """Two at once on streams of their own; two captured graphs over one workspace, in turn."""
    a, b = (Prefix(cuda_device, s, 4, 32, 8, 128, 9001, 300) for s in (1, 9))
    a.run()
    b.run()
    torch.cuda.synchronize()
    a.check()
    want = [(c.O.clone(), c.lse.clone()) for c in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.clear()
    b.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    assert a.same(want[0]) and b.same(want[1])
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s1):
            c.run(ws=a.ws)
        graphs.append(g)
    a.clear()
    b.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert a.same(want[0]) and b.same(want[1]) and status_of(a.ws) == 0


# B, H, Hk, d, Lq, N, W, A: with few queries a step of the bf16 kernel holds 2, 4 or 8 heads of the group
PACKED = [
    (2, 8, 1, 128, 1, 300, 90, 3), (1, 8, 1, 64, 13, 700, 300, 0), (2, 8, 2, 128, 30, 513, 100, 5), (1, 16, 2, 128, 16, 1025, 2000, 0),
    (1, 8, 1, 128, 20, 2000, 300, 150), (3, 12, 3, 64, 32, 999, 40, 1), (1, 6, 1, 128, 64, 800, 800, 0), (1, 8, 1, 128, 17, 2600, 70, 0),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,d,Lq,N,W,A", PACKED)
def test_weights_of_few_queries(cuda_device, B, H, Hk, d, Lq, N, W, A, dtype):
    by_call.test_weights(cuda_device, B, H, Hk, d, Lq, N, W, A, dtype)


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_random_weights_and_gradients(cuda_device, dtype, seed):
    g = torch.Generator().manual_seed(4000 + seed)

    def pick(lo, hi):
        return int(math.exp(torch.rand((), generator=g).item() * math.log(hi / lo)) * lo)

    G, Hk, B, d = pick(1, 8.99), pick(1, 4.99), pick(1, 3.99), 64 * pick(1, 2.99)
    N, W, A = pick(1, 900), pick(1, 1000) - 1, pick(1, 200) - 1
    Lq = pick(1, N + 0.99)
    by_call.test_weights(cuda_device, B, Hk * G, Hk, d, Lq, N, W, A, dtype)
    by_call.test_backward(cuda_device, B, Hk * G, Hk, d, N, W, A, dtype)
