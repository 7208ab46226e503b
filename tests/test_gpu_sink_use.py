"""The window-and-sink, shared-prefix and eviction calls as programs make them: on other
streams, captured and replayed, two at once, over workspaces used again, with views of other
layouts, far offsets, enough rows for several rounds of every CTA, and waits that run out."""
import math

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from oracle import sink as ref
from sink_testutil import check_prefill, forward_bounds, grad_bounds, make, params, prefill, status_of, weight_bound, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Calls:
    """One of each call on its own data, with workspaces that it keeps."""

    def __init__(self, dev, dtype, seed, B=2, H=4, Hk=2, d=64, N=300, W=70, A=3, P=700, budget=90):
        self.Q, self.K, self.V = make(B, H, Hk, N, N, d, dtype, seed, dev)
        self.p, self.A, self.budget = params(B, H, Hk, d, W, dtype), A, budget
        g = torch.Generator().manual_seed(seed + 1)
        self.dO = torch.randn(self.Q.shape, generator=g).to(dtype).to(dev)
        self.n = torch.tensor([N, N // 3], dtype=torch.int32, device=dev)[:B]
        _, kp, vp = make(1, H, Hk, 1, P, d, dtype, seed + 2, dev)
        self.Kp, self.Vp = kp, vp
        f = dict(dtype=F32, device=dev)
        self.O, self.lse = torch.empty_like(self.Q), torch.empty(B, H, N, **f)
        self.grads = [torch.empty_like(x) for x in (self.Q, self.K, self.V)]
        self.acc = torch.rand(B, Hk, N, generator=g).to(dev)
        self.w_out, self.d_out = torch.zeros_like(self.acc), torch.zeros_like(self.acc)
        self.q1 = self.Q[:, :, -1:].contiguous()
        self.o1, self.l1 = torch.empty_like(self.q1), torch.empty(B, H, **f)
        self.o2, self.l2 = torch.empty_like(self.q1), torch.empty(B, H, **f)
        self.Ko, self.Vo = (torch.zeros(B, Hk, budget, d, dtype=dtype, device=dev) for _ in range(2))
        self.ao = torch.zeros(B, Hk, budget, **f)
        self.idx = torch.empty(B, Hk, budget, dtype=torch.int32, device=dev)
        self.no = torch.empty(B, dtype=torch.int32, device=dev)
        ws = lambda c, r, o: hils.alloc_workspace(self.p, c, r, o, device=dev)
        self.ws = [ws(hils.HILS_CALL_SINK_PREFILL, N, A), ws(hils.HILS_CALL_SINK_BACKWARD, N, A), ws(hils.HILS_CALL_SINK_WEIGHTS, N, A),
                   ws(hils.HILS_CALL_SINK_DECODE_ACC, N, A), ws(hils.HILS_CALL_PREFIX_DECODE, N, P),
                   ws(hils.HILS_CALL_CACHE_EVICT, N, budget)]

    def run(self, ws=None, stream=None):
        w = ws or self.ws
        p, A, k = self.p, self.A, dict(stream=stream)
        hils.hils_sink_prefill(p, A, self.Q, self.K, self.V, self.O, self.lse, workspace=w[0], **k)
        hils.hils_sink_prefill_backward(p, A, self.Q, self.K, self.V, self.O, self.lse, self.dO, *self.grads, workspace=w[1], **k)
        hils.hils_sink_weights(p, A, self.Q, self.K, self.lse, self.acc, self.w_out, workspace=w[2], **k)
        hils.hils_sink_decode(p, A, self.q1, self.K, self.V, self.n, self.o1, self.l1, acc=self.acc, acc_out=self.d_out,
                              workspace=w[3], **k)
        hils.hils_prefix_decode(p, self.q1, self.Kp, self.Vp, self.K, self.V, self.n, self.o2, self.l2, workspace=w[4], **k)
        hils.hils_cache_evict(p, A, self.budget, self.K, self.V, self.acc, self.n, self.Ko, self.Vo, self.ao, self.idx, self.no,
                              workspace=w[5], **k)

    def outputs(self):
        return [self.O, self.lse, *self.grads, self.w_out, self.d_out, self.o1, self.l1, self.o2, self.l2, self.Ko, self.Vo, self.ao,
                self.idx, self.no]

    def clear(self):
        for t in self.outputs():
            t.fill_(5)


def _differ(a, b):
    """Which outputs are not the same bits."""
    return [i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [dict(), dict(B=2, H=8, Hk=1, d=128, P=3000)])
def test_streams_graphs_and_shared_workspaces(cuda_device, dtype, sizes):
    a, b = Calls(cuda_device, dtype, 1, **sizes), Calls(cuda_device, dtype, 50, **sizes)
    a.clear()  # (what a call leaves as it was compares too)
    b.clear()
    a.run()
    b.run()
    torch.cuda.synchronize()
    want_a, want_b = [t.clone() for t in a.outputs()], [t.clone() for t in b.outputs()]
    # another stream than the current one, and two at once, each with its own workspaces
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.clear()
    b.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    assert _differ(a.outputs(), want_a) == [] and _differ(b.outputs(), want_b) == []
    # two captured graphs over one set of workspaces, replayed in turn on one stream
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
    assert _differ(a.outputs(), want_a) == [] and _differ(b.outputs(), want_b) == []
    # new data in the captured buffers
    a.Q.copy_(b.Q)
    a.K.copy_(b.K)
    a.V.copy_(b.V)
    a.dO.copy_(b.dO)
    a.acc.copy_(b.acc)
    a.q1.copy_(b.q1)
    a.Kp.copy_(b.Kp)
    a.Vp.copy_(b.Vp)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert _differ(a.outputs(), want_b) == []
    assert all(status_of(w) == 0 for w in a.ws)


@pytest.mark.parametrize("d,G", [(128, 4), (64, 1), (128, 3)])
def test_several_rounds_of_every_cta(cuda_device, d, G):
    """More row tiles and key blocks than SMs; the check samples heads."""
    B, Hk, N, W, A = 2, 4, 2500, 300, 6
    H = Hk * G
    Q, K, V = make(B, H, Hk, N, N, d, BF, d + G, cuda_device)
    p = params(B, H, Hk, d, W, BF)
    O, lse = prefill(p, A, Q, K, V)
    dO = torch.randn(Q.shape, generator=torch.Generator().manual_seed(1)).to(BF).to(cuda_device)
    grads = [torch.full_like(x, 7.0) for x in (Q, K, V)]
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_BACKWARD, N, A, device=cuda_device)
    hils.hils_sink_prefill_backward(p, A, Q, K, V, O, lse, dO, *grads, workspace=ws)
    acc = torch.zeros(B, Hk, N, device=cuda_device)
    wsw = hils.alloc_workspace(p, hils.HILS_CALL_SINK_WEIGHTS, N, A, device=cuda_device)
    hils.hils_sink_weights(p, A, Q, K, lse, acc, workspace=wsw)
    torch.cuda.synchronize()
    assert status_of(ws) == status_of(wsw) == 0
    see, scale = ref.visible(N, N, W, A), 1 / math.sqrt(d)
    for b, hk in ((0, 1), (1, Hk - 1)):
        h = slice(hk * G, hk * G + G)
        sub = [x[b:b + 1, s].contiguous() for x, s in ((Q, h), (K, slice(hk, hk + 1)), (V, slice(hk, hk + 1)))]
        ps = params(1, G, 1, d, W, BF)
        o, l, do = O[b:b + 1, h], lse[b:b + 1, h], dO[b:b + 1, h]
        check_prefill(ps, A, *sub, o, l)
        val, mag, es = ref.backward(*sub, o, l, do, see, scale)
        L, lm = ref.attend(*sub, see, scale)[4].max().item(), l.abs().max().item()
        got = [grads[0][b:b + 1, h], grads[1][b:b + 1, hk:hk + 1], grads[2][b:b + 1, hk:hk + 1]]
        for x, v, t in zip(got, val, grad_bounds(val, mag, es, L, lm, d, N * G, BF)):
            within(x, v, t, "gradient")
        w = ref.weights(sub[0], sub[1], l, see, scale)
        within(acc[b:b + 1, hk:hk + 1], w, weight_bound(w, L, lm, d, N * G) + 2.0 ** -23 * w, "weights")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_expanded_and_padded_views(cuda_device, dtype):
    """Keys and values that a batch shares (stride 0), rows with a pitch, a head count of one
    in a larger allocation: all the calls that take views."""
    B, H, Hk, d, N, W, A = 3, 4, 2, 64, 150, 40, 2
    Q, K, V = make(B, H, Hk, N, N, d, dtype, 91, cuda_device)
    p = params(B, H, Hk, d, W, dtype)
    shared = [x[:1].expand(B, -1, -1, -1) for x in (K, V)]
    want = prefill(p, A, Q, *(x.contiguous() for x in shared))
    got = prefill(p, A, Q, *shared)
    # the expanded view may take the float32 kernel: its own bounds, and the same lse to float32
    check_prefill(p, A, Q, *shared, *got)
    assert (got[1] - want[1]).abs().max() < 1e-4
    pitch = torch.full((B, Hk, N, d + 16), math.nan, dtype=dtype, device=cuda_device)
    pitch[..., :d] = K
    got = prefill(p, A, Q, pitch[..., :d], V)
    want = prefill(p, A, Q, K, V)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    n = torch.tensor([N, 77, 5], dtype=torch.int32, device=cuda_device)
    O = torch.empty(B, H, 1, d, dtype=dtype, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_DECODE, N, A, device=cuda_device)
    hils.hils_sink_decode(p, A, Q[:, :, 5:6], pitch[..., :d], shared[1], n, O, workspace=ws)
    rO, rl, _, Om, L = ref.attend(Q[:, :, 5:6], K, shared[1], ref.decode_visible(n, N, W, A), 1 / math.sqrt(d))
    within(O, rO, forward_bounds(rO, Om, rl, L, d, N, dtype)[0], "O")


def test_offsets_beyond_32_bits(cuda_device):
    """A cache of 2^24 + 300 slots (2^31 elements and more): a later piece of a prompt, its
    token decoded, and the eviction, over the last slots and the sinks."""
    d, T, W, A, Lq = 128, 2 ** 24 + 300, 200, 3, 40
    K, V = (torch.zeros(1, 1, T, d, dtype=BF, device=cuda_device) for _ in range(2))
    Q, k, v = make(1, 2, 1, Lq, 300, d, BF, 7, cuda_device)
    K[:, :, -300:], V[:, :, -300:] = k, v
    K[:, :, :A], V[:, :, :A] = k[:, :, 5:5 + A], v[:, :, 5:5 + A]
    p = params(1, 2, 1, d, W, BF)
    O, lse = prefill(p, A, Q, K, V)
    # the same, with the slots that nothing sees left out
    small = [torch.cat([x[:, :, :A], x[:, :, -(W + Lq):]], 2) for x in (K, V)]
    sO, sl = prefill(p, A, Q, *small)
    assert torch.equal(O, sO) and torch.equal(lse, sl)
    n = torch.tensor([T], dtype=torch.int32, device=cuda_device)
    o, l = torch.empty_like(Q[:, :, :1]), torch.empty(1, 2, device=cuda_device)
    acc = torch.zeros(1, 1, T, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_DECODE_ACC, T, A, device=cuda_device)
    hils.hils_sink_decode(p, A, Q[:, :, -1:].contiguous(), K, V, n, o, l, acc=acc, workspace=ws)
    assert (l - lse[..., -1]).abs().max() < 1e-4
    assert abs(acc.sum().item() - 2) < 1e-4 and abs(acc[0, 0, -W:].sum() + acc[0, 0, :A].sum() - 2) < 1e-4
    budget = 400
    Ko, Vo = (torch.zeros(1, 1, budget, d, dtype=BF, device=cuda_device) for _ in range(2))
    ao, idx = torch.zeros(1, 1, budget, device=cuda_device), torch.zeros(1, 1, budget, dtype=torch.int32, device=cuda_device)
    hils.hils_cache_evict(p, A, budget, K, V, acc, n, Ko, Vo, ao, idx, n,
                          workspace=hils.alloc_workspace(p, hils.HILS_CALL_CACHE_EVICT, T, budget, device=cuda_device))
    # between the sinks and the window every weight is zero: the lowest slots stay
    assert idx[0, 0].tolist() == list(range(budget - W)) + list(range(T - W, T)) and n.item() == budget
    assert torch.equal(Ko[:, :, -W:], K[:, :, -W:]) and torch.equal(Vo[:, :, :A], V[:, :, :A])


def test_waits_that_run_out(cuda_device):
    """With every wait expiring at once, the tensor-core calls return with their status set and
    the next call on the same workspace, cleared, is whole."""
    c = Calls(cuda_device, BF, 3, B=2, H=8, Hk=2, d=128, N=600, P=9000)
    c.clear()
    c.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in c.outputs()]
    c.p.flags = hils.HILS_FLAG_DIAG_EXPIRE_WAITS
    c.run()
    torch.cuda.synchronize()
    assert all(status_of(w) == 1 for w in c.ws[:3])
    c.p.flags = 0
    for w in c.ws:
        hils.hils_workspace_init(w)
    c.run()
    torch.cuda.synchronize()
    assert _differ(c.outputs(), want) == [] and all(status_of(w) == 0 for w in c.ws)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_random_sizes(cuda_device, dtype, seed):
    """Sizes drawn over all calls' ranges at once (small ones: the check is float64)."""
    g = torch.Generator().manual_seed(900 + seed)

    def pick(lo, hi):
        return int(math.exp(torch.rand((), generator=g).item() * math.log(hi / lo)) * lo)

    G, Hk, B, d = pick(1, 8.99), pick(1, 4.99), pick(1, 3.99), 64 * pick(1, 2.99)
    N, W, A = pick(1, 900), pick(1, 1000) - 1, pick(1, 200) - 1
    Lq = pick(1, N + 0.99)
    Q, K, V = make(B, Hk * G, Hk, Lq, N, d, dtype, seed, cuda_device)
    p = params(B, Hk * G, Hk, d, W, dtype)
    O, lse = prefill(p, A, Q, K, V)
    check_prefill(p, A, Q, K, V, O, lse, f"{(G, Hk, B, d, N, W, A, Lq)}")
    n = torch.randint(0, N + 1, (B,), generator=g, dtype=torch.int32).to(cuda_device)
    o, l = torch.empty_like(Q[:, :, :1]), torch.empty(B, Hk * G, device=cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_SINK_DECODE, N, A, device=cuda_device)
    hils.hils_sink_decode(p, A, Q[:, :, :1].contiguous(), K, V, n, o, l, workspace=ws)
    rO, rl, _, Om, L = ref.attend(Q[:, :, :1], K, V, ref.decode_visible(n, N, W, A), 1 / math.sqrt(d))
    tO, tl = forward_bounds(rO, Om, rl, L, d, N, dtype)
    within(o, rO, tO, "decode O")
    within(l, rl[..., 0], tl[..., 0], "decode lse")
    P = pick(1, 3000)
    _, Kp, Vp = make(1, Hk * G, Hk, 1, P, d, dtype, seed + 50, cuda_device)
    ws = hils.alloc_workspace(p, hils.HILS_CALL_PREFIX_DECODE, N, P, device=cuda_device)
    hils.hils_prefix_decode(p, Q[:, :, :1].contiguous(), Kp, Vp, K, V, n, o, l, workspace=ws)
    assert status_of(ws) == 0
    rO, rl, _, Om, L = ref.prefix(Q[:, :, :1], Kp, Vp, K, V, n, 1 / math.sqrt(d))
    tO, tl = forward_bounds(rO, Om, rl, L, d, N + P, dtype)
    within(o, rO, tO, "prefix O")
    within(l, rl[..., 0], tl[..., 0], "prefix lse")
