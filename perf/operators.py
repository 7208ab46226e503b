"""Measured cases of the window-and-sink attention calls, the shared-prefix decode and the
cache eviction: their inputs, their plain form in elementary torch operations, the calls
of the library, what each has to read, write and compute, and a float64 evaluation.

A query at position t sees the first A tokens (the sinks) and the W newest up to its own:
    V(t) = { j <= t : j < A or j > t - W },    s_tj = scale q_t . k_j,
    lse_t = log sum_{j in V(t)} exp(s_tj),     p_tj = exp(s_tj - lse_t),
    o_t = sum_j p_tj v_j     (an empty V(t) gives o = 0, lse = -inf).
H query heads share Hk key-value heads in groups of G = H / Hk consecutive heads; the Lq
queries of a call are the last of N tokens, t = N - Lq + i.
    prefill   O, lse
    backward  D_t = dO_t . o_t, ds_tj = scale p_tj (dO_t . v_j - D_t), dQ = ds K,
              dK = ds^T Q, dV = p^T dO (summed over the group's heads), from given O and lse
    decode    one query per sequence at t = cache_len - 1; with `acc`, every visible slot's
              accumulated weight grows by the sum of the group's p_j
    weights   the same growth for the Lq newest queries of a prompt, from their lse
    prefix    one query per sequence over a prefix that the whole batch shares, then its
              own cache: softmax over both together
    evict     per key-value head keeps min(len, budget) slots: the first A, the W newest and
              the heaviest of the rest by acc (ties to the lower slot), in slot order
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one layer's prompt at the sizes of the benchmark's 8K prefill, with four sinks
        dict(name="prefill_8k", op="prefill", dtype="bf16", B=1, H=32, Hk=32, d=128, Lq=8192, N=8192, W=512, A=4),
        # a short later piece of a prompt (its keys already cached), odd sizes, groups of three
        dict(name="prefill_piece_fp32", op="prefill", dtype="fp32", B=2, H=6, Hk=2, d=64, Lq=333, N=1357, W=200, A=5),
        # its training step's backward, eight key-value heads for the 32 query heads
        dict(name="backward_8k", op="backward", dtype="bf16", B=1, H=32, Hk=8, d=128, Lq=8192, N=8192, W=512, A=4),
        # a small float32 training example
        dict(name="backward_small_fp32", op="backward", dtype="fp32", B=2, H=4, Hk=4, d=64, Lq=509, N=509, W=96, A=1),
        # a serving batch that attends to its whole ragged caches and keeps the weights for eviction
        dict(name="decode_batch", op="decode", dtype="bf16", B=8, H=32, Hk=8, d=128, T=131072, W=131072, A=0, acc=True),
        # one user's token: the sinks and the window of a long cache, where latency counts
        dict(name="decode_window", op="decode", dtype="bf16", B=1, H=32, Hk=32, d=128, T=131072, W=512, A=4, acc=False),
        # the weights of a whole prompt, before its cache is cut
        dict(name="weights_prompt", op="weights", dtype="bf16", B=1, H=32, Hk=8, d=128, Lq=8192, N=8192, W=8192, A=0),
        # the weights that the last 64 queries of a long prompt give
        dict(name="weights_recent", op="weights", dtype="bf16", B=1, H=32, Hk=8, d=128, Lq=64, N=65536, W=65536, A=0),
        # 32 users of one long document
        dict(name="prefix_batch", op="prefix", dtype="bf16", B=32, H=32, Hk=8, d=128, P=65536, T=512),
        # a few answers sampled from one prompt, float32
        dict(name="prefix_small_fp32", op="prefix", dtype="fp32", B=3, H=8, Hk=4, d=64, P=1000, T=70),
        # a serving batch's caches cut to a quarter
        dict(name="evict_batch", op="evict", dtype="bf16", B=8, H=8, Hk=8, d=128, T=32768, budget=8192, W=512, A=4),
        # a short cache cut while a small model answers
        dict(name="evict_small_fp32", op="evict", dtype="fp32", B=2, H=2, Hk=2, d=64, T=700, budget=256, W=32, A=1),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefill", "backward", "decode", "weights", "prefix", "evict"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    G = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8])
    Hk = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, dtype=dtype, B=rng.choice([1, 1, 2, 3, 4]), H=Hk * G, Hk=Hk, d=rng.choice([64, 128, 128]))
    if op in ("prefill", "backward", "weights"):
        N = _span(rng, 1, 8192)
        c |= dict(Lq=N if op == "backward" or rng.random() < 0.5 else _span(rng, 1, N), N=N,
                  W=rng.choice([0, N, _span(rng, 1, 4096), _span(rng, 1, 4096), _span(rng, 64, 1024)]),
                  A=rng.choice([0, 1, 4, 4, _span(rng, 1, 200)]))
        size, least = "N", 64
    elif op == "decode":
        T = _span(rng, 1, 131072)
        c |= dict(B=_span(rng, 1, 16), T=T, W=rng.choice([0, T, T, _span(rng, 1, 4096)]),
                  A=rng.choice([0, 1, 4, _span(rng, 1, 200)]), acc=rng.random() < 0.5)
        size, least = "T", 64
    elif op == "prefix":
        c |= dict(B=_span(rng, 1, 64), P=_span(rng, 1, 65536), T=_span(rng, 1, 1024))
        size, least = "P", 64
    else:
        T = _span(rng, 1, 65536)
        budget = _span(rng, 1, T)
        A = min(rng.choice([0, 1, 4, 16]), budget)
        c |= dict(B=_span(rng, 1, 8), T=T, budget=budget, W=rng.choice([0, _span(rng, 1, 512)]), A=A)
        c["W"] = min(c["W"], budget - A)
        size, least = "T", 64
    most = {k["op"]: work(k) for k in reversed(listed())}[op]  # an operator's first listed case is its largest
    part = 1 / 16 if dtype == "fp32" and op in ("prefill", "backward", "weights") else 1
    while c[size] > least and any(work(c)[k] > part * most[k] for k in most):
        c[size] -= c[size] // 5
        for k in ("Lq", "budget"):
            if k in c:
                c[k] = min(c[k], c[size])
        if op == "backward":
            c["Lq"] = c["N"]
        if op == "evict":
            c["A"] = min(c["A"], c["budget"])
            c["W"] = min(c["W"], c["budget"] - c["A"])
    return c


def _lens(c):
    """The sequences' cache lengths, ragged over the batch (the first one full)."""
    if c["op"] == "prefix":  # an own cache may still be empty
        return [(c["T"] * ((7 * b + 5) % 8)) // 7 if b else c["T"] for b in range(c["B"])]
    return [max(1, c["T"] - (c["T"] * ((5 * b) % 7)) // 16) for b in range(c["B"])]


def _visible(t, W, A):
    """How many tokens position t sees."""
    return min(t + 1, W) + min(A, max(0, t + 1 - W))


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    B, H, Hk, d = c["B"], c["H"], c["Hk"], c["d"]
    if c["op"] in ("prefill", "backward", "weights"):
        Lq, N, W, A = c["Lq"], c["N"], c["W"], c["A"]
        pairs = B * H * sum(_visible(t, W, A) for t in range(N - Lq, N))
        first = max(0, N - Lq - W + 1)  # keys that some query sees
        keys = B * Hk * ((N - first if W else 0) + min(A, first if W else N))
        q = B * H * Lq
        if c["op"] == "prefill":
            return {"bytes": 2 * q * d * e + 2 * keys * d * e + 4 * q, "flops": 4 * d * pairs}
        if c["op"] == "weights":
            return {"bytes": q * d * e + keys * d * e + 4 * q + 8 * keys, "flops": 2 * d * pairs}
        return {"bytes": 4 * q * d * e + 2 * keys * d * e + 2 * B * Hk * N * d * e + 4 * q, "flops": 10 * d * pairs}
    if c["op"] == "decode":
        keys = Hk * sum(_visible(n - 1, c["W"], c["A"]) for n in _lens(c))
        return {"bytes": 2 * keys * d * e + 2 * B * H * d * e + 4 * B * H + (8 * keys if c["acc"] else 0),
                "flops": 4 * d * keys * (H // Hk)}
    if c["op"] == "prefix":
        rest = sum(_lens(c))
        return {"bytes": 2 * Hk * (c["P"] + rest) * d * e + 2 * B * H * d * e + 4 * B * H,
                "flops": 4 * d * H * (B * c["P"] + rest)}
    kept = Hk * sum(min(n, c["budget"]) for n in _lens(c))
    return {"bytes": 4 * Hk * sum(_lens(c)) + kept * (4 * d * e + 4) + 4 * B * Hk * c["budget"] + 8 * B, "flops": 0}


# ------------------------------------------------------------------ inputs


def _qkv(c, g, Bq, Bk, Lq, tokens):
    """Queries and keys whose logits have the spread of a trained layer, and with it the
    first tokens that draw much of the weight; values with a mean and a spread."""
    dt, d = DTYPES[c["dtype"]], c["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    lean = normal(d)
    lean /= lean.norm()
    Q = (normal(Bq, c["H"], Lq, d) + 3.0 * lean).to(dt)
    K = normal(Bk, c["Hk"], tokens, d)
    K[:, :, :4] += 0.6 * math.sqrt(d) * lean
    V = normal(Bk, c["Hk"], tokens, d)
    V += 0.25 * normal(Bk, c["Hk"], 1, d)
    return Q, K.to(dt), V.to(dt)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, B, H, Hk, d = DTYPES[c["dtype"]], c["B"], c["H"], c["Hk"], c["d"]
    s = {"c": c}
    f32 = dict(dtype=torch.float32, device="cuda")

    def weights_so_far(T):
        """Accumulated weights: heavy-tailed, with many slots that no query has looked at."""
        a = torch.exp(1.5 * torch.randn(B, Hk, T, generator=g, device="cuda") - 2.0)
        return torch.where(torch.rand(B, Hk, T, generator=g, device="cuda") < 0.2, torch.zeros_like(a), a)

    if c["op"] in ("prefill", "backward", "weights"):
        s["Q"], s["K"], s["V"] = _qkv(c, g, B, B, c["Lq"], c["N"])
        if c["op"] == "prefill":
            s["O"], s["lse"] = torch.empty_like(s["Q"]), torch.empty(B, H, c["Lq"], **f32)
            return s
        s["O"], s["lse"] = _prefill(s)
        if c["op"] == "backward":
            s["dO"] = torch.randn(s["Q"].shape, generator=g, device="cuda").to(dt)
            s["dQ"], s["dK"], s["dV"] = torch.empty_like(s["Q"]), torch.empty_like(s["K"]), torch.empty_like(s["V"])
        else:
            s["acc"] = weights_so_far(c["N"])
            s["acc_out"] = s["acc"].clone()
        return s
    s["cache_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    if c["op"] == "evict":
        _, s["K"], s["V"] = _qkv(c, g, 1, B, 1, c["T"])
        s["acc"] = weights_so_far(c["T"])
        n = c["budget"]
        s["Kout"], s["Vout"] = torch.zeros(B, Hk, n, d, dtype=dt, device="cuda"), torch.zeros(B, Hk, n, d, dtype=dt, device="cuda")
        s["acc_out"] = torch.zeros(B, Hk, n, **f32)
        s["idx"] = torch.empty(B, Hk, n, dtype=torch.int32, device="cuda")
        s["len_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    if c["op"] == "prefix":
        s["Q"], s["Kp"], s["Vp"] = _qkv(c, g, B, 1, 1, c["P"])
        _, s["K"], s["V"] = _qkv(c, g, 1, B, 1, c["T"])
    else:
        s["Q"], s["K"], s["V"] = _qkv(c, g, B, B, 1, c["T"])
        if c["acc"]:
            s["acc"] = weights_so_far(c["T"])
            s["acc_out"] = s["acc"].clone()
    s["O"], s["lse"] = torch.empty_like(s["Q"]), torch.empty(B, H, **f32)
    return s


# ------------------------------------------------------------------ the plain form


def _softmax(x):
    """Softmax over the last axis and its log-sum, of rows that may be all -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z > 0, z, torch.ones_like(z)), (m + torch.log(z))[..., 0]


def _band(c, device):
    """The queries in blocks of 512 and, for each block, the keys that it may see: the
    sinks, then the window's span. Gives key indices [blocks, keys], which of them each
    query sees [blocks, 512, keys], and the number of blocks."""
    Lq, N, W, A = c["Lq"], c["N"], min(c["W"], c["N"]), min(c["A"], c["N"])
    rows = min(512, Lq)
    blocks = -(-Lq // rows)
    t = N - Lq + torch.arange(blocks * rows, device=device).view(blocks, rows)
    span = torch.arange(1 - W, rows, device=device) if W > 0 else torch.arange(0, device=device)
    j = torch.cat([torch.arange(A, device=device).expand(blocks, A), t[:, :1] + span], 1)
    sink = torch.arange(j.shape[1], device=device) < A
    t, k = t[..., None], j[:, None, :]
    in_window = (k > t - W) & (k <= t) & (k >= 0)
    seen = torch.where(sink, (k <= t - W) & (k <= t), in_window) & (t < N)
    return j.clamp(0, N - 1), seen, blocks, rows


def _blocks(c, x, blocks, rows):
    """[B, H, Lq, ..] in float32 as [B, Hk, G, blocks, rows, ..] (zeros behind the last query)."""
    out = x.new_zeros((x.shape[0], x.shape[1], blocks * rows) + x.shape[3:], dtype=torch.float32)
    out[:, :, :c["Lq"]] = x
    return out.view((x.shape[0], c["Hk"], c["H"] // c["Hk"], blocks, rows) + x.shape[3:])


def _rows(c, x):
    """The inverse: [B, Hk, G, blocks, rows, ..] -> [B, H, Lq, ..]."""
    return x.reshape((c["B"], c["H"], -1) + x.shape[5:])[:, :, :c["Lq"]]


def _logits(s, q, k, seen):
    x = torch.einsum("bkgnrd,bkntd->bkgnrt", q, k) / math.sqrt(s["c"]["d"])
    return x.masked_fill(~seen, -math.inf)


def _prefill(s):
    c = s["c"]
    j, seen, blocks, rows = _band(c, s["Q"].device)
    if j.shape[1] == 0:
        return torch.zeros_like(s["Q"]), torch.full((c["B"], c["H"], c["Lq"]), -math.inf, device=s["Q"].device)
    k, v = s["K"].float()[:, :, j], s["V"].float()[:, :, j]
    p, lse = _softmax(_logits(s, _blocks(c, s["Q"], blocks, rows), k, seen))
    o = torch.einsum("bkgnrt,bkntd->bkgnrd", p, v)
    return _rows(c, o).to(s["Q"].dtype).contiguous(), _rows(c, lse).contiguous()


def _probabilities(s, q, k, seen, blocks, rows):
    lse = _blocks(s["c"], s["lse"], blocks, rows)[..., None]
    p = torch.exp(_logits(s, q, k, seen) - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    return torch.where(seen, p, torch.zeros_like(p))


def _to_keys(c, x, j):
    """Sums of [B, Hk, blocks, keys, ..] into the keys' rows."""
    out = x.new_zeros((c["B"], c["Hk"], c["N"]) + x.shape[4:])
    return out.index_add_(2, j.reshape(-1), x.reshape((c["B"], c["Hk"], -1) + x.shape[4:]))


def _backward(s):
    c = s["c"]
    j, seen, blocks, rows = _band(c, s["Q"].device)
    if j.shape[1] == 0:
        return torch.zeros_like(s["Q"]), torch.zeros_like(s["K"]), torch.zeros_like(s["V"])
    k, v = s["K"].float()[:, :, j], s["V"].float()[:, :, j]
    q, do = _blocks(c, s["Q"], blocks, rows), _blocks(c, s["dO"], blocks, rows)
    p = _probabilities(s, q, k, seen, blocks, rows)
    D = (do * _blocks(c, s["O"], blocks, rows)).sum(-1, keepdim=True)
    ds = p * (torch.einsum("bkgnrd,bkntd->bkgnrt", do, v) - D) / math.sqrt(c["d"])
    dq = torch.einsum("bkgnrt,bkntd->bkgnrd", ds, k)
    dk = torch.einsum("bkgnrt,bkgnrd->bkntd", ds, q)
    dv = torch.einsum("bkgnrt,bkgnrd->bkntd", p, do)
    dt = s["Q"].dtype
    return _rows(c, dq).to(dt).contiguous(), _to_keys(c, dk, j).to(dt), _to_keys(c, dv, j).to(dt)


def _weights(s):
    c = s["c"]
    j, seen, blocks, rows = _band(c, s["Q"].device)
    if j.shape[1] == 0:
        return s["acc"].clone()
    p = _probabilities(s, _blocks(c, s["Q"], blocks, rows), s["K"].float()[:, :, j], seen, blocks, rows)
    return s["acc"] + _to_keys(c, p.sum((2, 4)), j)


def _decode(s):
    c = s["c"]
    B, Hk, T, d, W, A = c["B"], c["Hk"], c["T"], c["d"], c["W"], min(c["A"], c["T"])
    n = s["cache_len"].long()[:, None]
    j = torch.arange(T, device=n.device)[None]
    if W + A < T:  # the sinks, and the window's slots
        j = torch.cat([j[:, :A].expand(B, A), n - W + torch.arange(W, device=n.device)], 1)
        first = torch.arange(A + W, device=n.device) < A
        seen = (j >= 0) & (j < n) & torch.where(first, j < n - W, j >= n - W)
        j = j.clamp(0, T - 1)
        b = torch.arange(B, device=n.device)[:, None]
        k, v = s["K"][b, :, j].float().transpose(1, 2), s["V"][b, :, j].float().transpose(1, 2)
    else:
        seen = (j < n) & ((j < A) | (j >= n - W))
        k, v = s["K"].float(), s["V"].float()
    if j.shape[1] == 0:
        return torch.zeros_like(s["O"]), torch.full_like(s["lse"], -math.inf), s["acc"].clone() if c["acc"] else None
    q = s["Q"].float().view(B, Hk, c["H"] // Hk, d)
    x = (q @ k.transpose(2, 3) / math.sqrt(d)).masked_fill(~seen[:, None, None], -math.inf)
    p, lse = _softmax(x)
    o = (p @ v).view(B, c["H"], 1, d).to(s["Q"].dtype)
    acc = None
    if c["acc"]:
        acc = s["acc"].scatter_add(2, j[:, None].expand(B, Hk, j.shape[1]), p.sum(2))
    return o, lse.reshape(B, c["H"]), acc


def _prefix(s):
    c = s["c"]
    B, Hk, d, G = c["B"], c["Hk"], c["d"], c["H"] // c["Hk"]
    q = s["Q"].float().view(B, Hk, G, d)
    x = torch.einsum("bkgd,ktd->bkgt", q, s["Kp"][0].float())
    y = q @ s["K"].float().transpose(2, 3)
    gone = torch.arange(c["T"], device=q.device) >= s["cache_len"][:, None, None, None]
    p, lse = _softmax(torch.cat([x, y.masked_fill(gone, -math.inf)], 3) / math.sqrt(d))
    o = torch.einsum("bkgt,ktd->bkgd", p[..., :c["P"]], s["Vp"][0].float()) + p[..., c["P"]:] @ s["V"].float()
    return o.reshape(B, c["H"], 1, d).to(s["Q"].dtype), lse.reshape(B, c["H"])


def _evict(s):
    c = s["c"]
    n = s["cache_len"].long()[:, None, None]
    j = torch.arange(c["T"], device=n.device)
    x = torch.where((j < c["A"]) | (j >= n - c["W"]), torch.full_like(s["acc"], math.inf), s["acc"])
    x = torch.where(j < n, x, torch.full_like(x, -math.inf))
    order = torch.sort(x, dim=2, descending=True, stable=True).indices[:, :, :c["budget"]]
    kept = n.clamp(max=c["budget"])
    live = torch.arange(c["budget"], device=n.device) < kept
    order = torch.sort(torch.where(live, order, torch.full_like(order, c["T"])), dim=2).values
    at = order.clamp(max=c["T"] - 1)
    rows = at[..., None].expand(-1, -1, -1, c["d"])
    K = torch.where(live[..., None], torch.gather(s["K"], 2, rows), s["Kout"])
    V = torch.where(live[..., None], torch.gather(s["V"], 2, rows), s["Vout"])
    acc = torch.where(live, torch.gather(s["acc"], 2, at), s["acc_out"])
    return K, V, acc, torch.where(live, order, torch.full_like(order, -1)).int(), kept[:, 0, 0].int()


# ------------------------------------------------------------------ the calls


def _own(s):
    import hierarchical_chunk_sparse_b200 as hils

    c = s["c"]
    op = c["op"]
    if "p" not in s:  # what a program sets up once: the parameters and the workspace
        s["p"] = p = hils.Params(B=c["B"], H=c["H"], d=c["d"], K=0, W=c.get("W", 0), dtype=DTYPES[c["dtype"]], H_kv=c["Hk"])
        call, rows, other = {
            "prefill": (hils.HILS_CALL_SINK_PREFILL, c.get("Lq"), c.get("A")),
            "backward": (hils.HILS_CALL_SINK_BACKWARD, c.get("N"), c.get("A")),
            "weights": (hils.HILS_CALL_SINK_WEIGHTS, c.get("N"), c.get("A")),
            "decode": (hils.HILS_CALL_SINK_DECODE_ACC if c.get("acc") else hils.HILS_CALL_SINK_DECODE, c.get("T"), c.get("A")),
            "prefix": (hils.HILS_CALL_PREFIX_DECODE, c.get("T"), c.get("P")),
            "evict": (hils.HILS_CALL_CACHE_EVICT, c.get("T"), c.get("budget")),
        }[op]
        s["ws"] = hils.alloc_workspace(p, call, rows, other, device="cuda")
    p, ws = s["p"], s["ws"]
    if op == "prefill":
        hils.hils_sink_prefill(p, c["A"], s["Q"], s["K"], s["V"], s["O"], s["lse"], workspace=ws)
        return s["O"], s["lse"]
    if op == "backward":
        hils.hils_sink_prefill_backward(p, c["A"], s["Q"], s["K"], s["V"], s["O"], s["lse"], s["dO"], s["dQ"], s["dK"],
                                        s["dV"], workspace=ws)
        return s["dQ"], s["dK"], s["dV"]
    if op == "weights":
        hils.hils_sink_weights(p, c["A"], s["Q"], s["K"], s["lse"], s["acc"], s["acc_out"], workspace=ws)
        return s["acc_out"]
    if op == "decode":
        hils.hils_sink_decode(p, c["A"], s["Q"], s["K"], s["V"], s["cache_len"], s["O"], s["lse"], acc=s.get("acc"),
                              acc_out=s.get("acc_out"), workspace=ws)
        return (s["O"], s["lse"], s["acc_out"]) if c["acc"] else (s["O"], s["lse"])
    if op == "prefix":
        hils.hils_prefix_decode(p, s["Q"], s["Kp"], s["Vp"], s["K"], s["V"], s["cache_len"], s["O"], s["lse"], workspace=ws)
        return s["O"], s["lse"]
    hils.hils_cache_evict(p, c["A"], c["budget"], s["K"], s["V"], s["acc"], s["cache_len"], s["Kout"], s["Vout"],
                          s["acc_out"], s["idx"], s["len_out"], workspace=ws)
    return s["Kout"], s["Vout"], s["acc_out"], s["idx"], s["len_out"]


def run(state):
    if own:
        return _own(state)
    out = {"prefill": _prefill, "backward": _backward, "weights": _weights, "decode": _decode, "prefix": _prefix,
           "evict": _evict}[state["c"]["op"]](state)
    return out[:2] if state["c"]["op"] == "decode" and not state["c"]["acc"] else out


# ------------------------------------------------------------------ float64 values


def _exact_row(q, k, v, see):
    """[G, r, d] queries over [t, d] keys with visibility [r, t]: probabilities, outputs, lse."""
    x = (q @ k.T) * (1.0 / math.sqrt(q.shape[-1]))
    x[:, ~see] = -math.inf
    lse = torch.logsumexp(x, -1)
    p = torch.nan_to_num(torch.exp(x - lse[..., None]), nan=0.0)
    return p, (None if v is None else p @ v), lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    B, H, Hk, d = c["B"], c["H"], c["Hk"], c["d"]
    G = H // Hk
    if c["op"] == "evict":
        return _exact_evict(s)
    Q = s["Q"].double().view(B, Hk, G, -1, d)
    if c["op"] in ("decode", "prefix"):
        O, lse = torch.zeros_like(Q[..., 0, :]), torch.zeros(B, Hk, G, dtype=torch.float64, device="cuda")
        acc = s["acc"].double().clone() if c.get("acc") else None
        for b, n in enumerate(_lens(c)):
            first = max(0, n - c.get("W", n))  # the window's first slot
            at = torch.cat([torch.arange(min(c.get("A", 0), first), device="cuda"), torch.arange(first, n, device="cuda")])
            for h in range(Hk):
                k, v = s["K"][b, h, at].double(), s["V"][b, h, at].double()
                if c["op"] == "prefix":
                    k, v = torch.cat([s["Kp"][0, h].double(), k]), torch.cat([s["Vp"][0, h].double(), v])
                p, o, l = _exact_row(Q[b, h], k, v, torch.ones(1, k.shape[0], dtype=torch.bool, device="cuda"))
                O[b, h], lse[b, h] = o[:, 0], l[:, 0]
                if acc is not None:
                    acc[b, h, at] += p[:, 0].sum(0)
        out = (O.view(B, H, 1, d), lse.view(B, H))
        return out + (acc,) if acc is not None else out
    Lq, N, W, A = c["Lq"], c["N"], c["W"], c["A"]
    if work(c)["flops"] * (N / max(1, min(N, W + A + 1024))) > 3e13:
        return None
    O, lse = torch.zeros_like(Q), torch.zeros(B, Hk, G, Lq, dtype=torch.float64, device="cuda")
    dQ = torch.zeros_like(Q)
    dK, dV = (torch.zeros(B, Hk, N, d, dtype=torch.float64, device="cuda") for _ in range(2))
    acc = s["acc"].double().clone() if c["op"] == "weights" else None
    step = 1024
    for b in range(B):
        for h in range(Hk):
            K, V = s["K"][b, h].double(), s["V"][b, h].double()
            for i in range(0, Lq, step):
                e = min(Lq, i + step)
                t = torch.arange(N - Lq + i, N - Lq + e, device="cuda")[:, None]
                lo, hi = max(0, N - Lq + i - W + 1), N - Lq + e
                j = torch.cat([torch.arange(min(A, lo), device="cuda"), torch.arange(lo, hi, device="cuda")])
                see = (j <= t) & ((j < A) | (j > t - W))
                k, v = K[j], V[j]
                if c["op"] == "prefill":
                    _, O[b, h, :, i:e], lse[b, h, :, i:e] = _exact_row(Q[b, h, :, i:e], k, v, see)
                    continue
                q, L = Q[b, h, :, i:e], s["lse"].double().view(B, Hk, G, Lq)[b, h, :, i:e, None]
                p = torch.where(see, torch.exp(q @ k.T / math.sqrt(d) - L), 0.0)
                p = torch.where(torch.isfinite(L), p, 0.0)
                if c["op"] == "weights":
                    acc[b, h, j] += p.sum((0, 1))
                    continue
                do = s["dO"].double().view(B, Hk, G, Lq, d)[b, h, :, i:e]
                D = (do * s["O"].double().view(B, Hk, G, Lq, d)[b, h, :, i:e]).sum(-1, keepdim=True)
                ds = p * (do @ v.T - D) / math.sqrt(d)
                dQ[b, h, :, i:e] = ds @ k
                dK[b, h, j] += torch.einsum("grt,grd->td", ds, q)
                dV[b, h, j] += torch.einsum("grt,grd->td", p, do)
    if c["op"] == "prefill":
        return O.view(B, H, Lq, d), lse.view(B, H, Lq)
    return acc if c["op"] == "weights" else (dQ.view(B, H, Lq, d), dK, dV)


def _exact_evict(s):
    c = s["c"]
    out = [s[k].double().clone() for k in ("Kout", "Vout", "acc_out")]
    idx = torch.full((c["B"], c["Hk"], c["budget"]), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(_lens(c)):
        m = min(n, c["budget"])
        for h in range(c["Hk"]):
            mid = range(c["A"], n - c["W"])
            if n <= c["budget"]:
                kept = list(range(n))
            else:
                a = s["acc"][b, h].tolist()
                heavy = sorted(mid, key=lambda t: (-a[t], t))[:c["budget"] - c["A"] - c["W"]]
                kept = sorted(list(range(c["A"])) + heavy + list(range(n - c["W"], n)))
            at = torch.tensor(kept, dtype=torch.long, device="cuda")
            idx[b, h, :m] = at.int()
            out[0][b, h, :m], out[1][b, h, :m], out[2][b, h, :m] = s["K"][b, h, at].double(), s["V"][b, h, at].double(), s["acc"][b, h, at].double()
    return (*out, idx, torch.tensor([min(n, c["budget"]) for n in _lens(c)], dtype=torch.int32, device="cuda"))
