// C-ABI entry points of the window-and-sink attention, the shared-prefix decode and the
// cache eviction: argument checks, workspace layouts and dispatch. No call allocates,
// frees or synchronises.
#include "api_checks.cuh"
#include "sink_common.cuh"

namespace hils {
namespace {

View view(const hils_ctensor &t) { return {t.ptr, t.sb, t.sh, t.st}; }
MutView mut(const hils_tensor &t) { return {t.ptr, t.sb, t.sh, t.st}; }
template <typename V>
int check(const V &t, int64_t rows, const hils_params *p) {
    return check_view(t.ptr, t.sb, t.sh, t.st, rows, p);
}

// A view that is written: no two of its rows are one.
int check_out(const hils_tensor &t, int heads, int64_t rows, const hils_params *p) {
    HILS_TRY(check(t, rows, p));
    const bool twice = (t.sb == 0 && p->B > 1) || (t.sh == 0 && heads > 1) || (t.st == 0 && rows > 1);
    return twice && (int64_t)p->B * heads * rows > 0 ? HILS_ERR_INVALID_ARG : HILS_OK;
}

// The addresses [*lo, *hi) that a [B, H, T, d] view spans.
template <typename V>
void span_of(const V &t, int64_t B, int64_t H, int64_t T, const hils_params *p, uintptr_t *lo, uintptr_t *hi) {
    int64_t a = 0, e = p->d;
    const int64_t ext[3] = {(B - 1) * t.sb, (H - 1) * t.sh, (T - 1) * t.st};
    for (int64_t x : ext) (x < 0 ? a : e) += x;
    *lo = (uintptr_t)t.ptr + a * (int64_t)elem_size(p->dtype);
    *hi = (uintptr_t)t.ptr + e * (int64_t)elem_size(p->dtype);
}
bool disjoint(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a1 <= b0 || b1 <= a0; }

int clip(int64_t x, int64_t most) { return (int)(x < most ? x : most); }

// Rows of every (b, h) stay within int, and the shared checks of W and A.
int check_sink(const hils_params *p, int A, int64_t rows, float *scale) {
    HILS_TRY(check_params(p, scale));
    if (A < 0 || rows < 0) return HILS_ERR_INVALID_ARG;
    if ((int64_t)p->B * p->H * rows > 0x7fffffffll) return HILS_ERR_INVALID_ARG;
    return HILS_OK;
}
int check_tokens(int64_t n) { return n > kSinkMostTokens ? HILS_ERR_UNSUPPORTED : HILS_OK; }

// Longest key range of a prefill row tile.
int64_t prefill_keys(const hils_params *p, int A, int Lq) { return (int64_t)p->W + A + (Lq < 256 ? Lq : 256); }

hils_status forward(const hils_params *p, const SinkArgs &a, cudaStream_t s) {
    hils_status st;
    return launch_sink_forward_tc(p->dtype, p->d, a, s, &st) ? st : launch_sink_forward_general(p->dtype, p->d, a, s);
}

struct Carve {  // consecutive 256-byte aligned parts of a workspace
    uint8_t *base;
    size_t used = 0;
    template <typename T>
    T *take(size_t count) {
        T *r = reinterpret_cast<T *>(base + used);
        used += sink_align(count * sizeof(T));
        return r;
    }
};

size_t key_ws(const hils_params *p, int Lq, int N, int A, int per_key, SinkBwdArgs *a) {
    a->B = p->B;
    a->H = p->H;
    a->G = groups(p);
    sink_key_plan(p->dtype, p->B, p->H / a->G, a->G, Lq, N, clip(p->W, N), clip(A, N),
                  per_key == 1 && p->dtype == HILS_BF16 ? 2 * kSinkKeys : kSinkKeys, device_sm_count(), a);
    return sink_align(sink_key_part_floats(*a, per_key) * 4);
}

struct DecodePlan {
    int ctas, prefix_splits;
    int64_t keys, segs;  // longest visible range of a cache; segments of the CTAs' shares
    size_t bytes;
};
DecodePlan decode_plan(const hils_params *p, int64_t T, int64_t A, int64_t P, bool prefix, bool acc) {
    DecodePlan d{};
    const int Hk = p->H / groups(p), sms = device_sm_count();
    const int64_t rows = (int64_t)p->B * p->H;
    d.keys = prefix ? T : (T < A + p->W ? T : A + p->W);
    // a prefix that is cheaper read by each sequence than in a pass of its own
    const bool direct = prefix && sink_prefix_direct(p->dtype, p->d, p->B, p->H, groups(p), P);
    if (direct) d.keys = P + T;
    d.prefix_splits = prefix && !direct ? sink_prefix_splits(p->dtype, p->B, Hk, groups(p), (int)P, sms) : 0;
    d.ctas = sink_decode_ctas(p->dtype, p->B, Hk, d.keys, sms);
    d.segs = d.ctas + (int64_t)p->B * Hk;
    d.bytes = kSinkStatusBytes + sink_part_bytes(rows, d.prefix_splits, p->d) +
              sink_part_bytes(d.segs * groups(p), 1, p->d) + sink_align(rows * 4) +
              (acc ? sink_align((size_t)rows * d.keys * 4) : 0);
    return d;
}

// The decode kernel's parts of the workspace; the status word stays in front.
void decode_space(const hils_params *p, const DecodePlan &plan, Carve &ws, float *lse, SinkDecodeArgs *a) {
    const size_t rows = (size_t)p->B * p->H, segs = (size_t)plan.segs * a->G;
    ws.take<uint32_t>(kSinkStatusBytes / 4);
    a->slots = plan.prefix_splits;
    a->part_o = ws.take<float>(rows * a->slots * p->d);
    a->part_lse = ws.take<float>(rows * a->slots);
    a->seg_o = ws.take<float>(segs * p->d);
    a->seg_lse = ws.take<float>(segs);
    float *row_lse = ws.take<float>(rows);
    a->lse = lse ? lse : row_lse;
}

}  // namespace

size_t sink_ws_bytes(const hils_params *p, int call, int rows, int other) {
    float scale;
    // query rows: of the other calls `rows` counts cached tokens
    const int queries = call == HILS_CALL_SINK_PREFILL || call == HILS_CALL_SINK_BACKWARD ? rows : 1;
    const int64_t tokens = call == HILS_CALL_PREFIX_DECODE ? (int64_t)rows + other : rows;
    if (rows < 0 || tokens > kSinkMostTokens || check_sink(p, other, queries, &scale) != HILS_OK) return 0;
    const int64_t all = (int64_t)p->B * p->H * rows;
    SinkBwdArgs a{};
    switch (call) {
    case HILS_CALL_SINK_PREFILL: {
        const int s = sink_prefill_splits(p->dtype, p->B, p->H, groups(p), rows, prefill_keys(p, other, rows), device_sm_count());
        return kSinkStatusBytes + (s > 1 ? sink_part_bytes(all, s, p->d) : 0);
    }
    case HILS_CALL_SINK_BACKWARD:
        return kSinkStatusBytes + sink_align(all * 4) + key_ws(p, rows, rows, other, 2 * p->d, &a);
    case HILS_CALL_SINK_WEIGHTS: return kSinkStatusBytes + key_ws(p, rows, rows, other, 1, &a);
    case HILS_CALL_SINK_DECODE: return decode_plan(p, rows, other, 0, false, false).bytes;
    case HILS_CALL_SINK_DECODE_ACC: return decode_plan(p, rows, other, 0, false, true).bytes;
    case HILS_CALL_PREFIX_DECODE: return decode_plan(p, rows, 0, other, true, false).bytes;
    case HILS_CALL_CACHE_EVICT: return kSinkStatusBytes;
    default: return 0;
    }
}

}  // namespace hils

using namespace hils;

extern "C" {

int hils_sink_prefill(const hils_params *p, int A, hils_ctensor Q, int Lq, hils_ctensor K, hils_ctensor V, int N,
                      hils_tensor O, float *lse, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, A, Lq, &scale));
    if (N < Lq) return HILS_ERR_INVALID_ARG;
    HILS_TRY(check_tokens(N));
    HILS_TRY(check(Q, Lq, p));
    HILS_TRY(check(K, N, p));
    HILS_TRY(check(V, N, p));
    HILS_TRY(check_out(O, p->H, Lq, p));
    HILS_TRY(check_array(lse, 0));
    const int64_t rows = (int64_t)p->B * p->H * Lq;
    if (rows == 0) return HILS_OK;
    HILS_TRY(check_workspace(workspace, ws_bytes, sink_ws_bytes(p, HILS_CALL_SINK_PREFILL, Lq, A)));
    SinkArgs a{};
    a.Q = view(Q);
    a.K = view(K);
    a.V = view(V);
    a.O = mut(O);
    a.lse = lse;
    a.B = p->B;
    a.H = p->H;
    a.G = groups(p);
    a.Lq = Lq;
    a.N = N;
    a.W = clip(p->W, N);
    a.A = clip(A, N);
    a.scale = scale;
    a.wait_ns = work_wait_ns(p->flags);
    Carve ws{static_cast<uint8_t *>(workspace)};
    a.status = ws.take<uint32_t>(kSinkStatusBytes / 4);
    const int64_t keys = prefill_keys(p, A, Lq);
    a.splits = sink_prefill_splits(p->dtype, a.B, a.H, a.G, Lq, keys < N ? keys : N, device_sm_count());
    if (a.splits > 1) {
        a.slots = a.splits;
        a.part_o = ws.take<float>((size_t)rows * a.slots * p->d);
        a.part_lse = ws.take<float>((size_t)rows * a.slots);
    }
    HILS_TRY(forward(p, a, stream));
    if (a.splits == 1) return HILS_OK;
    return launch_sink_combine(p->dtype, p->d, {a.part_o, a.part_lse, rows, a.slots, a.H, Lq, a.O, lse}, stream);
}

int hils_sink_prefill_backward(const hils_params *p, int A, hils_ctensor Q, hils_ctensor K, hils_ctensor V, int N,
                               hils_ctensor O, const float *lse, hils_ctensor dO, hils_tensor dQ, hils_tensor dK,
                               hils_tensor dV, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, A, N, &scale));
    HILS_TRY(check_tokens(N));
    HILS_TRY(check(Q, N, p));
    HILS_TRY(check(K, N, p));
    HILS_TRY(check(V, N, p));
    HILS_TRY(check(O, N, p));
    HILS_TRY(check(dO, N, p));
    HILS_TRY(check_out(dQ, p->H, N, p));
    HILS_TRY(check_out(dK, p->H / groups(p), N, p));
    HILS_TRY(check_out(dV, p->H / groups(p), N, p));
    const int64_t rows = (int64_t)p->B * p->H * N;
    HILS_TRY(check_array(lse, rows));
    if (rows == 0) return HILS_OK;
    HILS_TRY(check_workspace(workspace, ws_bytes, sink_ws_bytes(p, HILS_CALL_SINK_BACKWARD, N, A)));
    SinkBwdArgs a{};
    const size_t part = key_ws(p, N, N, A, 2 * p->d, &a);
    a.Q = view(Q);
    a.K = view(K);
    a.V = view(V);
    a.O = view(O);
    a.dO = view(dO);
    a.dQ = mut(dQ);
    a.dK = mut(dK);
    a.dV = mut(dV);
    a.lse = lse;
    a.Lq = N;
    a.N = N;
    a.W = clip(p->W, N);
    a.A = clip(A, N);
    a.scale = scale;
    a.wait_ns = work_wait_ns(p->flags);
    Carve ws{static_cast<uint8_t *>(workspace)};
    a.status = ws.take<uint32_t>(kSinkStatusBytes / 4);
    float *Dv = ws.take<float>(rows);
    a.Dv = Dv;
    a.part = ws.take<float>(part / 4);
    HILS_TRY(launch_sink_dot(p->dtype, p->d, a, Dv, stream));
    hils_status st;
    if (!launch_sink_backward_tc(p->dtype, p->d, a, stream, &st)) st = launch_sink_backward_general(p->dtype, p->d, a, stream);
    HILS_TRY(st);
    return launch_sink_reduce(p->dtype, p->d, a, false, stream);
}

int hils_sink_weights(const hils_params *p, int A, hils_ctensor Q, int Lq, hils_ctensor K, int N, const float *lse,
                      const float *acc, float *acc_out, int T, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, A, Lq, &scale));
    if (N < Lq || T < N) return HILS_ERR_INVALID_ARG;
    HILS_TRY(check_tokens(N));
    HILS_TRY(check(Q, Lq, p));
    HILS_TRY(check(K, N, p));
    const int64_t rows = (int64_t)p->B * p->H * Lq;
    HILS_TRY(check_array(lse, rows));
    HILS_TRY(check_array(acc, rows > 0));
    HILS_TRY(check_array(acc_out, rows > 0));
    if (rows == 0) return HILS_OK;
    SinkBwdArgs a{};
    const size_t part = key_ws(p, Lq, N, A, 1, &a);
    HILS_TRY(check_workspace(workspace, ws_bytes, kSinkStatusBytes + part));
    a.Q = view(Q);
    a.K = view(K);
    a.lse = lse;
    a.acc = acc;
    a.acc_out = acc_out;
    a.T = T;
    a.Lq = Lq;
    a.N = N;
    a.W = clip(p->W, N);
    a.A = clip(A, N);
    a.scale = scale;
    a.wait_ns = work_wait_ns(p->flags);
    Carve ws{static_cast<uint8_t *>(workspace)};
    a.status = ws.take<uint32_t>(kSinkStatusBytes / 4);
    a.part = ws.take<float>(part / 4);
    hils_status st;
    if (!launch_sink_weights_tc(p->dtype, p->d, a, stream, &st)) st = launch_sink_weights_general(p->dtype, p->d, a, stream);
    HILS_TRY(st);
    return launch_sink_reduce(p->dtype, p->d, a, true, stream);
}

int hils_sink_decode(const hils_params *p, int A, hils_ctensor Q, hils_ctensor Kc, hils_ctensor Vc, int T,
                     const int32_t *cache_len, hils_tensor O, float *lse, const float *acc, float *acc_out,
                     void *workspace, size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, A, 1, &scale));
    if (T < 0 || (acc == nullptr) != (acc_out == nullptr)) return HILS_ERR_INVALID_ARG;
    HILS_TRY(check_tokens(T));
    HILS_TRY(check(Q, 1, p));
    HILS_TRY(check(Kc, T, p));
    HILS_TRY(check(Vc, T, p));
    HILS_TRY(check_out(O, p->H, 1, p));
    HILS_TRY(check_array(cache_len, p->B));
    HILS_TRY(check_array(lse, 0));
    HILS_TRY(check_array(acc, 0));
    HILS_TRY(check_array(acc_out, 0));
    const int64_t rows = (int64_t)p->B * p->H;
    if (rows == 0) return HILS_OK;
    const DecodePlan plan = decode_plan(p, T, A, 0, false, acc != nullptr);
    HILS_TRY(check_workspace(workspace, ws_bytes, plan.bytes));
    SinkDecodeArgs a{};
    a.Q = view(Q);
    a.K = view(Kc);
    a.V = view(Vc);
    a.O = mut(O);
    a.cache_len = cache_len;
    a.B = p->B;
    a.H = p->H;
    a.G = groups(p);
    a.T = T;
    a.W = clip(p->W, T);
    a.A = clip(A, T);
    a.scale = scale;
    Carve ws{static_cast<uint8_t *>(workspace)};
    decode_space(p, plan, ws, lse, &a);
    if (acc) {
        a.logits = ws.take<float>((size_t)rows * plan.keys);
        a.logit_stride = plan.keys;
    }
    // few slots a row: a second launch would cost more than sharing the rows saves
    a.whole = plan.keys <= kSinkWholeRow;
    HILS_TRY(launch_sink_decode(p->dtype, p->d, a, plan.ctas, stream));
    return acc ? launch_sink_decode_acc(a, a.lse, acc, acc_out, stream) : HILS_OK;
}

int hils_prefix_decode(const hils_params *p, hils_ctensor Q, hils_ctensor Kp, hils_ctensor Vp, int P, hils_ctensor Kc,
                       hils_ctensor Vc, int T, const int32_t *cache_len, hils_tensor O, float *lse, void *workspace,
                       size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, 0, 1, &scale));
    if (P < 0 || T < 0) return HILS_ERR_INVALID_ARG;
    HILS_TRY(check_tokens((int64_t)P + T));
    HILS_TRY(check(Q, 1, p));
    HILS_TRY(check(Kp, P, p));
    HILS_TRY(check(Vp, P, p));
    HILS_TRY(check(Kc, T, p));
    HILS_TRY(check(Vc, T, p));
    HILS_TRY(check_out(O, p->H, 1, p));
    HILS_TRY(check_array(cache_len, p->B));
    HILS_TRY(check_array(lse, 0));
    const int64_t rows = (int64_t)p->B * p->H;
    if (rows == 0) return HILS_OK;
    const DecodePlan plan = decode_plan(p, T, 0, P, true, false);
    HILS_TRY(check_workspace(workspace, ws_bytes, plan.bytes));
    SinkDecodeArgs s{};
    s.Q = view(Q);
    s.K = view(Kc);
    s.V = view(Vc);
    s.O = mut(O);
    s.cache_len = cache_len;
    s.B = p->B;
    s.H = p->H;
    s.G = groups(p);
    s.T = T;
    s.W = T;
    s.A = 0;
    s.scale = scale;
    Carve ws{static_cast<uint8_t *>(workspace)};
    decode_space(p, plan, ws, lse, &s);
    SinkArgs a{};
    a.status = static_cast<uint32_t *>(workspace);
    a.Q = s.Q;
    a.K = view(Kp);
    a.V = view(Vp);
    a.B = p->B;
    a.H = p->H;
    a.G = s.G;
    a.Lq = 1;
    a.N = P;
    a.W = P;
    a.A = 0;
    a.scale = scale;
    a.prefix = 1;
    a.splits = a.slots = s.slots;
    a.part_o = const_cast<float *>(s.part_o);
    a.part_lse = const_cast<float *>(s.part_lse);
    a.wait_ns = work_wait_ns(p->flags);
    if (plan.prefix_splits == 0) {  // each sequence reads the prefix before its own cache
        s.Kp = a.K;
        s.Vp = a.V;
        s.P = P;
        s.whole = (int64_t)P + T <= kSinkWholeRow;
    } else {
        s.whole = T <= kSinkWholeRow;
        HILS_TRY(forward(p, a, stream));
    }
    return launch_sink_decode(p->dtype, p->d, s, plan.ctas, stream);
}

int hils_cache_evict(const hils_params *p, int A, int budget, hils_ctensor K, hils_ctensor V, int T, const float *acc,
                     const int32_t *cache_len, hils_tensor Kout, hils_tensor Vout, float *acc_out, int32_t *idx,
                     int32_t *len_out, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    float scale;
    HILS_TRY(check_sink(p, A, 0, &scale));
    if (budget < 0 || T < 0 || (int64_t)A + p->W > budget) return HILS_ERR_INVALID_ARG;
    HILS_TRY(check_tokens(T > budget ? T : budget));
    if ((int64_t)p->B * p->H * budget > 0x7fffffffll) return HILS_ERR_INVALID_ARG;
    const int Hk = p->H / groups(p);
    const int64_t out = (int64_t)p->B * Hk * budget;
    HILS_TRY(check(K, T, p));
    HILS_TRY(check(V, T, p));
    HILS_TRY(check_out(Kout, Hk, budget, p));
    HILS_TRY(check_out(Vout, Hk, budget, p));
    HILS_TRY(check_array(acc, (int64_t)p->B * Hk * T));
    HILS_TRY(check_array(cache_len, p->B));
    HILS_TRY(check_array(acc_out, out));
    HILS_TRY(check_array(idx, out));
    HILS_TRY(check_array(len_out, p->B));
    if (p->B == 0) return HILS_OK;
    // the kept rows move to other places of their sequence: nothing that is read may be written
    if (out > 0 && T > 0) {
        uintptr_t r[3][2], w[3][2];
        span_of(K, p->B, Hk, T, p, &r[0][0], &r[0][1]);
        span_of(V, p->B, Hk, T, p, &r[1][0], &r[1][1]);
        r[2][0] = (uintptr_t)acc;
        r[2][1] = r[2][0] + (uintptr_t)p->B * Hk * T * 4;
        span_of(Kout, p->B, Hk, budget, p, &w[0][0], &w[0][1]);
        span_of(Vout, p->B, Hk, budget, p, &w[1][0], &w[1][1]);
        w[2][0] = (uintptr_t)acc_out;
        w[2][1] = w[2][0] + (uintptr_t)out * 4;
        for (int i = 0; i < 3; ++i)
            for (int j = 0; j < 3; ++j)
                if (!disjoint(r[i][0], r[i][1], w[j][0], w[j][1])) return HILS_ERR_INVALID_ARG;
    }
    HILS_TRY(check_workspace(workspace, ws_bytes, sink_ws_bytes(p, HILS_CALL_CACHE_EVICT, T, budget)));
    EvictArgs a{};
    a.K = view(K);
    a.V = view(V);
    a.Kout = mut(Kout);
    a.Vout = mut(Vout);
    a.acc = acc;
    a.cache_len = cache_len;
    a.acc_out = acc_out;
    a.idx = idx;
    a.len_out = len_out;
    a.B = p->B;
    a.Hk = Hk;
    a.T = T;
    a.budget = budget;
    a.W = p->W;
    a.A = A;
    return launch_cache_evict(p->dtype, p->d, a, stream);
}

}  // extern "C"
