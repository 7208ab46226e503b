// Arguments, work division and launchers of the window-and-sink attention (prefill, its
// backward, one-token decode, accumulated weights), the shared-prefix decode and the
// cache eviction.
//
// A query at position t sees V(t) = { j <= t : j < A or j > t - W }: the first A tokens
// (the sinks) and the W newest up to its own. With s_tj = scale q_t . k_j,
//   lse_t = log sum_{j in V(t)} exp(s_tj),  p_tj = exp(s_tj - lse_t),  o_t = sum_j p_tj v_j
// (an empty V(t): o = 0, lse = -inf). Backward, from O and lse:
//   D_t = dO_t . o_t,  ds_tj = scale p_tj (dO_t . v_j - D_t),
//   dQ = ds K,  dK = ds^T Q,  dV = p^T dO,  the last two summed over a group's heads.
#pragma once
#include "hils_internal.cuh"

namespace hils {

// Launches a kernel; `early`: it may be scheduled while the kernel before it on the stream ends,
// and calls pdl_wait() before it touches what that one writes. A CTA of each grid at least waits:
// a grid is then never over before the one that it follows.
template <typename... P, typename... A>
hils_status sink_launch(bool early, void (*kernel)(P...), int64_t grid, int threads, int smem, cudaStream_t s, const A &...args) {
    if (grid <= 0) return HILS_OK;
    if (grid > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return record_cuda_error(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// ------------------------------------------------------------------ forward

// One call's rows over one key range. Prefill: row (b, h, i) at position N - Lq + i. A
// shared prefix (`prefix`): the rows of every sequence, (b, h), over all N keys of key
// batch 0 (W = N, A = 0, Lq = 1).
struct SinkArgs {
    View Q, K, V;
    MutView O;
    float *lse;              // [B, H, Lq] or null
    int B, H, G, Lq, N, W, A;  // W, A <= N
    float scale;
    int prefix = 0;
    // split > 1 (or prefix): each row's partial results of key split s go to slot s of
    // `slots`: part_o [rows][slots][d] (normalised), part_lse [rows][slots] (natural log)
    int splits = 1, slots = 0;
    float *part_o = nullptr, *part_lse = nullptr;
    uint32_t *status = nullptr;
    long long wait_ns = kWaitLimitNs;
};

// The key tiles of one row tile: sinks [0, sinks) in ns tiles, then keys [lo, hi) in nw.
struct SinkSpan {
    int sinks, ns, lo, hi, nw;
};

// Rows at positions t0 .. t1, key tiles of `kt` keys. The window's tiles begin at its
// first visible key exactly, so that a slot that no row sees is never part of a tile.
__host__ __device__ inline SinkSpan sink_span(int t0, int t1, int W, int A, int kt) {
    SinkSpan s;
    s.hi = t1 + 1;
    s.lo = W > 0 ? (t0 - W + 1 > 0 ? t0 - W + 1 : 0) : s.hi;
    s.sinks = A < s.lo ? A : s.lo;
    s.ns = (s.sinks + kt - 1) / kt;
    s.nw = W > 0 ? (s.hi - s.lo + kt - 1) / kt : 0;
    return s;
}

// Tokens of a call (of the prefix and the own cache together): positions and tiles of them, and
// what rounds up to a tile, stay within int.
constexpr int64_t kSinkMostTokens = 0x7fffffffll - 1024;

constexpr size_t kSinkStatusBytes = 256;
inline size_t sink_align(size_t n) { return (n + 255) & ~(size_t)255; }

// Query heads packed into one row tile: the largest power of two <= 8 that divides G.
inline int sink_pack(int G) {
    int P = 1;
    while (P < 8 && G % (2 * P) == 0) P *= 2;
    return P;
}
// Key splits of a prefill call whose row tiles alone would leave most SMs idle. `keys`: the
// longest key range of a row tile (for the workspace's size, a bound of it). bf16: 256-row
// tiles, one an SM, 512 keys or more each; float32: 64-row tiles, three an SM, and a 64-key
// tile costs 7 us there, so that each may be a split (47 -> 16 us at 12 heads, 333 rows, W 200).
inline int sink_prefill_splits(hils_dtype dt, int B, int H, int G, int Lq, int64_t keys, int sms) {
    const bool f32 = dt == HILS_F32;
    const int P = f32 ? 1 : sink_pack(G), rows = f32 ? 64 : 256;
    const int64_t tiles = (int64_t)B * (H / P) * (((int64_t)Lq * P + rows - 1) / rows);
    const int64_t fill = tiles > 0 ? (f32 ? 3 : 1) * sms / tiles : 1;
    const int64_t most = f32 ? (keys + 63) / 64 : keys / 512;
    const int64_t s = fill < most ? fill : most;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}
// Key splits of a shared prefix of P tokens: two for each CTA of one wave over the row tiles
// (float32: 64-row tiles, three an SM, a 64-key tile each or more).
inline int sink_prefix_splits(hils_dtype dt, int B, int Hk, int G, int P, int sms) {
    const bool f32 = dt == HILS_F32;
    const int nb = (f32 ? 64 : 128) / G;
    const int64_t tiles = (int64_t)Hk * ((B + nb - 1) / nb);
    const int64_t fill = f32 ? (tiles > 0 ? 3 * sms / tiles : 1) : tiles > 0 && tiles < sms ? 2 * (sms / tiles) : 2;
    const int64_t most = f32 ? P / 64 : P / 256;
    const int64_t s = fill < most ? fill : most;
    return (int)(s < 1 ? 1 : s > 128 ? 128 : s);
}
// Whether each sequence reads a shared prefix by itself (from L2, after the first) instead of
// the prefix's own pass over all of them and a join. bf16 (d = 128): 19 against 24 us with 4 of
// 4096 tokens and 8 heads, 25.7 each at 8192, 37 against 43 us with 2 of 32K, 58 against 45 with 4;
// float32 is bound by its products, of which the pass spends 64 rows' a tile however few there
// are: 59 against 111 us with 8 rows, 62 against 45 with 16; small ones by their launches.
inline bool sink_prefix_direct(hils_dtype dt, int d, int B, int H, int G, int64_t P) {
    if (dt == HILS_F32) return B == 1 || (int64_t)B * G <= 12 || (int64_t)B * H * P * d <= (8ll << 20);
    return B <= 2 || (int64_t)B * (H / G) * P * d <= (24ll << 20);
}
inline size_t sink_part_bytes(int64_t rows, int slots, int d) {
    return sink_align((size_t)rows * slots * d * 4) + sink_align((size_t)rows * slots * 4);
}

hils_status launch_sink_forward_general(hils_dtype dt, int d, const SinkArgs &a, cudaStream_t s);
// On the tensor cores; false, and nothing launched, for a type or strides that it cannot take.
bool launch_sink_forward_tc(hils_dtype dt, int d, const SinkArgs &a, cudaStream_t s, hils_status *st);

// O and lse of every row from its partials: weights exp(lse_s - max) over the row's slots
// (slots with lse = -inf are skipped).
struct SinkCombineArgs {
    const float *part_o, *part_lse;
    int64_t rows;
    int slots, H, Lq;  // row = (b * H + h) * Lq + i
    MutView O;
    float *lse;
};
hils_status launch_sink_combine(hils_dtype dt, int d, const SinkCombineArgs &a, cudaStream_t s);

// ------------------------------------------------------------------ backward and weights

// Key-major items: a block of `keys` keys (kSinkKeys; 256 for bf16 weights) of one (b,
// key-value head) and a segment of its steps. Step s covers query rows [i0 + kSinkRows (s % tiles), ..) of group head
// s / tiles, where [i0, i1) are the rows that see a key of the block.
constexpr int kSinkKeys = 128, kSinkRows = 128;

struct SinkBwdArgs {
    View Q, K, V, O, dO;
    MutView dQ, dK, dV;
    const float *lse;       // [B, H, Lq]
    const float *Dv;        // [B, H, Lq] (backward)
    const float *acc;       // weights: [B, Hk, T]
    float *acc_out;
    int64_t T;
    int B, H, G, Lq, N, W, A;
    float scale;
    // key blocks [0, nsink) are cut into seg_s segments each, the others into seg_w
    int nblk, nsink, seg_s, seg_w, keys;
    float *part;            // partial sums of blocks with more than one segment
    uint32_t *status = nullptr;
    long long wait_ns = kWaitLimitNs;
};

// Query rows [i0, i1) that see a key of block [j0, j0 + keys).
__host__ __device__ inline void sink_rows_of_block(const SinkBwdArgs &a, int j0, int keys, int *i0, int *i1) {
    const int off = a.N - a.Lq;
    *i0 = j0 > off ? j0 - off : 0;
    if (j0 < a.A) {
        *i1 = a.Lq;
    } else if (a.W > 0) {
        const int64_t e = (int64_t)j0 + keys - 1 + a.W - off;
        *i1 = e < a.Lq ? (int)(e > 0 ? e : 0) : a.Lq;
    } else {
        *i1 = *i0;
    }
    if (*i1 < *i0) *i1 = *i0;
}

// The division of the key blocks: four items for every SM, at least eight steps each
// (float32: one 64-row tile, which costs more than its share of the reduction).
inline void sink_key_plan(hils_dtype dt, int B, int Hk, int G, int Lq, int N, int W, int A, int keys, int sms, SinkBwdArgs *a) {
    const int step = dt == HILS_F32 ? 64 : kSinkRows, least = dt == HILS_F32 ? 1 : 8;
    a->keys = keys;
    a->nblk = (N + keys - 1) / keys;
    a->nsink = (A + keys - 1) / keys;
    if (a->nsink > a->nblk) a->nsink = a->nblk;
    auto segments = [&](int blocks, int64_t rows) {
        const int64_t steps = (int64_t)G * ((rows + step - 1) / step);
        const int64_t items = (int64_t)B * Hk * blocks, fill = items > 0 ? 4 * sms / items : 1;
        int64_t s = steps / least < fill ? steps / least : fill;
        return (int)(s < 1 ? 1 : s);
    };
    a->seg_s = segments(a->nsink, Lq);
    const int64_t wr = (int64_t)W + keys;
    a->seg_w = segments(a->nblk - a->nsink, wr < Lq ? wr : Lq);
}
inline int64_t sink_key_items(const SinkBwdArgs &a) {
    return (int64_t)a.nsink * a.seg_s + (int64_t)(a.nblk - a.nsink) * a.seg_w;
}
// Floats of partial sums (`per_key` of each key: 2 d for dK and dV, 1 for weights).
inline size_t sink_key_part_floats(const SinkBwdArgs &a, int per_key) {
    if (a.seg_s <= 1 && a.seg_w <= 1) return 0;
    return (size_t)a.B * (a.H / a.G) * sink_key_items(a) * a.keys * per_key;
}

struct SinkItem {
    int blk, seg, nseg;
};
__host__ __device__ inline SinkItem sink_item(const SinkBwdArgs &a, int x) {
    SinkItem it;
    const int ns = a.nsink * a.seg_s;
    it.nseg = x < ns ? a.seg_s : a.seg_w;
    const int y = x < ns ? x : x - ns, q = it.nseg > 1 ? y / it.nseg : y;
    it.blk = x < ns ? q : a.nsink + q;
    it.seg = y - q * it.nseg;
    return it;
}

hils_status launch_sink_dot(hils_dtype dt, int d, const SinkBwdArgs &a, float *Dv, cudaStream_t s);
hils_status launch_sink_backward_general(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s);
// dQ, and dK and dV or their partials, on the tensor cores; false, and nothing launched, for
// a type or strides that it cannot take.
bool launch_sink_backward_tc(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s, hils_status *st);
bool launch_sink_weights_tc(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s, hils_status *st);
hils_status launch_sink_weights_general(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s);
// Sums the segments' partials in segment order into dK and dV, or acc_out.
hils_status launch_sink_reduce(hils_dtype dt, int d, const SinkBwdArgs &a, bool weights, cudaStream_t s);

// ------------------------------------------------------------------ decode

constexpr int kSinkWholeRow = 1024;  // longest row that one CTA takes by itself
struct SinkDecodeArgs {
    View Q, K, V;
    MutView O;
    float *lse;                // [B, H]
    const int32_t *cache_len;  // [B]
    int B, H, G, T, W, A;      // W, A <= T
    float scale;
    View Kp, Vp;               // P shared tokens before each sequence's own, read per sequence
    int P = 0;
    bool whole = false;        // no row is shared between CTAs: one launch, nothing to join
    // partial results of rows (b, h) from another kernel: part_o [rows][slots][d], part_lse [rows][slots]
    const float *part_o, *part_lse;
    int slots = 0;
    // this kernel's own: of CTA c's share of row r = (b, hk), head g, at (c + r) * G + g (a
    // staircase: no two pairs (c, r) that meet have the same sum)
    float *seg_o, *seg_lse;
    float *logits;             // with acc: [B, H, logit_stride] scaled logits in log2 units, by visible order
    int64_t logit_stride;
};
// The slots that a sequence of n tokens sees: [0, sinks), then [lo, n).
__host__ __device__ inline void sink_visible(int n, int W, int A, int *sinks, int *lo) {
    *lo = n > W ? n - W : 0;
    *sinks = A < *lo ? A : *lo;
}
int sink_decode_ctas(hils_dtype dt, int B, int Hk, int64_t keys, int sms);
hils_status launch_sink_decode(hils_dtype dt, int d, const SinkDecodeArgs &a, int ctas, cudaStream_t s);
// acc_out[b, hk, j] = acc[b, hk, j] + sum over the group's heads of p_j, for the visible
// slots j, from the call's logits and the rows' lse [B, H].
hils_status launch_sink_decode_acc(const SinkDecodeArgs &a, const float *lse, const float *acc, float *acc_out,
                                   cudaStream_t s);

// ------------------------------------------------------------------ eviction

struct EvictArgs {
    View K, V;
    MutView Kout, Vout;
    const float *acc;          // [B, Hk, T]
    const int32_t *cache_len;  // [B]
    float *acc_out;            // [B, Hk, budget]
    int32_t *idx;              // [B, Hk, budget]
    int32_t *len_out;          // [B]
    int B, Hk, T, budget, W, A;
};
hils_status launch_cache_evict(hils_dtype dt, int d, const EvictArgs &a, cudaStream_t s);

// Workspace sizes of the calls above (0: invalid parameters or another call).
size_t sink_ws_bytes(const hils_params *p, int call, int rows, int other);

}  // namespace hils
