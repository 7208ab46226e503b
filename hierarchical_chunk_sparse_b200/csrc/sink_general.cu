// Window-and-sink attention on the CUDA cores: prefill, shared prefix, backward and
// accumulated weights (formulas in sink_common.cuh). 64 x 64 tiles of scores, 256 threads
// with 4 x 4 of them each; every product and sum in float32, for float32 tensors and for bf16
// whose strides or scale the tensor-core kernels do not take. A tile's two products take 8192
// cycles of an SM at d = 128; small calls are bound by the latency of one tile (7 us
// at d = 64) and the launches, which is why their rows and keys are split to a tile a CTA: 2 x 6
// heads of 333 queries, W 200, d = 64 take 28 us with the binding, the backward of 2 x 4 heads of
// 509 tokens 49. Where products bind, 8 heads of 2048 causal tokens at d = 64 and 128: forward 338
// and 452 us (58 and 115 by their FMAs), backward 542 and 996 (144 and 289), weights 110 and 187 (29
// and 58); the FMA pipe is 47 to 51 % busy at d = 128, and its warps wait on shared-memory reads.
#include "sink_common.cuh"

namespace hils {
namespace {

constexpr int kT = 64;        // rows and keys per tile
constexpr int kThr = 256;
constexpr int kPS = kT + 4;   // row stride of the probability tiles in shared memory

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// 16 lanes' maximum / sum (the threads that share a row)
__device__ __forceinline__ float max16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Rows r of [64][D + 4] float tiles from element pointers row_ptr(r) (null: zeros): `fetch` has
// all of a thread's loads in flight (one after another they took half of a tile's time), `put`
// stores them.
template <typename T, int D>
struct TileLoad {
    static constexpr int kV = Vec<T>::kN, kU = D / kV, kN = kT * kU / kThr;  // 16-byte units of a row, of a thread
    uint4 v[kN];
    template <typename F>
    __device__ __forceinline__ void fetch(F row_ptr) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = threadIdx.x + i * kThr;
            const T *p = row_ptr(e / kU);
            v[i] = p ? __ldg(reinterpret_cast<const uint4 *>(p) + e % kU) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void put(float *dst) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = threadIdx.x + i * kThr;
            float f[kV];
            widen(v[i], f, T());
            float *d = dst + (e / kU) * (D + 4) + (e % kU) * kV;
#pragma unroll
            for (int k = 0; k < kV; k += 4) *reinterpret_cast<float4 *>(d + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
    }
};

// acc[r][c] = X row (4 ty + r) . Y row (tx + 16 c) over D
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float *X, const float *Y, int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
#pragma unroll 4
    for (int x = 0; x < D; x += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4 *>(X + (4 * ty + r) * (D + 4) + x);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4 *>(Y + (tx + 16 * c) * (D + 4) + x);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[r][c] = fmaf(a[r].x, b[c].x, acc[r][c]);
                acc[r][c] = fmaf(a[r].y, b[c].y, acc[r][c]);
                acc[r][c] = fmaf(a[r].z, b[c].z, acc[r][c]);
                acc[r][c] = fmaf(a[r].w, b[c].w, acc[r][c]);
            }
    }
}

// o[r][4 u + i] += sum_k P[4 ty + r][k] Y[k][64 u + 4 tx + i]
template <int D>
__device__ __forceinline__ void add_product(float (&o)[4][D / 16], const float *P, const float *Y, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < kT; ++k) {
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = P[(4 * ty + r) * kPS + k];
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float4 y = *reinterpret_cast<const float4 *>(Y + k * (D + 4) + 64 * u + 4 * tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                o[r][4 * u + 0] = fmaf(p[r], y.x, o[r][4 * u + 0]);
                o[r][4 * u + 1] = fmaf(p[r], y.y, o[r][4 * u + 1]);
                o[r][4 * u + 2] = fmaf(p[r], y.z, o[r][4 * u + 2]);
                o[r][4 * u + 3] = fmaf(p[r], y.w, o[r][4 * u + 3]);
            }
        }
    }
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16 *p, float a, float b, float c, float d) {
    uint2 v;
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    v.x = *reinterpret_cast<const uint32_t *>(&x);
    v.y = *reinterpret_cast<const uint32_t *>(&y);
    *reinterpret_cast<uint2 *>(p) = v;
}

template <int D>
constexpr int fwd_smem() {
    return (3 * kT * (D + 4) + kT * kPS) * 4;
}

// One CTA per (row tile, split): online softmax over the tile's keys. kPerSm CTAs an SM: three
// (d = 64; two more tiles' loads and chains in between) if there are more CTAs than SMs, 31 -> 28 us
// for 432 of a tile each; with one, the registers for deeper unrolling, 17 -> 15 us for 6.
template <typename T, int D, int kPerSm>
__global__ void __launch_bounds__(kThr, kPerSm) sink_fwd_kernel(SinkArgs a, int tiles) {
    extern __shared__ float sm[];
    float *Qs = sm, *Ks = Qs + kT * (D + 4), *Vs = Ks + kT * (D + 4), *Ps = Vs + kT * (D + 4);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int Hk = a.H / a.G;
    int x = blockIdx.x;
    const int split = x % a.splits;
    x /= a.splits;
    const int tile = a.prefix ? x % tiles : tiles - 1 - x % tiles;  // latest rows (most keys) first
    x /= tiles;
    const int nb = a.prefix ? kT / a.G : 1;
    const int h = a.prefix ? 0 : x % a.H, b = a.prefix ? 0 : x / a.H;
    const int hk = a.prefix ? x : h / a.G;
    // row r of this tile: its query, its place among all rows, its position (-1: no row)
    auto row = [&](int r, const T **q, int64_t *place) -> int {
        int bb = b, hh = h, i = tile * kT + r;
        if (a.prefix) {
            bb = tile * nb + r / a.G;
            hh = hk * a.G + r % a.G;
            i = 0;
            if (r >= nb * a.G || bb >= a.B) return -1;
        } else if (i >= a.Lq) {
            return -1;
        }
        *q = static_cast<const T *>(a.Q.ptr) + bb * a.Q.sb + hh * a.Q.sh + i * a.Q.st;
        *place = ((int64_t)bb * a.H + hh) * a.Lq + i;
        return a.prefix ? max(a.N - 1, 0) : a.N - a.Lq + i;
    };
    const T *Kb = static_cast<const T *>(a.K.ptr) + b * a.K.sb + hk * a.K.sh;
    const T *Vb = static_cast<const T *>(a.V.ptr) + b * a.V.sb + hk * a.V.sh;
    const int t0 = a.prefix ? a.N - 1 : a.N - a.Lq + tile * kT;
    const int t1 = a.prefix ? a.N - 1 : min(a.N - 1, t0 + kT - 1);
    SinkSpan sp = sink_span(t0, t1, a.W, a.A, kT);
    if (a.prefix) sp = {0, 0, 0, a.N, (a.N + kT - 1) / kT};
    const int nt = sp.ns + sp.nw;
    const int i0 = (int)((int64_t)nt * split / a.splits), i1 = (int)((int64_t)nt * (split + 1) / a.splits);

    TileLoad<T, D> first;
    first.fetch([&](int r) -> const T * {
        const T *q = nullptr;
        int64_t place;
        return row(r, &q, &place) >= 0 ? q : nullptr;
    });
    int tr[4];
    int64_t place[4];
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const T *q;
        place[r] = 0;
        tr[r] = row(4 * ty + r, &q, &place[r]);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[r][c] = 0.f;
    }
    const float scale2 = a.scale * 1.4426950408889634f;
    for (int i = i0; i < i1; ++i) {
        const bool sink = i < sp.ns;
        const int k0 = sink ? i * kT : sp.lo + (i - sp.ns) * kT;
        const int end = sink ? sp.sinks : sp.hi;
        TileLoad<T, D> lk, lv;
        lk.fetch([&](int r) -> const T * { return k0 + r < end ? Kb + (int64_t)(k0 + r) * a.K.st : nullptr; });
        lv.fetch([&](int r) -> const T * { return k0 + r < end ? Vb + (int64_t)(k0 + r) * a.V.st : nullptr; });
        __syncthreads();
        if (i == i0) first.put(Qs);
        lk.put(Ks);
        lv.put(Vs);
        __syncthreads();
        float s[4][4];
        dot_tile<D>(s, Qs, Ks, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float mt = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = k0 + tx + 16 * c;
                const bool in = j < end && j <= tr[r] && (sink || j < a.A || j > tr[r] - a.W);
                s[r][c] = in ? s[r][c] * scale2 : -INFINITY;
                mt = fmaxf(mt, s[r][c]);
            }
            mt = fmaxf(max16(mt), m[r]);
            const float f = mt == -INFINITY ? 1.f : exp2f(m[r] - mt);
            const float ref = mt == -INFINITY ? 0.f : mt;
            float z = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = exp2f(s[r][c] - ref);
                z += p;
                Ps[(4 * ty + r) * kPS + tx + 16 * c] = p;
            }
            l[r] = l[r] * f + sum16(z);
            m[r] = mt;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[r][c] *= f;
        }
        __syncwarp();  // a row's probabilities are written and read by one half-warp
        add_product<D>(o, Ps, Vs, ty, tx);
    }
    const bool part = a.part_o != nullptr;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (tr[r] < 0) continue;
        const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
        const float lse = l[r] > 0.f ? (m[r] + log2f(l[r])) * 0.6931471805599453f : -INFINITY;
        if (part) {
            float *dst = a.part_o + (place[r] * a.slots + split) * D;
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
                store4(dst + 64 * u + 4 * tx, o[r][4 * u] * inv, o[r][4 * u + 1] * inv, o[r][4 * u + 2] * inv, o[r][4 * u + 3] * inv);
            if (tx == 0) a.part_lse[place[r] * a.slots + split] = lse;
        } else {
            const int64_t i = place[r] % a.Lq, bh = place[r] / a.Lq;
            T *dst = static_cast<T *>(a.O.ptr) + (bh / a.H) * a.O.sb + (bh % a.H) * a.O.sh + i * a.O.st;
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
                store4(dst + 64 * u + 4 * tx, o[r][4 * u] * inv, o[r][4 * u + 1] * inv, o[r][4 * u + 2] * inv, o[r][4 * u + 3] * inv);
            if (tx == 0 && a.lse) a.lse[place[r]] = lse;
        }
    }
}

// D_i = dO_i . o_i: D / kV lanes a row, four rounds of rows a warp in flight (bound by HBM: 27 us,
// 5 TB/s, for 262144 rows of d = 128 in bf16).
template <typename T, int D>
__global__ void __launch_bounds__(256) sink_dot_kernel(SinkBwdArgs a, float *Dv) {
    constexpr int kL = D / Vec<T>::kN, kPer = 32 / kL, kRounds = 4;  // lanes of a row, rows of a round
    const int64_t rows = (int64_t)a.B * a.H * a.Lq;
    const int64_t r0 = ((int64_t)blockIdx.x * 8 + threadIdx.x / 32) * (kPer * kRounds) + threadIdx.x % 32 / kL;
    const int u = threadIdx.x % kL;
    uint4 x[kRounds], y[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int64_t row = min(r0 + k * kPer, rows - 1);
        const int64_t bh = row / a.Lq, i = row - bh * a.Lq;
        const int b = (int)bh / a.H, h = (int)bh - b * a.H;
        x[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.O.ptr) + b * a.O.sb + h * a.O.sh + i * a.O.st) + u);
        y[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.dO.ptr) + b * a.dO.sb + h * a.dO.sh + i * a.dO.st) + u);
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        float s = dot16<T>(x[k], y[k], 0.f);
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        if (u == 0 && r0 + k * kPer < rows) Dv[r0 + k * kPer] = s;
    }
}

// Whether any query row sees key j: the slots of acc_out that a weights call writes.
__device__ __forceinline__ bool seen_key(const SinkBwdArgs &a, int j) {
    int i0, i1;
    sink_rows_of_block(a, j, 1, &i0, &i1);
    return i0 < i1;
}

enum { kModeDq = 0, kModeDkv = 1, kModeWeights = 2 };

template <int D>
constexpr int bwd_smem(int mode) {
    return mode == kModeWeights ? 2 * kT * (D + 4) * 4 : (4 * kT * (D + 4) + 2 * kT * kPS + 2 * kT) * 4;
}

// Query-major (dQ): rows are 64 queries of one head, tiles are keys. Key-major (dK and dV,
// or the weights): rows are 64 keys of one key-value head, tiles are queries of the
// group's heads. X1, X2 are the rows' Q, dO or K, V; Y1, Y2 the tiles' K, V or Q, dO.
// `block`: the CTA among those of its mode.
template <int MODE, typename T, int D>
__device__ __forceinline__ void sink_bwd_rows(const SinkBwdArgs &a, int tiles, int block) {
    extern __shared__ float sm[];
    constexpr bool kTwo = MODE != kModeWeights;
    float *X1 = sm, *Y1 = X1 + kT * (D + 4);
    float *X2 = Y1 + kT * (D + 4), *Y2 = X2 + kT * (D + 4), *Ps = Y2 + kT * (D + 4), *Ss = Ps + kT * kPS;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int Hk = a.H / a.G, off = a.N - a.Lq;
    const float kLog2e = 1.4426950408889634f, scale2 = a.scale * kLog2e;
    auto at = [&](const View &v, int b, int h, int i) {
        return static_cast<const T *>(v.ptr) + b * v.sb + h * v.sh + (int64_t)i * v.st;
    };
    int b, h, hk, r0, nrows, s0, s1, qtiles = 1, i0 = 0, ilim = 0;
    SinkSpan sp{};
    SinkItem it{};
    int xb = 0;
    if (MODE == kModeDq) {
        const int tile = block % tiles, bh = block / tiles;
        b = bh / a.H;
        h = bh % a.H;
        hk = h / a.G;
        r0 = tile * kT;
        nrows = min(kT, a.Lq - r0);
        sp = sink_span(off + r0, off + r0 + nrows - 1, a.W, a.A, kT);
        s0 = 0;
        s1 = sp.ns + sp.nw;
    } else {
        // an item's key block in parts of 64 keys
        const int parts = a.keys / kT, part = block % parts, x = (block / parts) % tiles;
        xb = (block / parts) / tiles;
        b = xb / Hk;
        hk = xb % Hk;
        h = 0;
        it = sink_item(a, x);
        r0 = it.blk * a.keys + part * kT;
        nrows = max(0, min(kT, a.N - r0));
        if (nrows == 0) return;
        sink_rows_of_block(a, r0, kT, &i0, &ilim);
        qtiles = (ilim - i0 + kT - 1) / kT;
        const int64_t steps = (int64_t)a.G * qtiles;
        s0 = (int)(steps * it.seg / it.nseg);
        s1 = (int)(steps * (it.seg + 1) / it.nseg);
    }
    {
        TileLoad<T, D> x1, x2;
        x1.fetch([&](int r) -> const T * {
            return r < nrows ? (MODE == kModeDq ? at(a.Q, b, h, r0 + r) : at(a.K, b, hk, r0 + r)) : nullptr;
        });
        if (kTwo)
            x2.fetch([&](int r) -> const T * {
                return r < nrows ? (MODE == kModeDq ? at(a.dO, b, h, r0 + r) : at(a.V, b, hk, r0 + r)) : nullptr;
            });
        x1.put(X1);
        if (kTwo) x2.put(X2);
    }
    float o1[4][D / 16], o2[4][D / 16], w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o1[r][c] = o2[r][c] = 0.f;
    for (int st = s0; st < s1; ++st) {
        int k0 = 0, end = 0, hh = h, q0 = 0;
        bool sink = false;
        if (MODE == kModeDq) {
            sink = st < sp.ns;
            k0 = sink ? st * kT : sp.lo + (st - sp.ns) * kT;
            end = sink ? sp.sinks : sp.hi;
        } else {
            hh = hk * a.G + st / qtiles;
            q0 = i0 + (st % qtiles) * kT;
        }
        auto y = [&](const View &kv, const View &qv, int r) -> const T * {
            if (MODE == kModeDq) return k0 + r < end ? at(kv, b, hk, k0 + r) : nullptr;
            return q0 + r < ilim ? at(qv, b, hh, q0 + r) : nullptr;
        };
        TileLoad<T, D> y1, y2;
        y1.fetch([&](int r) { return y(a.K, a.Q, r); });
        if (kTwo) y2.fetch([&](int r) { return y(a.V, a.dO, r); });
        __syncthreads();
        y1.put(Y1);
        if (kTwo) y2.put(Y2);
        __syncthreads();
        float s[4][4], dp[4][4];
        dot_tile<D>(s, X1, Y1, ty, tx);
        if (kTwo) dot_tile<D>(dp, X2, Y2, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int rr = 4 * ty + r, cc = tx + 16 * c;
                const int i = MODE == kModeDq ? r0 + rr : q0 + cc;  // query row
                const int j = MODE == kModeDq ? k0 + cc : r0 + rr;  // key
                const int t = off + i;
                const bool in = (MODE == kModeDq ? rr < nrows && j < end : i < ilim && rr < nrows) && j <= t &&
                                (sink || j < a.A || j > t - a.W);
                const int64_t q = ((int64_t)b * a.H + hh) * a.Lq + i;
                const float L = in ? __ldg(a.lse + q) : -INFINITY;
                const float p = in && L != -INFINITY ? exp2f(s[r][c] * scale2 - L * kLog2e) : 0.f;
                if (kTwo) {
                    const float ds = in ? a.scale * p * (dp[r][c] - __ldcg(a.Dv + q)) : 0.f;
                    if (MODE == kModeDkv) Ps[rr * kPS + cc] = p;
                    Ss[rr * kPS + cc] = ds;
                } else {
                    w[r] += p;
                }
            }
        if (kTwo) {
            __syncwarp();
            add_product<D>(o1, Ss, Y1, ty, tx);
            if (MODE == kModeDkv) add_product<D>(o2, Ps, Y2, ty, tx);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int rr = 4 * ty + r;
        const float ws = MODE == kModeWeights ? sum16(w[r]) : 0.f;
        if (rr >= nrows) continue;
        const int64_t item = (int64_t)xb * tiles + (block / (a.keys / kT)) % tiles;  // key-major: partial sums' place
        const int kr = r0 + rr - it.blk * a.keys;
        if (MODE == kModeWeights) {
            if (tx == 0) {
                const int64_t g = ((int64_t)b * Hk + hk) * a.T + r0 + rr;
                if (it.nseg > 1) a.part[item * a.keys + kr] = ws;
                else if (seen_key(a, r0 + rr)) a.acc_out[g] = a.acc[g] + ws;
            }
            continue;
        }
        if (MODE == kModeDkv && it.nseg > 1) {
            float *d1 = a.part + (item * 2 * kSinkKeys + kr) * D, *d2 = d1 + kSinkKeys * D;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                store4(d1 + 64 * u + 4 * tx, o1[r][4 * u], o1[r][4 * u + 1], o1[r][4 * u + 2], o1[r][4 * u + 3]);
                store4(d2 + 64 * u + 4 * tx, o2[r][4 * u], o2[r][4 * u + 1], o2[r][4 * u + 2], o2[r][4 * u + 3]);
            }
            continue;
        }
        const MutView &v1 = MODE == kModeDq ? a.dQ : a.dK;
        T *d1 = static_cast<T *>(v1.ptr) + b * v1.sb + (MODE == kModeDq ? h : hk) * v1.sh + (int64_t)(r0 + rr) * v1.st;
        T *d2 = MODE == kModeDkv ? static_cast<T *>(a.dV.ptr) + b * a.dV.sb + hk * a.dV.sh + (int64_t)(r0 + rr) * a.dV.st : nullptr;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            store4(d1 + 64 * u + 4 * tx, o1[r][4 * u], o1[r][4 * u + 1], o1[r][4 * u + 2], o1[r][4 * u + 3]);
            if (MODE == kModeDkv)
                store4(d2 + 64 * u + 4 * tx, o2[r][4 * u], o2[r][4 * u + 1], o2[r][4 * u + 2], o2[r][4 * u + 3]);
        }
    }
}

// dQ's CTAs [0, nq), then those of dK and dV: side by side, each reads D once its grid is complete
// (in two kernels, dK and dV behind dQ, 2 x 4 heads of 509 tokens took 68 us, so 49). kPerSm CTAs an
// SM at d = 64; at d = 128 one fits.
template <typename T, int D, int kPerSm>
__global__ void __launch_bounds__(kThr, kPerSm) sink_bwd_kernel(SinkBwdArgs a, int qtiles, int nq, int items) {
    pdl_wait();
    if ((int)blockIdx.x < nq) sink_bwd_rows<kModeDq, T, D>(a, qtiles, blockIdx.x);
    else sink_bwd_rows<kModeDkv, T, D>(a, items, blockIdx.x - nq);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThr) sink_weights_kernel(SinkBwdArgs a, int items) {
    sink_bwd_rows<kModeWeights, T, D>(a, items, blockIdx.x);
}

// The partials of key blocks with several segments, in segment order: one warp per key row
// of dK and one of dV (weights: one thread per key). `keys`: the first keys of each head, that such blocks hold.
template <bool WEIGHTS, typename T, int D>
__global__ void __launch_bounds__(256) sink_reduce_kernel(SinkBwdArgs a, int items, int keys) {
    const int lane = threadIdx.x % 32, Hk = a.H / a.G;
    const int g_which = blockIdx.x & 1;
    const int64_t g = WEIGHTS ? (int64_t)blockIdx.x * 256 + threadIdx.x : (int64_t)(blockIdx.x / 2) * 8 + threadIdx.x / 32;
    pdl_wait();
    if (g >= (int64_t)a.B * Hk * keys) return;
    const int64_t xb = g / keys;
    const int j = (int)(g - xb * keys);
    const int blk = j / a.keys, kr = j % a.keys;
    const int nseg = blk < a.nsink ? a.seg_s : a.seg_w;
    if (nseg <= 1) return;
    const int64_t first = xb * items + (blk < a.nsink ? blk * a.seg_s : a.nsink * a.seg_s + (blk - a.nsink) * a.seg_w);
    if (WEIGHTS) {
        if (!seen_key(a, j)) return;
        float s = 0.f;
#pragma unroll 4
        for (int q = 0; q < nseg; ++q) s += a.part[(first + q) * a.keys + kr];
        const int64_t at = xb * a.T + j;
        a.acc_out[at] = a.acc[at] + s;
        return;
    }
    // a lane's D / 32 columns, 16 segments in flight
    constexpr int kE = D / 32;
    const int b = (int)(xb / Hk), hk = (int)(xb % Hk), which = g_which;
    const MutView &v = which ? a.dV : a.dK;
    T *dst = static_cast<T *>(v.ptr) + b * v.sb + hk * v.sh + (int64_t)j * v.st + lane * kE;
    const float *p = a.part + (first * 2 * kSinkKeys + which * kSinkKeys + kr) * D + lane * kE;
    float s[kE] = {};
#pragma unroll 16
    for (int q = 0; q < nseg; ++q) {
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
            const float2 x = load2(p + (int64_t)q * 2 * kSinkKeys * D + e);
            s[e] += x.x;
            s[e + 1] += x.y;
        }
    }
#pragma unroll
    for (int e = 0; e < kE; e += 2) store2(dst + e, s[e], s[e + 1]);
}

template <typename K, typename... A>
hils_status run(KernelSetup &setup, bool early, K kernel, int64_t grid, int threads, int smem, cudaStream_t s, const A &...args) {
    if (grid <= 0) return HILS_OK;
    const hils_status st = kernel_setup(setup, (const void *)kernel, threads, smem, nullptr);
    if (st != HILS_OK) return st;
    return sink_launch(early, kernel, grid, threads, smem, s, args...);
}

template <typename T, int D>
hils_status forward(const SinkArgs &a, cudaStream_t s) {
    static KernelSetup one, three;
    const int tiles = a.prefix ? (a.B + kT / a.G - 1) / (kT / a.G) : (a.Lq + kT - 1) / kT;
    const int64_t grid = (int64_t)tiles * a.splits * (a.prefix ? a.H / a.G : (int64_t)a.B * a.H);
    if (D == 64 && grid > device_sm_count())
        return run(three, false, sink_fwd_kernel<T, D, D == 64 ? 3 : 1>, grid, kThr, fwd_smem<D>(), s, a, tiles);
    return run(one, false, sink_fwd_kernel<T, D, 1>, grid, kThr, fwd_smem<D>(), s, a, tiles);
}
template <typename T, int D>
hils_status dot(const SinkBwdArgs &a, float *Dv, cudaStream_t s) {
    static KernelSetup setup;
    constexpr int kRows = 8 * 4 * 32 * Vec<T>::kN / D;  // of a CTA
    return run(setup, false, sink_dot_kernel<T, D>, ((int64_t)a.B * a.H * a.Lq + kRows - 1) / kRows, 256, 0, s, a, Dv);
}
template <typename T, int D>
hils_status backward(const SinkBwdArgs &a, cudaStream_t s) {
    static KernelSetup one, two;
    const int tiles = (a.Lq + kT - 1) / kT, items = (int)sink_key_items(a);
    const int64_t nq = (int64_t)tiles * a.B * a.H, nk = (int64_t)(a.keys / kT) * items * a.B * (a.H / a.G);
    if (nq > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
    // Two CTAs an SM, but for calls that wait for one CTA's walk (dQ's longest) rather than for all
    // steps of an SM: 8 heads of 2048 causal tokens 629 -> 540 us, 2 x 4 of 1000 with W 96 80 -> 72;
    // with one, and the registers for deeper unrolling, 4 heads of 2048 375 -> 321 us, 2 x 4 of 509
    // with W 96 57 -> 53.
    const int64_t see = ((int64_t)a.W + a.A + kT - 1 + kT - 1) / kT, longest = see < tiles ? see : tiles;
    const int64_t steps = 2 * (longest * (longest + 1) / 2 + (tiles - longest) * longest) * a.B * a.H;
    if (D == 64 && steps > longest * device_sm_count())
        return run(two, true, sink_bwd_kernel<T, D, D == 64 ? 2 : 1>, nq + nk, kThr, bwd_smem<D>(kModeDkv), s, a, tiles, (int)nq, items);
    return run(one, true, sink_bwd_kernel<T, D, 1>, nq + nk, kThr, bwd_smem<D>(kModeDkv), s, a, tiles, (int)nq, items);
}
template <typename T, int D>
hils_status weights(const SinkBwdArgs &a, cudaStream_t s) {
    static KernelSetup setup;
    const int items = (int)sink_key_items(a);
    return run(setup, false, sink_weights_kernel<T, D>, (int64_t)(a.keys / kT) * items * a.B * (a.H / a.G), kThr, bwd_smem<D>(kModeWeights), s,
               a, items);
}
template <typename T, int D>
hils_status reduce(const SinkBwdArgs &a, bool w, cudaStream_t s) {
    static KernelSetup s0, s1;
    if (a.seg_s <= 1 && a.seg_w <= 1) return HILS_OK;
    const int64_t last = (int64_t)a.nsink * a.keys;  // (without segments behind the sinks' blocks)
    const int keys = a.seg_w > 1 || last > a.N ? a.N : (int)last;
    const int64_t rows = (int64_t)a.B * (a.H / a.G) * keys;
    const int items = (int)sink_key_items(a);
    return w ? run(s0, true, sink_reduce_kernel<true, T, D>, (rows + 255) / 256, 256, 0, s, a, items, keys)
             : run(s1, true, sink_reduce_kernel<false, T, D>, (rows + 7) / 8 * 2, 256, 0, s, a, items, keys);
}

}  // namespace

#define BY_TYPE(fn, ...)                                                                              \
    (dt == HILS_BF16 ? (d == 64 ? fn<bf16, 64>(__VA_ARGS__) : fn<bf16, 128>(__VA_ARGS__))             \
                     : (d == 64 ? fn<float, 64>(__VA_ARGS__) : fn<float, 128>(__VA_ARGS__)))

hils_status launch_sink_forward_general(hils_dtype dt, int d, const SinkArgs &a, cudaStream_t s) { return BY_TYPE(forward, a, s); }
hils_status launch_sink_dot(hils_dtype dt, int d, const SinkBwdArgs &a, float *Dv, cudaStream_t s) { return BY_TYPE(dot, a, Dv, s); }
hils_status launch_sink_backward_general(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s) { return BY_TYPE(backward, a, s); }
hils_status launch_sink_weights_general(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s) { return BY_TYPE(weights, a, s); }
hils_status launch_sink_reduce(hils_dtype dt, int d, const SinkBwdArgs &a, bool w, cudaStream_t s) { return BY_TYPE(reduce, a, w, s); }

}  // namespace hils
