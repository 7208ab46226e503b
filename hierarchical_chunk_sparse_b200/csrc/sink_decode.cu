// One query per sequence over the visible slots of its cache (formulas in sink_common.cuh).
// Bound by HBM: 8 x 128K tokens of 8 key-value heads (32 heads, d = 128, bf16), 3.65 GB with the
// weights added to acc, take 632 us, 5.8 TB/s (the walk 571, the join 9, acc 38; 7840 in float32 on
// the CUDA cores). A window of 512 in one sequence takes 13 us, nearly all of it the launch.
// float32, 8 x 16K tokens of 8 key-value heads (32 heads, d = 128), 1.07 GB: 370 us, 2.9 TB/s, bound by
// the products' shuffles and shared-memory reads; 1131 with 64 heads.
#include "sink_common.cuh"

namespace hils {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// cp_async16, or 16 zero bytes where `in` is false (nothing is read then).
__device__ __forceinline__ void cp_async16_zfill(void *smem, const void *gmem, bool in) {
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(gmem), "r"(in ? 16 : 0) : "memory");
}

template <typename T>
constexpr int tile_keys() { return sizeof(T) == 2 ? 16 : 8; }
template <typename T, int D>
constexpr int tile_bytes() { return tile_keys<T>() * D * (int)sizeof(T); }  // of K, and of V
// stages of a warp's ring (what fits beside the results of eight warps and heads)
template <typename T, int kWarps>
constexpr int ring_stages() { return kWarps == 8 && sizeof(T) == 4 ? 2 : 3; }
// the warps' rings, their results of a row, and (float32) its queries
template <typename T, int D, int kWarps>
int decode_smem(int G) {
    return kWarps * ring_stages<T, kWarps>() * 2 * tile_bytes<T, D>() + kWarps * kMaxGroupHeads * 8 + kWarps * G * D * 4 +
           (sizeof(T) == 4 ? G * D * 4 : 0);
}

// What a sequence sees, in order: the shared prefix, the sinks, the window.
struct Visible {
    int n, prefix, sinks, lo;  // n in all
    int tiles;
};
template <int KT>
__device__ __forceinline__ Visible visible(const SinkDecodeArgs &a, int b) {
    Visible v;
    const int len = min(max(__ldg(a.cache_len + b), 0), a.T);
    sink_visible(len, a.W, a.A, &v.sinks, &v.lo);
    v.prefix = a.P;
    v.n = a.P + v.sinks + len - v.lo;
    v.tiles = max(1, (v.n + KT - 1) / KT);  // an empty row still gets its outputs
    return v;
}

// a / b of numbers that mostly fit 32 bits (a 64-bit division takes some 100 instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// A place in the flattened tiles of all (b, key-value head) rows.
template <int KT>
struct Place {
    int b, hk, k;  // tile k of row (b, hk)
    Visible v;
    __device__ __forceinline__ void advance(const SinkDecodeArgs &a, int Hk, int by) {
        k += by;
        while (k >= v.tiles && b < a.B) {
            k -= v.tiles;
            if (++hk == Hk) {
                hk = 0;
                if (++b < a.B) v = visible<KT>(a, b);
            }
        }
    }
};

// Tiles of all rows, and the place of tile `at` (every lane of the warp).
template <int KT>
__device__ int64_t all_tiles(const SinkDecodeArgs &a, int Hk) {
    int64_t t = 0;
    for (int b = threadIdx.x % 32; b < a.B; b += 32) t += visible<KT>(a, b).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
    return t * Hk;
}
template <int KT>
__device__ Place<KT> find_tile(const SinkDecodeArgs &a, int Hk, int64_t at) {
    const int lane = threadIdx.x % 32;
    int64_t before = 0;
    for (int b0 = 0;; b0 += 32) {
        int64_t t = b0 + lane < a.B ? (int64_t)visible<KT>(a, b0 + lane).tiles * Hk : 0, sum = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned hit = __ballot_sync(kFull, before + sum > at);
        if (hit == 0u && b0 + 32 < a.B) {
            before += __shfl_sync(kFull, sum, 31);
            continue;
        }
        const int l = hit ? __ffs(hit) - 1 : 31;
        before += __shfl_sync(kFull, sum - t, l);
        Place<KT> p;
        p.b = min(b0 + l, a.B - 1);
        p.v = visible<KT>(a, p.b);
        const int64_t in = at - before;
        p.hk = (int)divide(in, p.v.tiles);
        p.k = (int)(in - (int64_t)p.hk * p.v.tiles);
        return p;
    }
}

// The slots of one tile into a warp's stage, K then V: 16-byte unit u of row r at unit
// u ^ (r % 8); zeros for rows behind the last visible one.
template <typename T, int D, int KT>
__device__ __forceinline__ void load_kv(const SinkDecodeArgs &a, const Place<KT> &p, uint8_t *dst) {
    constexpr int kU = D * (int)sizeof(T) / 16, kPer = 32 / kU, kRounds = KT / kPer;
    static_assert(kU <= 32 && KT % kPer == 0, "a round of the warp is whole rows");
    const int lane = threadIdx.x % 32, u = lane % kU, r0 = lane / kU;
    const int v0 = p.k * KT, v1 = v0 + KT, own = v0 - p.v.prefix;
    const T *kc = static_cast<const T *>(a.K.ptr) + p.b * a.K.sb + p.hk * a.K.sh;
    const T *vc = static_cast<const T *>(a.V.ptr) + p.b * a.V.sb + p.hk * a.V.sh;
    uint8_t *to = dst + r0 * (kU * 16);
    if (v1 <= p.v.n && (own >= p.v.sinks || (own >= 0 && own + KT <= p.v.sinks) || v1 <= p.v.prefix)) {
        // all of one run of slots: the prefix, the sinks or the window
        const bool pre = own < 0;
        const int64_t j = (pre ? v0 : own < p.v.sinks ? own : p.v.lo + (own - p.v.sinks)) + r0;
        const int64_t ks = (pre ? a.Kp.st : a.K.st), vs = (pre ? a.Vp.st : a.V.st);
        const uint8_t *k = reinterpret_cast<const uint8_t *>((pre ? static_cast<const T *>(a.Kp.ptr) + p.hk * a.Kp.sh : kc) + j * ks) + u * 16;
        const uint8_t *w = reinterpret_cast<const uint8_t *>((pre ? static_cast<const T *>(a.Vp.ptr) + p.hk * a.Vp.sh : vc) + j * vs) + u * 16;
        const int64_t kstep = ks * kPer * (int)sizeof(T), vstep = vs * kPer * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int at = i * 512 + ((u ^ ((i * kPer + r0) & 7)) * 16);
            cp_async16(to + at, k);
            cp_async16(to + tile_bytes<T, D>() + at, w);
            k += kstep;
            w += vstep;
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < kRounds; ++i) {
        const int r = i * kPer + r0;
        int v = v0 + r;
        const bool in = v < p.v.n;
        const T *k = static_cast<const T *>(a.Q.ptr), *w = k;  // not read
        if (v < p.v.prefix) {
            k = static_cast<const T *>(a.Kp.ptr) + p.hk * a.Kp.sh + v * a.Kp.st;
            w = static_cast<const T *>(a.Vp.ptr) + p.hk * a.Vp.sh + v * a.Vp.st;
        } else if (in) {
            v -= p.v.prefix;
            const int64_t j = v < p.v.sinks ? v : p.v.lo + (v - p.v.sinks);
            k = kc + j * a.K.st;
            w = vc + j * a.V.st;
        }
        const int at = i * 512 + ((u ^ (r & 7)) * 16);
        cp_async16_zfill(to + at, reinterpret_cast<const uint8_t *>(k) + u * 16, in);
        cp_async16_zfill(to + tile_bytes<T, D>() + at, reinterpret_cast<const uint8_t *>(w) + u * 16, in);
    }
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 matrix of 16-bit elements
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float max8(float v) {  // over the lanes of equal lane % 4
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One warp's running softmax of a group's heads over its tiles: bf16 with mma.sync, the up to
// eight heads as the N of S^T = K Q^T and O^T = V^T P^T (a decode step reads each key once and
// is bound by that; tcgen05's 128 rows would be 15/16 padding). P is rounded to bf16 for it, at
// most 2^-8 of each.
template <typename T, int D>
struct Rows;

template <int D>
struct Rows<bf16, D> {
    uint32_t q[D / 16][2];  // Q^T fragments of head lane / 4
    float o[D / 16][4];     // O^T: dims lane / 4 (+ 8) of each 16, heads 2 (lane % 4) + {0, 1}
    float m[2], l[2];       // of those heads; l of this lane's keys only

    __device__ __forceinline__ void start(const SinkDecodeArgs &a, int b, int hk, float *) {
        const int lane = threadIdx.x % 32, g = lane / 4;
        const bf16 *p = static_cast<const bf16 *>(a.Q.ptr) + b * a.Q.sb + (int64_t)(hk * a.G + min(g, a.G - 1)) * a.Q.sh;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p + s * 16 + (lane % 4) * 2);
            q[s][0] = g < a.G ? __ldg(w) : 0u;
            q[s][1] = g < a.G ? __ldg(w + 4) : 0u;
        }
#pragma unroll
        for (int s = 0; s < D / 16; ++s) o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void tile(const SinkDecodeArgs &a, const Place<16> &p, const uint8_t *stage, float scale2,
                                         float *) {
        const int lane = threadIdx.x % 32, id = lane / 8, r7 = lane & 7;
        const uint32_t kb = (uint32_t)__cvta_generic_to_shared(stage), vb = kb + tile_bytes<bf16, D>();
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products
        const uint32_t kr = kb + (r7 + (id & 1) * 8) * (D * 2);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t f[4];
            ldsm4(f, kr + (((2 * k + (id >> 1)) ^ r7) * 16));
            mma16816(k & 1 ? s1 : s, f, q[k][0], q[k][1]);
        }
        const int left = p.v.n - p.k * 16;  // visible slots from this tile's first
        const int r = lane / 4;             // keys r (elements 0, 1) and r + 8 (2, 3) of heads g, g + 1
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = r + (e >> 1) * 8 < left ? (s[e] + s1[e]) * scale2 : -INFINITY;
        if (a.logits) {
            const int g = 2 * (lane % 4);
            float *out = a.logits + ((int64_t)p.b * a.H + p.hk * a.G + g) * a.logit_stride + p.k * 16 + r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + (e >> 1) * 8 < left && g + (e & 1) < a.G) out[(e & 1) * a.logit_stride + (e >> 1) * 8] = s[e];
        }
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float mx = fmaxf(m[i], max8(fmaxf(s[i], s[i + 2]))), ref = mx == -INFINITY ? 0.f : mx;
            f[i] = exp2f(m[i] - ref);
            m[i] = mx;
            s[i] = exp2f(s[i] - ref);
            s[i + 2] = exp2f(s[i + 2] - ref);
            l[i] = fmaf(l[i], f[i], s[i] + s[i + 2]);
        }
        if (__any_sync(kFull, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                o[c][0] *= f[0];
                o[c][1] *= f[1];
                o[c][2] *= f[0];
                o[c][3] *= f[1];
            }
        }
        // the probabilities rounded to bf16 as operands
        const uint32_t b0 = transpose8(pack2(s[0], s[1])), b1 = transpose8(pack2(s[2], s[3]));
        const uint32_t vr = vb + (r7 + (id >> 1) * 8) * (D * 2);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            uint32_t v[4];
            ldsm4_t(v, vr + (((2 * c + (id & 1)) ^ r7) * 16));
            mma16816(o[c], v, b0, b1);
        }
    }
    // this warp's results: row g of so [G][D], sm, sl [8]
    __device__ __forceinline__ void finish(float *sm, float *sl, float *so, int G) {
        const int lane = threadIdx.x % 32, g = 2 * (lane % 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float z = sum8(l[i]);
            if (lane < 4) {
                sm[g + i] = m[i];
                sl[g + i] = z;
            }
            if (g + i >= G) continue;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                so[(g + i) * D + c * 16 + lane / 4] = o[c][i];
                so[(g + i) * D + c * 16 + lane / 4 + 8] = o[c][2 + i];
            }
        }
    }
};

// float32 on the CUDA cores: a key's logits are four lanes' quarters of the dimensions; then a
// lane owns D / 32 dimensions of the output and runs over the keys.
template <int D>
struct Rows<float, D> {
    static constexpr int kE = D / 32;
    float o[kMaxGroupHeads][kE], m[kMaxGroupHeads], l[kMaxGroupHeads];  // m and l: of every lane alike

    __device__ __forceinline__ void start(const SinkDecodeArgs &a, int b, int hk, float *) {
#pragma unroll
        for (int g = 0; g < kMaxGroupHeads; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[g][e] = 0.f;
        }
    }
    __device__ __forceinline__ void tile(const SinkDecodeArgs &a, const Place<8> &p, const uint8_t *stage, float scale2,
                                         float *qs) {
        const int lane = threadIdx.x % 32, key = lane % 8, part = lane / 8;
        const float *kt = reinterpret_cast<const float *>(stage), *vt = kt + 8 * D;
        float s[kMaxGroupHeads];
#pragma unroll
        for (int g = 0; g < kMaxGroupHeads; ++g) s[g] = 0.f;
#pragma unroll 4
        for (int u = 0; u < D / 16; ++u) {
            const int uu = u * 4 + part;
            const float4 k = *reinterpret_cast<const float4 *>(kt + key * D + ((uu ^ key) * 4));
#pragma unroll
            for (int g = 0; g < kMaxGroupHeads; ++g) {
                if (g >= a.G) break;
                const float4 x = *reinterpret_cast<const float4 *>(qs + g * D + uu * 4);
                s[g] = fmaf(k.x, x.x, fmaf(k.y, x.y, fmaf(k.z, x.z, fmaf(k.w, x.w, s[g]))));
            }
        }
        const bool in = key < p.v.n - p.k * 8;
#pragma unroll
        for (int g = 0; g < kMaxGroupHeads; ++g) {
            if (g >= a.G) break;
            s[g] += __shfl_xor_sync(kFull, s[g], 8);
            s[g] += __shfl_xor_sync(kFull, s[g], 16);
            s[g] = in ? s[g] * scale2 : -INFINITY;
            if (a.logits && in && part == 0)
                a.logits[((int64_t)p.b * a.H + p.hk * a.G + g) * a.logit_stride + p.k * 8 + key] = s[g];
            float mx = s[g];
#pragma unroll
            for (int o_ = 4; o_ > 0; o_ >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o_));
            mx = fmaxf(mx, m[g]);
            const float ref = mx == -INFINITY ? 0.f : mx, f = exp2f(m[g] - ref);
            s[g] = exp2f(s[g] - ref);
            float z = s[g];
#pragma unroll
            for (int o_ = 4; o_ > 0; o_ >>= 1) z += __shfl_xor_sync(kFull, z, o_);
            m[g] = mx;
            l[g] = fmaf(l[g], f, z);
#pragma unroll
            for (int e = 0; e < kE; ++e) o[g][e] *= f;
        }
#pragma unroll 4
        for (int k = 0; k < 8; ++k) {
            float v[kE];
            const int unit = lane * kE / 4, at = k * D + ((unit ^ (k & 7)) * 4) + (lane * kE) % 4;
            if (kE == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(vt + at);
                v[0] = x.x;
                v[1] = x.y;
                v[kE - 2] = x.z;
                v[kE - 1] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(vt + at);
                v[0] = x.x;
                v[1] = x.y;
            }
#pragma unroll
            for (int g = 0; g < kMaxGroupHeads; ++g) {
                if (g >= a.G) break;
                const float w = __shfl_sync(kFull, s[g], k);
#pragma unroll
                for (int e = 0; e < kE; ++e) o[g][e] = fmaf(w, v[e], o[g][e]);
            }
        }
    }
    __device__ __forceinline__ void finish(float *sm, float *sl, float *so, int G) {
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int g = 0; g < kMaxGroupHeads; ++g) {
            if (g >= G) break;
            if (lane == 0) {
                sm[g] = m[g];
                sl[g] = l[g];
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) so[g * D + lane * kE + e] = o[g][e];
        }
    }
};

// The tiles of all rows are cut into one even share for each CTA, whatever the sequences'
// lengths. A row that is one CTA's alone gets its output here; of any other, each CTA leaves
// its share's result as a segment for the combine. With `whole`, the shares end at rows.
template <typename T, int D, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 8 / kWarps) sink_decode_kernel(SinkDecodeArgs a) {
    constexpr int KT = tile_keys<T>(), kE = D / 32, kThr = kWarps * 32, kStages = ring_stages<T, kWarps>();
    constexpr int kStage = 2 * tile_bytes<T, D>();
    extern __shared__ __align__(128) uint8_t smem[];
    const int Hk = a.H / a.G, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint8_t *ring = smem + warp * kStages * kStage;
    float *sm = reinterpret_cast<float *>(smem + kWarps * kStages * kStage), *sl = sm + kWarps * kMaxGroupHeads;
    float *so = sl + kWarps * kMaxGroupHeads, *qs = so + kWarps * a.G * D;
    const float scale2 = a.scale * kLog2e;
    const int64_t total = a.whole ? (int64_t)a.B * Hk : all_tiles<KT>(a, Hk), c = blockIdx.x;
    const int64_t n_cta = min((int64_t)gridDim.x, total);
    if (c < n_cta) {  // every CTA below n_cta has a tile
        int64_t t0 = divide(total * c, n_cta), t1 = divide(total * (c + 1), n_cta);
        Place<KT> cur;  // the CTA's current row, at its first tile here
        if (a.whole) {  // rows [t0, t1): their tiles, counted from 0
            cur.b = (int)(t0 / Hk);
            cur.hk = (int)(t0 % Hk);
            cur.k = 0;
            cur.v = visible<KT>(a, cur.b);
            int64_t n = 0;
            for (int64_t r = t0; r < t1; ++r) n += visible<KT>(a, (int)(r / Hk)).tiles;
            t0 = 0;
            t1 = n;
        } else {
            cur = find_tile<KT>(a, Hk, t0);
        }
        Place<KT> ld = cur;
        ld.advance(a, Hk, warp);
        int64_t at = t0 + warp;
        int put = 0, got = 0;  // stages written, read
        auto next_load = [&] {
            if (at < t1) {
                load_kv<T, D, KT>(a, ld, ring + put * kStage);
                ld.advance(a, Hk, kWarps);
                at += kWarps;
            }
            if (++put == kStages) put = 0;
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) next_load();
        for (int64_t t = t0; t < t1;) {  // a row, or what of it is this CTA's
            const int64_t row0 = t - cur.k;  // the row's first tile
            const int64_t end = min(t1, row0 + cur.v.tiles);
            if (sizeof(T) == 4) {  // (the row before has been joined)
                for (int e = threadIdx.x; e < a.G * D; e += kThr) {
                    const int g = e / D;
                    qs[e] = static_cast<const float *>(a.Q.ptr)[cur.b * a.Q.sb + (int64_t)(cur.hk * a.G + g) * a.Q.sh + e % D];
                }
                __syncthreads();
            }
            Rows<T, D> rows;
            rows.start(a, cur.b, cur.hk, qs);
            Place<KT> p = cur;
            const int skip = (int)((warp - (t - t0)) & (kWarps - 1));  // this warp's first tile at or after t
            p.k += skip;
            const int n = (int)(end - t);
#pragma unroll 1
            for (int x = skip; x < n; x += kWarps, p.k += kWarps) {
                next_load();
                cp_async_wait<kStages - 1>();
                __syncwarp();
                rows.tile(a, p, ring + got * kStage, scale2, qs);
                if (++got == kStages) got = 0;
                __syncwarp();
            }
            rows.finish(sm + warp * kMaxGroupHeads, sl + warp * kMaxGroupHeads, so + warp * a.G * D, a.G);
            __syncthreads();
            const int64_t rowidx = (int64_t)cur.b * Hk + cur.hk;
            const bool alone = a.slots == 0 && (a.whole || (row0 >= t0 && row0 + cur.v.tiles <= t1));
            for (int g = warp; g < a.G; g += kWarps) {
                float mx = -INFINITY, z = 0.f, r[kE] = {};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w * kMaxGroupHeads + g]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float lw = sl[w * kMaxGroupHeads + g], f = lw > 0.f ? exp2f(sm[w * kMaxGroupHeads + g] - mx) : 0.f;
                    z = fmaf(f, lw, z);
#pragma unroll
                    for (int e = 0; e < kE; ++e) r[e] = fmaf(f, so[(w * a.G + g) * D + lane * kE + e], r[e]);
                }
                const float inv = z > 0.f ? 1.f / z : 0.f, lse = z > 0.f ? (mx + log2f(z)) * kLn2 : -INFINITY;
                const int h = cur.hk * a.G + g;
                if (alone) {
                    T *dst = static_cast<T *>(a.O.ptr) + cur.b * a.O.sb + h * a.O.sh + lane * kE;
#pragma unroll
                    for (int e = 0; e < kE; e += 2) store2(dst + e, r[e] * inv, r[e + 1] * inv);
                    if (lane == 0) a.lse[(int64_t)cur.b * a.H + h] = lse;
                } else {
                    const int64_t seg = (a.whole ? rowidx : c + rowidx) * a.G + g;
#pragma unroll
                    for (int e = 0; e < kE; e += 2) store2(a.seg_o + seg * D + lane * kE + e, r[e] * inv, r[e + 1] * inv);
                    if (lane == 0) a.seg_lse[seg] = lse;
                }
            }
            __syncthreads();  // sm, sl, so, qs are free again
            cur.advance(a, Hk, n);
            t = end;
        }
        cp_async_wait<0>();
    }
    pdl_wait();  // the prefix kernel's partial results are complete when this grid is
}

// W warps per row (b, h; 4 / W rows a CTA): the partial results of the prefix kernel's slots and of the decode
// CTAs' segments, in that order; weights exp(lse_s - max). Rows that one CTA has finished are left.
template <typename T, int D, int W>
__global__ void __launch_bounds__(128) sink_decode_combine_kernel(SinkDecodeArgs a, int ctas) {
    constexpr int KT = tile_keys<T>(), kE = D / 32;
    const int Hk = a.H / a.G, lane = threadIdx.x % 32, part = threadIdx.x / 32 % W;
    const int64_t rows = (int64_t)a.B * a.H, at = (int64_t)blockIdx.x * (4 / W) + threadIdx.x / 32 / W, row = min(at, rows - 1);
    const int b = (int)divide(row, a.H), h = (int)(row - (int64_t)b * a.H), hk = h / a.G, g = h % a.G;
    int64_t before = 0, total = 0;
    for (int i = lane; i < a.B; i += 32) {
        const int64_t n = (int64_t)visible<KT>(a, i).tiles * Hk;
        total += n;
        before += i < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(kFull, total, o);
        before += __shfl_xor_sync(kFull, before, o);
    }
    const int tiles = visible<KT>(a, b).tiles;
    const int64_t first = before + (int64_t)hk * tiles, n_cta = min((int64_t)ctas, total);
    auto cta_of = [&](int64_t tile) { return divide((tile + 1) * n_cta - 1, total); };
    int64_t seg0 = (int64_t)b * Hk + hk;
    int ns = 1;
    if (!a.whole) {
        const int64_t c0 = cta_of(first);
        ns = (int)(cta_of(first + tiles - 1) - c0) + 1;
        seg0 += c0;
    }
    const int all = a.slots + ns;
    pdl_wait();  // every thread: this grid must not be over before the one that it follows
    if (all == 1 || at >= rows) return;
    auto lse_of = [&](int s) {
        return s < a.slots ? a.part_lse[row * a.slots + s] : a.seg_lse[(seg0 + (s - a.slots)) * a.G + g];
    };
    auto row_of = [&](int s) {
        return (s < a.slots ? a.part_o + (row * a.slots + s) * D : a.seg_o + ((seg0 + (s - a.slots)) * a.G + g) * D) + lane * kE;
    };
    float mx = -INFINITY, z = 0.f, r[kE] = {};
    for (int s = lane; s < all; s += 32) mx = fmaxf(mx, lse_of(s));
    mx = warp_max(mx);
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int s0 = 0; s0 < all; s0 += 32) {
        const float wl = s0 + lane < all ? expf(lse_of(s0 + lane) - ref) : 0.f;
        z += wl;
        const int m = min(32, all - s0);
#pragma unroll 8
        for (int i = part; i < m; i += W) {
            const float w = __shfl_sync(kFull, wl, i);
            const float *src = row_of(s0 + i);
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
                const float2 x = load2(src + e);
                r[e] = fmaf(w, x.x, r[e]);
                r[e + 1] = fmaf(w, x.y, r[e + 1]);
            }
        }
    }
    z = warp_sum(z);
    if (W > 1) {  // (the CTA's rows are one)
        __shared__ float rest[W][D];
#pragma unroll
        for (int e = 0; e < kE; ++e) rest[part][lane * kE + e] = r[e];
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int e = 0; e < kE; ++e) r[e] += rest[w][lane * kE + e];
    }
    const float inv = z > 0.f ? 1.f / z : 0.f;
    T *dst = static_cast<T *>(a.O.ptr) + b * a.O.sb + h * a.O.sh + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2) store2(dst + e, r[e] * inv, r[e + 1] * inv);
    if (lane == 0) a.lse[row] = z > 0.f ? mx + logf(z) : -INFINITY;
}

// One warp per row: weights exp(lse_s - max) over the row's slots, in slot order.
template <typename T, int D>
__global__ void __launch_bounds__(256) sink_combine_kernel(SinkCombineArgs a) {
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    pdl_wait();
    if (row >= a.rows) return;
    const float *lse = a.part_lse + row * a.slots;
    float mx = -INFINITY;
    for (int s = lane; s < a.slots; s += 32) mx = fmaxf(mx, lse[s]);
    mx = warp_max(mx);
    float z = 0.f;
    if (mx != -INFINITY)
        for (int s = lane; s < a.slots; s += 32) z += expf(lse[s] - mx);
    z = warp_sum(z);
    const float inv = z > 0.f ? 1.f / z : 0.f;
    float2 o[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[c] = make_float2(0.f, 0.f);
    for (int s = 0; s < a.slots; ++s) {
        const float x = lse[s];
        if (x == -INFINITY) continue;
        const float w = expf(x - mx) * inv;
        const float *p = a.part_o + (row * a.slots + s) * D + 2 * lane;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float2 v = load2(p + 64 * c);
            o[c].x = fmaf(w, v.x, o[c].x);
            o[c].y = fmaf(w, v.y, o[c].y);
        }
    }
    const int64_t i = row % a.Lq, bh = row / a.Lq;
    T *dst = static_cast<T *>(a.O.ptr) + (bh / a.H) * a.O.sb + (bh % a.H) * a.O.sh + i * a.O.st + 2 * lane;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) store2(dst + 64 * c, o[c].x, o[c].y);
    if (lane == 0 && a.lse) a.lse[row] = z > 0.f ? mx + logf(z) : -INFINITY;
}

// acc_out = acc + the weights of the group's heads, kAcc slots 256 apart for each thread (their
// loads in flight together).
constexpr int kAcc = 4;
__global__ void __launch_bounds__(256) sink_acc_kernel(SinkDecodeArgs a, const float *lse, const float *acc, float *acc_out,
                                                       int chunks) {
    const int Hk = a.H / a.G;
    const int bk = blockIdx.x / chunks, b = bk / Hk, hk = bk - b * Hk;
    const int v0 = (blockIdx.x - bk * chunks) * (256 * kAcc) + threadIdx.x;
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    int sinks, lo;
    sink_visible(n, a.W, a.A, &sinks, &lo);
    const int nvis = sinks + n - lo;
    const int64_t row = (int64_t)b * a.H + hk * a.G, out = ((int64_t)b * Hk + hk) * a.T;
    pdl_wait();
    if (v0 >= nvis) return;
    float w[kAcc] = {};
    for (int g = 0; g < a.G; ++g) {
        const float L = lse[row + g] * kLog2e;
        const float *s = a.logits + (row + g) * a.logit_stride + v0;
#pragma unroll
        for (int k = 0; k < kAcc; ++k)
            if (v0 + 256 * k < nvis) w[k] += exp2f(s[256 * k] - L);
    }
#pragma unroll
    for (int k = 0; k < kAcc; ++k) {
        const int v = v0 + 256 * k;
        if (v >= nvis) continue;
        const int64_t at = out + (v < sinks ? v : lo + (v - sinks));
        acc_out[at] = acc[at] + w[k];
    }
}

}  // namespace

// CTAs of a decode: two per SM, no more than there are tiles. (Both fit an SM's shared memory but in
// float32 with d = 128 and groups of seven or eight, where one does: its 116 KB; the others follow.)
int sink_decode_ctas(hils_dtype dt, int B, int Hk, int64_t keys, int sms) {
    const int kt = dt == HILS_BF16 ? tile_keys<bf16>() : tile_keys<float>();
    const int64_t tiles = (int64_t)B * Hk * (keys > kt ? (keys + kt - 1) / kt : 1);
    return (int)(tiles < 2 * sms ? tiles : 2 * sms);
}

namespace {
template <typename T, int D>
hils_status decode(const SinkDecodeArgs &a, int ctas, cudaStream_t s) {
    static KernelSetup setup, whole;  // (the latter: eight warps a CTA)
    hils_status st;
    const void *k = a.whole ? (const void *)sink_decode_kernel<T, D, 8> : (const void *)sink_decode_kernel<T, D, 4>;
    const int most = a.whole ? decode_smem<T, D, 8>(kMaxGroupHeads) : decode_smem<T, D, 4>(kMaxGroupHeads);
    const int smem = a.whole ? decode_smem<T, D, 8>(a.G) : decode_smem<T, D, 4>(a.G), threads = a.whole ? 256 : 128;
    st = kernel_setup(a.whole ? whole : setup, k, threads, most, nullptr);
    if (st != HILS_OK) return st;
    if (a.whole) {
        const int64_t rows = (int64_t)a.B * (a.H / a.G), sms = device_sm_count();
        ctas = (int)(rows < sms ? rows : sms);
    }
    // after a prefix kernel: it may begin while that one ends
    st = a.whole ? sink_launch(a.slots > 0, sink_decode_kernel<T, D, 8>, ctas, threads, smem, s, a)
                 : sink_launch(a.slots > 0, sink_decode_kernel<T, D, 4>, ctas, threads, smem, s, a);
    if (st != HILS_OK || (a.whole && a.slots == 0)) return st;
    // with a prefix's slots, or few rows for many CTAs, there is much to join
    const int64_t rows = (int64_t)a.B * a.H;
    return a.slots + ctas * (int64_t)a.G / rows >= 8 ? sink_launch(true, sink_decode_combine_kernel<T, D, 4>, rows, 128, 0, s, a, ctas)
                                                     : sink_launch(true, sink_decode_combine_kernel<T, D, 1>, (rows + 3) / 4, 128, 0, s, a, ctas);
}
}  // namespace

hils_status launch_sink_decode(hils_dtype dt, int d, const SinkDecodeArgs &a, int ctas, cudaStream_t s) {
    if (ctas == 0) return HILS_OK;
    if (dt == HILS_BF16) return d == 64 ? decode<bf16, 64>(a, ctas, s) : decode<bf16, 128>(a, ctas, s);
    return d == 64 ? decode<float, 64>(a, ctas, s) : decode<float, 128>(a, ctas, s);
}

hils_status launch_sink_combine(hils_dtype dt, int d, const SinkCombineArgs &a, cudaStream_t s) {
    const int64_t grid = (a.rows + 7) / 8;
    if (dt == HILS_BF16)
        return d == 64 ? sink_launch(true, sink_combine_kernel<bf16, 64>, grid, 256, 0, s, a)
                       : sink_launch(true, sink_combine_kernel<bf16, 128>, grid, 256, 0, s, a);
    return d == 64 ? sink_launch(true, sink_combine_kernel<float, 64>, grid, 256, 0, s, a)
                   : sink_launch(true, sink_combine_kernel<float, 128>, grid, 256, 0, s, a);
}

hils_status launch_sink_decode_acc(const SinkDecodeArgs &a, const float *lse, const float *acc, float *acc_out,
                                   cudaStream_t s) {
    const int chunks = (int)((a.logit_stride + 256 * kAcc - 1) / (256 * kAcc));
    const int64_t grid = (int64_t)a.B * (a.H / a.G) * chunks;
    return sink_launch(true, sink_acc_kernel, grid, 256, 0, s, a, lse, acc, acc_out, chunks);
}

}  // namespace hils
