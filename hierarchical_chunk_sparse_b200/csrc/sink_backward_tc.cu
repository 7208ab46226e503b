// Backward of the window-and-sink attention on the 5th-generation tensor cores (bf16;
// formulas in sink_common.cuh): two persistent kernels, so that no sum is an atomic.
//
// dQ, query-major: items of two 128-row query tiles A and B as in the prefill, 64-key tiles.
//   S = Q K^T, T = dO V^T (M = 128 rows, N = 64 keys), dS = p (T - D) in bf16 over S,
//   dQ += dS K with dS from TMEM; scale is applied once to the float32 sum.
//   TMEM: S_A [0,64), S_B [64,128), T_A [128,192), T_B [192,256), dQ_A [256,384), dQ_B [384,512).
// dK and dV, key-major: items of one 128-key block of a (b, key-value head) and a segment of
//   its steps, a step being 64 queries of one head of the group.
//   S^T = K Q^T, T^T = V dO^T (M = 128 keys, N = 64 queries), P^T and dS^T in bf16 over them,
//   dV += P^T dO, dK += dS^T Q with P^T, dS^T from TMEM. S^T and T^T are double-buffered: even
//   steps belong to softmax warps 0-3, odd ones to warps 4-7. lse and D of a step's queries
//   are staged in shared memory, since a thread owns a key and runs over the queries.
//   TMEM: S^T [0,64), [64,128), T^T [128,192), [192,256), dV [256,384), dK [384,512).
// Both recompute S and T: 7 products instead of the 5 of one kernel that would have to add
// dQ (or dK and dV) across CTAs with atomics, whose order changes the result.
// Warp roles and waits as in the prefill: 8 softmax warps, MMA, TMA.
#include "sink_tc.cuh"

namespace hils {
namespace {

using namespace tc;

constexpr int kThreads = 384, kMmaWarp = 8, kLoadWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// lse in log2 units; +inf for a row that sees nothing, so that exp2(s - L) = 0
__device__ __forceinline__ float log2_lse(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// 32 columns of p = exp2(s scale2 - L), 0 where masked, and ds = p (t - D).
template <typename LF, typename DF>
__device__ __forceinline__ void grad_columns(const uint32_t (&s)[32], const uint32_t (&t)[32], uint32_t mk, bool full,
                                             float scale2, LF L, DF Dv, uint32_t (&p)[16], uint32_t (&ds)[16]) {
#pragma unroll
    for (int q = 0; q < 32; q += 2) {
        float v0 = fmaf(__uint_as_float(s[q]), scale2, -L(q)), v1 = fmaf(__uint_as_float(s[q + 1]), scale2, -L(q + 1));
        if (!full) {
            v0 = (mk >> q) & 1u ? v0 : -INFINITY;
            v1 = (mk >> (q + 1)) & 1u ? v1 : -INFINITY;
        }
        v0 = exp2_ftz(v0);
        v1 = exp2_ftz(v1);
        float d0 = v0 * (__uint_as_float(t[q]) - Dv(q)), d1 = v1 * (__uint_as_float(t[q + 1]) - Dv(q + 1));
        if (!full) {  // t may be anything there
            d0 = (mk >> q) & 1u ? d0 : 0.f;
            d1 = (mk >> (q + 1)) & 1u ? d1 : 0.f;
        }
        p[q / 2] = pack_bf16(v0, v1);
        ds[q / 2] = pack_bf16(d0, d1);
    }
}

// ---------------------------------------------------------------------------- dQ

namespace dq {
constexpr int kM = 128, kKeys = 64, kStages = 3;
enum {
    kBarXfull = 0,   // + tile: Q, dO
    kBarXfree = 2,   // + tile
    kBarKfull = 4,   // + stage: K and V
    kBarKfree = 7,   // + stage (both tiles)
    kBarST = 10,     // + tile: S, T written
    kBarP = 12,      // + tile: dS written (4 warps)
    kBarPV = 14,     // + tile: dS K completed
    kBarOfree = 16,  // + tile: dQ read (4 warps)
    kBarDrain = 18,  // + tile
    kNumBars = 20
};
template <int D>
struct Smem {
    static constexpr int kX = kM * D * 2, kY = kKeys * D * 2;
    static constexpr int kQ = 0, kDO = 2 * kX, kK = 4 * kX, kV = kK + kStages * kY;
    static constexpr int kBars = kV + kStages * kY, kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 16 + 1024;  // + alignment slack
};
struct Args {
    SinkBwdArgs a;
    int P, qt, nqb, items, sink_box;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) sink_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                 const __grid_constant__ CUtensorMap tmDO,
                                                                 const __grid_constant__ CUtensorMap tmK,
                                                                 const __grid_constant__ CUtensorMap tmV,
                                                                 const __grid_constant__ CUtensorMap tmKs,
                                                                 const __grid_constant__ CUtensorMap tmVs, Args f) {
    extern __shared__ uint8_t smem_raw[];
    using L = Smem<D>;
    constexpr int kBlocks = D / 64, kXBlk = kM * 128, kYBlk = kKeys * 128;
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const SinkBwdArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;
    auto item = [&](int j) { return RowItem<kKeys>(j, a.B, a.H, a.G, f.P, f.qt, f.nqb, a.Lq, a.N, a.W, a.A, 1); };

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (i >= kBarKfree && i < kBarKfree + kStages) cnt = 2;
            if ((i >= kBarP && i < kBarP + 2) || (i >= kBarOfree && i < kBarOfree + 2)) cnt = 4;
            mbar_init(pipe.bar(i), cnt);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(sbase + L::kMisc, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp == kLoadWarp) {
        if (lane == 0) {
            int nx[2] = {0, 0}, g = 0;
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= f.items) break;
                const RowItem<kKeys> it = item(j);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (it.last(x) < 0) continue;
                    if (nx[x] > 0 && !(ok = pipe.wait(kBarXfree + x, (nx[x] - 1) & 1))) break;
                    mbar_expect_tx(pipe.bar(kBarXfull + x), 2 * L::kX);
                    ++nx[x];
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c) {
                        const uint32_t o = sbase + x * L::kX + c * kXBlk;
                        tma_load_4d(o + L::kQ, &tmQ, pipe.bar(kBarXfull + x), c * 64, it.i0 + x * f.qt, it.h, it.b);
                        tma_load_4d(o + L::kDO, &tmDO, pipe.bar(kBarXfull + x), c * 64, it.i0 + x * f.qt, it.h, it.b);
                    }
                }
                for (int e = it.e0; e < it.e1 && ok; ++e, ++g) {
                    const int s = g % kStages, k0 = it.first_key(e);
                    if (g >= kStages && !(ok = pipe.wait(kBarKfree + s, (g / kStages - 1) & 1))) break;
                    const bool sink = e < it.sp.ns;
                    mbar_expect_tx(pipe.bar(kBarKfull + s), 2u * (sink ? f.sink_box : kKeys) * D * 2);
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c) {
                        const uint32_t o = sbase + s * L::kY + c * kYBlk;
                        tma_load_4d(o + L::kK, sink ? &tmKs : &tmK, pipe.bar(kBarKfull + s), c * 64, k0, it.hk, it.b);
                        tma_load_4d(o + L::kV, sink ? &tmVs : &tmV, pipe.bar(kBarKfull + s), c * 64, k0, it.hk, it.b);
                    }
                }
            }
            for (int x = 0; x < 2; ++x) pipe.drain(kBarXfull + x, nx[x]);
            for (int s = 0; s < kStages; ++s) pipe.drain(kBarKfull + s, g > s ? (g - s + kStages - 1) / kStages : 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        const int x = warp - kMmaWarp;
        if (lane == 0) {
            int g = 0, c = 0, n = 0;
            bool ok = true;
            const uint32_t q = sbase + L::kQ + x * L::kX, go = sbase + L::kDO + x * L::kX;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= f.items) break;
                const RowItem<kKeys> it = item(j);
                const int last = it.last(x);
                if (last >= 0 && !(ok = pipe.wait(kBarXfull + x, n & 1))) break;
                tc_fence_after();
                bool first = true;
                for (int e = it.e0; e < it.e1; ++e, ++g) {
                    const int nk = it.keys(x, e), s = g % kStages;
                    if (!(ok = pipe.wait(kBarKfull + s, (g / kStages) & 1))) break;
                    if (nk <= 0) {
                        pipe.arrive(kBarKfree + s);
                        continue;
                    }
                    if (c > 0 && !(ok = pipe.wait(kBarPV + x, (c - 1) & 1))) break;
                    tc_fence_after();
                    const int n16 = (nk + 15) & ~15;
                    const uint32_t kb = sbase + L::kK + s * L::kY, vb = sbase + L::kV + s * L::kY;
                    const uint32_t id = idesc_bf16(kM, n16, false);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t xo = (k >> 2) * kXBlk + (k & 3) * 32, yo = (k >> 2) * kYBlk + (k & 3) * 32;
                        mma_ss(tmem + x * 64, smem_desc(q + xo, 16, 1024), smem_desc(kb + yo, 16, 1024), id, k > 0);
                    }
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t xo = (k >> 2) * kXBlk + (k & 3) * 32, yo = (k >> 2) * kYBlk + (k & 3) * 32;
                        mma_ss(tmem + 128 + x * 64, smem_desc(go + xo, 16, 1024), smem_desc(vb + yo, 16, 1024), id, k > 0);
                    }
                    mma_commit(pipe.bar(kBarST + x));
                    if (e == last) mma_commit(pipe.bar(kBarXfree + x));
                    if (!(ok = pipe.wait(kBarP + x, c & 1))) break;
                    if (first && n > 0 && !(ok = pipe.wait(kBarOfree + x, (n - 1) & 1))) break;
                    tc_fence_after();
                    for (int k = 0; k < n16 / 16; ++k)
                        mma_ts(tmem + 256 + x * 128, tmem + x * 64 + k * 8, smem_desc(kb + k * 2048, kYBlk, 1024),
                               idesc_bf16(kM, D, true), !first || k > 0);
                    mma_commit(pipe.bar(kBarKfree + s));
                    mma_commit(pipe.bar(kBarPV + x));
                    first = false;
                    ++c;
                }
                if (last >= 0) ++n;
            }
            mma_commit(pipe.bar(kBarDrain + x));
            pipe.drain(kBarDrain + x, 1);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int x = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_col = tmem + lanes + x * 64, t_col = s_col + 128, o_col = tmem + lanes + 256 + x * 128;
        const float scale2 = a.scale * kLog2e;
        bool ok = true;
        int c = 0;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.items) break;
            const RowItem<kKeys> it = item(j);
            const int h = it.h + row / f.qt, i = it.i0 + x * f.qt + row % f.qt, t = a.N - a.Lq + i;
            const bool have = i < a.Lq;
            const int64_t place = ((int64_t)it.b * a.H + h) * a.Lq + i;
            const float Lr = have ? log2_lse(__ldg(a.lse + place)) : INFINITY;
            const float Dr = have ? __ldg(a.Dv + place) : 0.f;
            bool any_tile = false;
            for (int e = it.e0; e < it.e1; ++e) {
                const int n = it.keys(x, e);
                if (n <= 0) continue;
                any_tile = true;
                int lo, hi, as;
                it.columns(e, n, t, a.W, &lo, &hi, &as);
                if (!have) hi = as = 0;
                const bool full = __all_sync(kFull, lo <= 0 && hi == kKeys);
                if (!(ok = pipe.wait_warp(kBarST + x, c & 1))) break;
                tc_fence_after();
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    if (ch * 32 >= n) continue;
                    const uint32_t mk = full ? kFull : range_bits(lo, hi, ch * 32) | range_bits(0, as, ch * 32);
                    uint32_t ds[16];
                    if (__any_sync(kFull, mk != 0)) {
                        uint32_t s[32], u[32], p[16];
                        tmem_ld32(s_col + ch * 32, s);
                        tmem_ld32(t_col + ch * 32, u);
                        tmem_wait_ld();
                        grad_columns(s, u, mk, full, scale2, [&](int) { return Lr; }, [&](int) { return Dr; }, p, ds);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) ds[q] = 0u;
                    }
                    tmem_st16(s_col + ch * 16, ds);  // columns whose S has been read
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarP + x);
                ++c;
            }
            if (!ok) break;
            if (any_tile) {
                if (!(ok = pipe.wait_warp(kBarPV + x, (c - 1) & 1))) break;
                tc_fence_after();
            }
            bf16 *orow = static_cast<bf16 *>(a.dQ.ptr) + it.b * a.dQ.sb + h * a.dQ.sh + (int64_t)i * a.dQ.st;
#pragma unroll
            for (int part = 0; part < D / 32; ++part) {
                uint32_t o[32];
                if (any_tile) {
                    tmem_ld32(o_col + part * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = 0u;
                }
                if (!have) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(orow + part * 32);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16(__uint_as_float(o[8 * q + 2 * k]) * a.scale, __uint_as_float(o[8 * q + 2 * k + 1]) * a.scale);
                    dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (any_tile) {
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarOfree + x);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, kTmemCols);
    }
}
}  // namespace dq

// ---------------------------------------------------------------------------- dK, dV

namespace dkv {
constexpr int kM = kSinkKeys, kRows = 64, kStages = 3;
enum {
    kBarXfull = 0,    // + buffer: K, V of an item
    kBarXfree = 2,    // + buffer: its last S, T completed
    kBarYfull = 4,    // + stage: Q, dO (bytes), lse and D (32 arrivals)
    kBarYfree = 7,    // + stage: the products that read it completed
    kBarST = 10,      // + buffer: S^T, T^T written
    kBarP = 12,       // + buffer: P^T, dS^T written (4 warps)
    kBarPV = 14,      // + buffer: the products that read them completed
    kBarDone = 16,    // dK, dV of an item final
    kBarOfree = 17,   // dK, dV read (8 warps)
    kBarDrain = 18,
    kNumBars = 19
};
template <int D>
struct Smem {
    static constexpr int kX = kM * D * 2, kY = kRows * D * 2;
    static constexpr int kK = 0, kV = 2 * kX, kQ = 4 * kX, kDO = kQ + kStages * kY;
    static constexpr int kSc = kDO + kStages * kY;  // per stage: lse (log2 units) [64], D [64]
    static constexpr int kBars = kSc + kStages * kRows * 8, kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 24 + 1024;  // + alignment slack
};
struct Args {
    SinkBwdArgs a;
    int items;  // of one (b, key-value head)
};
struct Item {
    int xb, b, hk, j0, i0, i1, tiles, s0, s1, nseg, index;
};
__device__ __forceinline__ Item decode(const Args &f, int j) {
    const SinkBwdArgs &a = f.a;
    const int Hk = a.H / a.G, heads = a.B * Hk;
    Item it;
    it.xb = j % heads;  // the blocks with most steps (the first ones of a causal range) come first
    const int x = j / heads;
    it.b = it.xb / Hk;
    it.hk = it.xb % Hk;
    const SinkItem k = sink_item(a, x);
    it.j0 = k.blk * kM;
    it.nseg = k.nseg;
    it.index = it.xb * f.items + x;
    sink_rows_of_block(a, it.j0, min(kM, a.N - it.j0), &it.i0, &it.i1);
    it.tiles = (it.i1 - it.i0 + kRows - 1) / kRows;
    const int64_t steps = (int64_t)a.G * it.tiles;
    it.s0 = (int)(steps * k.seg / k.nseg);
    it.s1 = (int)(steps * (k.seg + 1) / k.nseg);
    return it;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) sink_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                  const __grid_constant__ CUtensorMap tmDO,
                                                                  const __grid_constant__ CUtensorMap tmK,
                                                                  const __grid_constant__ CUtensorMap tmV, Args f,
                                                                  int total) {
    extern __shared__ uint8_t smem_raw[];
    using L = Smem<D>;
    constexpr int kBlocks = D / 64, kXBlk = kM * 128, kYBlk = kRows * 128;
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const SinkBwdArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    float *scal = reinterpret_cast<float *>(smem + L::kSc);
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (i >= kBarYfull && i < kBarYfull + kStages) cnt = 33;
            if (i >= kBarP && i < kBarP + 2) cnt = 4;
            if (i == kBarOfree) cnt = 8;
            mbar_init(pipe.bar(i), cnt);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(sbase + L::kMisc, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp == kLoadWarp) {
        int n = 0, g = 0;  // items with steps, steps
        bool ok = true;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            if (it.s0 >= it.s1) continue;
            const int xb = n & 1;
            if (n >= 2 && !(ok = pipe.wait_warp(kBarXfree + xb, ((n >> 1) - 1) & 1))) break;
            if (lane == 0) {
                mbar_expect_tx(pipe.bar(kBarXfull + xb), 2 * L::kX);
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
                    const uint32_t o = sbase + xb * L::kX + c * kXBlk;
                    tma_load_4d(o + L::kK, &tmK, pipe.bar(kBarXfull + xb), c * 64, it.j0, it.hk, it.b);
                    tma_load_4d(o + L::kV, &tmV, pipe.bar(kBarXfull + xb), c * 64, it.j0, it.hk, it.b);
                }
            }
            ++n;
            float sc[4];  // lse and D of rows lane, lane + 32 of the next step
            auto scalars = [&](int s) {
                const int64_t row0 = ((int64_t)it.b * a.H + it.hk * a.G + s / it.tiles) * a.Lq;
                const int q0 = it.i0 + (s % it.tiles) * kRows;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int i = q0 + lane + 32 * m;
                    sc[m] = i < it.i1 ? log2_lse(__ldg(a.lse + row0 + i)) : INFINITY;
                    sc[2 + m] = i < it.i1 ? __ldg(a.Dv + row0 + i) : 0.f;
                }
            };
            scalars(it.s0);
            for (int s = it.s0; s < it.s1; ++s, ++g) {
                const int st = g % kStages;
                if (g >= kStages && !(ok = pipe.wait_warp(kBarYfree + st, (g / kStages - 1) & 1))) break;
                if (lane == 0) {
                    mbar_expect_tx(pipe.bar(kBarYfull + st), 2 * L::kY);
                    const int h = it.hk * a.G + s / it.tiles, q0 = it.i0 + (s % it.tiles) * kRows;
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c) {
                        const uint32_t o = sbase + st * L::kY + c * kYBlk;
                        tma_load_4d(o + L::kQ, &tmQ, pipe.bar(kBarYfull + st), c * 64, q0, h, it.b);
                        tma_load_4d(o + L::kDO, &tmDO, pipe.bar(kBarYfull + st), c * 64, q0, h, it.b);
                    }
                }
                float *d = scal + st * 2 * kRows + lane;
                d[0] = sc[0];
                d[32] = sc[1];
                d[64] = sc[2];
                d[96] = sc[3];
                pipe.arrive(kBarYfull + st);
                if (s + 1 < it.s1) scalars(s + 1);
            }
        }
        if (lane == 0) {
            for (int x = 0; x < 2; ++x) pipe.drain(kBarXfull + x, n > x ? (n - x + 1) / 2 : 0);
            // on a stop, a stage's phase may lack this warp's own arrivals only if its copy was not started
            for (int s = 0; s < kStages; ++s) pipe.drain(kBarYfull + s, g > s ? (g - s + kStages - 1) / kStages : 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            int n = 0, c = 0;  // items with steps, steps
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= total) break;
                const Item it = decode(f, j);
                if (it.s0 >= it.s1) continue;
                const int xb = n & 1, steps = it.s1 - it.s0;
                const uint32_t kb = sbase + L::kK + xb * L::kX, vb = sbase + L::kV + xb * L::kX;
                if (!(ok = pipe.wait(kBarXfull + xb, (n >> 1) & 1))) break;
                // step i: S^T, T^T of step i, then the sums of step i - 1
                for (int i = 0; i <= steps && ok; ++i) {
                    if (i < steps) {
                        const int cc = c + i, st = cc % kStages, p = cc & 1;
                        if (!(ok = pipe.wait(kBarYfull + st, (cc / kStages) & 1))) break;
                        if (cc >= 2 && !(ok = pipe.wait(kBarPV + p, ((cc >> 1) - 1) & 1))) break;
                        tc_fence_after();
                        const uint32_t qb = sbase + L::kQ + st * L::kY, gb = sbase + L::kDO + st * L::kY;
                        const uint32_t id = idesc_bf16(kM, kRows, false);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t xo = (k >> 2) * kXBlk + (k & 3) * 32, yo = (k >> 2) * kYBlk + (k & 3) * 32;
                            mma_ss(tmem + p * 64, smem_desc(kb + xo, 16, 1024), smem_desc(qb + yo, 16, 1024), id, k > 0);
                        }
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t xo = (k >> 2) * kXBlk + (k & 3) * 32, yo = (k >> 2) * kYBlk + (k & 3) * 32;
                            mma_ss(tmem + 128 + p * 64, smem_desc(vb + xo, 16, 1024), smem_desc(gb + yo, 16, 1024), id, k > 0);
                        }
                        mma_commit(pipe.bar(kBarST + p));
                        if (i + 1 == steps) mma_commit(pipe.bar(kBarXfree + xb));
                    }
                    if (i > 0) {
                        const int cc = c + i - 1, st = cc % kStages, p = cc & 1;
                        if (!(ok = pipe.wait(kBarP + p, (cc >> 1) & 1))) break;
                        if (i == 1 && n > 0 && !(ok = pipe.wait(kBarOfree, (n - 1) & 1))) break;
                        tc_fence_after();
                        const uint32_t qb = sbase + L::kQ + st * L::kY, gb = sbase + L::kDO + st * L::kY;
                        const uint32_t id = idesc_bf16(kM, D, true);
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            mma_ts(tmem + 256, tmem + p * 64 + k * 8, smem_desc(gb + k * 2048, kYBlk, 1024), id, i > 1 || k > 0);
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            mma_ts(tmem + 384, tmem + 128 + p * 64 + k * 8, smem_desc(qb + k * 2048, kYBlk, 1024), id,
                                   i > 1 || k > 0);
                        mma_commit(pipe.bar(kBarPV + p));
                        mma_commit(pipe.bar(kBarYfree + st));
                        if (i == steps) mma_commit(pipe.bar(kBarDone));
                    }
                }
                c += steps;
                ++n;
            }
            mma_commit(pipe.bar(kBarDrain));
            pipe.drain(kBarDrain, 1);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;  // w: steps of its parity; then dV or dK
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_col = tmem + lanes + w * 64, t_col = s_col + 128, o_col = tmem + lanes + 256 + w * 128;
        const float scale2 = a.scale * kLog2e;
        const int off = a.N - a.Lq;
        bool ok = true;
        int c = 0, n = 0;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            const int key = it.j0 + row;
            const int steps = max(0, it.s1 - it.s0);
            for (int i = 0; i < steps; ++i) {
                const int cc = c + i;
                if ((cc & 1) != w) continue;
                const int st = cc % kStages, q0 = it.i0 + ((it.s0 + i) % it.tiles) * kRows;
                // columns (queries) that see this key
                const int lo = key - off - q0, end = min(kRows, it.i1 - q0);
                const int hi = key < a.A ? end : min(end, (int)min((int64_t)key + a.W - off - q0, (int64_t)kRows));
                const bool full = __all_sync(kFull, lo <= 0 && hi == kRows);
                if (!(ok = pipe.wait_warp(kBarYfull + st, (cc / kStages) & 1))) break;
                if (!(ok = pipe.wait_warp(kBarST + w, (cc >> 1) & 1))) break;
                tc_fence_after();
                const float *sc = scal + st * 2 * kRows;
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const uint32_t mk = full ? kFull : range_bits(lo, hi, ch * 32);
                    uint32_t p[16], ds[16];
                    if (__any_sync(kFull, mk != 0)) {
                        uint32_t s[32], u[32];
                        float Lc[32], Dc[32];
                        tmem_ld32(s_col + ch * 32, s);
                        tmem_ld32(t_col + ch * 32, u);
#pragma unroll
                        for (int q = 0; q < 32; q += 4) {
                            *reinterpret_cast<float4 *>(&Lc[q]) = *reinterpret_cast<const float4 *>(sc + ch * 32 + q);
                            *reinterpret_cast<float4 *>(&Dc[q]) = *reinterpret_cast<const float4 *>(sc + kRows + ch * 32 + q);
                        }
                        tmem_wait_ld();
                        grad_columns(s, u, mk, full, scale2, [&](int q) { return Lc[q]; }, [&](int q) { return Dc[q]; }, p, ds);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) p[q] = ds[q] = 0u;
                    }
                    tmem_st16(s_col + ch * 16, p);  // columns whose S, T have been read
                    tmem_st16(t_col + ch * 16, ds);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarP + w);
            }
            if (!ok) break;
            c += steps;
            if (steps > 0) {
                if (!(ok = pipe.wait_warp(kBarDone, n & 1))) break;
                tc_fence_after();
                ++n;
            }
            // ---- warps 0-3: dV, warps 4-7: dK
            const float f_out = w ? a.scale : 1.f;
            const MutView &v = w ? a.dK : a.dV;
            bf16 *orow = static_cast<bf16 *>(v.ptr) + it.b * v.sb + it.hk * v.sh + (int64_t)key * v.st;
            float *prow = it.nseg > 1 ? a.part + ((int64_t)it.index * 2 * kSinkKeys + (w ? 0 : kSinkKeys) + row) * D : nullptr;
#pragma unroll
            for (int part = 0; part < D / 32; ++part) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld32(o_col + part * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = 0u;
                }
                if (prow) {
#pragma unroll
                    for (int q = 0; q < 32; q += 4)
                        *reinterpret_cast<float4 *>(prow + part * 32 + q) =
                            make_float4(__uint_as_float(o[q]) * f_out, __uint_as_float(o[q + 1]) * f_out,
                                        __uint_as_float(o[q + 2]) * f_out, __uint_as_float(o[q + 3]) * f_out);
                } else if (key < a.N) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = pack_bf16(__uint_as_float(o[8 * q + 2 * k]) * f_out, __uint_as_float(o[8 * q + 2 * k + 1]) * f_out);
                        reinterpret_cast<uint4 *>(orow + part * 32)[q] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            if (steps > 0) {
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarOfree);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, kTmemCols);
    }
}
}  // namespace dkv

template <int D>
hils_status run(const SinkBwdArgs &a, const CUtensorMap (&m)[10], dq::Args q, dkv::Args k, int total, cudaStream_t s) {
    static KernelSetup s0, s1;
    int p0 = 0, p1 = 0;
    const auto f0 = dq::sink_dq_tc_kernel<D>;
    const auto f1 = dkv::sink_dkv_tc_kernel<D>;
    hils_status st = kernel_setup(s0, (const void *)f0, kThreads, dq::Smem<D>::kBytes, &p0);
    if (st != HILS_OK) return st;
    st = kernel_setup(s1, (const void *)f1, kThreads, dkv::Smem<D>::kBytes, &p1);
    if (st != HILS_OK) return st;
    if (p0 < 1 || p1 < 1) return HILS_ERR_CUDA;
    const int sms = device_sm_count();
    f0<<<q.items < sms ? q.items : sms, kThreads, dq::Smem<D>::kBytes, s>>>(m[0], m[1], m[2], m[3], m[4], m[5], q);
    st = record_cuda_error(cudaGetLastError());
    if (st != HILS_OK) return st;
    f1<<<total < sms ? total : sms, kThreads, dkv::Smem<D>::kBytes, s>>>(m[6], m[7], m[8], m[9], k, total);
    return record_cuda_error(cudaGetLastError());
}

}  // namespace

bool launch_sink_backward_tc(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s, hils_status *st) {
    if (dt != HILS_BF16 || a.N == 0) return false;
    const int Hk = a.H / a.G;
    dq::Args q{};
    q.a = a;
    q.P = sink_pack(a.G);
    q.qt = dq::kM / q.P;
    q.nqb = (a.Lq + 2 * q.qt - 1) / (2 * q.qt);
    const int64_t qi = (int64_t)a.B * (a.H / q.P) * q.nqb;
    dkv::Args k{};
    k.a = a;
    k.items = (int)sink_key_items(a);
    const int64_t ki = (int64_t)k.items * a.B * Hk;
    if (qi > 0x7fffffffll - 1024 || ki > 0x7fffffffll - 1024) return false;
    q.items = (int)qi;
    const int sinks = a.A > 0 ? a.A : 1;
    q.sink_box = sinks < dq::kKeys ? (sinks + 15) & ~15 : dq::kKeys;
    CUtensorMap m[10];
    if (!make_view_map(&m[0], a.Q, a.B, a.H, a.Lq, d, q.qt, q.P) || !make_view_map(&m[1], a.dO, a.B, a.H, a.Lq, d, q.qt, q.P) ||
        !make_view_map(&m[2], a.K, a.B, Hk, a.N, d, dq::kKeys, 1) || !make_view_map(&m[3], a.V, a.B, Hk, a.N, d, dq::kKeys, 1) ||
        !make_view_map(&m[4], a.K, a.B, Hk, sinks, d, q.sink_box, 1) ||
        !make_view_map(&m[5], a.V, a.B, Hk, sinks, d, q.sink_box, 1) ||
        !make_view_map(&m[6], a.Q, a.B, a.H, a.Lq, d, dkv::kRows, 1) || !make_view_map(&m[7], a.dO, a.B, a.H, a.Lq, d, dkv::kRows, 1) ||
        !make_view_map(&m[8], a.K, a.B, Hk, a.N, d, dkv::kM, 1) || !make_view_map(&m[9], a.V, a.B, Hk, a.N, d, dkv::kM, 1))
        return false;
    *st = d == 64 ? run<64>(a, m, q, k, (int)ki, s) : run<128>(a, m, q, k, (int)ki, s);
    return true;
}

}  // namespace hils
