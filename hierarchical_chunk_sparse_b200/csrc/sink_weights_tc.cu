// Accumulated attention weights on the 5th-generation tensor cores (bf16; formulas in
// sink_common.cuh), key-major: a thread owns a key and adds up exp2(s - lse) over the
// queries, so that no sum crosses threads.
//
// Items are 256 keys of one (b, key-value head), two 128-key tiles A and B, and a segment of
// their steps; a step is 128 query rows: of one head, or, in a call of few queries, of several
// heads of the group (the rows stay full). S^T = K Q^T (M = 128 keys, N = 128 rows, K = d) into
// TMEM, double-buffered per tile; the keys of the next item and the rows of the next steps are
// loaded meanwhile. The rows' lse (log2 units) are staged in shared memory.
// The exponentials bound it (16 a cycle and SM on the MUFU against 8192 products): every
// fourth one is evaluated on the FMA pipe instead.
// Warps 0-7, 8-15: the keys of tile A, B (TMEM lane quadrant w % 4), four warps for its even
// steps and four for the odd: with one warp per quadrant and tile the loads and exponentials
// waited on their latencies; 16, 17: tcgen05.mma of A, B; 18: TMA; 19: lse, fetched two steps
// ahead.
// A prompt of 8192 queries and keys (32 heads on 8, d = 128, causal) takes 342 us (10106 on the CUDA
// cores; 165 by its products, 240 by its exponentials on the MUFU alone): the MUFU is 66 % busy,
// the issue slots 58 %. 64 queries of 64K tokens take 72 us, 30 by the MUFU: an item has only two
// steps, and half its time goes into its keys' arrival and its sums' departure.
// TMEM: S_A [0,128), [128,256); S_B [256,384), [384,512).
#include "sink_tc.cuh"

namespace hils {
namespace {

using namespace tc;

// exp2_fma (fast_math.cuh; its polynomial) for two values that are at most 127, in packed float32 arithmetic: 13
// instructions for the pair. Below -126 the result is some subnormal number, below -127 (-inf too) 2^-149.
__device__ __forceinline__ float2 exp2_fma2(float2 x) {
    auto both = [](float c) { return make_float2(c, c); };
    x = make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
    const float2 t = add2(x, both(12582912.f));
    const float2 f = fma2(add2(t, both(-12582912.f)), both(-1.f), x);
    float2 p = fma2(both(1.327647129e-03f), f, both(9.675540961e-03f));
    p = fma2(p, f, both(5.550713092e-02f));
    p = fma2(p, f, both(2.402212024e-01f));
    p = fma2(p, f, both(6.931469440e-01f));
    p = fma2(p, f, both(1.000000119e+00f));
    // t holds 0x4b400000 + j: shifted left by 23 its upper bits fall away
    return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}

constexpr int kM = 128, kKeys = 2 * kM, kRows = 128, kStages = 3, kThreads = 640, kMmaWarp = 16, kLoadWarp = 18, kLseWarp = 19;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

enum {
    kBarXfull = 0,   // + buffer: the item's keys
    kBarXfree = 2,   // + buffer (both tiles)
    kBarYfull = 4,   // + stage: query rows (bytes) and lse (32 arrivals)
    kBarYfree = 7,   // + stage: lse read by both tiles' 4 warps (so the products are done too)
    kBarS = 10,      // + 2 * tile + buffer: S^T written
    kBarSfree = 14,  // + 2 * tile + buffer: S^T read (4 warps)
    kBarDrain = 18,  // + tile
    kBarHalf = 20,   // + 4 tile + quadrant: the odd steps' sums are in hsum
    kBarHalfFree = 28,  // + the same: read
    kNumBars = 36
};
template <int D>
struct Smem {
    static constexpr int kX = kM * D * 2, kY = kRows * D * 2;
    static constexpr int kK = 0, kQ = 4 * kX, kL = kQ + kStages * kY;
    static constexpr int kH = kL + kStages * kRows * 4;  // sums of the odd steps
    static constexpr int kBars = kH + kKeys * 4, kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 16;
};
struct Args {
    SinkBwdArgs a;
    int P, qn;   // heads and queries of each in a step
    int items;   // of one (b, key-value head)
    int Hk, heads, packs, qshift;  // key-value heads of a batch, of all; head packs of a group; qn = 1 << qshift
};
struct Item {
    int xb, b, hk, j0, i0, tiles, s0, s1, nseg, index;
    int a0, a1, b0, b1;  // the queries that see a key of A, B
};
__device__ __forceinline__ Item decode(const Args &f, int j) {
    const SinkBwdArgs &a = f.a;
    Item it;
    const int y = j / f.heads;
    it.xb = j - y * f.heads;  // the blocks with most steps (the first ones of a causal range) come first
    it.b = it.xb / f.Hk;
    it.hk = it.xb - it.b * f.Hk;
    const SinkItem k = sink_item(a, y);
    it.j0 = k.blk * kKeys;
    it.nseg = k.nseg;
    it.index = it.xb * f.items + y;
    it.b0 = it.b1 = 0;
    sink_rows_of_block(a, it.j0, min(kM, a.N - it.j0), &it.a0, &it.a1);
    if (it.j0 + kM < a.N) sink_rows_of_block(a, it.j0 + kM, min(kM, a.N - it.j0 - kM), &it.b0, &it.b1);
    const bool hasA = it.a0 < it.a1, hasB = it.b0 < it.b1;
    it.i0 = hasA ? it.a0 : it.b0;
    const int i1 = hasB ? max(it.b1, hasA ? it.a1 : 0) : it.a1;
    it.tiles = hasA || hasB ? (i1 - it.i0 + f.qn - 1) >> f.qshift : 0;
    const int steps = f.packs * it.tiles;
    it.s0 = 0;
    it.s1 = steps;
    if (k.nseg > 1) {
        it.s0 = (int)((int64_t)steps * k.seg / k.nseg);
        it.s1 = (int)((int64_t)steps * (k.seg + 1) / k.nseg);
    }
    return it;
}

// A walk over an item's steps: the step's query tile and head pack, and its stage with the
// stage's phase (kept over the items).
struct Walk {
    int st = 0;
    uint32_t ph = 0;
    int tile = 0, h = 0;
    __device__ __forceinline__ void start(const Item &it) {
        h = it.s0 > 0 ? it.s0 / it.tiles : 0;
        tile = it.s0 - h * it.tiles;
    }
    __device__ __forceinline__ void next(const Item &it) {
        if (++st == kStages) {
            st = 0;
            ph ^= 1u;
        }
        if (++tile == it.tiles) {
            tile = 0;
            ++h;
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) sink_weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                      const __grid_constant__ CUtensorMap tmK, Args f,
                                                                      int total) {
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's atoms: no room for slack
    using L = Smem<D>;
    constexpr int kBlocks = D / 64, kBlk = kM * 128;
    const SinkBwdArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    float *lse = reinterpret_cast<float *>(smem + L::kL), *hsum = reinterpret_cast<float *>(smem + L::kH);
    if (sbase & 1023u) {  // an alignment that the launch has to give
        if (tid == 0) atomicOr(a.status, 1u);
        return;
    }
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (i == kBarXfree || i == kBarXfree + 1) cnt = 2;
            if (i >= kBarYfull && i < kBarYfull + kStages) cnt = 33;
            if (i >= kBarYfree && i < kBarYfree + kStages) cnt = 8;
            if (i >= kBarSfree && i < kBarSfree + 4) cnt = 4;
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
        Walk w;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            if (it.s0 >= it.s1) continue;
            const int xb = n & 1;
            if (n >= 2 && !(ok = pipe.wait_warp(kBarXfree + xb, ((n >> 1) - 1) & 1))) break;
            if (elect_one()) {
                mbar_expect_tx(pipe.bar(kBarXfull + xb), 2 * L::kX);
#pragma unroll
                for (int x = 0; x < 2; ++x)  // B's keys may lie behind the last one: zeros
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c)
                        tma_load_4d(sbase + L::kK + (2 * xb + x) * L::kX + c * kBlk, &tmK, pipe.bar(kBarXfull + xb), c * 64,
                                    it.j0 + x * kM, it.hk, it.b);
            }
            __syncwarp();
            ++n;
            w.start(it);
            for (int s = it.s0; s < it.s1; ++s, ++g) {
                if (g >= kStages && !(ok = pipe.wait_warp(kBarYfree + w.st, w.ph ^ 1u))) break;
                if (elect_one()) {
                    mbar_expect_tx(pipe.bar(kBarYfull + w.st), L::kY);
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c)
                        tma_load_4d(sbase + L::kQ + w.st * L::kY + c * kBlk, &tmQ, pipe.bar(kBarYfull + w.st), c * 64,
                                    it.i0 + w.tile * f.qn, it.hk * a.G + w.h * f.P, it.b);
                }
                __syncwarp();
                w.next(it);
            }
        }
        if (lane == 0) {
            for (int x = 0; x < 2; ++x) pipe.drain(kBarXfull + x, n > x ? (n - x + 1) / 2 : 0);
            for (int s = 0; s < kStages; ++s) pipe.drain(kBarYfull + s, g > s ? (g - s + kStages - 1) / kStages : 0);
        }
        __syncwarp();
    } else if (warp == kLseWarp) {
        int g = 0;
        bool ok = true;
        Walk w;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            if (it.s0 >= it.s1) continue;
            w.start(it);
            int tile = w.tile, h = w.h, next = it.s0;
            float sc[2][4];  // lse of rows lane + 32 m of the next two steps
            auto fetch = [&](float(&d)[4]) {
                if (next >= it.s1) return;
                ++next;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int row = lane + 32 * m, i = it.i0 + tile * f.qn + (row & (f.qn - 1));
                    const int64_t bh = (int64_t)it.b * a.H + it.hk * a.G + h * f.P + (row >> f.qshift);
                    d[m] = i < a.Lq ? __ldg(a.lse + bh * a.Lq + i) : -INFINITY;
                }
                if (++tile == it.tiles) {
                    tile = 0;
                    ++h;
                }
            };
            auto put = [&](float(&d)[4]) {
                if (g >= kStages && !(ok = pipe.wait_warp(kBarYfree + w.st, w.ph ^ 1u))) return;
#pragma unroll
                for (int m = 0; m < 4; ++m)  // nothing seen: exp2(s - inf) = 0
                    lse[w.st * kRows + lane + 32 * m] = d[m] == -INFINITY ? d[m] : -d[m] * kLog2e;
                pipe.arrive(kBarYfull + w.st);
                ++g;
                w.next(it);
                fetch(d);
            };
            fetch(sc[0]);
            fetch(sc[1]);
            for (int s = it.s0; s < it.s1 && ok; s += 2) {
                put(sc[0]);
                if (ok && s + 1 < it.s1) put(sc[1]);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        const int x = warp - kMmaWarp;
        int n = 0, c = 0;  // items with steps, steps of x
        bool ok = true;
        Walk w;
        const uint64_t kd0 = tile_desc(sbase + L::kK + x * L::kX, 16), qd0 = tile_desc(sbase + L::kQ, 16);
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            if (it.s0 >= it.s1) continue;
            const uint64_t kd = kd0 + (n & 1) * (2 * L::kX / 16);
            if (!(ok = pipe.wait_warp(kBarXfull + (n & 1), (n >> 1) & 1))) break;
            w.start(it);
            // first queries of the steps that x takes part in
            const int q_lo = (x ? it.b0 : it.a0) - f.qn - it.i0, q_hi = (x ? it.b1 : it.a1) - it.i0;
            for (int s = it.s0; s < it.s1; ++s, w.next(it)) {
                const int q = w.tile * f.qn, sb = 2 * x + (c & 1);
                if (!(ok = pipe.wait_warp(kBarYfull + w.st, w.ph))) break;
                if (q <= q_lo || q >= q_hi) {  // for the softmax warps
                    pipe.arrive_if(lane == 0, kBarYfree + w.st, 4);
                    continue;
                }
                if (c >= 2 && !(ok = pipe.wait_warp(kBarSfree + sb, ((c >> 1) - 1) & 1))) break;
                tc_fence_after();
                const uint64_t qd = qd0 + w.st * (L::kY / 16);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t o = ((k >> 2) * kBlk + (k & 3) * 32) / 16;
                        mma_ss(tmem + sb * 128, kd + o, qd + o, idesc_bf16(kM, kRows, false), k > 0);
                    }
                    mma_commit(pipe.bar(kBarS + sb));
                }
                __syncwarp();
                ++c;
            }
            if (!ok) break;
            if (elect_one()) mma_commit(pipe.bar(kBarXfree + (n & 1)));
            __syncwarp();
            ++n;
        }
        if (elect_one()) {
            mma_commit(pipe.bar(kBarDrain + x));
            pipe.drain(kBarDrain + x, 1);
        }
        __syncwarp();
    } else {
        const int x = warp >> 3, quad = warp & 3, odd = (warp >> 2) & 1, row = quad * 32 + lane, pair = 4 * x + quad;
        const int sb = 2 * x + odd;
        const uint32_t s_col = tmem + ((uint32_t)(quad * 32) << 16) + sb * 128;
        const float scale2 = a.scale * kLog2e, lowest = scale2 > 0.f ? -INFINITY : INFINITY;  // its logit is -inf
        const float2 scale22 = make_float2(scale2, scale2);
        const int off = a.N - a.Lq, Hk = a.H / a.G;
        bool ok = true;
        int c = 0, n = 0;
        Walk walk;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= total) break;
            const Item it = decode(f, j);
            const int key = it.j0 + x * kM + row;
            // its weight so far, for the warp that adds to it
            const int64_t at = ((int64_t)it.b * Hk + it.hk) * a.T + key;
            float old = 0.f;
            bool seen = false;
            if (!odd && it.nseg == 1 && key < a.N) {
                int k0, k1;
                sink_rows_of_block(a, key, 1, &k0, &k1);
                seen = k0 < k1;
                if (seen) old = a.acc[at];
            }
            float w = 0.f;
            walk.start(it);
            const int q_lo = (x ? it.b0 : it.a0) - f.qn - it.i0, q_hi = (x ? it.b1 : it.a1) - it.i0;
            // queries that see this key, from the item's first on
            const int see0 = key - off - it.i0;
            const int see1 = (int)min(key < a.A ? (int64_t)a.Lq : (int64_t)key + a.W - off, (int64_t)a.Lq) - it.i0;
            for (int s = it.s0; s < it.s1; ++s, walk.next(it)) {
                const int q = walk.tile * f.qn;
                if (q <= q_lo || q >= q_hi || (c++ & 1) != odd) continue;
                const int lo = see0 - q, hi = min(f.qn, see1 - q);  // of each head
                const bool full = __all_sync(kFull, lo <= 0 && hi == f.qn);
                if (!(ok = pipe.wait_warp(kBarS + sb, ((c - 1) >> 1) & 1))) break;
                if (!(ok = pipe.wait_warp(kBarYfull + walk.st, walk.ph))) break;  // complete: S came of it
                tc_fence_after();
                const float *lr = lse + walk.st * kRows;
                float2 z0 = make_float2(0.f, 0.f), z1 = z0;
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint32_t v[64];
                    tmem_ld32(s_col + ch * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                    tmem_ld32(s_col + ch * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                    tmem_wait_ld();
                    if (ch == 1) {  // S is handed back before the last exponentials
                        tc_fence_before();
                        __syncwarp();
                        pipe.arrive_if(lane == 0, kBarSfree + sb);
                    }
                    if (!full) {
                        uint32_t mk0 = range_bits(lo, hi, (ch * 64) & (f.qn - 1)), mk1 = range_bits(lo, hi, (ch * 64 + 32) & (f.qn - 1));
                        if (f.qn == 16) {
                            mk0 |= mk0 << 16;
                            mk1 |= mk1 << 16;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            v[e] = (mk0 >> e) & 1u ? v[e] : __float_as_uint(lowest);
                            v[32 + e] = (mk1 >> e) & 1u ? v[32 + e] : __float_as_uint(lowest);
                        }
                    }
#pragma unroll
                    for (int q4 = 0; q4 < 64; q4 += 8) {
                        float2 e[4];
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            const float4 L4 = *reinterpret_cast<const float4 *>(lr + ch * 64 + q4 + 2 * k);
                            e[k] = fma2(as2(v + q4 + 2 * k), scale22, make_float2(L4.x, L4.y));
                            e[k + 1] = fma2(as2(v + q4 + 2 * k + 2), scale22, make_float2(L4.z, L4.w));
                        }
#pragma unroll
                        for (int k = 0; k < 3; ++k) e[k] = make_float2(exp2_ftz(e[k].x), exp2_ftz(e[k].y));
                        e[3] = exp2_fma2(e[3]);
                        z0 = add2(z0, add2(e[0], e[1]));
                        z1 = add2(z1, add2(e[2], e[3]));
                    }
                }
                w += (z0.x + z0.y) + (z1.x + z1.y);
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarYfree + walk.st);
            }
            if (!ok) break;
            // the sum of the even steps, then that of the odd ones
            if (odd) {
                if (n > 0 && !(ok = pipe.wait_warp(kBarHalfFree + pair, (n - 1) & 1))) break;
                hsum[x * kM + row] = w;
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarHalf + pair);
                ++n;
                continue;
            }
            if (!(ok = pipe.wait_warp(kBarHalf + pair, n & 1))) break;
            w += hsum[x * kM + row];
            __syncwarp();
            pipe.arrive_if(lane == 0, kBarHalfFree + pair);
            ++n;
            if (key >= a.N) continue;
            if (it.nseg > 1) {
                a.part[(int64_t)it.index * kKeys + x * kM + row] = w;
            } else if (seen) {
                a.acc_out[at] = old + w;
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

template <int D>
hils_status run(const Args &f, const CUtensorMap (&m)[2], int total, cudaStream_t s) {
    static KernelSetup setup;
    int per_sm = 0;
    const auto k = sink_weights_tc_kernel<D>;
    const hils_status st = kernel_setup(setup, (const void *)k, kThreads, Smem<D>::kBytes, &per_sm);
    if (st != HILS_OK) return st;
    if (per_sm < 1) return HILS_ERR_CUDA;
    const int sms = device_sm_count();
    return sink_launch(false, k, total < sms ? total : sms, kThreads, Smem<D>::kBytes, s, m[0], m[1], f, total);
}

}  // namespace

bool launch_sink_weights_tc(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s, hils_status *st) {
    if (dt != HILS_BF16 || a.N == 0 || a.keys != kKeys) return false;
    const int Hk = a.H / a.G;
    Args f{};
    f.a = a;
    // few queries: several heads of the group share a step
    f.P = 1;
    while (f.P < 8 && a.G % (2 * f.P) == 0 && (int64_t)a.Lq * 2 * f.P <= kRows) f.P *= 2;
    f.qn = kRows / f.P;
    f.Hk = Hk;
    f.heads = a.B * Hk;
    f.packs = a.G / f.P;
    for (f.qshift = 4; 1 << f.qshift < f.qn;) ++f.qshift;
    f.items = (int)sink_key_items(a);
    const int64_t total = (int64_t)f.items * a.B * Hk;
    if (total > 0x7fffffffll - 1024) return false;
    CUtensorMap m[2];
    if (!make_view_map(&m[0], a.Q, a.B, a.H, a.Lq, d, f.qn, f.P) || !make_view_map(&m[1], a.K, a.B, Hk, a.N, d, kM, 1))
        return false;
    *st = d == 64 ? run<64>(f, m, (int)total, s) : run<128>(f, m, (int)total, s);
    return true;
}

}  // namespace hils
