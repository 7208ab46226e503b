// Backward of the window-and-sink attention on the 5th-generation tensor cores (bf16;
// formulas in sink_common.cuh): one persistent kernel in two forms, so that no sum is an atomic.
//
// An item holds a tile X of 128 rows (TMEM lanes) and walks steps of 64 rows Y:
//   dQ      X = Q, dO of 128 query rows (P packed heads x 128 / P queries, as in the prefill),
//           Y = K, V of 64 keys;       acc: dQ += dS K
//   dK, dV  X = K, V of 128 keys (a block and a segment of its steps),
//           Y = Q, dO of 64 queries of one head of the group;   acc: dV += P^T dO, dK += dS^T Q
//   S = X1 Y1^T, T = X2 Y2^T (M = 128, N = 64, K = d), p = exp2(S scale2 - lse2),
//   dS = p (T - D); scale once on the float32 sums. P and dS are bf16 operands from TMEM. For dQ
//   a second product takes what dS lost in the rounding: a row's dS sum to zero, so that dQ is
//   small against its terms and their rounding showed (relative error 0.0026 instead of the
//   0.0017 of the result's own rounding; the 8K backward 411 -> 433 us). dK and dV are sums over
//   queries, without that cancellation.
// Both recompute S and T: 7 products instead of the 5 of one kernel that would have to add
// dQ (or dK and dV) across CTAs with atomics, whose order changes the result.
// Warps (640 threads), hand-offs through mbarriers:
//   0-15   a thread owns a row of X; steps alternate between warps 0-7 and 8-15, each step's
//          64 columns in two halves. S and T go into registers and are handed back before the
//          arithmetic; P and dS have two buffers of their own. The warps of an item's last step
//          write its sums while the others begin the next item.
//   16, 17 tcgen05.mma of S and T; of the sums;  18  TMA;  19  lse and D of a step's queries
//          (dK, dV: a thread owns a key and runs over the queries), fetched two steps ahead.
// TMEM, dK and dV: S [0,64), T [64,128), P [128,160), [160,192), dS [192,224), [224,256), dV
// [256,384), dK [384,512); dQ: S, T [0,128), [128,256), dS and its rest [256,320), [320,384), dQ
// [384,512).
// An 8K prompt (32 heads on 8 key-value heads, d = 128, W 512, A 4) takes 433 us in all from a cold
// L2 (9230 on the CUDA cores; 101 by its 5 products): D 27, dQ 164, dK and dV 217, the reduction
// 10. A step's products take 1280 cycles (S and T 48 an MMA with N = 64, whose operands come from
// shared memory) of the 2290 that it lasts: the tensor pipe is 46 and 51 % busy, and the rest is
// the round trip from S, T through the exponentials to the sums, which TMEM has no room to
// overlap further at d = 128 (dK, dV: one buffer of S and T). At d = 64 dV and dK leave 128 columns,
// which are not used: 303 us for the same prompt, with half the products.
#include "sink_tc.cuh"

namespace hils {
namespace {

using namespace tc;

// A step's rows stay until its sums are done, some 6000 cycles after their load began: with three
// stages that alone made a step 2000 cycles.
constexpr int kM = 128, kRows = 64, kStages = 5;
constexpr int kThreads = 640, kStWarp = 16, kSumWarp = 17, kLoadWarp = 18, kScalarWarp = 19;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kM == kSinkKeys, "a key block is a tile");

enum {
    kBarXfull = 0,
    kBarXfree = 1,   // the item's last S, T completed
    kBarYfull = 2,   // + stage: rows (bytes); dK, dV: lse and D (32 arrivals)
    kBarYfree = kBarYfull + kStages,    // + stage: the sums that read it completed
    kBarST = kBarYfree + kStages,       // + step parity: S, T written
    kBarSTfree = kBarST + 2,            // + buffer: S, T read (8 warps)
    kBarP = kBarSTfree + 2,             // + step parity: P, dS written (8 warps)
    kBarSum = kBarP + 2,                // + step parity: the sums that read them, and every one before, completed
    kBarOfree = kBarSum + 2,            // an item's sums read (8 warps)
    kBarDrain = kBarOfree + 1,          // + MMA warp
    kNumBars = kBarDrain + 2
};

// x less its rounding to bf16, rounded to bf16 itself.
__device__ __forceinline__ uint32_t rest_bf16(float2 x, uint32_t rounded) {
    const float2 r = fma2(make_float2(bf16lo(rounded), bf16hi(rounded)), make_float2(-1.f, -1.f), x);
    return pack_bf16(r.x, r.y);
}

template <int D>
struct Smem {
    static constexpr int kX = kM * D * 2, kY = kRows * D * 2;
    static constexpr int kX1 = 0, kX2 = kX, kY1 = 2 * kX, kY2 = kY1 + kStages * kY;
    static constexpr int kSc = kY2 + kStages * kY;  // per stage: -lse (log2 units) [64], -D [64]
    static constexpr int kBars = kSc + kStages * kRows * 8, kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 16;
};

struct Args {
    SinkBwdArgs a;
    int P, qt, tiles, sink_box;  // dQ: packed heads, queries of a tile, tiles of (b, packed heads)
    int items;                   // dK, dV: items of one (b, key-value head)
    int hp, units;               // head packs (dK, dV: key-value heads) of a batch, and of all
    int total;
};

struct Item {
    int b, h, hk;     // batch, first head (dQ), key-value head
    int row0;         // first query of the tile (dQ), first key of the block
    int steps;
    SinkSpan sp;      // dQ: the keys
    int i0, i1, tiles, s0, nseg, index;  // dK, dV: queries, their tiles, first step, segment
};

template <bool DQ>
__device__ __forceinline__ Item decode(const Args &f, int j) {
    const SinkBwdArgs &a = f.a;
    Item it;
    if (DQ) {
        const int q = j / f.units, u = j - q * f.units;
        it.b = u / f.hp;
        it.h = (u - it.b * f.hp) * f.P;
        it.hk = it.h / a.G;
        it.row0 = (f.tiles - 1 - q) * f.qt;  // latest queries (most keys) first
        const int t0 = a.N - a.Lq + it.row0;
        it.sp = sink_span(t0, min(a.N - 1, t0 + f.qt - 1), a.W, a.A, kRows);
        it.steps = it.sp.ns + it.sp.nw;
        it.i0 = it.i1 = it.tiles = it.s0 = it.index = 0;
        it.nseg = 1;
    } else {
        const int x = j / f.units, xb = j - x * f.units;
        it.b = xb / f.hp;
        it.hk = xb - it.b * f.hp;
        it.h = it.hk * a.G;
        const SinkItem k = sink_item(a, x);
        it.row0 = k.blk * kM;
        it.nseg = k.nseg;
        it.index = xb * f.items + x;
        sink_rows_of_block(a, it.row0, min(kM, a.N - it.row0), &it.i0, &it.i1);
        it.tiles = (it.i1 - it.i0 + kRows - 1) / kRows;
        const int steps = a.G * it.tiles;
        it.s0 = 0;
        it.steps = steps;
        if (k.nseg > 1) {
            it.s0 = (int)((int64_t)steps * k.seg / k.nseg);
            it.steps = (int)((int64_t)steps * (k.seg + 1) / k.nseg) - it.s0;
        }
        it.sp = SinkSpan{};
    }
    return it;
}

// A walk over an item's steps: their stage and its phase (kept over the items), and
// (dK, dV) the step's query tile and head.
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
// dQ: first key of step i, and its keys
__device__ __forceinline__ int step_key(const Item &it, int i) { return i < it.sp.ns ? i * kRows : it.sp.lo + (i - it.sp.ns) * kRows; }
__device__ __forceinline__ int step_keys(const Item &it, int i) {
    return min(kRows, (i < it.sp.ns ? it.sp.sinks : it.sp.hi) - step_key(it, i));
}

template <int D, bool DQ>
__global__ void __launch_bounds__(kThreads, 1) sink_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmX1,
                                                                  const __grid_constant__ CUtensorMap tmX2,
                                                                  const __grid_constant__ CUtensorMap tmY1,
                                                                  const __grid_constant__ CUtensorMap tmY2,
                                                                  const __grid_constant__ CUtensorMap tmS1,
                                                                  const __grid_constant__ CUtensorMap tmS2, Args f) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Smem<D>;
    constexpr int kBlocks = D / 64, kXBlk = kM * 128, kYBlk = kRows * 128;
    // TMEM columns; dQ's one sum leaves room for two buffers of S, T
    constexpr int kBufs = DQ ? 2 : 1, kP = 128, kDs = DQ ? 256 : 192, kDsStep = DQ ? 64 : 32, kAcc = DQ ? 384 : 256;
    const SinkBwdArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    float *scal = reinterpret_cast<float *>(smem + L::kSc);
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;
    if (sbase & 1023u) {  // an alignment that the launch has to give
        if (tid == 0) atomicOr(a.status, 1u);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (!DQ && i >= kBarYfull && i < kBarYfull + kStages) cnt = 33;
            if (i == kBarSTfree || i == kBarSTfree + 1 || i == kBarP || i == kBarP + 1 || i == kBarOfree) cnt = 8;
            mbar_init(pipe.bar(i), cnt);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kStWarp) tmem_alloc(sbase + L::kMisc, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp == kLoadWarp) {
        // ---------------------------------------------------------------- TMA
        int n = 0, g = 0;  // items with steps, steps
        bool ok = true;
        Walk w;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.total) break;
            const Item it = decode<DQ>(f, j);
            if (it.steps <= 0) continue;
            if (n > 0 && !(ok = pipe.wait_warp(kBarXfree, (n - 1) & 1))) break;
            if (elect_one()) {
                mbar_expect_tx(pipe.bar(kBarXfull), 2 * L::kX);
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
                    const uint32_t o = sbase + c * kXBlk;
                    tma_load_4d(o + L::kX1, &tmX1, pipe.bar(kBarXfull), c * 64, it.row0, DQ ? it.h : it.hk, it.b);
                    tma_load_4d(o + L::kX2, &tmX2, pipe.bar(kBarXfull), c * 64, it.row0, DQ ? it.h : it.hk, it.b);
                }
            }
            __syncwarp();
            ++n;
            w.start(it);
            for (int i = 0; i < it.steps; ++i, ++g) {
                if (g >= kStages && !(ok = pipe.wait_warp(kBarYfree + w.st, w.ph ^ 1u))) break;
                const bool sink = DQ && i < it.sp.ns;
                const int y = DQ ? step_key(it, i) : it.i0 + w.tile * kRows, h = DQ ? it.hk : it.h + w.h;
                if (elect_one()) {
                    mbar_expect_tx(pipe.bar(kBarYfull + w.st), 2u * (sink ? f.sink_box : kRows) * D * 2);
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c) {
                        const uint32_t o = sbase + w.st * L::kY + c * kYBlk;
                        tma_load_4d(o + L::kY1, sink ? &tmS1 : &tmY1, pipe.bar(kBarYfull + w.st), c * 64, y, h, it.b);
                        tma_load_4d(o + L::kY2, sink ? &tmS2 : &tmY2, pipe.bar(kBarYfull + w.st), c * 64, y, h, it.b);
                    }
                }
                __syncwarp();
                w.next(it);
            }
        }
        if (lane == 0) {  // what was started lands before the CTA's memory is released
            pipe.drain(kBarXfull, n);
            for (int s = 0; s < kStages; ++s) pipe.drain(kBarYfull + s, g > s ? (g - s + kStages - 1) / kStages : 0);
        }
        __syncwarp();
    } else if (warp == kScalarWarp) {
        // ---------------------------------------------------------------- lse and D of the queries
        if (!DQ) {
            pdl_wait();  // D (its kernel is over before dQ's, which this grid follows)
            int g = 0;
            bool ok = true;
            Walk w;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= f.total) break;
                const Item it = decode<DQ>(f, j);
                if (it.steps <= 0) continue;
                w.start(it);
                int tile = w.tile, h = w.h, next = 0;
                float sc[2][4];
                auto fetch = [&](float(&d)[4]) {
                    if (next >= it.steps) return;
                    ++next;
                    const int64_t row0 = ((int64_t)it.b * a.H + it.h + h) * a.Lq;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int i = it.i0 + tile * kRows + lane + 32 * m;
                        d[m] = i < it.i1 ? __ldg(a.lse + row0 + i) : -INFINITY;
                        d[2 + m] = i < it.i1 ? __ldg(a.Dv + row0 + i) : 0.f;
                    }
                    if (++tile == it.tiles) {
                        tile = 0;
                        ++h;
                    }
                };
                auto put = [&](float(&d)[4]) {
                    if (g >= kStages && !(ok = pipe.wait_warp(kBarYfree + w.st, w.ph ^ 1u))) return;
                    float *to = scal + w.st * 2 * kRows + lane;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {  // a query that sees nothing: exp2(s - inf) = 0
                        to[32 * m] = d[m] == -INFINITY ? d[m] : -d[m] * kLog2e;
                        to[64 + 32 * m] = -d[2 + m];
                    }
                    pipe.arrive(kBarYfull + w.st);
                    ++g;
                    w.next(it);
                    fetch(d);
                };
                fetch(sc[0]);
                fetch(sc[1]);
                for (int i = 0; i < it.steps && ok; i += 2) {
                    put(sc[0]);
                    if (ok && i + 1 < it.steps) put(sc[1]);
                }
            }
        }
        __syncwarp();
    } else if (warp == kStWarp) {
        // ---------------------------------------------------------------- S and T
        int n = 0, c = 0;
        bool ok = true;
        Walk w;
        const uint64_t x1 = tile_desc(sbase + L::kX1, 16), x2 = tile_desc(sbase + L::kX2, 16);
        const uint64_t y1 = tile_desc(sbase + L::kY1, 16), y2 = tile_desc(sbase + L::kY2, 16);
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.total) break;
            const Item it = decode<DQ>(f, j);
            if (it.steps <= 0) continue;
            if (!(ok = pipe.wait_warp(kBarXfull, n & 1))) break;
            auto shape = [&](int i) { return idesc_bf16(kM, DQ ? (step_keys(it, i) + 15) & ~15 : kRows, false); };
            uint32_t id = shape(0);
            for (int i = 0; i < it.steps; ++i, ++c) {
                const uint64_t yo = w.st * (L::kY / 16);
                const int buf = c & (kBufs - 1);
                if (!(ok = pipe.wait_warp(kBarYfull + w.st, w.ph))) break;
                if (c >= kBufs && !(ok = pipe.wait_warp(kBarSTfree + buf, (c / kBufs - 1) & 1))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(tmem + buf * 128, x1 + ((k >> 2) * kXBlk + (k & 3) * 32) / 16,
                               y1 + yo + ((k >> 2) * kYBlk + (k & 3) * 32) / 16, id, k > 0);
                }
                __syncwarp();
                // the next step's numbers while S is computed: T's issue waits for the pipe anyhow
                const uint32_t id_t = id;
                w.next(it);
                if (DQ && i + 1 < it.steps) id = shape(i + 1);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(tmem + buf * 128 + 64, x2 + ((k >> 2) * kXBlk + (k & 3) * 32) / 16,
                               y2 + yo + ((k >> 2) * kYBlk + (k & 3) * 32) / 16, id_t, k > 0);
                    mma_commit(pipe.bar(kBarST + (c & 1)));
                    if (i + 1 == it.steps) mma_commit(pipe.bar(kBarXfree));
                }
                __syncwarp();
            }
            ++n;
        }
        if (elect_one()) {
            mma_commit(pipe.bar(kBarDrain));  // what was issued completes before TMEM is released
            pipe.drain(kBarDrain, 1);
        }
        __syncwarp();
    } else if (warp == kSumWarp) {
        // ---------------------------------------------------------------- the sums
        int n = 0, c = 0;
        bool ok = true;
        Walk w;
        const uint64_t y1 = tile_desc(sbase + L::kY1, kYBlk), y2 = tile_desc(sbase + L::kY2, kYBlk);
        const uint32_t id = idesc_bf16(kM, D, true);
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.total) break;
            const Item it = decode<DQ>(f, j);
            if (it.steps <= 0) continue;
            for (int i = 0; i < it.steps; ++i, ++c) {
                const uint64_t yo = w.st * (L::kY / 16);
                const int k16 = DQ ? (step_keys(it, i) + 15) / 16 : kRows / 16;
                const uint32_t p = tmem + kP + (c & 1) * 32, ds = tmem + kDs + (c & 1) * kDsStep;
                if (!(ok = pipe.wait_warp(kBarP + (c & 1), (c >> 1) & 1))) break;
                if (!(ok = pipe.wait_warp(kBarYfull + w.st, w.ph))) break;  // (P came of it)
                if (i == 0 && n > 0 && !(ok = pipe.wait_warp(kBarOfree, (n - 1) & 1))) break;
                tc_fence_after();
                if (elect_one()) {
                    if (DQ) {
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            if (k < k16) {
                                mma_ts(tmem + kAcc, ds + k * 8, y1 + yo + k * (2048 / 16), id, i > 0 || k > 0);
                                mma_ts(tmem + kAcc, ds + 32 + k * 8, y1 + yo + k * (2048 / 16), id, 1u);
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k) mma_ts(tmem + kAcc, p + k * 8, y2 + yo + k * (2048 / 16), id, i > 0 || k > 0);
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k) mma_ts(tmem + kAcc + 128, ds + k * 8, y1 + yo + k * (2048 / 16), id, i > 0 || k > 0);
                    }
                    mma_commit(pipe.bar(kBarSum + (c & 1)));
                    mma_commit(pipe.bar(kBarYfree + w.st));
                }
                __syncwarp();
                w.next(it);
            }
            ++n;
        }
        if (elect_one()) {
            mma_commit(pipe.bar(kBarDrain + 1));
            pipe.drain(kBarDrain + 1, 1);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- rows of X
        const int w = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_col = lanes + (DQ ? w * 128 : 0) + half * 32, t_col = s_col + 64;
        const uint32_t p_col = lanes + kP + w * 32 + half * 16, d_col = lanes + kDs + w * kDsStep + half * 16;
        const float scale2 = a.scale * kLog2e, lowest = scale2 > 0.f ? -INFINITY : INFINITY;  // its logit is -inf
        const float2 scale22 = make_float2(scale2, scale2);
        const int off = a.N - a.Lq;
        bool ok = true;
        int c = 0;
        Walk walk;
        if (DQ) pdl_wait();  // D
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.total) break;
            const Item it = decode<DQ>(f, j);
            // dQ: this row's query; dK, dV: its key
            const int hrow = DQ ? row / f.qt : 0, i_q = it.row0 + (DQ ? row - hrow * f.qt : 0), t = off + i_q, key = it.row0 + row;
            const bool have = DQ ? i_q < a.Lq : key < a.N;
            float2 nl = make_float2(0.f, 0.f), nd = nl;
            int see0 = 0, see1 = 0;  // dK, dV: the queries that see the key, from the item's first on
            if (DQ) {
                const int64_t place = ((int64_t)it.b * a.H + it.h + hrow) * a.Lq + i_q;
                const float lse = have ? __ldg(a.lse + place) : -INFINITY, Dr = have ? a.Dv[place] : 0.f;
                nl.x = nl.y = lse == -INFINITY ? lse : -lse * kLog2e;
                nd.x = nd.y = -Dr;
            } else {
                see0 = key - off - it.i0;
                see1 = (int)min(key < a.A ? (int64_t)it.i1 : (int64_t)key + a.W - off, (int64_t)it.i1) - it.i0;
            }
            walk.start(it);
            for (int i = 0; i < it.steps; ++i, walk.next(it)) {
                const int cc = c + i;
                if ((cc & 1) != w) continue;
                uint32_t mk;  // visible columns of this half
                if (DQ) {
                    const int k0 = step_key(it, i) + half * 32, n = step_keys(it, i) - half * 32;
                    int hi = min(n, t + 1 - k0);
                    hi = have ? hi : 0;
                    mk = i < it.sp.ns ? range_bits(0, hi, 0) : range_bits(t - a.W + 1 - k0, hi, 0) | range_bits(0, min(a.A - k0, hi), 0);
                } else {
                    const int q = walk.tile * kRows + half * 32;
                    mk = range_bits(see0 - q, see1 - q, 0);
                }
                const bool full = __all_sync(kFull, mk == kFull);
                if (!(ok = pipe.wait_warp(kBarST + w, (cc >> 1) & 1))) break;
                tc_fence_after();
                uint32_t s[32], u[32];
                tmem_ld32(s_col, s);
                tmem_ld32(t_col, u);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarSTfree + (DQ ? w : 0));
                if (!full) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        s[q] = (mk >> q) & 1u ? s[q] : __float_as_uint(lowest);
                        u[q] = (mk >> q) & 1u ? u[q] : 0u;  // it may be anything there
                    }
                }
                const float *sc = scal + walk.st * 2 * kRows + half * 32;
                if (!DQ && !(ok = pipe.wait_warp(kBarYfull + walk.st, walk.ph))) break;  // complete: S came of it
                uint32_t p[16], ds[16];
#pragma unroll
                for (int q = 0; q < 32; q += 4) {
                    float2 l0 = nl, l1 = nl, d0 = nd, d1 = nd;
                    if (!DQ) {
                        const float4 x = *reinterpret_cast<const float4 *>(sc + q), y = *reinterpret_cast<const float4 *>(sc + kRows + q);
                        l0 = make_float2(x.x, x.y);
                        l1 = make_float2(x.z, x.w);
                        d0 = make_float2(y.x, y.y);
                        d1 = make_float2(y.z, y.w);
                    }
                    float2 e0 = fma2(as2(s + q), scale22, l0), e1 = fma2(as2(s + q + 2), scale22, l1);
                    e0 = make_float2(exp2_ftz(e0.x), exp2_ftz(e0.y));
                    e1 = make_float2(exp2_ftz(e1.x), exp2_ftz(e1.y));
                    const float2 g0 = mul2(e0, add2(as2(u + q), d0)), g1 = mul2(e1, add2(as2(u + q + 2), d1));
                    ds[q / 2] = pack_bf16(g0.x, g0.y);
                    ds[q / 2 + 1] = pack_bf16(g1.x, g1.y);
                    if (DQ) {  // what the rounding took
                        p[q / 2] = rest_bf16(g0, ds[q / 2]);
                        p[q / 2 + 1] = rest_bf16(g1, ds[q / 2 + 1]);
                    } else {
                        p[q / 2] = pack_bf16(e0.x, e0.y);
                        p[q / 2 + 1] = pack_bf16(e1.x, e1.y);
                    }
                }
                // the sums of two steps before have read this buffer
                if (cc >= 2 && !(ok = pipe.wait_warp(kBarSum + w, ((cc >> 1) - 1) & 1))) break;
                tc_fence_after();
                tmem_st16(DQ ? d_col + 32 : p_col, p);
                tmem_st16(d_col, ds);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarP + w);
            }
            if (!ok) break;
            c += it.steps;
            // ---- the item's sums, by the warps of its last step: dQ's halves of the columns, or dV and dK
            if (it.steps > 0 ? ((c - 1) & 1) != w : w != 0) continue;
            if (it.steps > 0) {
                if (!(ok = pipe.wait_warp(kBarSum + w, ((c - 1) >> 1) & 1))) break;
                tc_fence_after();
            }
            const float fac = DQ || half ? a.scale : 1.f;
            const uint32_t o_col = lanes + kAcc + (DQ ? half * (D / 2) : half * 128);
            const int cols = DQ ? D / 2 : D;
            const bool part = !DQ && it.nseg > 1;  // float32 partial rows
            const MutView &v = DQ ? a.dQ : half ? a.dK : a.dV;
            uint64_t mine = 0;
            if (part)
                mine = (uint64_t)(a.part + ((int64_t)it.index * 2 * kSinkKeys + (half ? 0 : kSinkKeys) + row) * D);
            else if (have)
                mine = (uint64_t)(static_cast<bf16 *>(v.ptr) + it.b * v.sb + (DQ ? it.h + hrow : it.hk) * v.sh +
                                  (int64_t)(DQ ? i_q : key) * v.st + (DQ ? half * (D / 2) : 0));
            char *to[4];  // the rows of a lane's group of four, at this lane's unit
            bool live[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t x = __shfl_sync(kFull, mine, (lane & ~3) + k);
                live[k] = x != 0;
                to[k] = reinterpret_cast<char *>(x) + (lane & 3) * 16;
            }
#pragma unroll 1
            for (int col = 0; col < cols; col += 32) {
                uint32_t o[32];
                if (it.steps > 0) {
                    tmem_ld32(o_col + col, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = 0u;
                }
#pragma unroll
                for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * fac);
                if (part) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint4 x[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            x[q] = make_uint4(o[16 * g + 4 * q], o[16 * g + 4 * q + 1], o[16 * g + 4 * q + 2], o[16 * g + 4 * q + 3]);
                        swap_units(x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4 *>(to[k] + col * 4 + g * 64) = x[k];
                    }
                } else {
                    uint4 x[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = pack_bf16(__uint_as_float(o[8 * q + 2 * k]), __uint_as_float(o[8 * q + 2 * k + 1]));
                        x[q] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    swap_units(x);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (live[k]) *reinterpret_cast<uint4 *>(to[k] + col * 2) = x[k];
                }
            }
            if (it.steps > 0) {
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarOfree);
            }
        }
    }
    if (!DQ) pdl_wait();  // the grid is not over before dQ's
    tc_fence_before();
    __syncthreads();
    if (warp == kStWarp) {
        tc_fence_after();
        tmem_free(tmem, kTmemCols);
    }
}

template <int D, bool DQ>
hils_status run(const Args &f, const CUtensorMap *m, cudaStream_t s) {
    static KernelSetup setup;
    int per_sm = 0;
    const auto k = sink_bwd_tc_kernel<D, DQ>;
    const hils_status st = kernel_setup(setup, (const void *)k, kThreads, Smem<D>::kBytes, &per_sm);
    if (st != HILS_OK) return st;
    if (per_sm < 1) return HILS_ERR_CUDA;
    const int sms = device_sm_count();
    // dQ follows the kernel of D; dK, dV begin, but for D, as dQ's CTAs end
    return sink_launch(true, k, f.total < sms ? f.total : sms, kThreads, Smem<D>::kBytes, s, m[0], m[1], m[2], m[3], m[4], m[5], f);
}

}  // namespace

bool launch_sink_backward_tc(hils_dtype dt, int d, const SinkBwdArgs &a, cudaStream_t s, hils_status *st) {
    if (dt != HILS_BF16 || a.N == 0) return false;
    const int Hk = a.H / a.G;
    Args q{}, k{};
    q.a = k.a = a;
    q.P = sink_pack(a.G);
    q.qt = kM / q.P;
    q.tiles = (a.Lq + q.qt - 1) / q.qt;
    q.hp = a.H / q.P;
    q.units = a.B * q.hp;
    k.hp = Hk;
    k.units = a.B * Hk;
    const int64_t qi = (int64_t)q.units * q.tiles;
    k.items = (int)sink_key_items(a);
    const int64_t ki = (int64_t)k.items * a.B * Hk;
    if (qi > 0x7fffffffll - 1024 || ki > 0x7fffffffll - 1024) return false;
    q.total = (int)qi;
    k.total = (int)ki;
    const int sinks = a.A > 0 ? a.A : 1;
    q.sink_box = sinks < kRows ? (sinks + 15) & ~15 : kRows;
    CUtensorMap mq[6], mk[6];
    if (!make_view_map(&mq[0], a.Q, a.B, a.H, a.Lq, d, q.qt, q.P) || !make_view_map(&mq[1], a.dO, a.B, a.H, a.Lq, d, q.qt, q.P) ||
        !make_view_map(&mq[2], a.K, a.B, Hk, a.N, d, kRows, 1) || !make_view_map(&mq[3], a.V, a.B, Hk, a.N, d, kRows, 1) ||
        // the sinks alone: their maps end at the last one
        !make_view_map(&mq[4], a.K, a.B, Hk, sinks, d, q.sink_box, 1) ||
        !make_view_map(&mq[5], a.V, a.B, Hk, sinks, d, q.sink_box, 1) ||
        !make_view_map(&mk[0], a.K, a.B, Hk, a.N, d, kM, 1) || !make_view_map(&mk[1], a.V, a.B, Hk, a.N, d, kM, 1) ||
        !make_view_map(&mk[2], a.Q, a.B, a.H, a.Lq, d, kRows, 1) || !make_view_map(&mk[3], a.dO, a.B, a.H, a.Lq, d, kRows, 1))
        return false;
    mk[4] = mk[2];  // not used
    mk[5] = mk[3];
    *st = d == 64 ? run<64, true>(q, mq, s) : run<128, true>(q, mq, s);
    if (*st == HILS_OK) *st = d == 64 ? run<64, false>(k, mk, s) : run<128, false>(k, mk, s);
    return true;
}

}  // namespace hils
