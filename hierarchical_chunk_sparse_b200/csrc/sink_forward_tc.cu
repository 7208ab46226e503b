// Window-and-sink attention on the 5th-generation tensor cores (bf16): prefill and the
// shared prefix of a decode batch (formulas in sink_common.cuh).
//
// A persistent CTA (one per SM) takes items of two 128-row query tiles A and B and walks
// 64-key tiles with an online softmax: S = Q K^T (M = 128 rows, N = keys, K = d) into TMEM,
// the softmax over it with P (bf16) written over S, O += P V with P read from TMEM.
//   prefill  a tile is P heads of a group (the largest power of two <= 8 that divides G)
//            with 128 / P consecutive queries each; A and B are neighbours and share each
//            key tile; a tile that only one of them sees is skipped by the other. The
//            sinks' tiles come first, from a tensor map that ends at the last sink, then
//            the window's from its first visible key: a slot that no query sees is never
//            loaded. The last tile's products cover only its keys, rounded up to 16.
//   prefix   a tile is 128 / G sequences with the G heads of a group each, so that the
//            prefix is read once for all of them; A and B are the same rows over two key
//            ranges, which are joined later.
// Warp roles (640 threads), hand-offs through mbarriers:
//   warps 0-15   softmax: two warpgroups for each of A and B, which take its key tiles in turn;
//                a thread owns a row (TMEM lane). Their maxima and sums are their own; the
//                row's reference goes from one to the other through shared memory, before the
//                exponentials, so that they overlap. It is raised, and O rescaled, only when a
//                tile's maximum passes it by more than 8 in log2 units (P <= 2^8: exact in the
//                float32 sums, rounded in bf16 as well as below 1). The warpgroup of an item's
//                last tile writes its output, while the other begins the next item.
//   warps 16, 17 tcgen05.mma of A, B;   warps 18, 19  TMA of Q and K, of V (one warp for both
//                held the keys of later tiles back until a PV had freed room for values).
// A softmax warp takes its 64 scores into registers and hands S back before anything else, and
// P has two buffers of its own, so that neither S of the next tile nor the next softmax waits
// for a PV. The MMA warp issues whatever product is ready, over the borders of items.
// An 8K prompt (32 heads, d = 128, W 512, A 4) takes 134 us from a cold L2 (2913 on the CUDA cores;
// 41 by its bytes, 40 by its products): the tensor pipe is 35 % busy and the MUFU 39 %, a key tile
// costs its warpgroup some 3570 cycles of which the softmax's dependent steps (TMEM load, maximum,
// exponentials, TMEM store) are three quarters, and the last wave about a tenth of the time. The
// prefix pass of 32 sequences over 64K tokens (8 key-value heads) takes 56 us, 4.8 TB/s.
// 64-key tiles with two warpgroups each took 131 us where 128-key tiles with one took 222.
// P is rounded to bf16 for its product (at most 2^-8 of each, averaged by the sum), as O is.
// TMEM of tile x, from 128 x: S [0,64), P [64,96), [96,128); O_A [256,384), O_B [384,512).
#include "sink_tc.cuh"

namespace hils {
namespace {

using namespace tc;

constexpr int kM = 128, kKeys = 64, kThreads = 640;
constexpr int kMmaWarp = 16, kLoadWarp = 18;  // K (and Q), V
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum {
    kBarQfull = 0,    // + tile (prefix: 0 for both)
    kBarQfree = 2,    // + tile
    kBarKfull = 4,    // + stage
    kBarKfree = 10,   // + stage: the S products that read it completed
    kBarVfull = 16,   // + stage
    kBarVfree = 20,   // + stage: the PV products that read it completed
    kBarS = 24,       // + 2 tile + warpgroup: S written
    kBarSfree = 28,   // + tile: S read (4 warps)
    kBarP = 30,       // + 2 tile + buffer: P written (4 warps)
    kBarPV = 34,      // + 2 tile + buffer: its PV, and every MMA before that, completed
    kBarOfree = 38,   // + tile: O read (4 warps)
    kBarRef = 40,     // + 4 tile + quadrant: the rows' reference after a tile (1 warp)
    kBarEnd = 48,     // + 8 item parity + 4 tile + quadrant: one warpgroup's sums, for the other (1 warp)
    kBarDrain = 64,   // + tile
    kNumBars = 66
};

// An entry's note for a tile (B's in the upper half of the word): its keys, and whether it is the
// item's first or last of the tile; 0 for an entry that is not the tile's.
constexpr uint32_t kNoteFirst = 128u, kNoteLast = 256u, kNoteEnd = 0x80000000u;

struct FwdTc {
    SinkArgs a;
    int P, qt, nqb;     // prefill: packed heads, queries of a tile, row items per (b, pack)
    int hp, units;      // packs of a batch, (b, pack) pairs
    int nb, tiles;      // prefix: sequences of a tile, tiles
    int items, sink_box;
};

template <int D, bool PREFIX>
struct Smem {
    static constexpr int kX = kM * D * 2, kY = kKeys * D * 2;
    // stages of one ring: one ring of each of K and V for both tiles, for a prefix one for each
    static constexpr int kKst = PREFIX ? 3 : 4, kVst = PREFIX ? 2 : 4, kRings = PREFIX ? 2 : 1;
    static constexpr int kQ = 0, kK = (PREFIX ? 1 : 2) * kX, kV = kK + kRings * kKst * kY;
    static constexpr int kRef = kV + kRings * kVst * kY;  // [2 tiles][128] references
    static constexpr int kEnd = kRef + 2 * kM * 4;        // [2 item parities][2 tiles][128] reference, sum
    static constexpr int kNote = kEnd + 4 * kM * 8;       // notes of the K stages [8], the V stages [8]
    static constexpr int kBars = kNote + 64, kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 16;
};

// The next stage of a ring and the phase of its full barrier.
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++st == stages) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// The key tiles of one row tile x of an item, in order: entries [a0, a1), then [b0, b1).
struct Own {
    int a0, n1, b0, n;  // n in all, n1 of them in the first run
    int sinks;          // how many of them are sinks' tiles
    __device__ __forceinline__ int entry(int i) const { return i < n1 ? a0 + i : b0 + (i - n1); }
    __device__ __forceinline__ int first_key(int i, const SinkSpan &sp) const {
        const int e = entry(i);
        return i < sinks ? e * kKeys : sp.lo + (e - sp.ns) * kKeys;
    }
};

struct PrefixItem {
    int hk, h, i0;      // key-value head, its first query head, first sequence
    int split;
    bool hasB;          // there is a second key range
    int r0, r1, r2;     // A's key tiles [r0, r1), B's [r1, r2)
};

template <bool PREFIX>
__device__ __forceinline__ auto decode_item(const FwdTc &f, int j) {
    const SinkArgs &a = f.a;
    if constexpr (PREFIX) {
        PrefixItem it;
        const int pairs = (a.splits + 1) / 2;
        it.split = j % pairs;
        const int u = j / pairs;
        it.i0 = (u % f.tiles) * f.nb;
        it.hk = u / f.tiles;
        it.h = it.hk * a.G;
        it.hasB = 2 * it.split + 1 < a.splits;
        const int nt = (a.N + kKeys - 1) / kKeys, r = 2 * it.split;
        it.r0 = (int)((int64_t)nt * r / a.splits);
        it.r1 = (int)((int64_t)nt * (r + 1) / a.splits);
        it.r2 = it.hasB ? (int)((int64_t)nt * (r + 2) / a.splits) : it.r1;
        return it;
    } else {
        return RowItem<kKeys>(j, f.hp, f.units, a.G, f.P, f.qt, f.nqb, a.Lq, a.N, a.W, a.A, a.splits);
    }
}
template <bool PREFIX, typename I>
__device__ __forceinline__ Own own_tiles(const I &it, int x) {
    Own o;
    if constexpr (PREFIX) {
        o.a0 = x ? it.r1 : it.r0;
        o.n = o.n1 = (x ? it.r2 : it.r1) - o.a0;
        o.b0 = 0;
    } else if (x == 0) {
        o.a0 = it.e0;
        o.n = o.n1 = max(0, min(it.e1, it.eA) - it.e0);
        o.b0 = 0;
    } else {
        const int w0 = it.sp.ns + it.wB;
        o.a0 = it.e0;
        o.n1 = max(0, min(it.e1, it.sp.ns) - it.e0);
        o.b0 = max(it.e0, w0);
        o.n = it.hasB ? o.n1 + max(0, it.e1 - o.b0) : 0;
        if (!it.hasB) o.n1 = 0;
    }
    o.sinks = 0;
    if constexpr (!PREFIX) o.sinks = min(o.n, max(0, it.sp.ns - it.e0));
    return o;
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1) sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                  const __grid_constant__ CUtensorMap tmK,
                                                                  const __grid_constant__ CUtensorMap tmV,
                                                                  const __grid_constant__ CUtensorMap tmKs,
                                                                  const __grid_constant__ CUtensorMap tmVs, FwdTc f) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Smem<D, PREFIX>;
    constexpr int kBlocks = D / 64;  // 64-column blocks of a row tile
    constexpr int kXBlk = kM * 128, kYBlk = kKeys * 128;
    const SinkArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile uint32_t *notes = reinterpret_cast<uint32_t *>(smem + L::kNote);
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;
    if (sbase & 1023u) {  // an alignment that the launch has to give
        if (tid == 0) atomicOr(a.status, 1u);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if ((i >= kBarP && i < kBarP + 4) || (i >= kBarSfree && i < kBarSfree + 2) || (i >= kBarOfree && i < kBarOfree + 2)) cnt = 4;
            // both tiles release what they share
            if (PREFIX ? i == kBarQfree : (i >= kBarKfree && i < kBarKfree + 6) || (i >= kBarVfree && i < kBarVfree + 4)) cnt = 2;
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

    if (warp >= kLoadWarp) {
        // ---------------------------------------------------------------- TMA
        const bool vals = warp > kLoadWarp;
        const int stages = vals ? L::kVst : L::kKst, full0 = vals ? kBarVfull : kBarKfull, free0 = vals ? kBarVfree : kBarKfree;
        const CUtensorMap *own_map = vals ? &tmV : &tmK, *sink_map = vals ? &tmVs : &tmKs;
        const uint32_t store = sbase + (vals ? L::kV : L::kK);
        volatile uint32_t *note_of_stage = notes + (vals ? 8 : 0);
        int nq[2] = {0, 0};
        bool ok = true;
        auto tile = [&](uint32_t dst, int blk, const CUtensorMap *m, int bar, int y, int z, int w) {
#pragma unroll
            for (int c = 0; c < kBlocks; ++c) tma_load_4d(dst + c * blk, m, pipe.bar(bar), c * 64, y, z, w);
        };
        Ring ring_at[2];  // of each ring: the next stage
        int loads[2] = {0, 0};
        // One entry: `note` tells the MMA warps which tiles take it (0: none).
        auto load = [&](int ring, uint32_t note, int k0, bool sink, int hk, int b) {
            const int s = ring * stages + ring_at[ring].st;
            if (loads[ring] >= stages && !(ok = pipe.wait_warp(free0 + s, ring_at[ring].ph ^ 1u))) return;
            if (elect_one()) {
                note_of_stage[s] = note;
                if (note & kNoteEnd) {
                    pipe.arrive(full0 + s);
                } else {
                    mbar_expect_tx(pipe.bar(full0 + s), (uint32_t)(sink ? f.sink_box : kKeys) * D * 2);
                    tile(store + s * L::kY, kYBlk, sink ? sink_map : own_map, full0 + s, k0, hk, b);
                }
            }
            __syncwarp();
            ring_at[ring].next(stages);
            ++loads[ring];
        };
        auto note_of = [](int keys, bool first, bool last) -> uint32_t {
            return keys > 0 ? (uint32_t)keys | (first ? kNoteFirst : 0u) | (last ? kNoteLast : 0u) : 0u;
        };
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.items) break;
            const auto it = decode_item<PREFIX>(f, j);
            if constexpr (PREFIX) {
                const int n0 = it.r1 - it.r0, n1 = it.r2 - it.r1;
                if (!vals) {
                    if (nq[0] > 0 && !(ok = pipe.wait_warp(kBarQfree, (nq[0] - 1) & 1))) break;
                    if (elect_one()) {
                        mbar_expect_tx(pipe.bar(kBarQfull), (uint32_t)(f.nb * a.G) * D * 2);
                        tile(sbase + L::kQ, kXBlk, &tmQ, kBarQfull, it.h, it.i0, 0);
                        // a range that is not there lets the queries go at once
                        if (n0 == 0) pipe.arrive(kBarQfree);
                        if (n1 == 0) pipe.arrive(kBarQfree);
                    }
                    __syncwarp();
                    ++nq[0];
                }
                for (int i = 0; i < max(n0, n1) && ok; ++i) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int n = x ? n1 : n0, e = (x ? it.r1 : it.r0) + i;
                        if (i < n && ok) load(x, note_of(min(kKeys, a.N - e * kKeys), i == 0, i + 1 == n), e * kKeys, false, it.hk, 0);
                    }
                }
            } else {
                const int l0 = it.last(0), l1 = it.last(1);
                if (!vals) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if ((x ? l1 : l0) < 0) continue;
                        if (nq[x] > 0 && !(ok = pipe.wait_warp(kBarQfree + x, (nq[x] - 1) & 1))) break;
                        if (elect_one()) {
                            mbar_expect_tx(pipe.bar(kBarQfull + x), L::kX);
                            tile(sbase + L::kQ + x * L::kX, kXBlk, &tmQ, kBarQfull + x, it.i0 + x * f.qt, it.h, it.b);
                        }
                        __syncwarp();
                        ++nq[x];
                    }
                }
                bool first0 = true, first1 = true;
                for (int e = it.e0; e < it.e1 && ok; ++e) {
                    const uint32_t n0 = note_of(it.keys(0, e), first0, e == l0), n1 = note_of(it.keys(1, e), first1, e == l1);
                    first0 = first0 && n0 == 0u;
                    first1 = first1 && n1 == 0u;
                    load(0, n0 | n1 << 16, it.first_key(e), e < it.sp.ns, it.hk, it.b);
                }
            }
        }
        for (int ring = 0; ring < L::kRings && ok; ++ring) load(ring, kNoteEnd, 0, false, 0, 0);
        // what was started lands before the CTA's memory is released
        if (lane == 0) {
            for (int x = 0; x < 2; ++x) pipe.drain(kBarQfull + x, nq[x]);
            for (int ring = 0; ring < L::kRings; ++ring)
                for (int q = 0; q < stages; ++q)
                    pipe.drain(full0 + ring * stages + q, loads[ring] > q ? (loads[ring] - q + stages - 1) / stages : 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ---------------------------------------------------------------- MMA of tile x
        const int x = warp - kMmaWarp, bq = PREFIX ? 0 : x;
        const int k_ring = PREFIX ? x * L::kKst : 0, v_ring = PREFIX ? x * L::kVst : 0;
        const uint64_t qd = tile_desc(sbase + L::kQ + (PREFIX ? 0 : x * L::kX), 16);
        const uint64_t kd0 = tile_desc(sbase + L::kK + k_ring * L::kY, 16), vd0 = tile_desc(sbase + L::kV + v_ring * L::kY, kYBlk);
        // S and PV go through the same entries, each in its own ring: c tiles and n items are done
        struct Side {
            Ring ring;
            int c = 0, n = 0;
            bool done = false;
        };
        Side S, V;
        // What the next S and the next PV need, one barrier a lane, so that one test serves all:
        // 0-2 its keys, S before it read, an item's queries; 3-5 P, its values, O of the item before
        // read. (Selects: a branch for each lane would cost more than the tests.)
        uint32_t my_bar, my_par;
        auto set_needs = [&] {
            const int s_full = kBarKfull + k_ring + S.ring.st, v_full = kBarVfull + v_ring + V.ring.st;
            const int p_full = kBarP + 2 * x + (V.c & 1);
            int i = lane == 0 ? s_full : kBarSfree + x;
            uint32_t par = lane == 0 ? S.ring.ph : (uint32_t)(S.c - 1);
            i = lane == 2 ? kBarQfull + bq : i;
            par = lane == 2 ? S.n : par;
            i = lane == 3 ? p_full : i;
            par = lane == 3 ? (uint32_t)V.c >> 1 : par;
            i = lane == 4 ? v_full : i;
            par = lane == 4 ? V.ring.ph : par;
            i = lane == 5 ? kBarOfree + x : i;
            par = lane == 5 ? (uint32_t)(V.n - 1) : par;
            my_bar = pipe.bar(i);
            my_par = par & 1u;
        };
        int spins = 0;
        uint64_t since = 0;
        while (!S.done || !V.done) {
            set_needs();
            const unsigned got = __ballot_sync(kFull, mbar_test_phase(my_bar, my_par)) | (S.c == 0 ? 2u : 0u);
            __syncwarp();
            bool progress = false;
            if (!S.done && (got & 1u)) {
                const uint32_t all = notes[k_ring + S.ring.st], note = PREFIX ? all : (all >> (16 * x)) & 0xffffu;
                if (all & kNoteEnd) {
                    S.done = progress = true;
                } else if (note == 0u) {  // not this tile's
                    pipe.arrive_if(lane == 0, kBarKfree + k_ring + S.ring.st);
                    S.ring.next(L::kKst);
                    progress = true;
                } else if ((got & 2u) && (!(note & kNoteFirst) || (got & 4u))) {
                    tc_fence_after();
                    const uint32_t id = idesc_bf16(kM, ((note & 127u) + 15) & ~15, false);
                    const uint64_t kd = kd0 + S.ring.st * (L::kY / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            mma_ss(tmem + x * 128, qd + ((s >> 2) * kXBlk + (s & 3) * 32) / 16,
                                   kd + ((s >> 2) * kYBlk + (s & 3) * 32) / 16, id, s > 0);
                        mma_commit(pipe.bar(kBarS + 2 * x + (S.c & 1)));
                        mma_commit(pipe.bar(kBarKfree + k_ring + S.ring.st));
                        if (note & kNoteLast) mma_commit(pipe.bar(kBarQfree + bq));
                    }
                    __syncwarp();
                    S.ring.next(L::kKst);
                    ++S.c;
                    if (note & kNoteLast) ++S.n;
                    progress = true;
                }
            }
            if (!V.done && (got & 16u)) {
                const uint32_t all = notes[8 + v_ring + V.ring.st], note = PREFIX ? all : (all >> (16 * x)) & 0xffffu;
                if (all & kNoteEnd) {
                    V.done = progress = true;
                } else if (note == 0u) {
                    pipe.arrive_if(lane == 0, kBarVfree + v_ring + V.ring.st);
                    V.ring.next(L::kVst);
                    progress = true;
                } else if ((got & 8u) && V.c < S.c && (!(note & kNoteFirst) || V.n == 0 || (got & 32u))) {
                    tc_fence_after();
                    const int k16 = ((note & 127u) + 15) / 16;
                    const uint32_t acc = note & kNoteFirst ? 0u : 1u;
                    const uint64_t vd = vd0 + V.ring.st * (L::kY / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < kKeys / 16; ++s)
                            if (s < k16)
                                mma_ts(tmem + 256 + x * 128, tmem + x * 128 + 64 + (V.c & 1) * 32 + s * 8, vd + s * (2048 / 16),
                                       idesc_bf16(kM, D, true), s > 0 ? 1u : acc);
                        mma_commit(pipe.bar(kBarPV + 2 * x + (V.c & 1)));
                        mma_commit(pipe.bar(kBarVfree + v_ring + V.ring.st));
                    }
                    __syncwarp();
                    V.ring.next(L::kVst);
                    ++V.c;
                    if (note & kNoteLast) ++V.n;
                    progress = true;
                }
            }
            if (progress) {
                spins = 0;
                since = 0;
            } else if (!pipe.idle(&spins, &since)) {
                break;
            }
        }
        if (elect_one()) {
            mma_commit(pipe.bar(kBarDrain + x));  // what was issued completes before TMEM is released
            pipe.drain(kBarDrain + x, 1);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax rows of tile x
        const int x = warp >> 3, w = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane, pair = 4 * x + quad;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_col = tmem + lanes + x * 128, p_col = s_col + 64 + w * 32, o_col = tmem + lanes + 256 + x * 128;
        float *refs = reinterpret_cast<float *>(smem + L::kRef) + x * kM + row;
        float2 *ends = reinterpret_cast<float2 *>(smem + L::kEnd) + x * kM + row;  // + item parity * 2 kM
        const float scale2 = a.scale * kLog2e;
        const float2 scale22 = make_float2(scale2, scale2);
        bool ok = true;
        int c = 0, n_items = 0;  // tiles and items of x
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.items) break;
            const auto it = decode_item<PREFIX>(f, j);
            const Own own = own_tiles<PREFIX>(it, x);
            int b, h, i, t;
            bool have;
            if constexpr (PREFIX) {
                b = it.i0 + row / a.G;
                h = it.h + row % a.G;
                i = 0;
                t = a.N;
                have = row < f.nb * a.G && b < a.B && (x == 0 || it.hasB);
            } else {
                b = it.b;
                h = it.h + row / f.qt;
                i = it.i0 + x * f.qt + row % f.qt;
                t = a.N - a.Lq + i;
                have = i < a.Lq;
            }
            int see_lo = 0, see_hi = 0, end = 0;  // the window and all that the row sees; the tile's last key
            if constexpr (!PREFIX) {
                see_lo = t - a.W + 1;
                see_hi = have ? t + 1 : 0;
                end = x ? it.sp.hi : min(it.sp.hi, it.tB);
            }
            float m = -INFINITY, l = 0.f;  // the reference of this warpgroup's last tile, and its sum
            for (int k = (c ^ w) & 1; k < own.n; k += 2) {  // tiles c + k of this warpgroup's parity
                const int cc = c + k;
                // this row's visible columns of the tile: [lo, hi) and (sinks in a window tile) [0, as)
                int lo, hi, as = 0;
                if constexpr (PREFIX) {
                    lo = 0;
                    hi = min(kKeys, a.N - own.entry(k) * kKeys);
                } else {
                    const int k0 = own.first_key(k, it.sp);
                    const bool sink = k < own.sinks;
                    lo = sink ? 0 : see_lo - k0;
                    hi = min(sink ? it.sp.sinks : end, see_hi) - k0;
                    as = sink ? 0 : min(a.A, see_hi) - k0;
                }
                const bool full = __all_sync(kFull, lo <= 0 && hi >= kKeys);
                if (!(ok = pipe.wait_warp(kBarS + 2 * x + w, (cc >> 1) & 1))) break;
                tc_fence_after();
                uint32_t s[64];
                tmem_ld32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));  // (behind the keys: anything, masked)
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarSfree + x);
                if (!full) {
                    const uint32_t mk0 = range_bits(lo, hi, 0) | range_bits(0, as, 0);
                    const uint32_t mk1 = range_bits(lo, hi, 32) | range_bits(0, as, 32);
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        s[q] = (mk0 >> q) & 1u ? s[q] : __float_as_uint(-INFINITY);
                        s[32 + q] = (mk1 >> q) & 1u ? s[32 + q] : __float_as_uint(-INFINITY);
                    }
                }
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int q = 0; q < 64; q += 8) {
                    m0 = fmax3(m0, __uint_as_float(s[q]), __uint_as_float(s[q + 1]));
                    m1 = fmax3(m1, __uint_as_float(s[q + 2]), __uint_as_float(s[q + 3]));
                    m2 = fmax3(m2, __uint_as_float(s[q + 4]), __uint_as_float(s[q + 5]));
                    m3 = fmax3(m3, __uint_as_float(s[q + 6]), __uint_as_float(s[q + 7]));
                }
                const float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * scale2;
                // the row's reference after the tile before, and after this one
                if (cc > 0 && !(ok = pipe.wait_warp(kBarRef + pair, (cc - 1) & 1))) break;
                const float ref = k > 0 ? *refs : -INFINITY;
                const bool raise = mt > ref + 8.f || (ref == -INFINITY && mt != -INFINITY);
                const float m_new = raise ? mt : ref;
                *refs = m_new;
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarRef + pair);
                if (__any_sync(kFull, raise && ref != -INFINITY)) {
                    // O holds the tiles before this one. The other buffer's PV of three tiles before may still
                    // be open, and by its parity the last one's would pass for complete: this buffer's of two
                    // tiles before, whose own phase before this warp has waited for, comes first.
                    if (cc >= 2 && !(ok = pipe.wait_warp(kBarPV + 2 * x + w, ((cc >> 1) - 1) & 1))) break;
                    if (!(ok = pipe.wait_warp(kBarPV + 2 * x + (w ^ 1), ((cc - 1) >> 1) & 1))) break;
                    tc_fence_after();
                    const float fac = raise && ref != -INFINITY ? exp2_ftz(ref - m_new) : 1.f;
#pragma unroll 1
                    for (int part = 0; part < D / 8; ++part) {
                        uint32_t o[8];
                        tmem_ld8(o_col + part * 8, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * fac);
                        tmem_st8(o_col + part * 8, o);
                    }
                }
                l *= m_new == m ? 1.f : exp2_ftz(m - m_new);  // 0 when m is -inf
                m = m_new;
                const float nb = m == -INFINITY ? 0.f : -m;
                const float2 nb2 = make_float2(nb, nb);
                float2 z0 = make_float2(0.f, 0.f), z1 = z0;
#pragma unroll
                for (int q = 0; q < 64; q += 8) {
                    float2 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] = fma2(as2(s + q + 2 * u), scale22, nb2);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] = make_float2(exp2_ftz(v[u].x), exp2_ftz(v[u].y));
                    z0 = add2(z0, add2(v[0], v[1]));
                    z1 = add2(z1, add2(v[2], v[3]));
#pragma unroll
                    for (int u = 0; u < 4; ++u) s[q / 2 + u] = pack_bf16(v[u].x, v[u].y);  // s[q / 2 ..] has been read
                }
                l += (z0.x + z0.y) + (z1.x + z1.y);
                // the PV of two tiles before has read this buffer
                if (cc >= 2 && !(ok = pipe.wait_warp(kBarPV + 2 * x + w, ((cc >> 1) - 1) & 1))) break;
                tc_fence_after();
                tmem_st32(p_col, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                pipe.arrive_if(lane == 0, kBarP + 2 * x + w);
            }
            if (!ok) break;
            c += own.n;
            // ---- O / l and lse: by the warpgroup of the last tile
            if (own.n > 0) {
                const int end = kBarEnd + 8 * (n_items & 1) + pair;
                float2 *e = ends + (n_items & 1) * 2 * kM;
                if (((c - 1) & 1) != w) {
                    *e = make_float2(m, l);
                    __syncwarp();
                    pipe.arrive_if(lane == 0, end);
                    ++n_items;
                    continue;
                }
                if (!(ok = pipe.wait_warp(end, (n_items >> 1) & 1))) break;
                ++n_items;
                const float2 y = *e;
                const float mf = fmaxf(m, y.x);  // references only rise
                if (mf != -INFINITY) l = l * exp2_ftz(m - mf) + y.y * exp2_ftz(y.x - mf);
                m = mf;
                if (!(ok = pipe.wait_warp(kBarPV + 2 * x + w, ((c - 1) >> 1) & 1))) break;
                tc_fence_after();
            } else if (w == 1) {
                continue;
            }
            const bool some = m != -INFINITY && l > 0.f;  // a split may hold nothing that the row sees
            const float inv = some ? __fdividef(1.f, l) : 0.f;
            const int64_t place = ((int64_t)b * a.H + h) * a.Lq + i;
            const int slot = PREFIX ? 2 * it.split + x : it.split;
            const bool part = a.part_o != nullptr;  // float32 partial rows, else bf16 outputs
            if (have && (part || a.lse))
                (part ? a.part_lse[place * a.slots + slot] : a.lse[place]) = some ? (m + log2f(l)) * kLn2 : -INFINITY;
            // the four rows of a lane's group of four (null: no row)
            char *to[4];
            {
                const uint64_t p = !have ? 0ull
                                   : part ? (uint64_t)(a.part_o + (place * a.slots + slot) * D)
                                          : (uint64_t)(static_cast<bf16 *>(a.O.ptr) + b * a.O.sb + h * a.O.sh + (int64_t)i * a.O.st);
#pragma unroll
                for (int k = 0; k < 4; ++k) to[k] = reinterpret_cast<char *>(__shfl_sync(kFull, p, (lane & ~3) + k)) + (lane & 3) * 16;
            }
            const bool live[4] = {(uint64_t)to[0] >= 64, (uint64_t)to[1] >= 64, (uint64_t)to[2] >= 64, (uint64_t)to[3] >= 64};
#pragma unroll 1
            for (int col = 0; col < D; col += 32) {
                uint32_t o[32];
                if (own.n > 0) {  // every lane loads
                    tmem_ld32(o_col + col, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = 0u;
                }
#pragma unroll
                for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * inv);
                if (part) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint4 u[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            u[q] = make_uint4(o[16 * g + 4 * q], o[16 * g + 4 * q + 1], o[16 * g + 4 * q + 2], o[16 * g + 4 * q + 3]);
                        swap_units(u);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (live[k]) *reinterpret_cast<uint4 *>(to[k] + col * 4 + g * 64) = u[k];
                    }
                } else {
                    uint4 u[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = pack_bf16(__uint_as_float(o[8 * q + 2 * k]), __uint_as_float(o[8 * q + 2 * k + 1]));
                        u[q] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    swap_units(u);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (live[k]) *reinterpret_cast<uint4 *>(to[k] + col * 2) = u[k];
                }
            }
            if (own.n > 0) {
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

template <int D, bool PREFIX>
hils_status run(const FwdTc &f, const CUtensorMap (&m)[5], cudaStream_t s) {
    static KernelSetup setup;
    int per_sm = 0;
    const auto k = sink_fwd_tc_kernel<D, PREFIX>;
    const hils_status st = kernel_setup(setup, (const void *)k, kThreads, Smem<D, PREFIX>::kBytes, &per_sm);
    if (st != HILS_OK) return st;
    if (per_sm < 1) return HILS_ERR_CUDA;
    const int sms = device_sm_count();
    return sink_launch(false, k, f.items < sms ? f.items : sms, kThreads, Smem<D, PREFIX>::kBytes, s, m[0], m[1], m[2], m[3], m[4], f);
}

}  // namespace

bool launch_sink_forward_tc(hils_dtype dt, int d, const SinkArgs &a, cudaStream_t s, hils_status *st) {
    if (dt != HILS_BF16 || a.N == 0 || !(a.scale > 0.f)) return false;  // (a negative scale: the largest product is not the largest logit)
    const int Hk = a.H / a.G;
    FwdTc f{};
    f.a = a;
    CUtensorMap m[5];
    int64_t items;
    if (a.prefix) {
        f.nb = kM / a.G;
        f.tiles = (a.B + f.nb - 1) / f.nb;
        items = (int64_t)Hk * f.tiles * ((a.splits + 1) / 2);
        if (!make_row_map(&m[0], a.Q.ptr, d, {a.H, a.B, 1}, {a.Q.sh, a.Q.sb, 0}, a.G, f.nb)) return false;
    } else {
        f.P = sink_pack(a.G);
        f.qt = kM / f.P;
        f.nqb = (a.Lq + 2 * f.qt - 1) / (2 * f.qt);
        f.hp = a.H / f.P;
        f.units = a.B * f.hp;
        items = (int64_t)f.units * f.nqb * a.splits;
        if (!make_view_map(&m[0], a.Q, a.B, a.H, a.Lq, d, f.qt, f.P)) return false;
    }
    if (items > 0x7fffffffll - 1024) return false;
    f.items = (int)items;
    const int B = a.prefix ? 1 : a.B;
    if (!make_view_map(&m[1], a.K, B, Hk, a.N, d, kKeys, 1) || !make_view_map(&m[2], a.V, B, Hk, a.N, d, kKeys, 1))
        return false;
    // the sinks alone: their maps end at the last one
    const int sinks = a.A > 0 ? a.A : 1;
    f.sink_box = sinks < kKeys ? (sinks + 15) & ~15 : kKeys;
    if (!make_view_map(&m[3], a.K, B, Hk, sinks, d, f.sink_box, 1) ||
        !make_view_map(&m[4], a.V, B, Hk, sinks, d, f.sink_box, 1))
        return false;
    *st = a.prefix ? (d == 64 ? run<64, true>(f, m, s) : run<128, true>(f, m, s))
                   : (d == 64 ? run<64, false>(f, m, s) : run<128, false>(f, m, s));
    return true;
}

}  // namespace hils
