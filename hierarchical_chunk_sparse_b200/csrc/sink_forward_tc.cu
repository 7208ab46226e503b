// Window-and-sink attention on the 5th-generation tensor cores (bf16): prefill and the
// shared prefix of a decode batch (formulas in sink_common.cuh).
//
// A persistent CTA (one per SM) takes items of two 128-row query tiles A and B and walks
// 128-key tiles with an online softmax: S = Q K^T (M = 128 rows, N = keys, K = d) into
// TMEM, the softmax over it with P (bf16) written over S, O += P V with P read from TMEM.
//   prefill  a tile is P heads of a group (the largest power of two <= 8 that divides G)
//            with 128 / P consecutive queries each; A and B are neighbours and share each
//            key tile; a tile that only one of them sees is skipped by the other. The
//            sinks' tiles come first, from a tensor map that ends at the last sink, then
//            the window's from its first visible key: a slot that no query sees is never
//            loaded. The last tile's products cover only its keys, rounded up to 16.
//   prefix   a tile is 128 / G sequences with the G heads of a group each, so that the
//            prefix is read once for all of them; A and B are the same rows over two key
//            ranges, which the combine joins.
// Warp roles (384 threads), hand-offs through mbarriers:
//   warps 0-3, 4-7  softmax of tile A, B: a thread owns a row (TMEM lane); its reference
//                   maximum is raised, and O rescaled, only when the tile's maximum passes
//                   it by more than 8 in log2 units (P <= 2^8: exact in the float32 sums,
//                   no worse rounded in bf16);
//   warps 8, 9      tcgen05.mma of tile A, B;   warp 10  TMA.
// S of a tile is single-buffered and its next S is issued once the PV that read P has
// completed: while A is in its softmax the tensor cores work for B, and the other way.
// TMEM: S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512).
#include "sink_tc.cuh"

namespace hils {
namespace {

using namespace tc;

constexpr int kM = 128, kKeys = 128, kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum {
    kBarQfull = 0,    // + tile (prefix: 0 for both)
    kBarQfree = 2,    // + tile
    kBarKfull = 4,    // + slot
    kBarKfree = 8,    // + slot
    kBarVfull = 12,   // + slot
    kBarVfree = 14,   // + slot
    kBarS = 16,       // + tile: S written
    kBarP = 18,       // + tile: P written over it (4 warps)
    kBarPV = 20,      // + tile: PV, and every MMA before it, completed
    kBarOfree = 22,   // + tile: O read (4 warps)
    kBarDrain = 24,   // + tile
    kNumBars = 26
};

struct FwdTc {
    SinkArgs a;
    int P, qt, nqb;     // prefill: packed heads, queries of a tile, row items per (b, packed heads)
    int nb, tiles;      // prefix: sequences of a tile, tiles
    int items, sink_box;
};

struct PrefixItem {
    int hk, h, i0;      // key-value head, its first query head, first sequence
    int split;
    bool hasB;          // there is a second key range
    int r0[2], r1[2];   // the key tiles of A's and B's range
};

template <int D, bool PREFIX>
struct Smem {
    static constexpr int kTileBytes = kM * D * 2;
    static constexpr int kQ = 0;
    static constexpr int kK = (PREFIX ? 1 : 2) * kTileBytes;
    static constexpr int kV = kK + (PREFIX ? 4 : 2) * kTileBytes;
    static constexpr int kBars = kV + 2 * kTileBytes;
    static constexpr int kMisc = kBars + 8 * kNumBars;
    static constexpr int kBytes = kMisc + 16 + 1024;  // + alignment slack
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
        const int nt = (a.N + kKeys - 1) / kKeys;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 2 * it.split + x;
            it.r0[x] = x == 0 || it.hasB ? (int)((int64_t)nt * r / a.splits) : 0;
            it.r1[x] = x == 0 || it.hasB ? (int)((int64_t)nt * (r + 1) / a.splits) : 0;
        }
        return it;
    } else {
        return RowItem<kKeys>(j, a.B, a.H, a.G, f.P, f.qt, f.nqb, a.Lq, a.N, a.W, a.A, a.splits);
    }
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1) sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                  const __grid_constant__ CUtensorMap tmK,
                                                                  const __grid_constant__ CUtensorMap tmV,
                                                                  const __grid_constant__ CUtensorMap tmKs,
                                                                  const __grid_constant__ CUtensorMap tmVs, FwdTc f) {
    extern __shared__ uint8_t smem_raw[];
    using L = Smem<D, PREFIX>;
    constexpr int kBlocks = D / 64;           // 64-column blocks of a row tile, 16 KB each
    constexpr int kBlk = kM * 128;
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const SinkArgs &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    const Pipe pipe{sbase + L::kBars, misc + 1, a.status, a.wait_ns};
    const int G = gridDim.x, cta = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t cnt = 1;
            if (i >= kBarP && i < kBarP + 2) cnt = 4;
            if (i >= kBarOfree && i < kBarOfree + 2) cnt = 4;
            // both tiles release what they share
            if (PREFIX && i == kBarQfree) cnt = 2;
            if (!PREFIX && ((i >= kBarKfree && i < kBarKfree + 4) || (i >= kBarVfree && i < kBarVfree + 2))) cnt = 2;
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
        // ---------------------------------------------------------------- TMA
        int nq[2] = {0, 0}, nk[4] = {0, 0, 0, 0}, nv[2] = {0, 0};  // copies into each slot
        if (lane == 0) {
            bool ok = true;
            auto tile = [&](uint32_t dst, const CUtensorMap *m, int bar, int y, int z, int w) {
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) tma_load_4d(dst + c * kBlk, m, pipe.bar(bar), c * 64, y, z, w);
            };
            auto load_kv = [&](int ks, int vs, int k0, bool sink, int hk, int b) {
                const uint32_t bytes = (uint32_t)(sink ? f.sink_box : kKeys) * D * 2;
                if (nk[ks] > 0 && !(ok = pipe.wait(kBarKfree + ks, (nk[ks] - 1) & 1))) return;
                mbar_expect_tx(pipe.bar(kBarKfull + ks), bytes);
                ++nk[ks];
                tile(sbase + L::kK + ks * L::kTileBytes, sink ? &tmKs : &tmK, kBarKfull + ks, k0, hk, b);
                if (nv[vs] > 0 && !(ok = pipe.wait(kBarVfree + vs, (nv[vs] - 1) & 1))) return;
                mbar_expect_tx(pipe.bar(kBarVfull + vs), bytes);
                ++nv[vs];
                tile(sbase + L::kV + vs * L::kTileBytes, sink ? &tmVs : &tmV, kBarVfull + vs, k0, hk, b);
            };
            int g = 0;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= f.items) break;
                const auto it = decode_item<PREFIX>(f, j);
                if constexpr (PREFIX) {
                    if (nq[0] > 0 && !(ok = pipe.wait(kBarQfree, (nq[0] - 1) & 1))) break;
                    mbar_expect_tx(pipe.bar(kBarQfull), (uint32_t)(f.nb * a.G) * D * 2);
                    ++nq[0];
                    tile(sbase + L::kQ, &tmQ, kBarQfull, it.h, it.i0, 0);
                    const int n0 = it.r1[0] - it.r0[0], n1 = it.r1[1] - it.r0[1];
                    for (int i = 0; i < max(n0, n1) && ok; ++i) {
                        if (i < n0) load_kv((nv[0] & 1), 0, (it.r0[0] + i) * kKeys, false, it.hk, 0);
                        if (ok && i < n1) load_kv(2 + (nv[1] & 1), 1, (it.r0[1] + i) * kKeys, false, it.hk, 0);
                    }
                } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (it.last(x) < 0) continue;
                    if (nq[x] > 0 && !(ok = pipe.wait(kBarQfree + x, (nq[x] - 1) & 1))) break;
                    mbar_expect_tx(pipe.bar(kBarQfull + x), kM * D * 2);
                    ++nq[x];
                    tile(sbase + L::kQ + x * L::kTileBytes, &tmQ, kBarQfull + x, it.i0 + x * f.qt, it.h, it.b);
                }
                for (int e = it.e0; e < it.e1 && ok; ++e, ++g) {
                    load_kv(g & 1, g & 1, it.first_key(e), e < it.sp.ns, it.hk, it.b);
                }
                }
            }
            // what was started lands before the CTA's memory is released
            for (int x = 0; x < 2; ++x) pipe.drain(kBarQfull + x, nq[x]);
            for (int x = 0; x < 4; ++x) pipe.drain(kBarKfull + x, nk[x]);
            for (int x = 0; x < 2; ++x) pipe.drain(kBarVfull + x, nv[x]);
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ---------------------------------------------------------------- MMA of tile x
        const int x = warp - kMmaWarp;
        if (lane == 0) {
            bool ok = true;
            int g = 0;   // entries, over all items (prefill)
            int c = 0;   // tiles of x
            int n = 0;   // items with tiles of x
            const uint32_t q = sbase + L::kQ + (PREFIX ? 0 : x * L::kTileBytes);
            const int bq = PREFIX ? 0 : x;
            auto run_tile = [&](int ks, uint32_t kpar, int vs, uint32_t vpar, int nkeys, bool first, bool last) {
                const int n16 = (nkeys + 15) & ~15;
                const uint32_t kb = sbase + L::kK + ks * L::kTileBytes, vb = sbase + L::kV + vs * L::kTileBytes;
                if (!(ok = pipe.wait(kBarKfull + ks, kpar))) return;
                if (c > 0 && !(ok = pipe.wait(kBarPV + x, (c - 1) & 1))) return;
                tc_fence_after();
                const uint32_t idS = idesc_bf16(kM, n16, false);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t o = (s >> 2) * kBlk + (s & 3) * 32;
                    mma_ss(tmem + x * 128, smem_desc(q + o, 16, 1024), smem_desc(kb + o, 16, 1024), idS, s > 0);
                }
                mma_commit(pipe.bar(kBarS + x));
                mma_commit(pipe.bar(kBarKfree + ks));
                if (last) mma_commit(pipe.bar(kBarQfree + bq));
                if (!(ok = pipe.wait(kBarP + x, c & 1))) return;
                if (!(ok = pipe.wait(kBarVfull + vs, vpar))) return;
                if (first && n > 0 && !(ok = pipe.wait(kBarOfree + x, (n - 1) & 1))) return;
                tc_fence_after();
                for (int s = 0; s < n16 / 16; ++s)
                    mma_ts(tmem + 256 + x * 128, tmem + x * 128 + s * 8, smem_desc(vb + s * 2048, kBlk, 1024),
                           idesc_bf16(kM, D, true), !first || s > 0);
                mma_commit(pipe.bar(kBarVfree + vs));
                mma_commit(pipe.bar(kBarPV + x));
                ++c;
            };
            int nqx = 0;
            for (int r = 0; ok; ++r) {
                const int j = item_of_round(r, cta, G);
                if (j >= f.items) break;
                const auto it = decode_item<PREFIX>(f, j);
                if constexpr (PREFIX) {
                    if (!(ok = pipe.wait(kBarQfull, r & 1))) break;
                    const int nt = it.r1[x] - it.r0[x];
                    if (nt == 0) {
                        pipe.arrive(kBarQfree);
                        continue;
                    }
                    tc_fence_after();
                    for (int i = 0; i < nt && ok; ++i)
                        run_tile(2 * x + (c & 1), (c >> 1) & 1, x, c & 1, min(kKeys, a.N - (it.r0[x] + i) * kKeys), i == 0,
                                 i + 1 == nt);
                    ++n;
                } else {
                const int last = it.last(x);
                if (last >= 0) {
                    if (!(ok = pipe.wait(kBarQfull + x, nqx & 1))) break;
                    ++nqx;
                    tc_fence_after();
                }
                bool first = true;
                for (int e = it.e0; e < it.e1 && ok; ++e, ++g) {
                    const int nk = it.keys(x, e), s = g & 1;
                    const uint32_t par = (g >> 1) & 1;
                    if (nk > 0) {
                        run_tile(s, par, s, par, nk, first, e == last);
                        first = false;
                    } else {  // not this tile's: release it once it has landed
                        if (!(ok = pipe.wait(kBarKfull + s, par))) break;
                        pipe.arrive(kBarKfree + s);
                        if (!(ok = pipe.wait(kBarVfull + s, par))) break;
                        pipe.arrive(kBarVfree + s);
                    }
                }
                if (last >= 0) ++n;
                }
            }
            mma_commit(pipe.bar(kBarDrain + x));  // what was issued completes before TMEM is released
            pipe.drain(kBarDrain + x, 1);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---------------------------------------------------------------- softmax rows of tile x
        const int x = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t s_col = tmem + lanes + x * 128, o_col = tmem + lanes + 256 + x * 128;
        const float scale2 = a.scale * kLog2e;
        bool ok = true;
        int c = 0;
        for (int r = 0; ok; ++r) {
            const int j = item_of_round(r, cta, G);
            if (j >= f.items) break;
            const auto it = decode_item<PREFIX>(f, j);
            int b, h, i, t;
            bool have;
            int first_e, end_e;
            if constexpr (PREFIX) {
                first_e = it.r0[x];
                end_e = it.r1[x];
                b = it.i0 + row / a.G;
                h = it.h + row % a.G;
                i = 0;
                t = a.N;
                have = row < f.nb * a.G && b < a.B && (x == 0 || it.hasB);
            } else {
                first_e = it.e0;
                end_e = it.e1;
                b = it.b;
                h = it.h + row / f.qt;
                i = it.i0 + x * f.qt + row % f.qt;
                t = a.N - a.Lq + i;
                have = i < a.Lq;
            }
            float m = -INFINITY, l = 0.f;
            bool any_tile = false;
            for (int e = first_e; e < end_e; ++e) {
                int n, lo, hi, as;  // visible columns: [lo, hi) and [0, as)
                if constexpr (PREFIX) {
                    n = hi = min(kKeys, a.N - e * kKeys);
                    lo = as = 0;
                } else {
                    n = it.keys(x, e);
                    if (n <= 0) continue;
                    it.columns(e, n, t, a.W, &lo, &hi, &as);
                    if (!have) hi = as = 0;
                }
                any_tile = true;
                const bool full = __all_sync(kFull, lo <= 0 && hi == kKeys);
                if (!(ok = pipe.wait_warp(kBarS + x, c & 1))) break;
                tc_fence_after();
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
                uint32_t seen = 0;  // 32-column chunks that some row of the warp sees
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    const uint32_t mk = full ? kFull : range_bits(lo, hi, ch * 32) | range_bits(0, as, ch * 32);
                    if (!__any_sync(kFull, mk != 0)) continue;
                    seen |= 1u << ch;
                    uint32_t s[32];
                    tmem_ld32(s_col + ch * 32, s);
                    tmem_wait_ld();
                    if (!full) {
#pragma unroll
                        for (int q = 0; q < 32; ++q) s[q] = (mk >> q) & 1u ? s[q] : __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int q = 0; q < 32; q += 8) {
                        m0 = fmax3(m0, __uint_as_float(s[q]), __uint_as_float(s[q + 1]));
                        m1 = fmax3(m1, __uint_as_float(s[q + 2]), __uint_as_float(s[q + 3]));
                        m2 = fmax3(m2, __uint_as_float(s[q + 4]), __uint_as_float(s[q + 5]));
                        m3 = fmax3(m3, __uint_as_float(s[q + 6]), __uint_as_float(s[q + 7]));
                    }
                }
                float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
                if (scale2 < 0.f) {  // the largest logit is the smallest product: no reference from the maximum
                    mt = INFINITY;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        if (!((seen >> ch) & 1u)) continue;
                        const uint32_t mk = full ? kFull : range_bits(lo, hi, ch * 32) | range_bits(0, as, ch * 32);
                        uint32_t s[32];
                        tmem_ld32(s_col + ch * 32, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) mt = fminf(mt, (mk >> q) & 1u ? __uint_as_float(s[q]) : INFINITY);
                    }
                }
                const bool none = isinf(mt);  // no visible key in this tile
                mt = none ? -INFINITY : mt * scale2;
                const bool raise = !none && (m == -INFINITY || mt > m + 8.f);
                const float fac = raise ? exp2_ftz(m - mt) : 1.f;  // 0 when m is -inf
                if (__any_sync(kFull, raise && l > 0.f)) {
                    // S of this tile was issued after the PV of the one before had completed
#pragma unroll 1
                    for (int part = 0; part < D / 32; ++part) {
                        uint32_t o[32];
                        tmem_ld32(o_col + part * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * fac);
                        tmem_st32(o_col + part * 32, o);
                    }
                }
                if (raise) {
                    l *= fac;
                    m = mt;
                }
                const float nb = m == -INFINITY ? 0.f : -m;
                float z0 = 0.f, z1 = 0.f, z2 = 0.f, z3 = 0.f;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    if (ch * 32 >= n) continue;
                    uint32_t p[16];
                    if ((seen >> ch) & 1u) {
                        const uint32_t mk = full ? kFull : range_bits(lo, hi, ch * 32) | range_bits(0, as, ch * 32);
                        uint32_t s[32];
                        tmem_ld32(s_col + ch * 32, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; q += 4) {
                            float v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[k] = fmaf(__uint_as_float(s[q + k]), scale2, nb);
                            if (!full) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) v[k] = (mk >> (q + k)) & 1u ? v[k] : -INFINITY;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[k] = exp2_ftz(v[k]);
                            z0 += v[0];
                            z1 += v[1];
                            z2 += v[2];
                            z3 += v[3];
                            p[q / 2] = pack_bf16(v[0], v[1]);
                            p[q / 2 + 1] = pack_bf16(v[2], v[3]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) p[q] = 0u;
                    }
                    tmem_st16(s_col + ch * 16, p);  // columns whose S has been read
                }
                l += (z0 + z1) + (z2 + z3);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pipe.arrive(kBarP + x);
                ++c;
            }
            if (!ok) break;
            // ---- O / l and lse
            if (any_tile) {
                if (!(ok = pipe.wait_warp(kBarPV + x, (c - 1) & 1))) break;
                tc_fence_after();
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const float lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            const int64_t place = ((int64_t)b * a.H + h) * a.Lq + i;
            const int slot = PREFIX ? 2 * it.split + x : it.split;
            bf16 *orow = static_cast<bf16 *>(a.O.ptr) + b * a.O.sb + h * a.O.sh + (int64_t)i * a.O.st;
            float *prow = a.part_o ? a.part_o + (place * a.slots + slot) * D : nullptr;
#pragma unroll
            for (int part = 0; part < D / 32; ++part) {
                uint32_t o[32];
                if (any_tile) {  // every lane loads
                    tmem_ld32(o_col + part * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = 0u;
                }
                if (!have) continue;
                if (prow) {
                    float4 *dst = reinterpret_cast<float4 *>(prow + part * 32);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q] = make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                                             __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(orow + part * 32);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[8 * q + 0]) * inv, __uint_as_float(o[8 * q + 1]) * inv);
                        v.y = pack_bf16(__uint_as_float(o[8 * q + 2]) * inv, __uint_as_float(o[8 * q + 3]) * inv);
                        v.z = pack_bf16(__uint_as_float(o[8 * q + 4]) * inv, __uint_as_float(o[8 * q + 5]) * inv);
                        v.w = pack_bf16(__uint_as_float(o[8 * q + 6]) * inv, __uint_as_float(o[8 * q + 7]) * inv);
                        dst[q] = v;
                    }
                }
            }
            if (have) {
                if (prow) a.part_lse[place * a.slots + slot] = lse;
                else if (a.lse) a.lse[place] = lse;
            }
            if (any_tile) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pipe.arrive(kBarOfree + x);
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
    k<<<f.items < sms ? f.items : sms, kThreads, Smem<D, PREFIX>::kBytes, s>>>(m[0], m[1], m[2], m[3], m[4], f);
    return record_cuda_error(cudaGetLastError());
}

}  // namespace

bool launch_sink_forward_tc(hils_dtype dt, int d, const SinkArgs &a, cudaStream_t s, hils_status *st) {
    if (dt != HILS_BF16 || a.N == 0) return false;
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
        items = (int64_t)a.B * (a.H / f.P) * f.nqb * a.splits;
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
