// What the tcgen05 kernels of the window-and-sink calls share: bounded waits, tensor maps
// of the row tiles, and the masks of a tile's columns.
#pragma once
#include "sink_common.cuh"
#include "tc_common.cuh"

namespace hils {
namespace tc {

// Non-blocking test of an mbarrier phase.
__device__ __forceinline__ bool mbar_test_phase(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The CTA's waits. Each is bounded by the global timer; the first one that expires sets
// the abort flag and bit 0 of the call's status word, after which every wait fails, the
// roles stop issuing, and the CTA drains what it started and returns.
// A wait knows its phase by the parity alone: with the phase before that one still open it
// returns at once. So whoever waits has to know that the phase before is complete: from its
// own earlier wait, or from an event that came after it.
struct Pipe {
    uint32_t bars;                  // shared address of the first mbarrier
    volatile uint32_t *abort_flag;  // shared
    uint32_t *status;
    long long wait_ns;

    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        const uint32_t b = bar(i);
        if (wait_ns > 0) {
            // a short wait never reads the timer
            for (int it = 0; it < 64; ++it)
                if (mbar_try_wait(b, parity)) return true;
            const uint64_t t0 = global_ns();
            for (int it = 0;; ++it) {
                if (mbar_try_wait(b, parity)) return true;
                if ((it & 15) == 15) {
                    if (*abort_flag) return false;
                    if ((long long)(global_ns() - t0) > wait_ns) break;
                }
            }
        }
        *abort_flag = 1u;
        atomicOr(status, 1u);
        return false;
    }
    // For a loop over several barriers: false once it has made no progress for the limit since
    // *since (0: none yet) or the CTA stops. `spins` counts the idle rounds.
    __device__ __forceinline__ bool idle(int *spins, uint64_t *since) const {
        bool ok = true;
        if (wait_ns == 0) {
            ok = false;
        } else if ((++*spins & 63) == 0) {
            const uint64_t now = global_ns();
            if (*since == 0) *since = now;
            if (*abort_flag) return false;
            ok = (long long)(now - *since) <= wait_ns;
        }
        ok = __all_sync(kFull, ok);
        if (!ok) {
            *abort_flag = 1u;
            atomicOr(status, 1u);
        }
        return ok;
    }
    // A converged warp waits; true if the phase completed. The loop's condition is a vote, so that
    // no branch diverges (one that does costs about 100 cycles, as does a branch around one lane's
    // arrival).
    __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
        const uint32_t b = bar(i);
        if (wait_ns > 0) {
            for (int it = 0; it < 64; ++it)
                if (__all_sync(kFull, mbar_try_wait(b, parity))) return true;
        }
        return __all_sync(kFull, wait(i, parity));
    }
    __device__ __forceinline__ void arrive(int i) const {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar(i)) : "memory");
    }
    // one lane's arrival (count times), without a branch
    __device__ __forceinline__ void arrive_if(bool on, int i, uint32_t count = 1) const {
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar(i)),
            "r"(count), "r"((uint32_t)on)
            : "memory");
    }
    // bounded wait for this CTA's own copies or MMAs while it stops: `uses` phases of barrier i
    __device__ __forceinline__ void drain(int i, int uses) const {
        if (uses == 0) return;
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(bar(i), (uint32_t)(uses - 1) & 1u))
            if ((long long)(global_ns() - t0) > kDrainLimitNs) break;
    }
};

// One lane of a converged warp. The tcgen05 instructions take their operands from uniform
// registers: under a per-lane condition like lane == 0 the compiler has to move each of them
// there and the issue of 16 products took 3200 cycles instead of some hundred.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// Descriptor of a tile at a shared address; an offset of o bytes within the CTA's memory adds o / 16.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo) { return smem_desc(addr, lbo, 1024); }

__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_slot), "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 2^x with the hardware approximation, results below 2^-126 flushed to 0 (without the flush
// each costs a compare and two products more).
__device__ __forceinline__ float exp2_ftz(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 as2(const uint32_t *r) { return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])); }
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Four lanes that hold 16-byte units 0..3 of their own rows (one row a lane) exchange them:
// afterwards unit k of lane j (of each four) is unit j of the row of lane k, so that one store
// of the warp writes 64 consecutive bytes of eight rows instead of 16 of 32.
__device__ __forceinline__ void swap_units(uint4 (&u)[4]) {
    const int lane = threadIdx.x % 32;
    auto step = [&](uint4 &a, uint4 &b, int mask) {  // a: kept by lanes without the bit, b: by those with it
        const bool up = lane & mask;
        uint4 s = up ? a : b;
        s.x = __shfl_xor_sync(kFull, s.x, mask);
        s.y = __shfl_xor_sync(kFull, s.y, mask);
        s.z = __shfl_xor_sync(kFull, s.z, mask);
        s.w = __shfl_xor_sync(kFull, s.w, mask);
        if (up) a = s;
        else b = s;
    };
    step(u[0], u[2], 2);
    step(u[1], u[3], 2);
    step(u[0], u[1], 1);
    step(u[2], u[3], 1);
}

// Bit q is set where lo <= c0 + q < hi.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int c0) {
    const int l = max(lo - c0, 0), h = min(hi - c0, 32);
    if (h <= l) return 0u;
    return (0xffffffffu >> (32 - (h - l))) << l;
}

// The work item of round r for CTA c of n: rounds alternate direction, so that every CTA
// gets a similar share of the expensive items, which come first.
__device__ __forceinline__ int item_of_round(int r, int c, int n) { return r * n + ((r & 1) ? (n - 1 - c) : c); }

// Two neighbouring row tiles A and B (P packed heads x qt queries each) of one (b, head
// pack), and the KT-key tiles that they see: the sinks' first, then the window's.
template <int KT>
struct RowItem {
    int b, h, hk, i0;   // batch, first packed head, its key-value head, first query of A
    int tA, tB;         // first positions
    SinkSpan sp;
    int e0, e1, eA, wB; // entries of this split; A sees entries < eA, B the sinks' and window tiles >= wB
    int split;
    bool hasB;          // B has rows

    RowItem() = default;
    __device__ __forceinline__ RowItem(int j, int hp, int units, int G, int P, int qt, int nqb, int Lq, int N, int W, int A,
                                       int splits) {
        split = 0;
        if (splits > 1) {
            const int q = j / splits;
            split = j - q * splits;
            j = q;
        }
        const int q = j / units, u = j - q * units;  // units: (b, pack) pairs, hp: packs of a batch
        const int qb = nqb - 1 - q;  // latest queries (most keys) first
        b = u / hp;
        h = (u - b * hp) * P;
        hk = h / G;
        i0 = qb * 2 * qt;
        tA = N - Lq + i0;
        tB = tA + qt;
        hasB = tB < N;
        sp = sink_span(tA, min(N - 1, tB + qt - 1), W, A, KT);
        const int nt = sp.ns + sp.nw;
        e0 = 0;
        e1 = nt;
        if (splits > 1) {
            e0 = (int)((int64_t)nt * split / splits);
            e1 = (int)((int64_t)nt * (split + 1) / splits);
        }
        eA = sp.ns + (sp.nw > 0 ? (min(sp.hi, tB) - sp.lo + KT - 1) / KT : 0);
        const int gone = tB - W - sp.lo - (KT - 1);  // >= 0: B sees no key of the first window tile
        wB = sp.lo >= A && gone >= 0 ? gone / KT + 1 : 0;
    }
    __device__ __forceinline__ int first_key(int e) const { return e < sp.ns ? e * KT : sp.lo + (e - sp.ns) * KT; }
    // keys of entry e that tile x multiplies (0: it skips the entry)
    __device__ __forceinline__ int keys(int x, int e) const {
        const int k0 = first_key(e);
        if (e < sp.ns) return x == 0 || hasB ? min(KT, sp.sinks - k0) : 0;
        if (x == 0) return e < eA ? min(KT, min(sp.hi, tB) - k0) : 0;
        return hasB && e - sp.ns >= wB ? min(KT, sp.hi - k0) : 0;
    }
    // the last entry that tile x sees (-1: none)
    __device__ __forceinline__ int last(int x) const {
        if (x == 0) return min(e1, eA) > e0 ? min(e1, eA) - 1 : -1;
        if (!hasB) return -1;
        int l = e1 - 1;
        if (l >= sp.ns && l - sp.ns < wB) l = min(l, sp.ns - 1);
        return l >= e0 ? l : -1;
    }
};

// A map of a bf16 tensor with extents dims[0] = d elements (contiguous) and three outer
// dimensions with strides in elements, in boxes of 64 x b1 x b2 x 1 with the 128-byte
// swizzle; what lies outside the extents reads as zero. False if it cannot be described.
inline bool make_row_map(CUtensorMap *m, const void *ptr, int d, const int64_t (&dims)[3], const int64_t (&strides)[3],
                         int b1, int b2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dm[4] = {(cuuint64_t)d}, st[3];
    for (int i = 0; i < 3; ++i) {
        if (dims[i] <= 0 || dims[i] > 0x7fffffffll) return false;
        dm[i + 1] = (cuuint64_t)dims[i];
        const int64_t s = dims[i] == 1 ? (int64_t)d : strides[i];  // the stride of one row is of no matter
        if (s <= 0 || s >= (1ll << 38)) return false;
        st[i] = (cuuint64_t)s * 2;
    }
    const cuuint32_t box[4] = {64u, (cuuint32_t)b1, (cuuint32_t)b2, 1u}, estr[4] = {1u, 1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dm, st, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows of a [B, H, T, d] view: boxes of `rows` rows of `heads` heads.
inline bool make_view_map(CUtensorMap *m, const View &v, int64_t B, int64_t H, int64_t T, int d, int rows, int heads) {
    return make_row_map(m, v.ptr, d, {T, H, B}, {v.st, v.sh, v.sb}, rows, heads);
}

}  // namespace tc
}  // namespace hils
