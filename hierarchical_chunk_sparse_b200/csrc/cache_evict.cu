// Eviction from a KV cache by accumulated attention weight. Per (b, key-value head) with
// n = cache_len[b] tokens, n > budget: keep the slots [0, A), the W newest and, of the
// slots between, the m = budget - A - W with the largest acc (equal ones: the lower slot;
// NaN counts as the smallest). The kept rows are written in slot order.
#include "sink_common.cuh"

namespace hils {
namespace {

// Order of the accumulated weights: larger float, larger key; -0 equals +0, NaN is lowest.
__device__ __forceinline__ unsigned weight_key(float f) { return f != f ? 0u : ordered_key(f + 0.f); }

// A cluster of C CTAs per (b, head): the m-th largest key by histograms of 2048 bins over the
// keys' range, then over the bin that holds it (three at most), with the keys in registers. Each
// CTA counts its share of the slots and reads the others' counts over distributed shared memory,
// so that all come to the same threshold. It ends early once a bin's lower border leaves exactly
// m keys. Equal bins within a warp are counted by one lane: many weights are zero, and their
// atomics on one address took 70 us of the 77 at 64 x 32K slots. Warp w of CTA c holds the keys of
// R * 32 consecutive slots; those behind C * THR * R slots are read again for each histogram. Slots
// are counted unsigned: a step past the last one may pass 2^31.
// Bound by the latencies of its steps.
constexpr int kBins = 2048;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}
// The address of a shared variable in CTA `rank` of the cluster, and a load from there.
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ int2 load_int2(uint32_t at) {
    int2 v;
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

template <int THR, int R, int C>
__global__ void __cluster_dims__(C) __launch_bounds__(THR) evict_select_kernel(EvictArgs a) {
    constexpr int kW = THR / 32, kPer = kBins / THR;  // kPer: 2, 4 or 8 bins a thread
    __shared__ __align__(16) int hist[kBins];
    __shared__ int sh[2][kW];
    __shared__ int2 base[kW];
    __shared__ int2 range;
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rank = blockIdx.x % C, gwarp = rank * kW + warp;
    const int64_t bk = blockIdx.x / C;
    const int b = (int)(bk / a.Hk);
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    const float *acc = a.acc + bk * a.T;
    int32_t *idx = a.idx + bk * a.budget;
    if (n <= a.budget) {
        for (unsigned i = rank * THR + tid; i < (unsigned)a.budget; i += C * THR) idx[i] = i < (unsigned)n ? (int)i : -1;
        return;
    }
    const int m0 = a.A, m1 = n - a.W, m = a.budget - a.A - a.W;  // m of [m0, m1), fewer than there are
    for (unsigned i = rank * THR + tid; i < (unsigned)a.A; i += C * THR) idx[i] = i;
    for (unsigned i = rank * THR + tid; i < (unsigned)a.W; i += C * THR) idx[a.budget - a.W + i] = n - a.W + i;
    if (m == 0) return;
    const unsigned mid = m1 - m0, far = C * THR * R;  // slots [far, mid) of the middle stay in memory
    unsigned key[R];
    unsigned low = 0xffffffffu, high = 0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const unsigned i = (gwarp * R + r) * 32 + lane;
        key[r] = i < mid ? weight_key(__ldg(acc + m0 + i)) : 0u;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = (gwarp * R + r) * 32 + lane < mid;
        low = min(low, in ? key[r] : 0xffffffffu);
        high = max(high, key[r]);
    }
    for (unsigned i = far + rank * THR + tid; i < mid; i += C * THR) {
        const unsigned k = weight_key(__ldg(acc + m0 + i));
        low = min(low, k);
        high = max(high, k);
    }
    low = __reduce_min_sync(kFull, low);
    high = __reduce_max_sync(kFull, high);
    if (lane == 0) {
        sh[0][warp] = (int)low;
        sh[1][warp] = (int)high;
    }
    __syncthreads();
    low = __reduce_min_sync(kFull, lane < kW ? (unsigned)sh[0][lane] : 0xffffffffu);
    high = __reduce_max_sync(kFull, lane < kW ? (unsigned)sh[1][lane] : 0u);
    if (tid == 0) range = make_int2((int)low, (int)high);
    cluster_sync();
    for (int c = 0; c < C; ++c) {
        const int2 x = load_int2(in_cta(&range, c));
        low = min(low, (unsigned)x.x);
        high = max(high, (unsigned)x.y);
    }
    unsigned thr = low;  // the keys of the bins: [thr, high]
    int shift = high > low ? max(0, 32 - __clz(high - low) - 11) : 0, left = m;
    bool exact = false;  // exactly the keys from thr on are kept
    auto count = [&](bool in, unsigned k) {
        const unsigned bin = (k - thr) >> shift;
        in = in && k >= thr && k <= high;
        const unsigned act = __ballot_sync(kFull, in);
        if (act == 0u) return;
        const unsigned first = __shfl_sync(kFull, bin, __ffs(act) - 1);
        const unsigned same = __ballot_sync(kFull, in && bin == first);
        if (lane == __ffs(act) - 1) atomicAdd(&hist[first], __popc(same));
        else if (in && bin != first) atomicAdd(&hist[bin], 1);
    };
    while (true) {
        for (int i = tid; i < kBins; i += THR) hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) count((gwarp * R + r) * 32 + lane < mid, key[r]);
        for (unsigned i0 = far + rank * THR; i0 < mid; i0 += C * THR) {
            const unsigned i = i0 + tid;
            count(i < mid, i < mid ? weight_key(__ldg(acc + m0 + i)) : 0u);
        }
        cluster_sync();
        // thread t has bins [kBins - kPer (t + 1), kBins - kPer t): sums from the top
        const int top = kBins - kPer * tid;
        int bins[kPer] = {}, mine = 0;  // bins[q]: bin top - kPer + q
        for (int c = 0; c < C; ++c) {
            const uint32_t at = in_cta(&hist[top - kPer], c);
#pragma unroll
            for (int q = 0; q < kPer; q += 2) {
                const int2 x = load_int2(at + 4 * q);
                bins[q] += x.x;
                bins[q + 1] += x.y;
            }
        }
#pragma unroll
        for (int q = 0; q < kPer; ++q) mine += bins[q];
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sh[0][warp] = sum;
        __syncthreads();
        const int before = __reduce_add_sync(kFull, lane < warp ? sh[0][lane] : 0);
        int cum = before + sum - mine;  // in the bins above this thread's
        if (cum < left && cum + mine >= left) {
            bool open = true;
#pragma unroll
            for (int q = kPer - 1; q >= 0; --q) {
                if (!open) continue;
                if (cum + bins[q] >= left) {
                    found[0] = top - kPer + q;
                    found[1] = cum;
                    found[2] = bins[q];
                    open = false;
                } else {
                    cum += bins[q];
                }
            }
        }
        __syncthreads();
        thr += (unsigned)found[0] << shift;
        high = min(high, thr + ((1u << shift) - 1u));  // (thr + 2^shift - 1 does not wrap: thr <= the bin's keys)
        left -= found[1];
        exact = found[2] == left;
        if (exact || shift == 0) break;
        shift = max(0, shift - 11);
        cluster_sync();  // hist and found are free again
    }
    // keys above thr are kept, and of those equal to it the first need (all of them if exact)
    auto kind = [&](unsigned i, unsigned k) { return i >= mid ? 0 : k > thr || (exact && k == thr) ? 2 : k == thr ? 1 : 0; };
    int2 mine = make_int2(0, 0);  // of this warp's register slots: above, equal
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = kind((gwarp * R + r) * 32 + lane, key[r]);
        mine.x += __popc(__ballot_sync(kFull, t == 2));
        mine.y += __popc(__ballot_sync(kFull, t == 1));
    }
    if (lane == 0) base[warp] = mine;
    cluster_sync();
    const int need = left;  // of the keys equal to thr
    int2 at = make_int2(0, 0), all = make_int2(0, 0);  // in the warps before this one; in all
#pragma unroll
    for (int w0 = 0; w0 < C * kW; w0 += 32) {
        const int w = w0 + lane;
        const int2 x = w < C * kW ? load_int2(in_cta(&base[w % kW], w / kW)) : make_int2(0, 0);
        all.x += __reduce_add_sync(kFull, x.x);
        all.y += __reduce_add_sync(kFull, x.y);
        at.x += __reduce_add_sync(kFull, w < gwarp ? x.x : 0);
        at.y += __reduce_add_sync(kFull, w < gwarp ? x.y : 0);
    }
    cluster_sync();  // nobody's shared memory is read any more
    auto keep = [&](unsigned i, int t, int2 &p) {
        const unsigned up = __ballot_sync(kFull, t == 2), eq = __ballot_sync(kFull, t == 1), lower = (1u << lane) - 1u;
        const int gt = p.x + __popc(up & lower), eb = p.y + __popc(eq & lower);
        if (t == 2 || (t == 1 && eb < need)) idx[a.A + gt + min(eb, need)] = m0 + i;
        p.x += __popc(up);
        p.y += __popc(eq);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const unsigned i = (gwarp * R + r) * 32 + lane;
        keep(i, kind(i, key[r]), at);
    }
    if (rank > 0) return;
    // the slots that stayed in memory: THR at a time, in order
    for (unsigned i0 = far; i0 < mid; i0 += THR) {
        const unsigned i = i0 + tid;
        const int t = i < mid ? kind(i, weight_key(__ldg(acc + m0 + i))) : 0;
        const int2 x = make_int2(__popc(__ballot_sync(kFull, t == 2)), __popc(__ballot_sync(kFull, t == 1)));
        __syncthreads();
        if (lane == 0) base[warp] = x;
        __syncthreads();
        int2 p = all;
        for (int w = 0; w < kW; ++w) {
            const int2 y = base[w];
            if (w < warp) p = make_int2(p.x + y.x, p.y + y.y);
            all = make_int2(all.x + y.x, all.y + y.y);
        }
        keep(i, t, p);
    }
}

// Copies the kept rows: a warp takes 256 / U rows of U 16-byte units (K's, then V's), so that
// each lane has eight loads in flight; bound by HBM (5.3 TB/s, 95 us, for 64 x 8192 rows of
// d = 128). Block 0 also writes the new lengths.
template <int U>
__global__ void __launch_bounds__(256) evict_gather_kernel(EvictArgs a, int esize) {
    constexpr int kRows = 256 / U;
    const int lane = threadIdx.x % 32;
    const int64_t rows = (int64_t)a.B * a.Hk * a.budget, r0 = ((int64_t)blockIdx.x * 8 + threadIdx.x / 32) * kRows;
    pdl_wait();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += 256) a.len_out[b] = min(min(max(a.cache_len[b], 0), a.T), a.budget);
    if (r0 >= rows) return;
    const int my = lane < kRows && r0 + lane < rows ? a.idx[r0 + lane] : -1;
    // the first row's (b, head) and place; rows number less than 2^31
    const unsigned bk0 = (unsigned)r0 / (unsigned)a.budget, b0 = bk0 / (unsigned)a.Hk;
    const int r = (int)((unsigned)r0 - bk0 * (unsigned)a.budget), h0 = (int)(bk0 - b0 * (unsigned)a.Hk);
    // of a row `on` further: heads passed, and its place
    auto place = [&](int on, int *rr) {
        int k = 0;
        for (*rr = r + on; *rr >= a.budget; ++k) *rr -= a.budget;
        return k;
    };
    if ((unsigned)my < (unsigned)a.T) {
        int rr;
        const int64_t bk = (int64_t)bk0 + place(lane, &rr);
        a.acc_out[r0 + lane] = __ldg(a.acc + bk * a.T + my);
    }
    uint4 v[8];
    char *to[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = i * 32 + lane, row = e / U, u = e % U;
        const int j = __shfl_sync(kFull, my, row);
        int rr, h = h0 + place(row, &rr), b = (int)b0;
        for (; h >= a.Hk; ++b) h -= a.Hk;
        const bool val = u >= U / 2;
        const View &s = val ? a.V : a.K;
        const MutView &d = val ? a.Vout : a.Kout;
        to[i] = nullptr;
        if ((unsigned)j < (unsigned)a.T) {
            const int x = (val ? u - U / 2 : u) * 16;
            v[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(s.ptr) +
                                                         (b * s.sb + h * s.sh + (int64_t)j * s.st) * esize + x));
            to[i] = static_cast<char *>(d.ptr) + (b * d.sb + h * d.sh + (int64_t)rr * d.st) * esize + x;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (to[i]) *reinterpret_cast<uint4 *>(to[i]) = v[i];
}

template <int THR, int R, int C>
hils_status select(const EvictArgs &a, cudaStream_t s) {
    const int64_t grid = (int64_t)a.B * a.Hk * C;
    if (grid > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
    evict_select_kernel<THR, R, C><<<(unsigned)grid, THR, 0, s>>>(a);
    return record_cuda_error(cudaGetLastError());
}

template <int U>
hils_status gather(const EvictArgs &a, int esize, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.Hk * a.budget, per = 8 * (256 / U), grid = rows > 0 ? (rows + per - 1) / per : 1;
    return sink_launch(rows > 0, evict_gather_kernel<U>, grid, 256, 0, s, a, esize);
}

}  // namespace

// The select's CTAs hold T slots in registers, 8192 a CTA up to 32K slots: clusters of four
// instead of a CTA of 1024 threads took 46 -> 36 us for 64 rows of 32K and 309 -> 45 us with the
// copy for 8 rows of 128K; with no more CTAs than T needs, since idle slots cost as much as others
// (512 rows of 4096: 252 -> 74 us).
hils_status launch_cache_evict(hils_dtype dt, int d, const EvictArgs &a, cudaStream_t s) {
    if ((int64_t)a.B * a.Hk * a.budget > 0) {
        const hils_status st = a.T <= 2048    ? select<256, 8, 1>(a, s)
                               : a.T <= 4096  ? select<512, 8, 1>(a, s)
                               : a.T <= 8192  ? select<512, 16, 1>(a, s)
                               : a.T <= 16384 ? select<512, 16, 2>(a, s)
                               : a.T <= 32768 ? select<512, 16, 4>(a, s)
                               : a.T <= 65536 ? select<1024, 32, 2>(a, s)
                                              : select<1024, 32, 4>(a, s);
        if (st != HILS_OK) return st;
    }
    if (a.B == 0) return HILS_OK;
    const int esize = dt == HILS_BF16 ? 2 : 4, units = 2 * d * esize / 16;
    return units == 16 ? gather<16>(a, esize, s) : units == 32 ? gather<32>(a, esize, s) : gather<64>(a, esize, s);
}

}  // namespace hils
