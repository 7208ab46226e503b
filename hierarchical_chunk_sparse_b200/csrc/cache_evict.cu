// Eviction from a KV cache by accumulated attention weight. Per (b, key-value head) with
// n = cache_len[b] tokens, n > budget: keep the slots [0, A), the W newest and, of the
// slots between, the m = budget - A - W with the largest acc (equal ones: the lower slot;
// NaN counts as the smallest). The kept rows are written in slot order.
#include "sink_common.cuh"

namespace hils {
namespace {

// Order of the accumulated weights: larger float, larger key; -0 equals +0, NaN is lowest.
__device__ __forceinline__ unsigned weight_key(float f) { return f != f ? 0u : ordered_key(f + 0.f); }

// One CTA per (b, head): the m-th largest key by histograms of 2048 bins over the keys' range,
// then over the bin that holds it (three at most), with the keys in registers. It ends early
// once a bin's lower border leaves exactly m keys. Equal bins within a warp are counted by one
// lane: many weights are zero, and their atomics on one address took 70 us of the 77 at 64 x 32K
// slots. Warp w holds the keys of R * 32 consecutive slots; those behind THR * R slots are read
// again for each histogram.
constexpr int kBins = 2048;

template <int THR, int R>
__global__ void __launch_bounds__(THR) evict_select_kernel(EvictArgs a) {
    constexpr int kW = THR / 32, kPer = kBins / THR;
    __shared__ int hist[kBins];
    __shared__ int sh[2][kW];
    __shared__ int2 base[kW];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t bk = blockIdx.x;
    const int b = (int)(bk / a.Hk);
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    const float *acc = a.acc + bk * a.T;
    int32_t *idx = a.idx + bk * a.budget;
    if (n <= a.budget) {
        for (int i = tid; i < a.budget; i += THR) idx[i] = i < n ? i : -1;
        return;
    }
    const int m0 = a.A, m1 = n - a.W, m = a.budget - a.A - a.W;  // m of [m0, m1), fewer than there are
    for (int i = tid; i < a.A; i += THR) idx[i] = i;
    for (int i = tid; i < a.W; i += THR) idx[a.budget - a.W + i] = n - a.W + i;
    if (m == 0) return;
    const int mid = m1 - m0, far = THR * R;  // slots [far, mid) of the middle stay in memory
    unsigned key[R];
    unsigned low = 0xffffffffu, high = 0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = (warp * R + r) * 32 + lane;
        key[r] = i < mid ? weight_key(__ldg(acc + m0 + i)) : 0u;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = (warp * R + r) * 32 + lane < mid;
        low = min(low, in ? key[r] : 0xffffffffu);
        high = max(high, key[r]);
    }
    for (int i = far + tid; i < mid; i += THR) {
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
        for (int r = 0; r < R; ++r) count((warp * R + r) * 32 + lane < mid, key[r]);
        for (int i0 = far; i0 < mid; i0 += THR) {
            const int i = i0 + tid;
            count(i < mid, i < mid ? weight_key(__ldg(acc + m0 + i)) : 0u);
        }
        __syncthreads();
        // thread t has bins [kBins - kPer (t + 1), kBins - kPer t): sums from the top
        const int top = kBins - kPer * tid;
        int mine = 0;
#pragma unroll
        for (int q = 1; q <= kPer; ++q) mine += hist[top - q];
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
            int q = 1;
            while (cum + hist[top - q] < left) cum += hist[top - q++];
            found[0] = top - q;
            found[1] = cum;
            found[2] = hist[top - q];
        }
        __syncthreads();
        thr += (unsigned)found[0] << shift;
        high = min(high, thr + ((1u << shift) - 1u));  // (thr + 2^shift - 1 does not wrap: thr <= the bin's keys)
        left -= found[1];
        exact = found[2] == left;
        if (exact || shift == 0) break;
        shift = max(0, shift - 11);
        __syncthreads();  // hist and found are free again
    }
    // keys above thr are kept, and of those equal to it the first need (all of them if exact)
    auto kind = [&](int i, unsigned k) { return i >= mid ? 0 : k > thr || (exact && k == thr) ? 2 : k == thr ? 1 : 0; };
    int2 mine = make_int2(0, 0);  // of this warp's register slots: above, equal
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = kind((warp * R + r) * 32 + lane, key[r]);
        mine.x += __popc(__ballot_sync(kFull, t == 2));
        mine.y += __popc(__ballot_sync(kFull, t == 1));
    }
    if (lane == 0) base[warp] = mine;
    __syncthreads();
    const int need = left;  // of the keys equal to thr
    int2 at = make_int2(0, 0), all = make_int2(0, 0);
    for (int w = 0; w < kW; ++w) {
        const int2 x = base[w];
        if (w < warp) at = make_int2(at.x + x.x, at.y + x.y);
        all = make_int2(all.x + x.x, all.y + x.y);
    }
    auto keep = [&](int i, int t, int2 &p) {
        const unsigned up = __ballot_sync(kFull, t == 2), eq = __ballot_sync(kFull, t == 1), lower = (1u << lane) - 1u;
        const int gt = p.x + __popc(up & lower), eb = p.y + __popc(eq & lower);
        if (t == 2 || (t == 1 && eb < need)) idx[a.A + gt + min(eb, need)] = m0 + i;
        p.x += __popc(up);
        p.y += __popc(eq);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = (warp * R + r) * 32 + lane;
        keep(i, kind(i, key[r]), at);
    }
    // the slots that stayed in memory: THR at a time, in order
    for (int i0 = far; i0 < mid; i0 += THR) {
        const int i = i0 + tid, t = i < mid ? kind(i, weight_key(__ldg(acc + m0 + i))) : 0;
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
// each lane has eight loads in flight; bound by HBM. Block 0 also writes the new lengths.
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

template <int THR, int R>
hils_status select(const EvictArgs &a, cudaStream_t s) {
    evict_select_kernel<THR, R><<<(unsigned)(a.B * a.Hk), THR, 0, s>>>(a);
    return record_cuda_error(cudaGetLastError());
}

template <int U>
hils_status gather(const EvictArgs &a, int esize, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.Hk * a.budget, per = 8 * (256 / U), grid = rows > 0 ? (rows + per - 1) / per : 1;
    return sink_launch(rows > 0, evict_gather_kernel<U>, grid, 256, 0, s, a, esize);
}

}  // namespace

hils_status launch_cache_evict(hils_dtype dt, int d, const EvictArgs &a, cudaStream_t s) {
    if ((int64_t)a.B * a.Hk * a.budget > 0) {
        const hils_status st = a.T <= 2048 ? select<256, 8>(a, s) : a.T <= 16384 ? select<512, 32>(a, s) : select<1024, 32>(a, s);
        if (st != HILS_OK) return st;
    }
    if (a.B == 0) return HILS_OK;
    const int esize = dt == HILS_BF16 ? 2 : 4, units = 2 * d * esize / 16;
    return units == 16 ? gather<16>(a, esize, s) : units == 32 ? gather<32>(a, esize, s) : gather<64>(a, esize, s);
}

}  // namespace hils
