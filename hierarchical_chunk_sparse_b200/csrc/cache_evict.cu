// Eviction from a KV cache by accumulated attention weight. Per (b, key-value head) with
// n = cache_len[b] tokens, n > budget: keep the slots [0, A), the W newest and, of the
// slots between, the budget - A - W with the largest acc (equal ones: the lower slot; NaN
// counts as the smallest). The kept rows are written in slot order.
#include "sink_common.cuh"

namespace hils {
namespace {

constexpr int kThr = 1024;

// Order of the accumulated weights: larger float, larger key; -0 equals +0, NaN is lowest.
__device__ __forceinline__ unsigned weight_key(float f) { return f != f ? 0u : ordered_key(f + 0.f); }

// Exclusive sum over the block of (x, y); the totals in *tx, *ty.
__device__ __forceinline__ void block_scan(int &x, int &y, int *total_x, int *total_y, int2 *sh) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ax = __shfl_up_sync(kFull, ix, o), ay = __shfl_up_sync(kFull, iy, o);
        if (lane >= o) {
            ix += ax;
            iy += ay;
        }
    }
    __syncthreads();
    if (lane == 31) sh[warp] = make_int2(ix, iy);
    __syncthreads();
    int bx = 0, by = 0, tx = 0, ty = 0;
    for (int w = 0; w < kThr / 32; ++w) {
        if (w == warp) {
            bx = tx;
            by = ty;
        }
        tx += sh[w].x;
        ty += sh[w].y;
    }
    x = bx + ix - x;
    y = by + iy - y;
    *total_x = tx;
    *total_y = ty;
}

// One CTA per (b, head): the threshold by a radix select of 8 bits a pass, then the kept
// slots in order.
__global__ void __launch_bounds__(kThr) evict_select_kernel(EvictArgs a) {
    __shared__ unsigned hist[256];
    __shared__ unsigned s_digit;
    __shared__ int s_need;
    __shared__ int2 sh[kThr / 32];
    const int tid = threadIdx.x;
    const int64_t bk = blockIdx.x;
    const int b = (int)(bk / a.Hk);
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    const float *acc = a.acc + bk * a.T;
    int32_t *idx = a.idx + bk * a.budget;
    if (n <= a.budget) {
        for (int i = tid; i < a.budget; i += kThr) idx[i] = i < n ? i : -1;
        return;
    }
    const int m0 = a.A, m1 = n - a.W, m = a.budget - a.A - a.W;  // m of [m0, m1), fewer than there are
    unsigned prefix = 0u, mask = 0u;
    int need = m;  // of the slots whose key has the prefix
    for (int shift = 24; shift >= 0 && m > 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThr) hist[i] = 0u;
        __syncthreads();
        for (int i = m0 + tid; i < m1; i += kThr) {
            const unsigned k = weight_key(acc[i]);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, dgt = 255;
            while (dgt > 0 && (int)hist[dgt] < left) left -= (int)hist[dgt--];
            s_digit = (unsigned)dgt;
            s_need = left;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= 255u << shift;
        need = s_need;
        __syncthreads();
    }
    for (int i = tid; i < a.A; i += kThr) idx[i] = i;
    for (int i = tid; i < a.W; i += kThr) idx[a.budget - a.W + i] = n - a.W + i;
    if (m == 0) return;
    int kept = 0, equal = 0;  // before this round: above the threshold, at it
    for (int i0 = m0; i0 < m1; i0 += kThr) {
        const int i = i0 + tid;
        const unsigned k = i < m1 ? weight_key(acc[i]) : 0u;
        int gt = i < m1 && k > prefix, eq = i < m1 && k == prefix, tg, te;
        const bool is_gt = gt != 0, is_eq = eq != 0;
        block_scan(gt, eq, &tg, &te, sh);
        const int before_eq = equal + eq;
        if (is_gt || (is_eq && before_eq < need)) idx[a.A + kept + gt + min(before_eq, need)] = i;
        kept += tg;
        equal += te;
        __syncthreads();
    }
}

// One warp per kept row; row 0 of head 0 also writes the sequence's new length.
__global__ void __launch_bounds__(256) evict_gather_kernel(EvictArgs a, int units, int esize) {
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= (int64_t)a.B * a.Hk * a.budget) return;
    const int r = (int)(row % a.budget);
    const int64_t bk = row / a.budget;
    const int b = (int)(bk / a.Hk), h = (int)(bk % a.Hk);
    const int j = a.idx[row];
    if (j < 0) return;
    if (lane == 0) a.acc_out[row] = a.acc[bk * a.T + j];
    const char *ks = static_cast<const char *>(a.K.ptr) + (b * a.K.sb + h * a.K.sh + (int64_t)j * a.K.st) * esize;
    const char *vs = static_cast<const char *>(a.V.ptr) + (b * a.V.sb + h * a.V.sh + (int64_t)j * a.V.st) * esize;
    char *kd = static_cast<char *>(a.Kout.ptr) + (b * a.Kout.sb + h * a.Kout.sh + (int64_t)r * a.Kout.st) * esize;
    char *vd = static_cast<char *>(a.Vout.ptr) + (b * a.Vout.sb + h * a.Vout.sh + (int64_t)r * a.Vout.st) * esize;
    for (int u = lane; u < 2 * units; u += 32) {
        const bool v = u >= units;
        const int x = (v ? u - units : u) * 16;
        *reinterpret_cast<uint4 *>((v ? vd : kd) + x) = __ldg(reinterpret_cast<const uint4 *>((v ? vs : ks) + x));
    }
}

__global__ void evict_len_kernel(EvictArgs a) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < a.B) a.len_out[b] = min(min(max(a.cache_len[b], 0), a.T), a.budget);
}

}  // namespace

hils_status launch_cache_evict(hils_dtype dt, int d, const EvictArgs &a, cudaStream_t s) {
    const int64_t heads = (int64_t)a.B * a.Hk, rows = heads * a.budget;
    if (rows > 0) {
        evict_select_kernel<<<(unsigned)heads, kThr, 0, s>>>(a);
        const int esize = dt == HILS_BF16 ? 2 : 4;
        evict_gather_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, d * esize / 16, esize);
    }
    if (a.B > 0) evict_len_kernel<<<(a.B + 255) / 256, 256, 0, s>>>(a);
    return record_cuda_error(cudaGetLastError());
}

}  // namespace hils
