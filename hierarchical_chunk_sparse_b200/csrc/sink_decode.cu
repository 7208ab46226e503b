// One query per sequence over the visible slots of its cache (formulas in sink_common.cuh):
// the slots are cut into splits, one CTA each, whose partial results meet in the combine.
#include "sink_common.cuh"

namespace hils {
namespace {

constexpr int kThr = 128, kWarps = kThr / 32;

template <typename T, int D>
__global__ void __launch_bounds__(kThr) sink_decode_kernel(SinkDecodeArgs a) {
    constexpr int kE = D / 32;  // elements of a row per lane
    const int Hk = a.H / a.G;
    const int split = blockIdx.x % a.splits, bk = blockIdx.x / a.splits;
    const int b = bk / Hk, hk = bk % Hk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    int sinks, lo;
    sink_visible(n, a.W, a.A, &sinks, &lo);
    const int nvis = sinks + n - lo;
    const int v0 = (int)((int64_t)nvis * split / a.splits), v1 = (int)((int64_t)nvis * (split + 1) / a.splits);
    __shared__ float sm[kWarps][kMaxGroupHeads], sl[kWarps][kMaxGroupHeads], so[kWarps][kMaxGroupHeads][D];
    float q[kMaxGroupHeads][kE], o[kMaxGroupHeads][kE], m[kMaxGroupHeads], l[kMaxGroupHeads];
    const float scale2 = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int g = 0; g < kMaxGroupHeads; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
        const T *qp = static_cast<const T *>(a.Q.ptr) + b * a.Q.sb + (hk * a.G + min(g, a.G - 1)) * a.Q.sh;
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
            const float2 v = load2(qp + lane * kE + e);
            q[g][e] = v.x;
            q[g][e + 1] = v.y;
            o[g][e] = o[g][e + 1] = 0.f;
        }
    }
    for (int v = v0 + warp; v < v1; v += kWarps) {
        const int64_t j = v < sinks ? v : lo + (v - sinks);
        const T *kp = static_cast<const T *>(a.K.ptr) + b * a.K.sb + hk * a.K.sh + j * a.K.st + lane * kE;
        const T *vp = static_cast<const T *>(a.V.ptr) + b * a.V.sb + hk * a.V.sh + j * a.V.st + lane * kE;
        float k[kE], u[kE];
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
            const float2 x = load2(kp + e), y = load2(vp + e);
            k[e] = x.x;
            k[e + 1] = x.y;
            u[e] = y.x;
            u[e + 1] = y.y;
        }
#pragma unroll
        for (int g = 0; g < kMaxGroupHeads; ++g) {
            if (g >= a.G) break;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(q[g][e], k[e], s);
            s = warp_sum(s) * scale2;
            if (a.logits && lane == 0) a.logits[((int64_t)b * a.H + hk * a.G + g) * a.logit_stride + v] = s;
            const float mt = fmaxf(m[g], s);
            const float ref = mt == -INFINITY ? 0.f : mt;
            const float f = exp2f(m[g] - ref), p = exp2f(s - ref);
            m[g] = mt;
            l[g] = fmaf(l[g], f, p);
#pragma unroll
            for (int e = 0; e < kE; ++e) o[g][e] = fmaf(o[g][e], f, p * u[e]);
        }
    }
#pragma unroll
    for (int g = 0; g < kMaxGroupHeads; ++g) {
        if (lane == 0) {
            sm[warp][g] = m[g];
            sl[warp][g] = l[g];
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) so[warp][g][lane * kE + e] = o[g][e];
    }
    __syncthreads();
    for (int g = warp; g < a.G; g += kWarps) {
        float mx = -INFINITY, z = 0.f;
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w][g]);
        float r[kE] = {};
        for (int w = 0; w < kWarps; ++w) {
            const float f = sl[w][g] > 0.f ? exp2f(sm[w][g] - mx) : 0.f;
            z = fmaf(f, sl[w][g], z);
#pragma unroll
            for (int e = 0; e < kE; ++e) r[e] = fmaf(f, so[w][g][lane * kE + e], r[e]);
        }
        const int64_t slot = ((int64_t)b * a.H + hk * a.G + g) * a.slots + a.slot0 + split;
        const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) a.part_o[slot * D + lane * kE + e] = r[e] * inv;
        if (lane == 0) a.part_lse[slot] = z > 0.f ? (mx + log2f(z)) * 0.6931471805599453f : -INFINITY;
    }
}

// One warp per row: weights exp(lse_s - max) over the row's slots, in slot order.
template <typename T, int D>
__global__ void __launch_bounds__(256) sink_combine_kernel(SinkCombineArgs a) {
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
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

__global__ void __launch_bounds__(256) sink_acc_kernel(SinkDecodeArgs a, const float *lse, const float *acc, float *acc_out,
                                                       int chunks) {
    const int Hk = a.H / a.G;
    const int bk = blockIdx.x / chunks, b = bk / Hk, hk = bk % Hk;
    const int v = (blockIdx.x % chunks) * 256 + threadIdx.x;
    const int n = min(max(__ldg(a.cache_len + b), 0), a.T);
    int sinks, lo;
    sink_visible(n, a.W, a.A, &sinks, &lo);
    if (v >= sinks + n - lo) return;
    const int64_t j = v < sinks ? v : lo + (v - sinks);
    const int64_t row = (int64_t)b * a.H + hk * a.G;
    float w = 0.f;
    for (int g = 0; g < a.G; ++g)
        w += exp2f(a.logits[(row + g) * a.logit_stride + v] - __ldg(lse + row + g) * 1.4426950408889634f);
    const int64_t at = ((int64_t)b * Hk + hk) * a.T + j;
    acc_out[at] = acc[at] + w;
}

}  // namespace

// Splits of a sequence's visible slots: about two CTAs per SM, 64 slots or more each.
int sink_decode_splits(int B, int Hk, int64_t keys, int sms) {
    const int64_t rows = (int64_t)B * Hk;
    int64_t s = rows > 0 ? (2 * (int64_t)sms + rows - 1) / rows : 1;
    if (s > keys / 64) s = keys / 64;
    return (int)(s < 1 ? 1 : s > 128 ? 128 : s);
}

hils_status launch_sink_decode(hils_dtype dt, int d, const SinkDecodeArgs &a, cudaStream_t s) {
    const int64_t grid = (int64_t)a.B * (a.H / a.G) * a.splits;
    if (grid == 0) return HILS_OK;
    if (grid > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
    if (dt == HILS_BF16) {
        if (d == 64) sink_decode_kernel<bf16, 64><<<(unsigned)grid, kThr, 0, s>>>(a);
        else sink_decode_kernel<bf16, 128><<<(unsigned)grid, kThr, 0, s>>>(a);
    } else {
        if (d == 64) sink_decode_kernel<float, 64><<<(unsigned)grid, kThr, 0, s>>>(a);
        else sink_decode_kernel<float, 128><<<(unsigned)grid, kThr, 0, s>>>(a);
    }
    return record_cuda_error(cudaGetLastError());
}

hils_status launch_sink_combine(hils_dtype dt, int d, const SinkCombineArgs &a, cudaStream_t s) {
    const int64_t grid = (a.rows + 7) / 8;
    if (grid == 0) return HILS_OK;
    if (dt == HILS_BF16) {
        if (d == 64) sink_combine_kernel<bf16, 64><<<(unsigned)grid, 256, 0, s>>>(a);
        else sink_combine_kernel<bf16, 128><<<(unsigned)grid, 256, 0, s>>>(a);
    } else {
        if (d == 64) sink_combine_kernel<float, 64><<<(unsigned)grid, 256, 0, s>>>(a);
        else sink_combine_kernel<float, 128><<<(unsigned)grid, 256, 0, s>>>(a);
    }
    return record_cuda_error(cudaGetLastError());
}

hils_status launch_sink_decode_acc(const SinkDecodeArgs &a, const float *lse, const float *acc, float *acc_out,
                                   cudaStream_t s) {
    const int chunks = (int)((a.logit_stride + 255) / 256);
    const int64_t grid = (int64_t)a.B * (a.H / a.G) * chunks;
    if (grid == 0) return HILS_OK;
    if (grid > 0x7fffffffll) return HILS_ERR_UNSUPPORTED;
    sink_acc_kernel<<<(unsigned)grid, 256, 0, s>>>(a, lse, acc, acc_out, chunks);
    return record_cuda_error(cudaGetLastError());
}

}  // namespace hils
