// Argument checks shared by the C-ABI entry points: parameters, strided views, dense
// arrays and workspaces. Host only; nothing here launches or touches device memory.
#pragma once
#include <math.h>

#include "hils_internal.cuh"

#define HILS_TRY(expr)                 \
    do {                               \
        const int _rc = (expr);        \
        if (_rc != HILS_OK) return _rc; \
    } while (0)

namespace hils {

inline size_t elem_size(hils_dtype dt) { return dt == HILS_BF16 ? 2 : 4; }

// Common parameter checks; fills the effective scale.
inline int check_params(const hils_params *p, float *scale) {
    if (!p) return HILS_ERR_INVALID_ARG;
    if (p->B < 0 || p->H < 0 || p->K < 0 || p->W < 0) return HILS_ERR_INVALID_ARG;
    if (p->dtype != HILS_F32 && p->dtype != HILS_BF16) return HILS_ERR_UNSUPPORTED;
    if (p->d != 64 && p->d != 128) return HILS_ERR_UNSUPPORTED;
    if (p->S != kChunk) return HILS_ERR_UNSUPPORTED;
    if (p->K > 32) return HILS_ERR_UNSUPPORTED;
    if (p->flags & ~(uint32_t)(HILS_FLAG_EXCLUDE_WINDOW_CHUNKS | HILS_FLAG_DIAG_EXPIRE_WAITS))
        return HILS_ERR_UNSUPPORTED;
    if (!isfinite(p->scale)) return HILS_ERR_INVALID_ARG;
    if (p->H_kv < 0 || (p->H_kv > 0 && p->H % p->H_kv != 0)) return HILS_ERR_INVALID_ARG;
    if (p->H_kv > 0 && p->H / p->H_kv > kMaxGroupHeads) return HILS_ERR_UNSUPPORTED;
    *scale = p->scale != 0.f ? p->scale : (float)(1.0 / sqrt((double)p->d));
    return HILS_OK;
}

// Query heads per key-value head (parameters already checked).
inline int groups(const hils_params *p) { return p->H_kv > 0 && p->H > 0 ? p->H / p->H_kv : 1; }

inline bool aligned16(const void *ptr) { return ((uintptr_t)ptr & 15u) == 0; }

// A [B, H, T, d] view with T rows used: non-null when it holds elements, 16-byte
// aligned base and strides.
inline int check_view(const void *ptr, int64_t sb, int64_t sh, int64_t st, int64_t rows, const hils_params *p) {
    if ((int64_t)p->B * p->H * rows == 0) return HILS_OK;
    if (!ptr) return HILS_ERR_INVALID_ARG;
    const int64_t es = (int64_t)elem_size(p->dtype);
    if (!aligned16(ptr)) return HILS_ERR_ALIGNMENT;
    if ((sb * es) % 16 || (sh * es) % 16 || (st * es) % 16) return HILS_ERR_ALIGNMENT;
    return HILS_OK;
}

inline int check_array(const void *ptr, int64_t count) {
    if (count > 0 && !ptr) return HILS_ERR_INVALID_ARG;
    if (ptr && ((uintptr_t)ptr & 3u)) return HILS_ERR_ALIGNMENT;
    return HILS_OK;
}

inline int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return HILS_OK;
    if (!ws || have < need) return HILS_ERR_WORKSPACE;
    if (!aligned16(ws)) return HILS_ERR_ALIGNMENT;
    return HILS_OK;
}

}  // namespace hils
