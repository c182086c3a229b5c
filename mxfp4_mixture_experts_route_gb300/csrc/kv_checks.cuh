// Argument checks that the cache calls' C entries share (kv_abi.cu, qkv_abi.cu).
#pragma once

#include "kv.cuh"

#include <math.h>

namespace moe {

static inline bool a16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Checks a shape and fills in the packed strides.
static inline int kv_dims(const moe_kv_shape* s, KvDims& d) {
    if (!s) return MOE_ERR_INVALID_ARG;
    if (s->flags & ~MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
    if (s->B < 1 || s->T < 1 || s->Hq < 1 || s->Hkv < 1 || s->page < 1 || s->n_pages < 1 || s->max_pages < 1 ||
        s->W < 0)
        return MOE_ERR_INVALID_ARG;
    if (!(s->scale > 0.0f) || !isfinite(s->scale)) return MOE_ERR_INVALID_ARG;
    if (s->page_stride < 0 || s->head_stride < 0 || s->token_stride < 0 || s->q_stride < 0 || s->kv_stride < 0)
        return MOE_ERR_INVALID_ARG;
    if (s->D != 64 && s->D != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (s->B > KV_MAX_B || s->T > (1 << 20) || s->Hq > 4096 || s->Hq % s->Hkv || s->Hq / s->Hkv > 128)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (s->page % 8 || s->page > 1024 || s->W > KV_MAX_W) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)s->n_pages * s->page >= (int64_t)1 << 31 || (int64_t)s->max_pages * s->page > (int64_t)1 << 30)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    d = KvDims{s->B, s->T, s->Hq, s->Hkv, s->D, s->page, s->n_pages, s->max_pages, s->W, (s->flags & MOE_KV_E4M3) != 0,
               s->scale, s->page_stride, s->head_stride, s->token_stride, s->q_stride, s->kv_stride};
    // packed: [n_pages][Hkv][page][D]
    if (!d.token_stride) d.token_stride = d.D;
    if (!d.head_stride) d.head_stride = (int64_t)d.page * d.D;
    if (!d.page_stride) d.page_stride = (int64_t)d.Hkv * d.page * d.D;
    if (!d.q_stride) d.q_stride = (int64_t)d.Hq * d.D;
    if (!d.kv_stride) d.kv_stride = (int64_t)d.Hkv * d.D;
    if (d.token_stride < d.D || d.head_stride < d.D || d.page_stride < d.D || d.q_stride < (int64_t)d.Hq * d.D ||
        d.kv_stride < (int64_t)d.Hkv * d.D)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t cache_el = d.e4m3 ? 16 : 8;   // elements of 16 bytes
    if (d.token_stride % cache_el || d.head_stride % cache_el || d.page_stride % cache_el || d.q_stride % 8 ||
        d.kv_stride % 8)
        return MOE_ERR_ALIGNMENT;
    // tensor-map strides are below 2^40 bytes
    const int64_t most = ((int64_t)1 << 39) / 2;
    if (d.token_stride >= most || d.head_stride >= most || d.page_stride >= most || d.q_stride >= most ||
        d.kv_stride >= most)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

static inline int check_kv_ws(const KvDims& d, void* ws, size_t ws_bytes) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if ((uintptr_t)ws & 255) return MOE_ERR_ALIGNMENT;
    if (ws_bytes < tree_attn_ws_bytes(d)) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

// the scale vectors: given with an e4m3 cache, absent otherwise
static inline int check_scales(const KvDims& d, const float* ks, const float* vs) {
    return d.e4m3 == (ks != nullptr) && d.e4m3 == (vs != nullptr) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

}  // namespace moe
