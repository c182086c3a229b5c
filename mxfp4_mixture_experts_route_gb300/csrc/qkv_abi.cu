// The C ABI of moe_qkv_append: argument checks, then the launch.
// Declaration and contract: include/moe.h.
#include "kv_checks.cuh"

using namespace moe;

extern "C" {

int moe_qkv_append(const moe_kv_shape* shape, const moe_rope* rope, const void* q_in, const void* k_new,
                   const void* v_new, const int32_t* positions, const int64_t* slots, const float* q_norm,
                   const float* k_norm, const float* cos_sin, const float* k_scale, const float* v_scale, void* q,
                   void* k_cache, void* v_cache, void* ws, size_t ws_bytes, void* stream) {
    KvDims d;
    int rc = kv_dims(shape, d);
    if (rc) return rc;
    if (!rope || rope->flags & ~MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
    if (rope->R < 0 || rope->q_in_stride < 0 || !(rope->eps >= 0.0f) || !isfinite(rope->eps)) return MOE_ERR_INVALID_ARG;
    if (rope->R > 0 && rope->max_pos < 1) return MOE_ERR_INVALID_ARG;
    if (rope->R % 16 || rope->R > d.D) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t q_in_stride = rope->q_in_stride ? rope->q_in_stride : (int64_t)d.Hq * d.D;
    if (q_in_stride < (int64_t)d.Hq * d.D || q_in_stride >= (int64_t)1 << 38) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (q_in_stride % 8) return MOE_ERR_ALIGNMENT;
    if (!q_in || !k_new || !v_new || !positions || !slots || !q || !k_cache || !v_cache) return MOE_ERR_INVALID_ARG;
    if ((cos_sin != nullptr) != (rope->R > 0)) return MOE_ERR_INVALID_ARG;
    if (q == q_in && q_in_stride != d.q_stride) return MOE_ERR_INVALID_ARG;
    rc = check_scales(d, k_scale, v_scale);
    if (rc) return rc;
    for (const void* p : {q_in, k_new, v_new, (const void*)positions, (const void*)slots, (const void*)q_norm,
                          (const void*)k_norm, (const void*)cos_sin, (const void*)k_scale, (const void*)v_scale,
                          (const void*)q, (const void*)k_cache, (const void*)v_cache})
        if (!a16(p)) return MOE_ERR_ALIGNMENT;
    rc = check_kv_ws(d, ws, ws_bytes);
    if (!rc) rc = check_device();
    if (rc) return rc;
    const QkvArgs a{q_in, k_new, v_new, positions, slots, q_norm, k_norm, cos_sin, k_scale, v_scale, q, k_cache, v_cache,
                    reinterpret_cast<StatusBlock*>(ws), rope->R, rope->max_pos,
                    (rope->flags & MOE_ROPE_INTERLEAVED) != 0, rope->eps, q_in_stride};
    return cuda_rc(launch_qkv_append(d, a, (cudaStream_t)stream));
}

}  // extern "C"
