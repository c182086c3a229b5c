// The C ABI of the cache-side calls: argument checks, then the launches.
// Declarations and contracts: include/moe.h.
#include "kv_checks.cuh"

using namespace moe;

extern "C" {

int moe_kv_workspace_bytes(const moe_kv_shape* shape, size_t* bytes) {
    KvDims d;
    const int rc = kv_dims(shape, d);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = tree_attn_ws_bytes(d);
    return MOE_OK;
}

int moe_kv_plan(const moe_kv_shape* shape, const int32_t* ctx_len, const int32_t* n_new, const int32_t* parents,
                const int32_t* free_pages, int32_t n_free, int32_t* block_table, int32_t* row_start, int64_t* slots,
                int32_t* positions, uint32_t* mask, int32_t* used, void* ws, size_t ws_bytes, void* stream) {
    KvDims d;
    int rc = kv_dims(shape, d);
    if (rc) return rc;
    if (!ctx_len || !n_new || !block_table || !row_start || !slots || !positions || !used) return MOE_ERR_INVALID_ARG;
    if (n_free < 0 || (n_free > 0 && !free_pages)) return MOE_ERR_INVALID_ARG;
    if ((parents != nullptr) != (d.W > 0) || (mask != nullptr) != (d.W > 0)) return MOE_ERR_INVALID_ARG;
    if (!a16(ctx_len) || !a16(n_new) || (parents && !a16(parents)) || (free_pages && !a16(free_pages)) ||
        !a16(block_table) || !a16(row_start) || !a16(slots) || !a16(positions) || (mask && !a16(mask)) || !a16(used))
        return MOE_ERR_ALIGNMENT;
    rc = check_kv_ws(d, ws, ws_bytes);
    if (!rc) rc = check_device();
    if (rc) return rc;
    const PlanArgs a{ctx_len, n_new, parents, free_pages, n_free, block_table, row_start,
                     slots,   positions, mask, used, reinterpret_cast<StatusBlock*>(ws)};
    return cuda_rc(launch_kv_plan(d, a, (cudaStream_t)stream));
}

int moe_kv_append(const moe_kv_shape* shape, const void* k_new, const void* v_new, const int64_t* slots,
                  const float* k_scale, const float* v_scale, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                  void* stream) {
    KvDims d;
    int rc = kv_dims(shape, d);
    if (rc) return rc;
    if (!k_new || !v_new || !slots || !k_cache || !v_cache) return MOE_ERR_INVALID_ARG;
    rc = check_scales(d, k_scale, v_scale);
    if (rc) return rc;
    if (!a16(k_new) || !a16(v_new) || !a16(slots) || !a16(k_cache) || !a16(v_cache) || (k_scale && !a16(k_scale)) ||
        (v_scale && !a16(v_scale)))
        return MOE_ERR_ALIGNMENT;
    rc = check_kv_ws(d, ws, ws_bytes);
    if (!rc) rc = check_device();
    if (rc) return rc;
    const AppendArgs a{k_new, v_new, slots, k_scale, v_scale, k_cache, v_cache, reinterpret_cast<StatusBlock*>(ws)};
    return cuda_rc(launch_kv_append(d, a, (cudaStream_t)stream));
}

int moe_tree_attention(const moe_kv_shape* shape, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* ctx_len, const int32_t* row_start,
                       const uint32_t* mask, const float* k_scale, const float* v_scale, void* out, float* lse,
                       void* ws, size_t ws_bytes, void* stream) {
    KvDims d;
    int rc = kv_dims(shape, d);
    if (rc) return rc;
    if (!q || !k_cache || !v_cache || !block_table || !ctx_len || !row_start || !out) return MOE_ERR_INVALID_ARG;
    if ((mask != nullptr) != (d.W > 0)) return MOE_ERR_INVALID_ARG;
    rc = check_scales(d, k_scale, v_scale);
    if (rc) return rc;
    if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(block_table) || !a16(ctx_len) || !a16(row_start) ||
        (mask && !a16(mask)) || (k_scale && !a16(k_scale)) || (v_scale && !a16(v_scale)) || !a16(out) ||
        (lse && !a16(lse)))
        return MOE_ERR_ALIGNMENT;
    rc = check_kv_ws(d, ws, ws_bytes);
    if (!rc) rc = check_device();
    if (rc) return rc;
    const AttnArgs a{q, k_cache, v_cache, block_table, ctx_len, row_start, mask, k_scale, v_scale, out, lse, (char*)ws};
    const cudaError_t e = launch_tree_attn(d, a, (cudaStream_t)stream);
    // too few SMs for the launch, whose CTAs wait for one another: nothing was enqueued
    if (e == cudaErrorNotSupported || e == cudaErrorCooperativeLaunchTooLarge) {
        cudaGetLastError();
        return MOE_ERR_NO_DEVICE;
    }
    return cuda_rc(e);
}

}  // extern "C"
