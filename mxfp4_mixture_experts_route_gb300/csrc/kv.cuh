// Shared by the cache-side calls (kv_abi.cu, kv_plan.cu, kv_append.cu,
// tree_attn.cu); the contracts are in include/moe.h.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int KV_MAX_B = 4096;      // requests a call
constexpr int KV_MAX_W = 32;        // mask words a row

// The shape with its strides filled in (elements).
struct KvDims {
    int B, T, Hq, Hkv, D, page, n_pages, max_pages, W;
    bool e4m3;
    float scale;
    int64_t page_stride, head_stride, token_stride, q_stride, kv_stride;
};

// One request as the attention reads it: c cached tokens, n new ones, whose
// first row is r0.  Lengths come from device memory, so they are checked here
// before anything is indexed with them; a request that does not fit has no rows.
struct KvReq {
    int c, n, r0;
    bool ok;
};
__device__ __forceinline__ KvReq kv_request(const KvDims& d, const int32_t* ctx_len, const int32_t* row_start, int b) {
    KvReq r;
    r.c = ld_dep(ctx_len + b);
    r.r0 = ld_dep(row_start + b);
    const int e = ld_dep(row_start + b + 1);
    r.ok = r.c >= 0 && r.r0 >= 0 && e >= r.r0 && e <= d.T && (int64_t)r.c + (e - r.r0) <= (int64_t)d.max_pages * d.page &&
           (d.W == 0 || e - r.r0 <= 32 * d.W);
    r.n = r.ok ? e - r.r0 : 0;
    return r;
}

// host checks and error reporting of the library (moe_abi.cu)
int check_device();
int cuda_rc(cudaError_t e);

struct PlanArgs {
    const int32_t *ctx_len, *n_new, *parents, *free_pages;
    int n_free;
    int32_t *block_table, *row_start;
    int64_t* slots;
    int32_t* positions;
    uint32_t* mask;
    int32_t* used;
    StatusBlock* sb;
};
cudaError_t launch_kv_plan(const KvDims& d, const PlanArgs& a, cudaStream_t st);

struct AppendArgs {
    const void *k_new, *v_new;
    const int64_t* slots;
    const float *k_scale, *v_scale;
    void *k_cache, *v_cache;
    StatusBlock* sb;
};
cudaError_t launch_kv_append(const KvDims& d, const AppendArgs& a, cudaStream_t st);

struct QkvArgs {
    const void *q_in, *k_new, *v_new;
    const int32_t* positions;
    const int64_t* slots;
    const float *q_norm, *k_norm, *cos_sin, *k_scale, *v_scale;
    void *q, *k_cache, *v_cache;
    StatusBlock* sb;
    int R, max_pos;
    bool interleaved;
    float eps;
    int64_t q_in_stride;
};
cudaError_t launch_qkv_append(const KvDims& d, const QkvArgs& a, cudaStream_t st);

struct AttnArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *block_table, *ctx_len, *row_start;
    const uint32_t* mask;
    const float *k_scale, *v_scale;
    void* out;
    float* lse;
    char* ws;
};
size_t tree_attn_ws_bytes(const KvDims& d);
cudaError_t launch_tree_attn(const KvDims& d, const AttnArgs& a, cudaStream_t st);

}  // namespace moe
