// Attention of a tree of drafted tokens (or a chain) over the paged cache.
//
// One CTA a row and query head: its warps take keys in turn, each with a
// running maximum m and sum l of exp2 (the softmax in one pass:
// o <- o 2^(m - m') + 2^(x - m') v), joined through shared memory.
#include "kv.cuh"
#include "tc_ptx.cuh"

#include <math_constants.h>

namespace moe {
namespace {

constexpr int SIMPLE_WARPS = 8;

__device__ __forceinline__ bool sees(const KvDims& d, const AttnArgs& a, int row, int i, int j) {
    if (d.W == 0) return j <= i;
    return (ld_dep(a.mask + (int64_t)row * d.W + (j >> 5)) >> (j & 31)) & 1;
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_kv(const void* base, int64_t off, float* x) {
    constexpr int V = D / 32;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (E4M3) {
            float lo, hi;
            ptx::e4m3x2_to_f32(reinterpret_cast<const uint8_t*>(base)[off + i], lo, hi);
            x[i] = lo;
        } else {
            x[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[off + i] << 16);
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * SIMPLE_WARPS) k_tree_attn_rows(const KvDims d, const AttnArgs a) {
    constexpr int V = D / 32;
    __shared__ float sh_m[SIMPLE_WARPS], sh_l[SIMPLE_WARPS], sh_o[SIMPLE_WARPS][D];
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    StatusBlock* sb = reinterpret_cast<StatusBlock*>(a.ws);
    pdl_wait();
    // the request: the last b with row_start[b] <= row
    int lo = 0, hi = d.B;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (ld_dep(a.row_start + m) <= row) lo = m; else hi = m;
    }
    const KvReq r = kv_request(d, a.ctx_len, a.row_start, lo);
    if (!r.ok) {
        if (threadIdx.x == 0) latch_status(sb, MOE_ERR_BAD_LENGTHS, lo);
        return;
    }
    const int i = row - r.r0;
    if (i < 0 || i >= r.n) return;
    const int kvh = h / (d.Hq / d.Hkv);
    const float c = d.scale * 1.44269504f * (E4M3 ? ld_dep(a.k_scale + kvh) : 1.f);
    float q[V], o[V], m = -CUDART_INF_F, l = 0.f;
    load_kv<D, false>(a.q, row * d.q_stride + (int64_t)h * D + lane * V, q);
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    for (int key = warp; key < r.c + r.n; key += SIMPLE_WARPS) {
        if (key >= r.c && !sees(d, a, row, i, key - r.c)) continue;
        const int pg = ld_dep(a.block_table + (int64_t)lo * d.max_pages + key / d.page);
        if (pg < 0 || pg >= d.n_pages) {
            if (lane == 0) latch_status(sb, MOE_ERR_BAD_PAGE, pg);
            continue;
        }
        const int64_t off = pg * d.page_stride + kvh * d.head_stride + (key % d.page) * d.token_stride + lane * V;
        float k[V], x = 0.f;
        load_kv<D, E4M3>(a.k_cache, off, k);
#pragma unroll
        for (int v = 0; v < V; ++v) x += q[v] * k[v];
#pragma unroll
        for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        x *= c;
        const float m2 = fmaxf(m, x), base = m2 == -CUDART_INF_F ? 0.f : m2;
        const float f = exp2f(m - base), p = exp2f(x - base);
        load_kv<D, E4M3>(a.v_cache, off, k);
        l = l * f + p;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = o[v] * f + p * k[v];
        m = m2;
    }
    if (lane == 0) {
        sh_m[warp] = m;
        sh_l[warp] = l;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sh_o[warp][lane * V + v] = o[v];
    __syncthreads();
    float top = -CUDART_INF_F;
    for (int w = 0; w < SIMPLE_WARPS; ++w) top = fmaxf(top, sh_m[w]);
    const float base = top == -CUDART_INF_F ? 0.f : top;
    float total = 0.f;
    for (int w = 0; w < SIMPLE_WARPS; ++w) total += sh_l[w] * exp2f(sh_m[w] - base);
    for (int e = threadIdx.x; e < D; e += 32 * SIMPLE_WARPS) {
        float s = 0.f;
        for (int w = 0; w < SIMPLE_WARPS; ++w) s += sh_o[w][e] * exp2f(sh_m[w] - base);
        s = total == 0.f ? 0.f : s / total;
        if (E4M3) s *= ld_dep(a.v_scale + kvh);
        reinterpret_cast<__nv_bfloat16*>(a.out)[((int64_t)row * d.Hq + h) * D + e] = __float2bfloat16_rn(s);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(int64_t)row * d.Hq + h] = total == 0.f ? -CUDART_INF_F : (base + log2f(total)) * 0.69314718f;
}

}  // namespace

size_t tree_attn_ws_bytes(const KvDims&) { return 8192; }

cudaError_t launch_tree_attn(const KvDims& d, const AttnArgs& a, cudaStream_t st) {
    timing_begin(K_TREE_ATTN, st);
    const dim3 grid(d.T, d.Hq), block(32 * SIMPLE_WARPS);
    cudaError_t e;
    if (d.D == 128)
        e = d.e4m3 ? launch_pdl(k_tree_attn_rows<128, true>, grid, block, 0, st, d, a)
                   : launch_pdl(k_tree_attn_rows<128, false>, grid, block, 0, st, d, a);
    else
        e = d.e4m3 ? launch_pdl(k_tree_attn_rows<64, true>, grid, block, 0, st, d, a)
                   : launch_pdl(k_tree_attn_rows<64, false>, grid, block, 0, st, d, a);
    timing_end(st);
    return e;
}

}  // namespace moe
