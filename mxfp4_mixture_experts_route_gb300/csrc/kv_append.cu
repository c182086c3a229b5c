// The new tokens' K and V rows into the paged cache.
//
//   bf16 cache: cache[slot] = x;   e4m3: code = rn_e4m3(x / scale_h)
//
// Bound: HBM (each row read once, written once) for prompts, latency for a
// step's few rows.  A thread moves 16-byte pieces, blockIdx.y picks K or V.
#include "kv.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int APPEND_THREADS = 256;

// The division by the scale is IEEE's (not a product with the reciprocal), so
// that a code is the one the formula gives; cvt saturates at +-448.
__device__ __forceinline__ uint32_t quant4(uint32_t lo, uint32_t hi, float s) {
    const float a = __fdiv_rn(__uint_as_float(lo << 16), s), b = __fdiv_rn(__uint_as_float(lo & 0xFFFF0000u), s);
    const float c = __fdiv_rn(__uint_as_float(hi << 16), s), e = __fdiv_rn(__uint_as_float(hi & 0xFFFF0000u), s);
    return ptx::cvt_e4m3x2(a, b) | ptx::cvt_e4m3x2(c, e) << 16;
}

template <bool E4M3>
__global__ void __launch_bounds__(APPEND_THREADS) k_kv_append(const KvDims d, const AppendArgs a) {
    constexpr int EL = E4M3 ? 16 : 8;                 // elements a piece
    const int per_head = d.D / EL, per_row = d.Hkv * per_head;
    const bool is_v = blockIdx.y != 0;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? a.v_new : a.k_new);
    uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
    const float* scale = is_v ? a.v_scale : a.k_scale;
    const int64_t n = (int64_t)d.T * per_row;
    KT_MARK(K_KV_APPEND, 0);
    pdl_wait();
    KT_MARK(K_KV_APPEND, 1);
    for (int64_t i = (int64_t)blockIdx.x * APPEND_THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * APPEND_THREADS) {
        const int t = (int)(i / per_row), p = (int)(i - (int64_t)t * per_row);
        const int h = p / per_head, e = (p - h * per_head) * EL;
        const int64_t slot = ld_dep(reinterpret_cast<const long long*>(a.slots) + t);
        if (slot < 0) continue;
        if (slot >= (int64_t)d.n_pages * d.page) {
            latch_status(a.sb, MOE_ERR_BAD_PAGE, (int)(slot / d.page));
            continue;
        }
        const int pg = (int)slot / d.page, o = (int)slot - pg * d.page;
        const int64_t to = pg * d.page_stride + h * d.head_stride + o * d.token_stride + e;
        const uint4* from = reinterpret_cast<const uint4*>(src + t * d.kv_stride + (int64_t)h * d.D + e);
        uint4 x = ld_dep(from);
        if (E4M3) {
            const uint4 y = ld_dep(from + 1);
            const float s = ld_dep(scale + h);
            x = make_uint4(quant4(x.x, x.y, s), quant4(x.z, x.w, s), quant4(y.x, y.y, s), quant4(y.z, y.w, s));
            *reinterpret_cast<uint4*>(dst + to) = x;
        } else {
            *reinterpret_cast<uint4*>(dst + 2 * to) = x;
        }
    }
    KT_MARK(K_KV_APPEND, 2);
}

}  // namespace

cudaError_t launch_kv_append(const KvDims& d, const AppendArgs& a, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_KV_APPEND, st);
    const int64_t n = (int64_t)d.T * d.Hkv * d.D / (d.e4m3 ? 16 : 8);
    const int64_t want = (n + APPEND_THREADS - 1) / APPEND_THREADS, most = 8 * num_sms();
    const dim3 grid((unsigned)(want < most ? want : most), 2);
    const cudaError_t e = d.e4m3 ? launch_pdl(k_kv_append<true>, grid, dim3(APPEND_THREADS), 0, st, d, a)
                                 : launch_pdl(k_kv_append<false>, grid, dim3(APPEND_THREADS), 0, st, d, a);
    timing_end(st);
    return e;
}

}  // namespace moe
