// The new tokens' K and V rows into the paged cache.
//
//   bf16 cache: cache[slot] = x;   e4m3: code = rn_e4m3(x / scale_h)
//
// Bound: HBM (each row read once, written once) for prompts, latency for a
// step's few rows.  A thread moves 16-byte pieces, blockIdx.y picks K or V.
#include "kv_codes.cuh"

namespace moe {
namespace {

constexpr int APPEND_THREADS = 256;

__device__ __forceinline__ uint32_t quant4(uint32_t lo, uint32_t hi, const KvScale& k) {
    return kv_codes4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
                     __uint_as_float(hi & 0xFFFF0000u), k);
}

// U pieces a thread at once, their loads under way together.  Measured: 16,411 rows of
// 8 heads x 128 to e4m3 21.0 us with two, 21.9 with one, more with four or eight (0.70 of
// the measured copy bandwidth; what is left is the codes' arithmetic, 73% of the issue
// slots; 26.4 us when every code was a division); 8 rows to bf16 1.3 us with one, 1.7 with two.
template <bool E4M3, int U>
__global__ void __launch_bounds__(APPEND_THREADS) k_kv_append(const KvDims d, const AppendArgs a) {
    constexpr int EL = E4M3 ? 16 : 8;                 // elements a piece
    const int per_head = d.D / EL, per_row = d.Hkv * per_head;
    const bool is_v = blockIdx.y != 0;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? a.v_new : a.k_new);
    uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
    const float* scale = is_v ? a.v_scale : a.k_scale;
    // pieces first, first + step, ... as (row, piece in the row), counted on without divisions
    const int step = gridDim.x * APPEND_THREADS, step_t = step / per_row, step_p = step - step_t * per_row;
    const int first = blockIdx.x * APPEND_THREADS + threadIdx.x;
    int t = first / per_row, p = first - t * per_row;
    KT_MARK(K_KV_APPEND, 0);
    pdl_wait();
    KT_MARK(K_KV_APPEND, 1);
    while (t < d.T) {
        uint4 x[U], y[U];
        float s[U];
        int64_t to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u] = -1;
            if (t < d.T) {
                const int h = p / per_head, e = (p - h * per_head) * EL;
                const int64_t slot = ld_dep(reinterpret_cast<const long long*>(a.slots) + t);
                const uint4* from = reinterpret_cast<const uint4*>(src + t * d.kv_stride + (int64_t)h * d.D + e);
                x[u] = ld_dep(from);
                if (E4M3) {
                    y[u] = ld_dep(from + 1);
                    s[u] = ld_dep(scale + h);
                }
                if (slot >= (int64_t)d.n_pages * d.page) {
                    latch_status(a.sb, MOE_ERR_BAD_PAGE, (int)(slot / d.page));
                } else if (slot >= 0) {
                    const int pg = (int)slot / d.page, o = (int)slot - pg * d.page;
                    to[u] = pg * d.page_stride + h * d.head_stride + o * d.token_stride + e;
                }
            }
            t += step_t;
            p += step_p;
            if (p >= per_row) {
                p -= per_row;
                ++t;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (to[u] < 0) continue;
            if (E4M3) {
                const KvScale k(s[u]);
                *reinterpret_cast<uint4*>(dst + to[u]) = make_uint4(quant4(x[u].x, x[u].y, k), quant4(x[u].z, x[u].w, k),
                                                                    quant4(y[u].x, y[u].y, k), quant4(y[u].z, y[u].w, k));
            } else {
                *reinterpret_cast<uint4*>(dst + 2 * to[u]) = x[u];
            }
        }
    }
    KT_MARK(K_KV_APPEND, 2);
}

}  // namespace

cudaError_t launch_kv_append(const KvDims& d, const AppendArgs& a, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_KV_APPEND, st);
    const int64_t n = (int64_t)d.T * d.Hkv * d.D / (d.e4m3 ? 16 : 8);
    // one piece a thread while that is at most one round of the SMs' threads
    // (shortest path), two otherwise; every piece has its thread: no loop to run dry
    // (but for the largest calls, whose pieces' numbers pass 31 bits)
    const int64_t one = (n + APPEND_THREADS - 1) / APPEND_THREADS;
    const bool few = one <= 8 * num_sms();
    const int64_t want = few ? one : (one + 1) / 2, most = ((int64_t)1 << 30) / APPEND_THREADS;
    const dim3 grid((unsigned)(want < most ? want : most), 2), block(APPEND_THREADS);
    cudaError_t e;
    if (d.e4m3)
        e = few ? launch_pdl(k_kv_append<true, 1>, grid, block, 0, st, d, a)
                : launch_pdl(k_kv_append<true, 2>, grid, block, 0, st, d, a);
    else
        e = few ? launch_pdl(k_kv_append<false, 1>, grid, block, 0, st, d, a)
                : launch_pdl(k_kv_append<false, 2>, grid, block, 0, st, d, a);
    timing_end(st);
    return e;
}

}  // namespace moe
