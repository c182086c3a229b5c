// Norms and rotation of query and key heads, and the append of K and V.
//
//   y = x rsqrt(mean x^2 + eps) w;   z_i = y_i cos_i - y_j sin_i,  z_j = y_j cos_i + y_i sin_i
//
// Bound: HBM (each row read once, written once) for prompts, latency for a
// step's few rows.  D / 8 lanes hold a head, 8 elements each, and take
// some heads of one token: the angles and weights are the same for all of
// them, so a lane keeps w cos and w' sin of its elements in registers
// (z = r (x (w cos) + x' (w' sin)), x' the pair's other element, r the head's rsqrt) and a
// head costs it one load, one sum over the lanes, four shuffles and one store.
#include "kv_codes.cuh"

namespace moe {
namespace {

constexpr int QKV_THREADS = 128;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// four and eight fp32 of a table or weight row: in shared memory, or as an earlier kernel may have written it
template <bool SHARED>
__device__ __forceinline__ float4 load4(const float* p) {
    return SHARED ? *reinterpret_cast<const float4*>(p) : ld_dep(reinterpret_cast<const float4*>(p));
}
template <bool SHARED>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = load4<SHARED>(p), b = load4<SHARED>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// LPH lanes a head; a warp takes CH heads of one kind (query, key or value) of one token, 32 / LPH side by side, U
// of each group of lanes loaded at a time.  With most heads a warp is a block of its own, a token's
// next to one another: a block of all of them holds its place until the last one (often one of query heads beside
// two of few key and value heads) is done, and 64 registers let 32 blocks run at once (16,411 rows of 56 + 2 x 8 heads:
// to bf16 102 us, in blocks of four warps 112, with 71 registers 116; a token's warps far apart in the grid 117).
constexpr bool lone(int heads) { return heads == 32; }
template <int LPH, int CH, int U, bool E4M3, bool INTER>
__global__ void __launch_bounds__(lone(CH) ? 32 : QKV_THREADS, lone(CH) ? 32 : 1) k_qkv_append(const KvDims d, const QkvArgs a) {
    constexpr int D = LPH * 8, SIDE = 32 / LPH;
    constexpr bool STAGED = CH == 8 || CH == 16;
    const int qc = (d.Hq + CH - 1) / CH, kc = (d.Hkv + CH - 1) / CH, chunks = qc + 2 * kc;
    const int t = lone(CH) ? blockIdx.x / chunks : blockIdx.x;
    int c = lone(CH) ? blockIdx.x - t * chunks : blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;
    const int p = threadIdx.x % LPH;                 // the lane's piece of the head
    KT_MARK(K_QKV_APPEND, 0);
    pdl_wait();
    KT_MARK(K_QKV_APPEND, 1);
    const int pos = ld_dep(a.positions + t);
    const int64_t slot = ld_dep(reinterpret_cast<const long long*>(a.slots) + t);
    const int what = c < qc ? 0 : c < qc + kc ? 1 : 2;   // q, K, V: the same for the warp
    bool live = c < chunks;
    c -= what == 0 ? 0 : what == 1 ? qc : qc + kc;
    const int end = min(what == 0 ? d.Hq : d.Hkv, (c + 1) * CH);   // the warp's heads end here
    const int h0 = c * CH + threadIdx.x % 32 / LPH;                // this lane's: h0, h0 + SIDE, ...
    if (pos < 0) return;
    if (a.R > 0 && pos >= a.max_pos) {
        latch_status(a.sb, MOE_ERR_BAD_LENGTHS, t);
        return;
    }
    int64_t to = 0;
    if (what != 0 && live) {
        if (slot >= (int64_t)d.n_pages * d.page) latch_status(a.sb, MOE_ERR_BAD_PAGE, (int)(slot / d.page));
        live = slot >= 0 && slot < (int64_t)d.n_pages * d.page;
        if (live) {
            const int pg = (int)slot / d.page, o = (int)slot - pg * d.page;
            to = pg * d.page_stride + o * d.token_stride + 8 * p;
        }
    }
    const uint16_t* src = reinterpret_cast<const uint16_t*>(what == 0 ? a.q_in : what == 1 ? a.k_new : a.v_new) +
                          t * (what == 0 ? a.q_in_stride : d.kv_stride) + 8 * p;
    const float* scale = what == 1 ? a.k_scale : a.v_scale;
    uint4 x[U], ahead[U];
    float sc[U], sc_ahead[U];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int head = h + i * SIDE;
            if (head < end) {
                ahead[i] = ld_dep(reinterpret_cast<const uint4*>(src + (int64_t)head * D));
                if (E4M3 && what != 0) sc_ahead[i] = ld_dep(scale + head);
            } else {
                ahead[i] = make_uint4(0, 0, 0, 0);
                sc_ahead[i] = 1.f;
            }
        }
    };
    if (live) load(h0);

    // the token's angles and the weights: by way of shared memory, once a block instead of once a warp, where a warp has
    // some heads (500 rows of 56 + 2 x 8: 5.1 us, without 7.3; with fewer heads its latency counts, with more
    // it gains nothing: 16,411 rows in blocks of four warps 122 us, without 116)
    const float *w = what == 0 ? a.q_norm : a.k_norm, *row = a.cos_sin + (int64_t)pos * a.R;
    if constexpr (STAGED) {
        __shared__ float4 stage[3][D / 4];
        for (int i = threadIdx.x; i < 3 * D / 4; i += blockDim.x) {
            const int n = i / (D / 4), j = i % (D / 4);
            const float* from = n == 0 ? a.q_norm : n == 1 ? a.k_norm : row;
            if (n < 2 ? from != nullptr : 4 * j < a.R) stage[n][j] = ld_dep(reinterpret_cast<const float4*>(from) + j);
        }
        __syncthreads();
        if (w) w = reinterpret_cast<const float*>(stage[what == 0 ? 0 : 1]);
        row = reinterpret_cast<const float*>(stage[2]);
    }
    if (!live) return;
    // own[j] = w cos, other[j] = +- w' sin of the lane's element j; partner: the piece that holds x'
    float own[8], other[8];
    const bool turned = what != 2 && 8 * p < a.R;
    const int half = a.R / 16;                       // pieces of half the rotated part
    const int partner = INTER || !turned ? p : p < half ? p + half : p - half;
#pragma unroll
    for (int j = 0; j < 8; ++j) own[j] = 1.f, other[j] = 0.f;
    if (what != 2 && w) load8<STAGED>(w + 8 * p, own);
    if (turned) {
        float cs[8], sn[8], wp[8];
        if (INTER) {
            const float4 u = load4<STAGED>(row + 4 * p);
            const float4 v = load4<STAGED>(row + a.R / 2 + 4 * p);
            cs[0] = cs[1] = u.x, cs[2] = cs[3] = u.y, cs[4] = cs[5] = u.z, cs[6] = cs[7] = u.w;
            sn[1] = v.x, sn[3] = v.y, sn[5] = v.z, sn[7] = v.w;
#pragma unroll
            for (int j = 0; j < 8; j += 2) sn[j] = -sn[j + 1], wp[j] = own[j + 1], wp[j + 1] = own[j];
        } else {
            const int i = 8 * (p < half ? p : p - half);
            load8<STAGED>(row + i, cs);
            load8<STAGED>(row + a.R / 2 + i, sn);
#pragma unroll
            for (int j = 0; j < 8; ++j) wp[j] = 1.f, sn[j] = p < half ? -sn[j] : sn[j];
            if (w) load8<STAGED>(w + 8 * partner, wp);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) other[j] = wp[j] * sn[j], own[j] *= cs[j];
    }
    const bool norm = what != 2 && w;
    // (the same number of rounds for the warp's lanes, which exchange elements)
#pragma unroll 1
    for (int hb = h0; hb - h0 < end - c * CH; hb += U * SIDE) {
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = ahead[i], sc[i] = sc_ahead[i];
        if (CH > U * SIDE) load(hb + U * SIDE);      // the next heads' loads under way meanwhile
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = hb + i * SIDE;
            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[2 * j] = lo_f(v[j]), f[2 * j + 1] = hi_f(v[j]);
            float r = 1.f;
            if (norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
                for (int o = LPH / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrtf(ss * (1.f / D) + a.eps);
            }
            if (what != 2) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t o = INTER ? __byte_perm(v[j], 0, 0x1032) : __shfl_sync(0xffffffffu, v[j], partner, LPH);
                    // (no product with the other element where nothing turns: it may be an infinity)
                    float a0 = f[2 * j] * own[2 * j], a1 = f[2 * j + 1] * own[2 * j + 1];
                    if (turned) a0 = fmaf(lo_f(o), other[2 * j], a0), a1 = fmaf(hi_f(o), other[2 * j + 1], a1);
                    f[2 * j] = a0 * r, f[2 * j + 1] = a1 * r;
                }
            }
            if (h >= end) continue;
            if (what == 0 || !E4M3) {
                uint16_t* dst = what == 0 ? reinterpret_cast<uint16_t*>(a.q) + t * d.q_stride + (int64_t)h * D + 8 * p
                                          : reinterpret_cast<uint16_t*>(what == 1 ? a.k_cache : a.v_cache) + to + h * d.head_stride;
                *reinterpret_cast<uint4*>(dst) = make_uint4(ptx::cvt_bf16x2(f[0], f[1]), ptx::cvt_bf16x2(f[2], f[3]),
                                                            ptx::cvt_bf16x2(f[4], f[5]), ptx::cvt_bf16x2(f[6], f[7]));
            } else {
                const KvScale k(sc[i]);
                uint8_t* dst = reinterpret_cast<uint8_t*>(what == 1 ? a.k_cache : a.v_cache) + to + h * d.head_stride;
                *reinterpret_cast<uint2*>(dst) = make_uint2(kv_codes4(f[0], f[1], f[2], f[3], k), kv_codes4(f[4], f[5], f[6], f[7], k));
            }
        }
    }
    KT_MARK(K_QKV_APPEND, 2);
}

template <int LPH, int CH, int U>
cudaError_t launch_heads(const KvDims& d, const QkvArgs& a, cudaStream_t st) {
    // a token's warps in equal blocks, or a block each
    const int chunks = (d.Hq + CH - 1) / CH + 2 * ((d.Hkv + CH - 1) / CH);
    const int ny = (chunks * 32 + QKV_THREADS - 1) / QKV_THREADS;
    const dim3 grid = lone(CH) ? dim3((unsigned)d.T * chunks) : dim3(d.T, ny), block(lone(CH) ? 32 : (chunks + ny - 1) / ny * 32);
    if (d.e4m3)
        return a.interleaved ? launch_pdl(k_qkv_append<LPH, CH, U, true, true>, grid, block, 0, st, d, a)
                             : launch_pdl(k_qkv_append<LPH, CH, U, true, false>, grid, block, 0, st, d, a);
    return a.interleaved ? launch_pdl(k_qkv_append<LPH, CH, U, false, true>, grid, block, 0, st, d, a)
                         : launch_pdl(k_qkv_append<LPH, CH, U, false, false>, grid, block, 0, st, d, a);
}

// The heads of a warp: two to four while an SM has few warps (short chains), more where the angles and
// weights that every warp needs come to count (rows of 56 + 2 x 8 heads to bf16: 32 rows 2.8 us with two, 3.0 with 8; 64 rows 4.1 and
// 3.3; 200 rows 3.6 with 8, 4.2 with 16; 500 rows 6.7 and 5.1; 1000 rows 9.7 with 16, 12.2 with 32; 3000 rows 25.0 and 24.6; of
// 32 + 2 x 4 heads to e4m3: 3000 rows 21.7 and 19.0).
template <int LPH>
cudaError_t launch_lph(const KvDims& d, const QkvArgs& a, cudaStream_t st) {
    constexpr int SIDE = 32 / LPH;
    const int64_t heads = (int64_t)d.T * (d.Hq + 2 * d.Hkv), sms = num_sms();
    if (heads <= sms * 10 * SIDE) return launch_heads<LPH, SIDE, 1>(d, a, st);
    if (heads <= sms * 128) return launch_heads<LPH, 8, 2>(d, a, st);
    if (heads <= sms * 768) return launch_heads<LPH, 16, 2>(d, a, st);
    return launch_heads<LPH, 32, 2>(d, a, st);
}

}  // namespace

cudaError_t launch_qkv_append(const KvDims& d, const QkvArgs& a, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_QKV_APPEND, st);
    const cudaError_t e = d.D == 128 ? launch_lph<16>(d, a, st) : launch_lph<8>(d, a, st);
    timing_end(st);
    return e;
}

}  // namespace moe
