// Rows to MXFP4 and back.
//
//   scale byte b = max(E - 2, 0), E the biased exponent of the block's largest magnitude
//   code = rn_e2m1(x 2^(127 - b)), saturated at 6;   y = e2m1(code) 2^(b - 127)
//
// The scale is a power of two whose reciprocal is one too, so the product with it is exact
// and the code is the nearest of x / scale.  A block with E = 255 (NaN, infinity)
// has byte 255 and codes 0.
//
// Bound: HBM.  A thread takes pieces of 16 bytes of the wide side (8 elements of 16 bits,
// 4 of 32), neighbouring threads neighbouring pieces, so that every access of a warp is to
// consecutive bytes; a block's 4 or 8 threads find its maximum by shuffles.
#include "mx.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int MXQ_THREADS = 256;

template <int DT>
constexpr int piece_elems() { return DT == MOE_F32 ? 4 : 8; }

// a piece as fp32
template <int DT>
__device__ __forceinline__ void widen(const uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (DT == MOE_F32) {
            f[j] = __uint_as_float(w[j]);
        } else if (DT == MOE_BF16) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        } else {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        }
    }
}

// fp32 values -> a piece (round to nearest even)
template <int DT>
__device__ __forceinline__ uint4 narrow(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (DT == MOE_F32) {
            w[j] = __float_as_uint(f[j]);
        } else if (DT == MOE_BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __half2 p = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// four fp32 -> four e2m1 codes, the first in the lowest bits (round to nearest even, saturating)
__device__ __forceinline__ uint32_t e2m1x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b8 lo, hi, z;\n\t.reg .b16 p, q;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\t"
        "mov.b16 p, {lo, hi};\n\t"
        "mov.b16 q, 0;\n\t"
        "mov.b32 %0, {p, q};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// two e2m1 codes (bits 0..3 and 4..7 of v) -> two fp32 (exact)
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t v) {
    uint32_t h;
    asm("{\n\t.reg .b8 c, z;\n\t.reg .b16 s;\n\t"
        "cvt.u16.u32 s, %1;\n\t"
        "mov.b16 {c, z}, s;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(h)
        : "r"(v));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^(b - 127); 255: NaN
__device__ __forceinline__ float e8m0(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// Piece `i` of all rows stands at row i / per_row; PACKED rows need no row number.
template <bool PACKED>
__device__ __forceinline__ int64_t wide_offset(int64_t i, int per_row, int64_t stride, int elems) {
    if (PACKED) return i * elems;
    const int64_t row = (i >> 32) ? i / per_row : (int64_t)((uint32_t)i / (uint32_t)per_row);
    return row * stride + (i - row * per_row) * elems;
}

template <int DT, bool PACKED, int U>
__global__ void __launch_bounds__(MXQ_THREADS) k_mx_quantize(const uint8_t* x, int64_t stride, int64_t pieces, int per_row,
                                                             uint8_t* codes, uint8_t* scales) {
    constexpr int EL = piece_elems<DT>(), SIZE = 16 / EL, LANES = 32 / EL;   // lanes of a block of 32
    const int64_t first = ((int64_t)blockIdx.x * U) * MXQ_THREADS + threadIdx.x;
    KT_MARK(K_MX_QUANT, 0);
    pdl_wait();
    KT_MARK(K_MX_QUANT, 1);
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * MXQ_THREADS;
        v[u] = make_uint4(0, 0, 0, 0);
        if (i < pieces)
            v[u] = ld_dep(reinterpret_cast<const uint4*>(x + SIZE * wide_offset<PACKED>(i, per_row, stride, EL)));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * MXQ_THREADS;
        float f[EL];
        widen<DT>(v[u], f);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < EL; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < LANES; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t e = top >> 23;
        const bool bad = e == 255;
        const uint32_t b = bad ? 255u : e > 2 ? e - 2 : 0u;
        const float inv = __uint_as_float((254u - (bad ? 0u : b)) << 23);      // 2^(127 - b)
        uint32_t c = e2m1x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        if (EL == 8) c |= e2m1x4(f[EL - 4] * inv, f[EL - 3] * inv, f[EL - 2] * inv, f[EL - 1] * inv) << 16;
        if (bad) c = 0;
        if (i >= pieces) continue;
        if (EL == 8)
            reinterpret_cast<uint32_t*>(codes)[i] = c;
        else
            reinterpret_cast<uint16_t*>(codes)[i] = (uint16_t)c;
        if (threadIdx.x % LANES == 0) scales[i / LANES] = (uint8_t)b;
    }
    KT_MARK(K_MX_QUANT, 2);
}

template <int DT, bool PACKED, int U>
__global__ void __launch_bounds__(MXQ_THREADS) k_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t pieces,
                                                               int per_row, uint8_t* y, int64_t stride) {
    constexpr int EL = piece_elems<DT>(), SIZE = 16 / EL, LANES = 32 / EL;
    const int64_t first = ((int64_t)blockIdx.x * U) * MXQ_THREADS + threadIdx.x;
    KT_MARK(K_MX_DEQUANT, 0);
    pdl_wait();
    KT_MARK(K_MX_DEQUANT, 1);
    uint32_t c[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * MXQ_THREADS;
        c[u] = b[u] = 0;
        if (i < pieces) {
            c[u] = EL == 8 ? ld_dep(reinterpret_cast<const uint32_t*>(codes) + i)
                           : (uint32_t)ld_dep(reinterpret_cast<const uint16_t*>(codes) + i);
            b[u] = ld_dep(scales + i / LANES);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * MXQ_THREADS;
        if (i >= pieces) break;
        const float s = e8m0(b[u]);
        float f[EL];
#pragma unroll
        for (int j = 0; j < EL / 2; ++j) {
            const float2 p = e2m1x2_to_f32(c[u] >> (8 * j) & 0xFF);
            f[2 * j] = p.x * s;
            f[2 * j + 1] = p.y * s;
        }
        *reinterpret_cast<uint4*>(y + SIZE * wide_offset<PACKED>(i, per_row, stride, EL)) = narrow<DT>(f);
    }
    KT_MARK(K_MX_DEQUANT, 2);
}

// One launch over all pieces: with few, one a thread (shortest path); else U, their loads under way together.
template <int DT, bool PACKED, bool BACK>
cudaError_t launch_pieces(int64_t rows, int K, uint8_t* wide, int64_t stride, uint8_t* codes, uint8_t* scales,
                          cudaStream_t st) {
    constexpr int U = 4;
    const int per_row = K / piece_elems<DT>();
    const int64_t pieces = rows * per_row;
    const bool few = pieces <= (int64_t)num_sms() * 2048;
    const int64_t per = (int64_t)MXQ_THREADS * (few ? 1 : U), blocks = (pieces + per - 1) / per;
    const dim3 grid((unsigned)blocks), block(MXQ_THREADS);
    if (BACK)
        return few ? launch_pdl(k_mx_dequantize<DT, PACKED, 1>, grid, block, 0, st, codes, scales, pieces, per_row, wide, stride)
                   : launch_pdl(k_mx_dequantize<DT, PACKED, U>, grid, block, 0, st, codes, scales, pieces, per_row, wide, stride);
    return few ? launch_pdl(k_mx_quantize<DT, PACKED, 1>, grid, block, 0, st, wide, stride, pieces, per_row, codes, scales)
               : launch_pdl(k_mx_quantize<DT, PACKED, U>, grid, block, 0, st, wide, stride, pieces, per_row, codes, scales);
}

template <bool BACK>
cudaError_t launch_rows(int64_t rows, int K, int dtype, uint8_t* wide, int64_t stride, uint8_t* codes, uint8_t* scales,
                        cudaStream_t st) {
    // (at most 2^30 threads' pieces a launch, so that the grid fits)
    const int64_t most = ((int64_t)1 << 38) / K;
    for (int64_t at = 0; at < rows; at += most) {
        const int64_t n = rows - at < most ? rows - at : most;
        uint8_t *w = wide + at * stride * (dtype == MOE_F32 ? 4 : 2), *c = codes + at * (K / 2), *s = scales + at * (K / 32);
        const bool packed = stride == K;
        cudaError_t e;
        if (dtype == MOE_BF16)
            e = packed ? launch_pieces<MOE_BF16, true, BACK>(n, K, w, stride, c, s, st)
                       : launch_pieces<MOE_BF16, false, BACK>(n, K, w, stride, c, s, st);
        else if (dtype == MOE_F16)
            e = packed ? launch_pieces<MOE_F16, true, BACK>(n, K, w, stride, c, s, st)
                       : launch_pieces<MOE_F16, false, BACK>(n, K, w, stride, c, s, st);
        else
            e = packed ? launch_pieces<MOE_F32, true, BACK>(n, K, w, stride, c, s, st)
                       : launch_pieces<MOE_F32, false, BACK>(n, K, w, stride, c, s, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_mx_quantize(int64_t rows, int K, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                               uint8_t* scales, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_MX_QUANT, st);
    const cudaError_t e = launch_rows<false>(rows, K, dtype, (uint8_t*)const_cast<void*>(x), x_stride, codes, scales, st);
    timing_end(st);
    return e;
}

cudaError_t launch_mx_dequantize(int64_t rows, int K, int dtype, const uint8_t* codes, const uint8_t* scales, void* y,
                                 int64_t y_stride, cudaStream_t st) {
    KT_BIND();
    timing_begin(K_MX_DEQUANT, st);
    const cudaError_t e = launch_rows<true>(rows, K, dtype, (uint8_t*)y, y_stride, const_cast<uint8_t*>(codes),
                                            const_cast<uint8_t*>(scales), st);
    timing_end(st);
    return e;
}

}  // namespace moe
