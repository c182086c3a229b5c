// The e4m3 codes of the paged cache (kv_append.cu, qkv_append.cu).
#pragma once

#include "kv.cuh"
#include "tc_ptx.cuh"

#include <math_constants.h>

namespace moe {

// The code of x / s is that of the division's correctly rounded quotient, not of
// a product with the reciprocal, so that a code is the one the formula gives.  The
// product with the approximate reciprocal (off by 2^-23) and a factor next to one (two roundings, 2^-24 each)
// is off by less than 2^-21 of itself, so where a little more and a little
// less than it give the same code, that is the quotient's code too (rounding
// is monotonic); only next to a tie between two codes the division is made.
struct KvScale {
    float s, lo, hi;
    __device__ __forceinline__ explicit KvScale(float v) : s(v) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
        // (a scale whose reciprocal is not an ordinary number: always by division)
        const bool fine = v > 0x1p-120f && v < 0x1p120f;
        lo = fine ? r * (1.f - 0x1p-21f) : 1.f;
        hi = fine ? r * (1.f + 0x1p-21f) : CUDART_NAN_F;
    }
};
// the codes of four values, saturating at +-448
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float e) {
    return ptx::cvt_e4m3x2(a, b) | ptx::cvt_e4m3x2(c, e) << 16;
}
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float e, const KvScale& k) {
    const uint32_t u = kv_codes4(a * k.lo, b * k.lo, c * k.lo, e * k.lo);
    const uint32_t v = kv_codes4(a * k.hi, b * k.hi, c * k.hi, e * k.hi);
    if (u == v) return u;
    return kv_codes4(__fdiv_rn(a, k.s), __fdiv_rn(b, k.s), __fdiv_rn(c, k.s), __fdiv_rn(e, k.s));
}

}  // namespace moe
