// Dense MXFP4 (mx_abi.cu, mx_quant.cu, mx_linear.cu); the contracts are in include/moe.h.
#pragma once

#include "moe_internal.cuh"

namespace moe {

cudaError_t launch_mx_quantize(int64_t rows, int K, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                               uint8_t* scales, cudaStream_t st);
cudaError_t launch_mx_dequantize(int64_t rows, int K, int dtype, const uint8_t* codes, const uint8_t* scales, void* y,
                                 int64_t y_stride, cudaStream_t st);

// The product's shape with its strides filled in (elements), and how it is cut (mx_cut, of the rest).
struct MxDims {
    int T, N, K;
    bool x_mx;
    int64_t x_stride, out_stride;
    int cg, nt, split;   // CTAs and tokens a tile; CTAs of a cluster that share a tile's K
};
void mx_cut(MxDims& d);
struct MxArgs {
    const void* x;
    const uint8_t *xs, *w, *w_scales;
    void* out;
    char* ws;
};
size_t mx_linear_ws_bytes(const MxDims& d);
cudaError_t launch_mx_linear(const MxDims& d, const MxArgs& a, cudaStream_t st);

// host checks and error reporting of the library (moe_abi.cu)
int check_device();
int cuda_rc(cudaError_t e);

}  // namespace moe
