// The C ABI of the dense MXFP4 calls: argument checks, then the launches.
// Declarations and contracts: include/moe.h.
#include "mx.cuh"

namespace moe {
namespace {

bool a16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// What quantise and dequantise share: sizes, the wide side's type and stride.
int check_rows(int64_t rows, int32_t K, int dtype, const void* wide, int64_t& stride, const void* codes,
               const void* scales) {
    if (rows < 1 || K < 1 || stride < 0) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_BF16 && dtype != MOE_F16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (K % 32 || K > (1 << 20) || rows >= ((int64_t)1 << 44) / K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!stride) stride = K;
    if (stride < K || stride >= (int64_t)1 << 40 || (rows > 1 && stride >= ((int64_t)1 << 60) / rows))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!wide || !codes || !scales) return MOE_ERR_INVALID_ARG;
    if (stride % (dtype == MOE_F32 ? 4 : 8) || !a16(wide) || !a16(codes) || !a16(scales)) return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

int mx_dims(const moe_mx_shape* s, MxDims& d) {
    if (!s || s->flags & ~MOE_MX_X_MXFP4) return MOE_ERR_INVALID_ARG;
    if (s->T < 1 || s->N < 1 || s->K < 1 || s->x_stride < 0 || s->out_stride < 0) return MOE_ERR_INVALID_ARG;
    if (s->T > (1 << 20) || s->N > (1 << 20) || s->N % 8 || s->K % 128 || s->K > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
    d = MxDims{s->T, s->N, s->K, (s->flags & MOE_MX_X_MXFP4) != 0, s->x_stride ? s->x_stride : s->K,
               s->out_stride ? s->out_stride : s->N, 0, 0, 0};
    const int64_t most = (int64_t)1 << 38;
    if (d.x_stride < d.K || d.out_stride < d.N || d.x_stride >= most || d.out_stride >= most)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (d.x_mx && d.x_stride != d.K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (d.x_stride % 8 || d.out_stride % 8) return MOE_ERR_ALIGNMENT;
    mx_cut(d);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_mx_quantize(int64_t rows, int32_t K, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                    uint8_t* scales, void* stream) {
    int rc = check_rows(rows, K, dtype, x, x_stride, codes, scales);
    if (!rc) rc = check_device();
    if (rc) return rc;
    return cuda_rc(launch_mx_quantize(rows, K, dtype, x, x_stride, codes, scales, (cudaStream_t)stream));
}

int moe_mx_dequantize(int64_t rows, int32_t K, int dtype, const uint8_t* codes, const uint8_t* scales, void* y,
                      int64_t y_stride, void* stream) {
    int rc = check_rows(rows, K, dtype, y, y_stride, codes, scales);
    if (!rc) rc = check_device();
    if (rc) return rc;
    return cuda_rc(launch_mx_dequantize(rows, K, dtype, codes, scales, y, y_stride, (cudaStream_t)stream));
}

int moe_mx_workspace_bytes(const moe_mx_shape* shape, size_t* bytes) {
    MxDims d;
    const int rc = mx_dims(shape, d);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = mx_linear_ws_bytes(d);
    return MOE_OK;
}

int moe_mx_linear_cut(const moe_mx_shape* shape, int32_t* ctas, int32_t* tokens, int32_t* parts) {
    MxDims d;
    const int rc = mx_dims(shape, d);
    if (rc) return rc;
    if (ctas) *ctas = d.cg;
    if (tokens) *tokens = d.nt;
    if (parts) *parts = d.split;
    return MOE_OK;
}

int moe_mx_linear(const moe_mx_shape* shape, const void* x, const uint8_t* xs, const uint8_t* w,
                  const uint8_t* w_scales, void* out, void* ws, size_t ws_bytes, void* stream) {
    MxDims d;
    int rc = mx_dims(shape, d);
    if (rc) return rc;
    if (!x || !w || !w_scales || !out || !ws) return MOE_ERR_INVALID_ARG;
    if ((xs != nullptr) != d.x_mx) return MOE_ERR_INVALID_ARG;
    if (!a16(x) || !a16(xs) || ((uintptr_t)w & 31) || !a16(w_scales) || !a16(out) || ((uintptr_t)ws & 255))
        return MOE_ERR_ALIGNMENT;
    if (ws_bytes < mx_linear_ws_bytes(d)) return MOE_ERR_WORKSPACE;
    rc = check_device();
    if (rc) return rc;
    const MxArgs a{x, xs, w, w_scales, out, (char*)ws};
    return cuda_rc(launch_mx_linear(d, a, (cudaStream_t)stream));
}

}  // extern "C"
