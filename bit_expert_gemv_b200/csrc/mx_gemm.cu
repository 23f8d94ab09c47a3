// Product of MXFP4 weights with MXFP8 tokens: y[t][r] = sum_c W[r][c] X[t][c].
#include "mx.cuh"

namespace gale {
namespace {

// One output per thread, blocks of 32 columns at a time: the products of a
// block summed in fp32, then the two scales.
__global__ void __launch_bounds__(256) mx_gemm_simple_kernel(const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws,
                                                             const uint8_t* __restrict__ x,
                                                             const uint8_t* __restrict__ xs, int64_t rows,
                                                             int64_t tokens, int64_t nt, void* __restrict__ y, int dtype,
                                                             int64_t ldy) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * tokens) return;
    const int64_t r = i % rows, t = i / rows;
    float acc = 0.f;
    for (int64_t b = 0; b < nt * 4; ++b) {
        const uint4 q = *reinterpret_cast<const uint4*>(w + ((r / kMxTile) * nt + b / 4) * kMx4TileBytes +
                                                        (r % kMxTile) * (kMxTile / 2) + b % 4 * 16);
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
        const uint8_t* xr = x + t * nt * kMxTile + b * kMxBlock;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 wv = __half22float2(
                    __half2(__nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(qw[k] >> (8 * n)), __NV_E2M1)));
                const float2 xv = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
                    *reinterpret_cast<const __nv_fp8x2_storage_t*>(xr + k * 8 + n * 2), __NV_E4M3)));
                sum = fmaf(wv.x, xv.x, sum);
                sum = fmaf(wv.y, xv.y, sum);
            }
        }
        acc = fmaf(sum, mx_scale_value(ws[mx_scale_at(r, b, nt)]) * mx_scale_value(xs[mx_scale_at(t, b, nt)]), acc);
    }
    store_rn(y, dtype, t * ldy + r, acc);
}

}  // namespace
}  // namespace gale

extern "C" size_t gale_mx_gemm_workspace_size(int64_t rows, int64_t cols, int64_t tokens) {
    gale_mx_layout_t L;
    if (gale_mx4_layout(rows, cols, &L) != GALE_OK || gale_mx8_layout(tokens, cols, &L) != GALE_OK) return 0;
    return 256;   // the status word
}

extern "C" int gale_mx_gemm(const void* w4, int64_t rows, int64_t cols, const void* x8, int64_t tokens, void* y,
                            int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    using namespace gale;
    gale_mx_layout_t W, X;
    if (!valid_dtype(y_dtype) || gale_mx4_layout(rows, cols, &W) != GALE_OK || tokens < 0) return GALE_ERR_ARG;
    if (tokens == 0) return GALE_OK;
    if (gale_mx8_layout(tokens, cols, &X) != GALE_OK || !w4 || !x8 || !y || ldy < rows) return GALE_ERR_ARG;
    if (!aligned(w4, 256) || !aligned(x8, 256) || !aligned(y, dtype_size(y_dtype))) return GALE_ERR_ALIGN;
    if (!ws || ws_bytes < gale_mx_gemm_workspace_size(rows, cols, tokens)) return GALE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GALE_ERR_ALIGN;
    const uint8_t* w = static_cast<const uint8_t*>(w4);
    const uint8_t* x = static_cast<const uint8_t*>(x8);
    mx_gemm_simple_kernel<<<unsigned((rows * tokens + 255) / 256), 256, 0, as_stream(stream)>>>(
        w, w + W.s_offset, x, x + X.s_offset, rows, tokens, W.cols_padded / kMxTile, y, y_dtype, ldy);
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}
