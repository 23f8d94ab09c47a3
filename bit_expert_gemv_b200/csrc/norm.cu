// RMSNorm with the residual's addition:  h = x + r,  y = h / sqrt(mean h^2 + eps) * w.
//
// One pass: a row's h stays in registers between the sum of squares and the
// outputs, so every input is read once and every output written once; the
// kernel is bound by HBM (by latency for a few tokens).  h enters the norm in
// fp32, before its rounding to the residual's type.  y leaves in 16 or 32 bits
// and / or as MXFP8 (e4m3 codes, one power-of-two scale per 32 columns).
#include "mx.cuh"

namespace gale {
namespace {

struct NormArgs {
    const void* x;
    const void* r;       // or null
    const void* w;       // or null: unit weight
    void* h;             // or null
    void* y;             // or null
    uint8_t* q;          // MXFP8 codes, or null
    uint8_t* s;
    int64_t ldx, ldr, ldh, ldy;
    int64_t tokens;
    int64_t nt;          // padded columns / 128
    int cols, span;      // span: columns written (the padded ones with MXFP8)
    int dt, wt, yt;
    int vw;              // w may be read 16 bytes at a time
    float eps;
};

__device__ __forceinline__ void mx8_store_vec(const NormArgs& a, int64_t row, int c, const float (&v)[8], bool live) {
    // four neighbouring threads hold a block; all 32 lanes take part
    uint32_t m = amax8_bits(v);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = mx8_scale_byte(m);
    const float inv = mx_inverse(b);
    uint32_t word = b << (8 * ((threadIdx.x >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (!live) return;
    uint2 q = make_uint2(0u, 0u);
    if (b != 255u)
        q = make_uint2(mx8_codes(v[0], v[1], v[2], v[3], inv), mx8_codes(v[4], v[5], v[6], v[7], inv));
    *reinterpret_cast<uint2*>(a.q + row * a.nt * kMxTile + c) = q;
    if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(a.s + mx_scale_at(row, c / kMxBlock, a.nt)) = word;
}

__device__ __forceinline__ void mx8_store_scalar(const NormArgs& a, int64_t row, int c, float v, bool live) {
    // a warp's 32 consecutive columns are one block
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
    if (!live) return;
    const uint32_t b = mx8_scale_byte(m);
    const float f = b == 255u ? 0.f : v * mx_inverse(b);
    a.q[row * a.nt * kMxTile + c] = uint8_t(__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3));
    if ((threadIdx.x & 31) == 0) a.s[mx_scale_at(row, c / kMxBlock, a.nt)] = uint8_t(b);
}

// A row per group of `threads` threads (a warp, or the CTA), CH * 8 columns per
// thread.  VEC: thread t holds columns (j * threads + t) * 8 + i, read and
// written 16 bytes at a time; otherwise (j * 8 + i) * threads + t, single
// elements, for rows that are not 16-byte aligned.
template <bool VEC, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_kernel(NormArgs a) {
    __shared__ float part[32];
    const int lane = threadIdx.x & 31;
    const int threads = WARP ? 32 : blockDim.x;
    const int t = WARP ? lane : threadIdx.x;
    const int64_t row = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.tokens) return;      // whole warps (a CTA always has its row)
    float h[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if constexpr (VEC) {
            const int c = (j * threads + t) * 8;
            load8(a.x, a.dt, row * a.ldx + c, a.cols - c, true, h[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = (j * 8 + i) * threads + t;
                h[j][i] = c < a.cols ? load_as_f32(a.x, a.dt, row * a.ldx + c) : 0.f;
            }
        }
    }
    if (a.r) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float r[8];
            if constexpr (VEC) {
                const int c = (j * threads + t) * 8;
                load8(a.r, a.dt, row * a.ldr + c, a.cols - c, true, r);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = (j * 8 + i) * threads + t;
                    r[i] = c < a.cols ? load_as_f32(a.r, a.dt, row * a.ldr + c) : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] += r[i];
        }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    ss = warp_sum(ss);
    if constexpr (!WARP) {
        if (lane == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = warp_sum(lane < (threads >> 5) ? part[lane] : 0.f);
    }
    const float inv = 1.0f / sqrtf(ss / float(a.cols) + a.eps);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if constexpr (VEC) {
            const int c = (j * threads + t) * 8;
            const int n = a.cols - c;
            if (a.h && n > 0) store8(a.h, a.dt, row * a.ldh + c, n, true, h[j]);
            float w[8];
            if (a.w) load8(a.w, a.wt, c, n, a.vw, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = h[j][i] * inv;
                h[j][i] = i < n ? (a.w ? y * w[i] : y) : 0.f;
            }
            if (a.y && n > 0) store8(a.y, a.yt, row * a.ldy + c, n, true, h[j]);
            if (a.q) mx8_store_vec(a, row, c, h[j], c < a.span);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = (j * 8 + i) * threads + t;
                const bool in = c < a.cols;
                if (a.h && in) store_rn(a.h, a.dt, row * a.ldh + c, h[j][i]);
                float y = in ? h[j][i] * inv : 0.f;
                if (a.w && in) y *= load_as_f32(a.w, a.wt, c);
                if (a.y && in) store_rn(a.y, a.yt, row * a.ldy + c, y);
                if (a.q) mx8_store_scalar(a, row, c, y, c < a.span);
            }
        }
    }
}

constexpr int kNormMaxCols = 32768;

template <bool VEC>
int launch_norm(const NormArgs& a, cudaStream_t st) {
    const int chunks = (a.span + 7) / 8;             // eight-column chunks of a row
    if (chunks <= 128) {                             // up to 1024 columns: a warp per row, eight rows per CTA
        const unsigned grid = unsigned((a.tokens + 7) / 8);
        if (chunks <= 32) rmsnorm_kernel<VEC, 1, true><<<grid, 256, 0, st>>>(a);
        else if (chunks <= 64) rmsnorm_kernel<VEC, 2, true><<<grid, 256, 0, st>>>(a);
        else rmsnorm_kernel<VEC, 4, true><<<grid, 256, 0, st>>>(a);
    } else {                                         // a CTA per row
        const unsigned grid = unsigned(a.tokens);
        const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
        const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
        if (ch == 1) rmsnorm_kernel<VEC, 1, false><<<grid, threads, 0, st>>>(a);
        else if (ch == 2) rmsnorm_kernel<VEC, 2, false><<<grid, threads, 0, st>>>(a);
        else rmsnorm_kernel<VEC, 4, false><<<grid, threads, 0, st>>>(a);
    }
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}

}  // namespace
}  // namespace gale

extern "C" int gale_rmsnorm(const void* x, const void* residual, int dtype, int64_t ldx, int64_t ldr,
                            const void* weight, int w_dtype, float eps, int64_t tokens, int64_t cols, void* sum_out,
                            int64_t ldsum, void* y, int y_dtype, int64_t ldy, void* mx8, void* stream) {
    using namespace gale;
    if (!valid_dtype(dtype) || (weight && !valid_dtype(w_dtype)) || (y && !valid_dtype(y_dtype))) return GALE_ERR_ARG;
    if (tokens < 0 || tokens > INT32_MAX || cols < 1 || !(eps >= 0.f)) return GALE_ERR_ARG;
    if (!y && !mx8 && !sum_out) return GALE_ERR_ARG;
    if (cols > kNormMaxCols) return GALE_ERR_UNSUPPORTED;
    if (tokens == 0) return GALE_OK;
    if (!x || ldx < cols || (residual && ldr < cols) || (sum_out && ldsum < cols) || (y && ldy < cols))
        return GALE_ERR_ARG;
    const size_t es = dtype_size(dtype);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(sum_out, es) ||
        (weight && !aligned(weight, dtype_size(w_dtype))) || (y && !aligned(y, dtype_size(y_dtype))) ||
        !aligned(mx8, 256))
        return GALE_ERR_ALIGN;
    NormArgs a{};
    a.x = x;
    a.r = residual;
    a.w = weight;
    a.h = sum_out;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldsum;
    a.ldy = ldy;
    a.tokens = tokens;
    a.cols = int(cols);
    a.span = int(cols);
    a.dt = dtype;
    a.wt = w_dtype;
    a.yt = y_dtype;
    a.eps = eps;
    if (mx8) {
        gale_mx_layout_t L;
        if (gale_mx8_layout(tokens, cols, &L) != GALE_OK) return GALE_ERR_ARG;
        a.q = static_cast<uint8_t*>(mx8);
        a.s = a.q + L.s_offset;
        a.nt = L.cols_padded / kMxTile;
        a.span = int(L.cols_padded);
    }
    const bool vec = rows_vec(x, dtype, ldx) && (!residual || rows_vec(residual, dtype, ldr)) &&
                     (!sum_out || rows_vec(sum_out, dtype, ldsum)) && (!y || rows_vec(y, y_dtype, ldy));
    a.vw = weight && aligned(weight, 16);
    return vec ? launch_norm<true>(a, as_stream(stream)) : launch_norm<false>(a, as_stream(stream));
}
