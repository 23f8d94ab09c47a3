// Microscaled matrices: layouts, quantisers and the unpacker.
//
// Weights (MXFP4) are stored as 128 x 128 tiles, 8 KB each and contiguous, so
// that a product streams them in order whatever the row length; tokens (MXFP8)
// as plain rows.  The scales of both sit in 512-byte atoms per 128 x 128 tile,
// in the byte order in which the tensor core's scale columns take them.
#include "mx.cuh"
#include "ptx.cuh"

namespace gale {
namespace {

// One 128 x 128 tile per CTA: 16 threads of 8 columns per row, 16 rows a pass,
// all eight passes' loads in flight before the first is used.  Bound by HBM:
// it reads the matrix once and writes 0.53 bytes per element.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void* __restrict__ w, int64_t ld, int64_t rows,
                                                           int64_t cols, uint8_t* __restrict__ q,
                                                           uint32_t* __restrict__ s) {
    const int64_t nt = (cols + kMxTile - 1) / kMxTile;
    const int64_t tile = blockIdx.x;
    const int64_t r0 = tile / nt * kMxTile, c0 = tile % nt * kMxTile;
    const int tr = threadIdx.x >> 4, tc = (threadIdx.x & 15) * 8;
    const int64_t left = cols - c0 - tc;
    const int n = left >= 8 ? 8 : left > 0 ? int(left) : 0;
    Raw8<DT> raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + p * 16 + tr;
        load_raw8<DT, VEC>(w, r * ld + c0 + tc, r < rows ? n : 0, raw[p]);
    }
    uint8_t* qt = q + tile * kMx4TileBytes;
    uint32_t* st = s + tile * (kMxAtomBytes / 4);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = p * 16 + tr;
        float v[8];
        raw8_f32<DT>(raw[p], v);
        uint32_t m = amax8_bits(v);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t b = mx4_scale_byte(m);
        *reinterpret_cast<uint32_t*>(qt + r * (kMxTile / 2) + tc / 2) = b == 255u ? 0u : mx4_codes(v, mx_inverse(b));
        // the row's four scale bytes, one per four threads, as one word
        uint32_t word = b << (8 * ((threadIdx.x >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((threadIdx.x & 15) == 0) st[(r & 31) * 4 + (r >> 5)] = word;
    }
}

// The reverse: 16 threads of 8 columns per row, a tile per CTA.  Rows that are
// not 16-byte aligned leave through shared memory, so that a warp writes
// neighbouring elements (2050 x 1001 in 16 bits: 9.6 us element by element).
template <bool VEC>
__global__ void __launch_bounds__(256) mx4_unpack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                         int64_t rows, int64_t cols, void* __restrict__ out, int dtype,
                                                         int64_t ld) {
    const int64_t nt = (cols + kMxTile - 1) / kMxTile;
    const int64_t tile = blockIdx.x;
    const int64_t r0 = tile / nt * kMxTile, c0 = tile % nt * kMxTile;
    const int tr = threadIdx.x >> 4, tc = (threadIdx.x & 15) * 8;
    const int64_t left = cols - c0 - tc;
    const int n = left >= 8 ? 8 : left > 0 ? int(left) : 0;
    const uint8_t* qt = q + tile * kMx4TileBytes;
    const uint8_t* st = s + tile * kMxAtomBytes;
    uint32_t word[8], sc[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = p * 16 + tr;
        word[p] = __ldg(reinterpret_cast<const uint32_t*>(qt + r * (kMxTile / 2) + tc / 2));
        sc[p] = __ldg(st + (r & 31) * 16 + (r >> 5) * 4 + tc / kMxBlock);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + p * 16 + tr;
        const float f = mx_scale_value(sc[p]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(word[p] >> (8 * i)), __NV_E2M1);
            const float2 g = __half22float2(__half2(h));
            v[2 * i] = g.x * f;
            v[2 * i + 1] = g.y * f;
        }
        if constexpr (VEC) {
            if (r < rows && n > 0) store8(out, dtype, r * ld + c0 + tc, n, true, v);
        } else {
            __shared__ float tile_row[16][kMxTile + 4];
            __syncthreads();      // the last pass has been written
#pragma unroll
            for (int i = 0; i < 8; ++i) tile_row[tr][tc + i] = v[i];
            __syncthreads();
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rr = warp * 2 + i / 4, c = i % 4 * 32 + lane;
                const int64_t row = r0 + p * 16 + rr;
                if (row < rows && c0 + c < cols) store_rn(out, dtype, row * ld + c0 + c, tile_row[rr][c]);
            }
        }
    }
}

// Tokens: 16 rows by 512 columns per CTA, 16 threads of 8 columns per row and 128
// columns; the columns up to the next multiple of 128 are written as zeros with
// scale byte 0.
constexpr int kQ8Rows = 16, kQ8Tiles = 4;
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) mx8_quantize_kernel(const void* __restrict__ x, int64_t ld, int64_t tokens,
                                                           int64_t cols, uint8_t* __restrict__ q,
                                                           uint8_t* __restrict__ s) {
    pdl_launch_dependents();      // a product behind this kernel may set itself up meanwhile
    const int64_t nt = (cols + kMxTile - 1) / kMxTile;
    const int64_t nc = (nt + kQ8Tiles - 1) / kQ8Tiles;
    const int64_t ct = blockIdx.x % nc * kQ8Tiles;
    const int64_t r = blockIdx.x / nc * kQ8Rows + (threadIdx.x >> 4);
    const int tc = (threadIdx.x & 15) * 8;
    Raw8<DT> raw[kQ8Tiles];
#pragma unroll
    for (int p = 0; p < kQ8Tiles; ++p) {
        const int64_t c = (ct + p) * kMxTile + tc, left = cols - c;
        const int n = r >= tokens || left <= 0 ? 0 : left >= 8 ? 8 : int(left);
        load_raw8<DT, VEC>(x, r * ld + c, n, raw[p]);
    }
#pragma unroll
    for (int p = 0; p < kQ8Tiles; ++p) {
        float v[8];
        raw8_f32<DT>(raw[p], v);
        uint32_t m = amax8_bits(v);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t b = mx8_scale_byte(m);
        const float inv = mx_inverse(b);
        uint2 c = make_uint2(0u, 0u);
        if (b != 255u)
            c = make_uint2(mx8_codes(v[0], v[1], v[2], v[3], inv), mx8_codes(v[4], v[5], v[6], v[7], inv));
        uint32_t word = b << (8 * ((threadIdx.x >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (r < tokens && ct + p < nt) {
            *reinterpret_cast<uint2*>(q + (r * nt + ct + p) * kMxTile + tc) = c;
            if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(s + mx_scale_at(r, (ct + p) * 4, nt)) = word;
        }
    }
}

constexpr int64_t kMxMaxRows = int64_t(1) << 24, kMxMaxCols = int64_t(1) << 20;

bool mx_sizes(int64_t rows, int64_t cols) {
    // the tensor-map rows of all tiles stay well below 2^31
    return rows >= 1 && rows <= kMxMaxRows && cols >= 1 && cols <= kMxMaxCols &&
           align_up(rows, kMxTile) / kMxTile * align_up(cols, kMxTile) < (int64_t(1) << 30);
}

}  // namespace
}  // namespace gale

extern "C" int gale_mx4_layout(int64_t rows, int64_t cols, gale_mx_layout_t* out) {
    using namespace gale;
    if (!out || !mx_sizes(rows, cols)) return GALE_ERR_ARG;
    out->rows = rows;
    out->cols = cols;
    out->cols_padded = align_up(cols, kMxTile);
    out->q_offset = 0;
    out->q_bytes = align_up(rows, kMxTile) * out->cols_padded / 2;
    out->s_offset = align_up(out->q_bytes, kAlign);
    out->s_bytes = align_up(rows, kMxTile) * out->cols_padded / kMxBlock;
    out->total = align_up(out->s_offset + out->s_bytes, kAlign);
    return GALE_OK;
}

extern "C" int gale_mx8_layout(int64_t tokens, int64_t cols, gale_mx_layout_t* out) {
    using namespace gale;
    if (!out || !mx_sizes(tokens, cols)) return GALE_ERR_ARG;
    out->rows = tokens;
    out->cols = cols;
    out->cols_padded = align_up(cols, kMxTile);
    out->q_offset = 0;
    out->q_bytes = tokens * out->cols_padded;
    out->s_offset = align_up(out->q_bytes, kAlign);
    out->s_bytes = align_up(tokens, kMxTile) * out->cols_padded / kMxBlock;
    out->total = align_up(out->s_offset + out->s_bytes, kAlign);
    return GALE_OK;
}

extern "C" int gale_mx4_quantize(const void* w, int w_dtype, int64_t ld, int64_t rows, int64_t cols, void* packed,
                                 void* stream) {
    using namespace gale;
    gale_mx_layout_t L;
    if (!w || !packed || !valid_dtype(w_dtype) || gale_mx4_layout(rows, cols, &L) != GALE_OK || ld < cols)
        return GALE_ERR_ARG;
    if (!aligned(packed, 256) || !aligned(w, dtype_size(w_dtype))) return GALE_ERR_ALIGN;
    uint8_t* b = static_cast<uint8_t*>(packed);
    const int64_t tiles = L.q_bytes / kMx4TileBytes;
    by_dtype_vec(w_dtype, rows_vec(w, w_dtype, ld), [&](auto dt, auto vec) {
        mx4_quantize_kernel<decltype(dt)::value, decltype(vec)::value><<<unsigned(tiles), 256, 0, as_stream(stream)>>>(
            w, ld, rows, cols, b, reinterpret_cast<uint32_t*>(b + L.s_offset));
    });
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}

extern "C" int gale_mx4_unpack(const void* packed, int64_t rows, int64_t cols, void* out, int out_dtype, int64_t ld,
                               void* stream) {
    using namespace gale;
    gale_mx_layout_t L;
    if (!out || !packed || !valid_dtype(out_dtype) || gale_mx4_layout(rows, cols, &L) != GALE_OK || ld < cols)
        return GALE_ERR_ARG;
    if (!aligned(packed, 256) || !aligned(out, dtype_size(out_dtype))) return GALE_ERR_ALIGN;
    const uint8_t* b = static_cast<const uint8_t*>(packed);
    const int64_t tiles = L.q_bytes / kMx4TileBytes;
    auto kern = rows_vec(out, out_dtype, ld) ? mx4_unpack_kernel<true> : mx4_unpack_kernel<false>;
    kern<<<unsigned(tiles), 256, 0, as_stream(stream)>>>(b, b + L.s_offset, rows, cols, out, out_dtype, ld);
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}

extern "C" int gale_mx8_quantize(const void* x, int x_dtype, int64_t ld, int64_t tokens, int64_t cols, void* packed,
                                 void* stream) {
    using namespace gale;
    if (tokens == 0 && cols >= 1 && valid_dtype(x_dtype)) return GALE_OK;
    gale_mx_layout_t L;
    if (!x || !packed || !valid_dtype(x_dtype) || gale_mx8_layout(tokens, cols, &L) != GALE_OK || ld < cols)
        return GALE_ERR_ARG;
    if (!aligned(packed, 256) || !aligned(x, dtype_size(x_dtype))) return GALE_ERR_ALIGN;
    uint8_t* b = static_cast<uint8_t*>(packed);
    const int64_t nc = (L.cols_padded / kMxTile + kQ8Tiles - 1) / kQ8Tiles;
    const int64_t grid = (tokens + kQ8Rows - 1) / kQ8Rows * nc;
    by_dtype_vec(x_dtype, rows_vec(x, x_dtype, ld), [&](auto dt, auto vec) {
        mx8_quantize_kernel<decltype(dt)::value, decltype(vec)::value><<<unsigned(grid), 256, 0, as_stream(stream)>>>(
            x, ld, tokens, cols, b, b + L.s_offset);
    });
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}
