// RMSNorm with the residual's addition:  h = x + r,  y = h / sqrt(mean h^2 + eps) * w.
//
// One pass: a row's h stays in registers between the sum of squares and the
// outputs, so every input is read once and every output written once; the
// kernel is bound by HBM (by latency for a few tokens).  h enters the norm in
// fp32, before its rounding to the residual's type.  y leaves in 16 or 32 bits
// and / or as MXFP8 (e4m3 codes, one power-of-two scale per 32 columns).
//
// A row goes straight into registers: of a warp up to 512 columns, of a CTA
// beyond.  Many wide rows in 16 bits cost more instructions per byte than that
// hides: theirs arrive by bulk copies in a ring of shared-memory stages (4096 x
// 4096 with residual 24 us, 31 us without the ring).
#include "mx.cuh"
#include "ptx.cuh"
#include "tma.cuh"

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
    int wt, yt;
    int vw;              // w may be read 16 bytes at a time
    float inv_cols;
    int stages, stage_bytes, r_off;      // ring: stages, bytes of one, where the residual's row starts in it
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

// MXFP8 of four columns per thread: eight neighbouring threads hold a block.
__device__ __forceinline__ void mx8_store_vec(const NormArgs& a, int64_t row, int c, const float (&v)[4], bool live) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
    const uint32_t b = mx8_scale_byte(m);
    uint32_t word = b << (8 * ((threadIdx.x >> 3) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    if (!live) return;
    *reinterpret_cast<uint32_t*>(a.q + row * a.nt * kMxTile + c) =
        b != 255u ? mx8_codes(v[0], v[1], v[2], v[3], mx_inverse(b)) : 0u;
    if ((threadIdx.x & 31) == 0) *reinterpret_cast<uint32_t*>(a.s + mx_scale_at(row, c / kMxBlock, a.nt)) = word;
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

// What a thread takes at a time: 16 bytes of a row, E columns, so that a warp's accesses are contiguous.
template <int DT>
struct Unit {
    static constexpr int E = DT == GALE_F32 ? 4 : 8;
    uint4 v;
    __device__ __forceinline__ void f32(float (&h)[E]) const {
        if constexpr (DT == GALE_F32) {
            h[0] = __uint_as_float(v.x); h[1] = __uint_as_float(v.y);
            h[2] = __uint_as_float(v.z); h[3] = __uint_as_float(v.w);
        } else {
            const Raw8<DT> r{{v.x, v.y, v.z, v.w}};
            raw8_f32<DT>(r, h);
        }
    }
};

template <int E>
__device__ __forceinline__ void store_unit(void* p, int dtype, int64_t at, const float (&v)[E]) {
    if constexpr (E == 8) {
        store8(p, dtype, at, 8, true, v);
    } else if (dtype == GALE_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
            make_uint2(pack16(dtype, v[0], v[1]), pack16(dtype, v[2], v[3]));
    }
}

// How a row is read and written: units of neighbouring columns, the row starting
// on a unit (kVec) or anywhere (kPhased: units that are aligned in memory, the
// first and the last of which the row may fill in part); or single elements
// `threads` apart (kSingle).
enum { kSingle, kVec, kPhased };

// A unit of a row as loaded, from column c (kSingle: c + i * threads); zero outside the row.
template <int DT, int HOW>
__device__ __forceinline__ void norm_load(const void* p, int64_t at, int cols, int c, int threads, Unit<DT>& v) {
    constexpr int E = Unit<DT>::E;
    if (HOW != kSingle && (HOW == kVec || c >= 0) && c + E <= cols) {
        v.v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + (at + c) * (16 / E));
    } else {
        uint32_t u[4] = {};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = HOW == kSingle ? c + i * threads : c + i;
            if (e >= cols || (HOW == kPhased && e < 0)) continue;
            if constexpr (DT == GALE_F32) u[i] = static_cast<const uint32_t*>(p)[at + e];
            else u[i / 2] |= uint32_t(static_cast<const uint16_t*>(p)[at + e]) << (16 * (i % 2));
        }
        v.v = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// The weights of columns c .. c + E - 1, `lo` to `n` - 1 of which exist.
template <int E>
__device__ __forceinline__ void norm_weights(const NormArgs& a, int c, int lo, int n, float (&w)[E]) {
    const bool whole = lo == 0 && n >= E && a.vw;
    if (a.wt == GALE_F32 && whole && (c & 3) == 0) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.w) + c + 4 * q);
            w[4 * q] = f.x; w[4 * q + 1] = f.y; w[4 * q + 2] = f.z; w[4 * q + 3] = f.w;
        }
    } else if (a.wt == GALE_F32 && whole && c >= 4 && n >= E + 4) {
        // E of the E + 4 from the 16-byte boundary before
        float f[E + 4];
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.w) + (c & ~3));
#pragma unroll
        for (int i = 0; i < E / 4 + 1; ++i) {
            const float4 v = q[i];
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
        if (c & 2) {
#pragma unroll
            for (int i = 0; i < E + 1; ++i) f[i] = f[i + 2];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = c & 1 ? f[i + 1] : f[i];
    } else if (a.wt != GALE_F32 && whole && (c & (E - 1)) == 0) {
        uint32_t u[E / 2];
        const uint16_t* q = static_cast<const uint16_t*>(a.w) + c;
        if constexpr (E == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(q);
            u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(q);
            u[0] = v.x; u[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 f = a.wt == GALE_BF16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u))
                                               : __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            w[2 * i] = f.x;
            w[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = i >= lo && i < n ? load_as_f32(a.w, a.wt, c + i) : 0.f;
    }
}

// The columns c .. c + E - 1 of a row, `n` of them up to the row's end (a phased row's first unit begins before it).
template <int E>
__device__ __forceinline__ void norm_store(void* p, int dtype, int64_t at, int c, int n, const float (&v)[E]) {
    if (c >= 0 && n >= E) {
        store_unit<E>(p, dtype, at, v);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (c + i >= 0 && i < n) store_rn(p, dtype, at + i, v[i]);
    }
}

// A row per group of `threads` threads (a warp, or the CTA), CH * 8 columns per
// thread: (j * threads + t) * E + i less the row's phase, or, kSingle, (j * E +
// i) * threads + t.  Units of 16 bytes in fp32 too, so that a warp's access is
// one run of 512 bytes; all of a row's loads, then all of its residual's, are
// asked for before the first is used (10,007 x 5000 fp32: 67 -> 62 us, with
// residual 95 -> 89).  Registers are bounded for as many CTAs as keep HBM busy:
// 50 instead of 48 of them for two chunks cost a fourth CTA at 5000 columns, 74
// us.  (Chosen on rows in units: kSingle spills 20 to 650 bytes a thread under them.)
template <int DT, int HOW, int CH, bool WARP>
__global__ void __maxnreg__(CH == 1 ? 40 : CH == 2 ? 48 : CH == 4 ? 64 : 128) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float part[16];
    if (a.q) pdl_launch_dependents();      // a product behind this kernel may set itself up meanwhile
    constexpr int E = Unit<DT>::E, N = CH * 8 / E;
    const int lane = threadIdx.x & 31;
    const int threads = WARP ? 32 : blockDim.x;
    const int t = WARP ? lane : threadIdx.x;
    const int64_t row = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.tokens) return;      // whole warps (a CTA always has its row)
    float h[N][E];
    float ss = 0.f;
    const int ph = HOW == kPhased ? int((row * a.ldx) & 7) : 0;
    auto column = [&](int j) { return HOW == kSingle ? j * E * threads + t : (j * threads + t) * E - ph; };
    Unit<DT> x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) norm_load<DT, HOW>(a.x, row * a.ldx, a.cols, column(j), threads, x[j]);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j].f32(h[j]);
    if (a.r) {
        constexpr int B = N < 8 ? N : 8;      // so many loads at once
#pragma unroll
        for (int j0 = 0; j0 < N; j0 += B) {
            Unit<DT> raw[B];
#pragma unroll
            for (int j = 0; j < B; ++j)
                norm_load<DT, HOW>(a.r, row * a.ldr, a.cols, column(j0 + j), threads, raw[j]);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                float r[E];
                raw[j].f32(r);
#pragma unroll
                for (int i = 0; i < E; ++i) h[j0 + j][i] += r[i];
            }
        }
    }
    // no more than 32 squares are added in order: an addition may lose half a unit of the sum
    constexpr int kRun = N * E <= 32 ? N : 32 / E;
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += kRun) {
        float part_ss = 0.f;
#pragma unroll
        for (int j = j0; j < j0 + kRun; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) part_ss = fmaf(h[j][i], h[j][i], part_ss);
        ss += part_ss;
    }
    ss = warp_sum(ss);
    if constexpr (!WARP) {
        if (lane == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = warp_sum(lane < (threads >> 5) ? part[lane] : 0.f);
    }
    const float inv = rsqrtf(fmaf(ss, a.inv_cols, a.eps));
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if constexpr (HOW != kSingle) {
            const int c = column(j);
            const int n = a.cols - c;
            float w[E];
            if (a.w) norm_weights<E>(a, c, c < 0 ? -c : 0, n, w);
            if (a.h) norm_store<E>(a.h, DT, row * a.ldh + c, c, n, h[j]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float y = h[j][i] * inv;
                h[j][i] = i < n ? (a.w ? y * w[i] : y) : 0.f;
            }
            if (a.y) norm_store<E>(a.y, a.yt, row * a.ldy + c, c, n, h[j]);
            if (HOW == kVec && a.q) mx8_store_vec(a, row, c, h[j], c < a.span);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = column(j) + i * threads;
                const bool in = c < a.cols;
                if (a.h && in) store_rn(a.h, DT, row * a.ldh + c, h[j][i]);
                float y = in ? h[j][i] * inv : 0.f;
                if (a.w && in) y *= load_as_f32(a.w, a.wt, c);
                if (a.y && in) store_rn(a.y, a.yt, row * a.ldy + c, y);
                if (a.q) mx8_store_scalar(a, row, c, y, c < a.span);
            }
        }
    }
}

// A CTA per row, rows blockIdx.x, + gridDim.x, ...: thread 0 keeps the next
// `stages` rows' bulk copies in flight.  Rows whose length is no multiple of
// eight start at any element; every tensor's row starts at the same element
// modulo 8 (its phase), so chunks of eight that are aligned in one are in all: a
// copy takes the aligned bytes around its row (inside the tensor for every row
// but the last, whose last columns are fetched one by one), and the first and
// the last chunk hold columns of the neighbouring rows, which are masked.
//
// The weights stay in registers, loaded once: a load behind the stores waited
// thousands of cycles in the saturated memory pipeline.  So a CTA's rows have
// one phase, the grid being a multiple of eight CTAs; registers are bounded so that
// the CTAs the launch counts on fit.  A row held in registers between its two passes
// beats one read twice from its stage by fewer warps (4096 x 4096 in 16 bits 24
// against 34 us: half the unpacking).
template <int DT, int CH, bool PHASED>
__global__ void __launch_bounds__(CH == 1 ? 256 : 512, CH == 1 ? 6 : CH == 2 ? 2 : 1) rmsnorm_ring_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float part[2][16];
    __shared__ uint64_t full[8];
    static_assert(DT != GALE_F32, "16-bit rows");
    constexpr int ES = 2;
    if (a.q) pdl_launch_dependents();
    const int lane = threadIdx.x & 31, t = threadIdx.x, threads = blockDim.x;
    if (t == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    const int ph = PHASED ? int((blockIdx.x * a.ldx) & 7) : 0;
    auto issue = [&](int64_t row, int s) {
        int bytes = ((ph + a.cols) * ES + 15) & ~15;
        if (row + 1 == a.tokens) bytes = (ph + a.cols) * ES & ~15;
        uint8_t* st = ring + s * a.stage_bytes;
        mbar_arrive_expect_tx(&full[s], a.r ? 2 * bytes : bytes);
        if (bytes) {
            bulk_load(st, static_cast<const uint8_t*>(a.x) + (row * a.ldx - ph) * ES, bytes, &full[s]);
            if (a.r) bulk_load(st + a.r_off, static_cast<const uint8_t*>(a.r) + (row * a.ldr - ph) * ES, bytes, &full[s]);
        }
    };
    if (t == 0)
        for (int s = 0; s < a.stages; ++s) {
            const int64_t row = blockIdx.x + int64_t(s) * gridDim.x;
            if (row < a.tokens) issue(row, s);
        }
    float w[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = (j * threads + t) * 8 - ph;
        if (a.w) {
            norm_weights<8>(a, c, c < 0 ? -c : 0, a.cols - c, w[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[j][i] = 1.0f;
        }
    }
    int s = 0, turn = 0;
    uint32_t parity = 0;
    for (int64_t row = blockIdx.x; row < a.tokens; row += gridDim.x) {
        const bool here = mbar_wait_cycles(&full[s], parity);
        uint8_t* st = ring + s * a.stage_bytes;
        if (row + 1 == a.tokens && (ph + a.cols) * ES % 16) {      // what the copy left out
            for (int e = ((ph + a.cols) * ES & ~15) / ES + t; e < ph + a.cols; e += threads) {
                reinterpret_cast<uint16_t*>(st)[e] = static_cast<const uint16_t*>(a.x)[row * a.ldx - ph + e];
                if (a.r)
                    reinterpret_cast<uint16_t*>(st + a.r_off)[e] = static_cast<const uint16_t*>(a.r)[row * a.ldr - ph + e];
            }
            __syncthreads();
        }
        float h[CH][8];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int k = j * threads + t;
            const int c = k * 8 - ph;
            if (c < a.cols) {
                Raw8<DT> x;
                load_raw8<DT, true>(st, k * 8, 8, x);
                raw8_f32<DT>(x, h[j]);
                if (a.r) {
                    float r[8];
                    load_raw8<DT, true>(st + a.r_off, k * 8, 8, x);
                    raw8_f32<DT>(x, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] += r[i];
                }
                if (c < 0 || c + 8 > a.cols) {      // columns that are not the row's
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] = c + i >= 0 && c + i < a.cols ? h[j][i] : 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
            }
            if (!here) h[j][0] = __uint_as_float(0x7FC00000u);      // the bounded wait ran out: the row is NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
        }
        ss = warp_sum(ss);
        // (two buffers: a fast warp's next row does not reach into a slow one's read)
        if (lane == 0) part[turn][t >> 5] = ss;
        __syncthreads();
        if (t == 0) {      // every thread has its row in registers: the stage is free
            const int64_t ahead = row + int64_t(a.stages) * gridDim.x;
            if (ahead < a.tokens) issue(ahead, s);
        }
        ss = warp_sum(lane < (threads >> 5) ? part[turn][lane] : 0.f);
        turn ^= 1;
        if (++s == a.stages) {
            s = 0;
            parity ^= 1;
        }
        const float inv = rsqrtf(fmaf(ss, a.inv_cols, a.eps));
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = (j * threads + t) * 8 - ph;
            if (c >= 0 && c + 8 <= a.cols) {
                if (a.h) store8(a.h, DT, row * a.ldh + c, 8, true, h[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * inv * w[j][i];
                if (a.y && a.yt == DT) store8(a.y, DT, row * a.ldy + c, 8, true, h[j]);
                else if (a.y) store8(a.y, a.yt, row * a.ldy + c, 8, true, h[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (c + i < 0 || c + i >= a.cols) continue;
                    if (a.h) store_rn(a.h, DT, row * a.ldh + c + i, h[j][i]);
                    h[j][i] = h[j][i] * inv * w[j][i];
                    if (a.y) store_rn(a.y, a.yt, row * a.ldy + c + i, h[j][i]);
                }
            }
            if (a.q) mx8_store_vec(a, row, c, h[j], c < a.span);      // (phase 0)
        }
    }
}

constexpr int kNormMaxCols = 32768;

// Rows straight into registers.
template <int DT, int HOW>
void launch_norm(const NormArgs& a, cudaStream_t st) {
    const int chunks = (a.span + 7) / 8 + (HOW == kPhased ? 1 : 0);             // eight-column chunks of a row
    if (chunks <= 64) {                              // up to 512 columns: a warp per row, eight rows per CTA
        const unsigned grid = unsigned((a.tokens + 7) / 8);
        if (chunks <= 32) rmsnorm_kernel<DT, HOW, 1, true><<<grid, 256, 0, st>>>(a);
        else rmsnorm_kernel<DT, HOW, 2, true><<<grid, 256, 0, st>>>(a);
    } else {                                         // a CTA per row (148 rows of 704 columns: 2.4 us, a warp each 4.7)
        const unsigned grid = unsigned(a.tokens);
        const int ch = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
        const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
        if (ch == 1) rmsnorm_kernel<DT, HOW, 1, false><<<grid, threads, 0, st>>>(a);
        else if (ch == 2) rmsnorm_kernel<DT, HOW, 2, false><<<grid, threads, 0, st>>>(a);
        else if (ch == 4) rmsnorm_kernel<DT, HOW, 4, false><<<grid, threads, 0, st>>>(a);
        else rmsnorm_kernel<DT, HOW, 8, false><<<grid, threads, 0, st>>>(a);
    }
}

// Rows through the ring; false if it does not take them.
template <int DT>
int launch_norm_ring(NormArgs& a, cudaStream_t st, bool& taken) {
    const int es = 2;
    taken = false;
    const int chunks = (a.span + 7) / 8 + (a.ldx % 8 ? 1 : 0);
    const int row_bytes = chunks * 8 * es;
    a.r_off = row_bytes;
    a.stage_bytes = a.r ? 2 * row_bytes : row_bytes;
    // columns per thread: what a row costs every thread (barrier, sums, addresses) weighs least with many, the latency
    // of a row least with few (4096 x 4096 in 16 bits: 16 of them 17.4 us, 32 19.5; 4000 x 6000: 24.5
    // and 30.5)
    const int ch = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
    const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    // CTAs of an SM by its registers; two stages each
    auto room = [](int ctas) { return 228 * 1024 / ctas - 1536; };      // shared memory of each, static and reserved off
    int per_sm = (ch == 4 ? 512 : ch == 2 ? 1024 : 1536) / threads;
    if (per_sm < 1) per_sm = 1;
    while (per_sm > 1 && room(per_sm) < 2 * a.stage_bytes) --per_sm;
    a.stages = room(per_sm) / a.stage_bytes;
    if (a.stages > 8) a.stages = 8;
    const int64_t most = int64_t(sm_count()) * per_sm;
    if (chunks > 2048 || a.stages < 2) return GALE_OK;
    taken = true;
    // a multiple of eight CTAs takes rows of one phase each
    const unsigned grid = unsigned(a.tokens <= most ? a.tokens : a.ldx % 8 ? most / 8 * 8 : most);
    if (a.tokens <= most) a.stages = 1;
    const int smem = a.stages * a.stage_bytes;
    auto go = [&](auto kern) {
        if (ensure_smem(reinterpret_cast<const void*>(kern), smem) != GALE_OK) return GALE_ERR_CUDA;
        kern<<<grid, threads, smem, st>>>(a);
        return GALE_OK;
    };
    if (a.ldx % 8)
        return ch == 1   ? go(rmsnorm_ring_kernel<DT, 1, true>)
               : ch == 2 ? go(rmsnorm_ring_kernel<DT, 2, true>)
                         : go(rmsnorm_ring_kernel<DT, 4, true>);
    return ch == 1   ? go(rmsnorm_ring_kernel<DT, 1, false>)
           : ch == 2 ? go(rmsnorm_ring_kernel<DT, 2, false>)
                     : go(rmsnorm_ring_kernel<DT, 4, false>);
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
    a.wt = w_dtype;
    a.yt = y_dtype;
    a.eps = eps;
    a.inv_cols = 1.0f / float(cols);
    if (mx8) {
        gale_mx_layout_t L;
        if (gale_mx8_layout(tokens, cols, &L) != GALE_OK) return GALE_ERR_ARG;
        a.q = static_cast<uint8_t*>(mx8);
        a.s = a.q + L.s_offset;
        a.nt = L.cols_padded / kMxTile;
        a.span = int(L.cols_padded);
    }
    a.vw = weight && aligned(weight, 16);
    cudaStream_t st = as_stream(stream);
    const bool vec = rows_vec(x, dtype, ldx) && (!residual || rows_vec(residual, dtype, ldr)) &&
                     (!sum_out || rows_vec(sum_out, dtype, ldsum)) && (!y || rows_vec(y, y_dtype, ldy));
    // bases on 16 bytes and row strides that agree modulo 8 elements: rows in aligned chunks (with MXFP8, whose blocks
    // start with the row, only if rows start on chunks of eight)
    auto agrees = [&](const void* p, int64_t ld) { return !p || (aligned(p, 16) && (ld - ldx) % 8 == 0); };
    // (and a row with the chunk that its phase may add has to fit 512 threads of 64 columns)
    const bool phased = a.span > 256 && a.span <= kNormMaxCols - 8 && agrees(x, ldx) && agrees(residual, ldr) && agrees(sum_out, ldsum) &&
                        agrees(y, ldy) && (!mx8 || ldx % 8 == 0);
    // The ring pays where a row costs many instructions per byte and there are rows enough: in 16 bits, from 1024
    // columns and 4.5 M elements on (with residual: 4736 x 4096 21 us, straight into registers 32; 20,000 x 704 20 each;
    // 592 x 5000 5.9 and 5.2).  In fp32 registers are ahead everywhere (10,007 x 5000: 62 us, ring 78).
    if (phased && dtype != GALE_F32 && cols >= 1024 && tokens * cols >= 4500000) {
        bool taken = false;
        const int rc = dtype == GALE_BF16 ? launch_norm_ring<GALE_BF16>(a, st, taken)
                                          : launch_norm_ring<GALE_F16>(a, st, taken);
        if (rc != GALE_OK) return rc;
        if (taken) {
            GALE_LAUNCH_CHECK();
            return GALE_OK;
        }
    }
    auto direct = [&](auto how) {
        constexpr int HOW = decltype(how)::value;
        if (dtype == GALE_F32) launch_norm<GALE_F32, HOW>(a, st);
        else if (dtype == GALE_BF16) launch_norm<GALE_BF16, HOW>(a, st);
        else launch_norm<GALE_F16, HOW>(a, st);
    };
    if (vec) direct(std::integral_constant<int, kVec>());
    else if (phased) direct(std::integral_constant<int, kPhased>());
    else direct(std::integral_constant<int, kSingle>());
    GALE_LAUNCH_CHECK();
    return GALE_OK;
}
