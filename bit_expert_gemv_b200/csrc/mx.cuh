// Microscaled formats: blocks of 32 consecutive columns share one power-of-two
// scale (an 8-bit exponent with bias 127; 255 stands for NaN).  Codes are e2m1
// (4 bits: 0, .5, 1, 1.5, 2, 3, 4, 6) or e4m3 (8 bits, largest 448).
//
// The scale of a block is the smallest 2^k with max|v| <= 2^k * largest code, so
// no value is clipped; the codes are v / 2^k rounded to nearest even.  The
// division is by a power of two, so every decision is exact in fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"

namespace gale {

constexpr int kMxBlock = 32;      // columns of a scale
constexpr int kMxTile = 128;      // rows and columns of a storage tile
constexpr int kMx4TileBytes = kMxTile * kMxTile / 2;
constexpr int kMxAtomBytes = kMxTile * (kMxTile / kMxBlock);   // scales of a 128 x 128 tile

// Byte of the scale of (row, block) in the scale section, nt = padded cols / 128.
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t row, int64_t blk, int64_t nt) {
    return ((row / kMxTile) * nt + blk / 4) * kMxAtomBytes + (row % 32) * 16 + (row % kMxTile) / 32 * 4 + blk % 4;
}

// Scale byte of a block from the largest magnitude's bits (sign bit cleared):
// k = floor(log2 max) - TOP_EXP, one more if the mantissa is above the largest
// code's (TOP_MANT: its 23 fraction bits), clamped to [-127, 127], stored + 127.
template <uint32_t TOP_MANT, int TOP_EXP>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;      // infinity or NaN in the block
    int e = int(amax_bits >> 23);
    uint32_t m = amax_bits & 0x7FFFFFu;
    if (e == 0) return 0u;                           // zero, or so small that 2^-127 holds it
    const int k = e - TOP_EXP + (m > TOP_MANT ? 1 : 0);   // biased by 127
    return uint32_t(k < 0 ? 0 : k);                  // at most 254 - TOP_EXP + 1
}
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) { return mx_scale_byte<0x400000u, 2>(amax_bits); }
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) { return mx_scale_byte<0x600000u, 8>(amax_bits); }

// 2^(127 - byte): the factor that divides by the scale (byte 0..254; the
// result is at least 2^-127, a subnormal for byte 254).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte < 254u ? __uint_as_float((254u - byte) << 23) : __uint_as_float(0x00400000u);
}
// 2^(byte - 127)
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// Eight values as e2m1 nibbles, value i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t mx4_codes(const float (&v)[8], float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_E2M1,
                                               cudaRoundNearest))
             << (8 * i);
    return w;
}
// Four values as e4m3 bytes, value i in byte i.
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// Eight consecutive elements of type DT as loaded: several rows' loads can be in
// flight before the first is converted.
template <int DT>
struct Raw8 {
    uint32_t u[DT == GALE_F32 ? 8 : 4];
};
// The elements from offset `at`, of which the first `n` exist; the others are
// zero.  VEC: they may be read 16 bytes at a time.
template <int DT, bool VEC>
__device__ __forceinline__ void load_raw8(const void* p, int64_t at, int n, Raw8<DT>& v) {
    if (VEC && n >= 8) {
        if constexpr (DT == GALE_F32) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
            const uint4 a = q[0], b = q[1];
            v.u[0] = a.x; v.u[1] = a.y; v.u[2] = a.z; v.u[3] = a.w;
            v.u[4] = b.x; v.u[5] = b.y; v.u[6] = b.z; v.u[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
            v.u[0] = a.x; v.u[1] = a.y; v.u[2] = a.z; v.u[3] = a.w;
        }
    } else if constexpr (DT == GALE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.u[i] = i < n ? static_cast<const uint32_t*>(p)[at + i] : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t* q = static_cast<const uint16_t*>(p) + at + 2 * i;
            v.u[i] = (2 * i < n ? uint32_t(q[0]) : 0u) | (2 * i + 1 < n ? uint32_t(q[1]) << 16 : 0u);
        }
    }
}
template <int DT>
__device__ __forceinline__ void raw8_f32(const Raw8<DT>& r, float (&v)[8]) {
    if constexpr (DT == GALE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == GALE_BF16) {
                v[2 * i] = __uint_as_float(r.u[i] << 16);
                v[2 * i + 1] = __uint_as_float(r.u[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}
// Calls f with the dtype code and the alignment case as compile-time constants.
template <typename F>
inline void by_dtype_vec(int dtype, bool vec, F f) {
    auto v = [&](auto dt) {
        if (vec) f(dt, std::true_type());
        else f(dt, std::false_type());
    };
    if (dtype == GALE_F32) v(std::integral_constant<int, GALE_F32>());
    else if (dtype == GALE_BF16) v(std::integral_constant<int, GALE_BF16>());
    else v(std::integral_constant<int, GALE_F16>());
}

// One value rounded to nearest even into dtype (NaN and infinities kept).
__device__ __forceinline__ void store_rn(void* p, int dtype, int64_t i, float v) {
    if (dtype == GALE_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == GALE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
__device__ __forceinline__ uint32_t pack16(int dtype, float a, float b) {
    if (dtype == GALE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(void* p, int dtype, int64_t at, int n, bool vec, const float (&v)[8]) {
    if (vec && n >= 8) {
        if (dtype == GALE_F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
                make_uint4(pack16(dtype, v[0], v[1]), pack16(dtype, v[2], v[3]), pack16(dtype, v[4], v[5]),
                           pack16(dtype, v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store_rn(p, dtype, at + i, v[i]);
    }
}

// Largest magnitude's bits of eight values.
__device__ __forceinline__ uint32_t amax8_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    return m;
}

inline bool valid_dtype(int d) { return d == GALE_F32 || d == GALE_BF16 || d == GALE_F16; }
inline int dtype_size(int d) { return d == GALE_F32 ? 4 : 2; }
// Whether rows of `ld` elements from p can be read and written eight elements (16 or 32 bytes) at a time.
inline bool rows_vec(const void* p, int dtype, int64_t ld) {
    return aligned(p, 16) && (ld * dtype_size(dtype)) % 16 == 0;
}

}  // namespace gale
