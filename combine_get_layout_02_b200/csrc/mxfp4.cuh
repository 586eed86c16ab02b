// Device helpers for MXFP4 rows: blocks of 32 values, each E2M1 (sign, two
// exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times one power
// of two 2^(byte - 127) per block (UE8M0; byte 255 is NaN).  Two codes a byte,
// the lower index in the low four bits.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace cgl {

constexpr int kMxBlock = 32;

// The scale byte for a block whose largest |value| has these binary32 bits:
// the smallest e >= -127 with 6 * 2^e >= amax.  amax = m * 2^E with 1 <= m < 2,
// and 6 * 2^e = 1.5 * 2^(e + 2), so e = E - 2 where m <= 1.5, else E - 1:
// adding 0x3FFFFF carries into the exponent field exactly where the mantissa
// field is above 0x400000.  No value saturates.  Infinities and NaN (bits
// compared as integers, so a NaN is above everything) give 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;
    const int b = (int)((amax_bits + 0x3FFFFFu) >> 23) - 2;
    return b > 0 ? (uint32_t)b : 0u;
}

// 2^(127 - byte), the factor that brings a block into E2M1's range (exact for
// every byte mx_scale_byte gives below 255: 2^127 down to 2^-126).
__device__ __forceinline__ float mx_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127): byte 0 is the subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Eight floats -> eight E2M1 codes in one word, nearest, ties to even, past 6
// clamped (no value is).  v[0] lands in bits 3:0.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float v[8]) {
    uint32_t r;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 codes -> eight floats (exact).
__device__ __forceinline__ void cvt_f32x8_e2m1(uint32_t codes, float v[8]) {
    uint32_t h[4];
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n"
            ".reg .f16 l, u;\n"
            "mov.b32 {l, u}, %2;\n"
            "cvt.f32.f16 %0, l;\n"
            "cvt.f32.f16 %1, u;\n"
            "}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(h[i]));
}

// Four E2M1 codes -> four floats (exact).
__device__ __forceinline__ void cvt_f32x4_e2m1(uint16_t codes, float v[4]) {
    uint32_t h[2];
    asm("{\n"
        ".reg .b8 b0, b1;\n"
        "mov.b16 {b0, b1}, %2;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "}"
        : "=r"(h[0]), "=r"(h[1])
        : "h"(codes));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[2 * i] = __half2float(__ushort_as_half((unsigned short)(h[i] & 0xFFFFu)));
        v[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(h[i] >> 16)));
    }
}

// Eight values of a row by type: loaded as 16-byte words, widened exactly.
template <int DT>
struct Vec8;

template <>
struct Vec8<CGL_BF16> {
    uint4 a;
    __device__ __forceinline__ void load(const void *x, int64_t i) {
        a = ld_nc_v4(static_cast<const uint16_t *>(x) + i * 8);
    }
    __device__ __forceinline__ void widen(float v[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float v[8]) {
        st_cs_v4(static_cast<uint16_t *>(p) + i * 8, make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                                               cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])));
    }
};

template <>
struct Vec8<CGL_F16> {
    uint4 a;
    __device__ __forceinline__ void load(const void *x, int64_t i) {
        a = ld_nc_v4(static_cast<const uint16_t *>(x) + i * 8);
    }
    __device__ __forceinline__ void widen(float v[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __half2float(__ushort_as_half((unsigned short)(w[j] & 0xFFFFu)));
            v[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(w[j] >> 16)));
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float v[8]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
        st_cs_v4(static_cast<uint16_t *>(p) + i * 8, make_uint4(w[0], w[1], w[2], w[3]));
    }
};

template <>
struct Vec8<CGL_F32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *x, int64_t i) {
        const float *p = static_cast<const float *>(x) + i * 8;
        a = ld_nc_l1_v4(p);   // L1 keeps the sector for its other half
        b = ld_nc_l1_v4(p + 4);
    }
    __device__ __forceinline__ void widen(float v[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    }
    static __device__ __forceinline__ void store(void *p, int64_t i, const float v[8]) {
        float *q = static_cast<float *>(p) + i * 8;
        st_cs_v4(q, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        st_cs_v4(q + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    }
};

// Quantise this lane's eight values; the four lanes of each aligned group of
// four hold one block of 32.  Returns the codes; `byte` is the block's scale.
__device__ __forceinline__ uint32_t mx_quantize8(float v[8], uint32_t &byte) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    byte = mx_scale_byte(m);
    if (byte == 255u) return 0u;
    const float inv = mx_inverse(byte);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fmul_rn(v[j], inv);
    return cvt_e2m1x8(q);
}

// Quantise this lane's sixteen BF16 values (a, b); each aligned pair of lanes holds one block.
__device__ __forceinline__ uint2 mx_quantize16(const uint4 a, const uint4 b, uint32_t &byte) {
    // The largest |value| by its bits, NaN above everything: pairs compared as 16-bit integers.
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs)),
                          __vmaxu2(__vmaxu2(b.x & kAbs, b.y & kAbs), __vmaxu2(b.z & kAbs, b.w & kAbs)));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    byte = mx_scale_byte(max(m << 16, m & 0xFFFF0000u));
    if (byte == 255u) return make_uint2(0u, 0u);
    const float inv = mx_inverse(byte);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __fmul_rn(bf16_lo(w[i]), inv);
        v[2 * i + 1] = __fmul_rn(bf16_hi(w[i]), inv);
    }
    return make_uint2(cvt_e2m1x8(v), cvt_e2m1x8(v + 8));
}

}  // namespace cgl
