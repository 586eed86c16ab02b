// What the BF16 product and the gradient of its activation share.
#pragma once

#include "common.cuh"

namespace cgl {

__device__ __forceinline__ float widen16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// 1 / (1 + e^-z): 0 where e^-z overflows.  Approximate exponential and reciprocal, each
// within two steps of binary32, and the rounded exponent, |z| 2^-24: far below the
// half step of the BF16 result.
__device__ __forceinline__ float sigmoid(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
// The normal distribution function; erfc keeps it exact where it is near 0.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }
__device__ __forceinline__ float relu(float z) { return z > 0.0f || z != z ? z : 0.0f; }   // NaN stays

// Rows [r0, r0 + m) of expert e.  `bad`: offsets that run backwards or out of the
// buffer.  Where no expert's are, the experts' rows are apart and in the buffer.
__device__ __forceinline__ void expert_rows(const int32_t *off, int64_t rows, int64_t cap, int e, int &r0, int &m, bool &bad) {
    if (off == nullptr) {
        r0 = 0;
        m = (int)rows;
        return;
    }
    const int64_t a = __ldg(off + e), b = __ldg(off + e + 1), n = b - a;
    if (a < 0 || n < 0 || (cap == 0 && b > rows)) bad = true;
    r0 = (int)(cap > 0 ? e * cap : a);
    m = (int)(cap > 0 && n > cap ? cap : n);
}

}  // namespace cgl
