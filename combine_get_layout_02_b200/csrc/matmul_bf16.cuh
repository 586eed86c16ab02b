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
// The normal distribution function and, in `bell`, e^(-z^2 / 2).  For z <= 0 it is
// half erfc(|z| / sqrt(2)) = half e^(-z^2 / 2) t p(t) with t = 1 / (1 + 0.375 |z| / sqrt(2)):
// p of degree 6, fitted to e^(x^2) erfc(x) / t over x in [0, 10] for the least relative
// error (6.4e-7).  So the far negative side, where the function is near 0, stays exact
// in relation to it (2.4e-6 down to -6, from the rounded exponent).  erfcf took 40 us
// more of 300 (8192 rows, 2048 -> 7168).
__device__ __forceinline__ float normal_cdf(float z, float &bell) {
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.26516504f, fabsf(z), 1.0f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell) : "f"(-0.72134752f * z * z));
    float p = -0.06754669576f;
    p = fmaf(p, t, 0.19396447858f);
    p = fmaf(p, t, -0.06479228701f);
    p = fmaf(p, t, 0.14152602816f);
    p = fmaf(p, t, 0.08333421921f);
    p = fmaf(p, t, 0.10784417987f);
    p = fmaf(p, t, 0.10566975951f);
    const float half = p * t * bell;
    return z > 0.0f ? 1.0f - half : half;
}
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
