// The experts' product on BF16 rows with bias, activation and residual, and its
// gradients (formulas at cgl_matmul_bf16 in cgl.h).
//
// One thread a result, operands through shared memory, sums in binary32.
#include "common.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kT = 16;   // a block's tile is kT x kT results

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t narrow(float v) { return (uint16_t)cvt_bf16x2(v, 0.0f); }

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case CGL_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
        case CGL_ACT_GELU: return 0.5f * z * erfcf(-0.70710678f * z);
        case CGL_ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}
// The activation's derivative.
__device__ __forceinline__ float slope(float z, int act) {
    switch (act) {
        case CGL_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case CGL_ACT_GELU: return 0.5f * erfcf(-0.70710678f * z) + z * 0.39894228f * expf(-0.5f * z * z);
        case CGL_ACT_SILU: {
            const float s = sigmoid(z);
            return s * (1.0f + z * (1.0f - s));
        }
        default: return 1.0f;
    }
}

// Whether the offsets run forwards and inside the buffer, asked by a whole block.
__device__ bool offsets_ok(const MatmulArgs &m) {
    bool bad = false;
    if (m.off != nullptr)
        for (int e = threadIdx.x + threadIdx.y * blockDim.x; e < m.E; e += blockDim.x * blockDim.y) {
            const int64_t a = m.off[e], b = m.off[e + 1];
            bad = bad || a < 0 || b < a || (m.cap == 0 && b > m.rows);
        }
    bad = __syncthreads_or(bad) != 0;
    if (bad && threadIdx.x + threadIdx.y == 0) report(m.status, kErrRange);
    return !bad;
}
__device__ void rows_of(const MatmulArgs &m, int e, int64_t &r0, int64_t &r1) {
    if (m.off == nullptr) {
        r0 = 0, r1 = m.rows;
        return;
    }
    const int64_t a = m.off[e], n = m.off[e + 1] - a;
    r0 = m.cap > 0 ? e * m.cap : a;
    r1 = r0 + (m.cap > 0 && n > m.cap ? m.cap : n);
}

// sum_c x(i, c) y(j, c) for this thread's i, j; x and y give 0 outside.
template <typename X, typename Y>
__device__ __forceinline__ float product(int64_t n, X x, Y y) {
    __shared__ float sx[kT][kT + 1], sy[kT][kT + 1];
    float sum = 0.0f;
    for (int64_t c = 0; c < n; c += kT) {
        sx[threadIdx.y][threadIdx.x] = c + threadIdx.x < n ? x(threadIdx.y, c + threadIdx.x) : 0.0f;
        sy[threadIdx.y][threadIdx.x] = c + threadIdx.x < n ? y(threadIdx.y, c + threadIdx.x) : 0.0f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kT; ++i) sum = fmaf(sx[threadIdx.y][i], sy[threadIdx.x][i], sum);
        __syncthreads();
    }
    return sum;
}

// blockIdx: features, rows (strided), expert.
__global__ void __launch_bounds__(kT *kT)
forward_kernel(const MatmulArgs m, const uint16_t *bias, const uint16_t *residual, uint16_t *y, uint16_t *preact) {
    griddep_wait();
    if (!offsets_ok(m)) return;
    const int e = blockIdx.z;
    const bool gated = m.act == CGL_ACT_SWIGLU;
    const int cols = gated ? m.F / 2 : m.F;
    const int64_t f0 = (int64_t)blockIdx.x * kT;
    int64_t r0, r1;
    rows_of(m, e, r0, r1);
    const uint16_t *w = m.w + (int64_t)e * m.F * m.K;
    for (r0 += (int64_t)blockIdx.y * kT; r0 < r1; r0 += (int64_t)gridDim.y * kT) {
        const auto rows = [&](int i, int64_t c) { return r0 + i < r1 ? widen(m.a[(r0 + i) * m.K + c]) : 0.0f; };
        const auto weights = [&](int64_t first) {
            return [=](int i, int64_t c) { return f0 + i < cols ? widen(w[(first + f0 + i) * m.K + c]) : 0.0f; };
        };
        float z = product(m.K, rows, weights(0)), up = 0.0f;
        if (gated) up = product(m.K, rows, weights(cols));
        const int64_t r = r0 + threadIdx.y, f = f0 + threadIdx.x;
        if (r >= r1 || f >= cols) continue;
        if (bias != nullptr) {
            z += widen(bias[(int64_t)e * m.F + f]);
            if (gated) up += widen(bias[(int64_t)e * m.F + cols + f]);
        }
        if (preact != nullptr) {
            preact[r * m.F + f] = narrow(z);
            if (gated) preact[r * m.F + cols + f] = narrow(up);
        }
        float v = gated ? z * sigmoid(z) * up : activate(z, m.act);
        if (residual != nullptr) v += widen(residual[r * cols + f]);
        y[r * cols + f] = narrow(v);
    }
}

// dz of the experts' rows in binary32, its BF16 values to the workspace.
__device__ __forceinline__ float slope_at(const MatmulArgs &m, const uint16_t *g, const uint16_t *z, int64_t r, int64_t f) {
    if (m.act != CGL_ACT_SWIGLU) return widen(g[r * m.F + f]) * (m.act == CGL_ACT_NONE ? 1.0f : slope(widen(z[r * m.F + f]), m.act));
    const int64_t cols = m.F / 2, h = f % cols;
    const float gate = widen(z[r * m.F + h]), up = widen(z[r * m.F + cols + h]), d = widen(g[r * cols + h]);
    return f < cols ? d * up * slope(gate, CGL_ACT_SILU) : d * (gate * sigmoid(gate));
}

__global__ void __launch_bounds__(kT *kT)
slope_kernel(const MatmulArgs m, const uint16_t *g, const uint16_t *z, uint16_t *dz, uint16_t *grad_bias) {
    griddep_wait();
    if (!offsets_ok(m)) return;
    const int e = blockIdx.z;
    const int64_t f = (int64_t)blockIdx.x * kT * kT + threadIdx.y * kT + threadIdx.x;
    int64_t r0, r1;
    rows_of(m, e, r0, r1);
    if (f >= m.F) return;
    float sum = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float v = slope_at(m, g, z, r, f);
        dz[r * m.F + f] = narrow(v);
        sum += v;
    }
    if (grad_bias != nullptr) grad_bias[(int64_t)e * m.F + f] = narrow(sum);
}

__global__ void __launch_bounds__(kT *kT)
grad_a_kernel(const MatmulArgs m, const uint16_t *dz, uint16_t *grad_a) {
    griddep_wait();
    if (!offsets_ok(m)) return;
    const int e = blockIdx.z;
    const int64_t k0 = (int64_t)blockIdx.x * kT;
    int64_t r0, r1;
    rows_of(m, e, r0, r1);
    const uint16_t *w = m.w + (int64_t)e * m.F * m.K;
    for (r0 += (int64_t)blockIdx.y * kT; r0 < r1; r0 += (int64_t)gridDim.y * kT) {
        const float v = product(m.F, [&](int i, int64_t c) { return r0 + i < r1 ? widen(dz[(r0 + i) * m.F + c]) : 0.0f; },
                                [&](int i, int64_t c) { return k0 + i < m.K ? widen(w[c * m.K + k0 + i]) : 0.0f; });
        const int64_t r = r0 + threadIdx.y, k = k0 + threadIdx.x;
        if (r < r1 && k < m.K) grad_a[r * m.K + k] = narrow(v);
    }
}

__global__ void __launch_bounds__(kT *kT)
grad_w_kernel(const MatmulArgs m, const uint16_t *dz, uint16_t *grad_w) {
    griddep_wait();
    if (!offsets_ok(m)) return;
    const int e = blockIdx.z;
    const int64_t k0 = (int64_t)blockIdx.x * kT;
    int64_t r0, r1;
    rows_of(m, e, r0, r1);
    for (int64_t f0 = (int64_t)blockIdx.y * kT; f0 < m.F; f0 += (int64_t)gridDim.y * kT) {
        const float v = product(r1 - r0, [&](int i, int64_t c) { return f0 + i < m.F ? widen(dz[(r0 + c) * m.F + f0 + i]) : 0.0f; },
                                [&](int i, int64_t c) { return k0 + i < m.K ? widen(m.a[(r0 + c) * m.K + k0 + i]) : 0.0f; });
        const int64_t f = f0 + threadIdx.y, k = k0 + threadIdx.x;
        if (f < m.F && k < m.K) grad_w[((int64_t)e * m.F + f) * m.K + k] = narrow(v);
    }
}

dim3 tiles(int64_t x, int64_t y, int64_t z) {
    y = (y + kT - 1) / kT;
    return dim3((unsigned)((x + kT - 1) / kT), (unsigned)(y < 64 ? (y < 1 ? 1 : y) : 64), (unsigned)z);
}

}  // namespace

cgl_status launch_matmul_bf16(const MatmulArgs &m, const uint16_t *bias, const uint16_t *residual, uint16_t *y,
                              uint16_t *preact, cudaStream_t stream) {
    if (m.rows == 0) return CGL_OK;
    const int cols = m.act == CGL_ACT_SWIGLU ? m.F / 2 : m.F;
    return launch_pdl(forward_kernel, tiles(cols, m.rows, m.E), dim3(kT, kT), 0, stream, m, bias, residual, y, preact) == cudaSuccess
               ? CGL_OK : CGL_ECUDA;
}

size_t matmul_bf16_backward_workspace_bytes(int64_t rows, int E, int F) { return (size_t)(rows > 0 ? rows : 1) * F * 2 + 16; }

cgl_status launch_matmul_bf16_backward(const MatmulArgs &m, const uint16_t *grad_y, const uint16_t *preact, uint16_t *grad_a,
                                       uint16_t *grad_w, uint16_t *grad_bias, void *ws, cudaStream_t stream) {
    uint16_t *dz = static_cast<uint16_t *>(ws);
    bool ok = launch_pdl(slope_kernel, dim3((m.F + kT * kT - 1) / (kT * kT), 1, m.E), dim3(kT, kT), 0, stream, m, grad_y, preact, dz,
                         grad_bias) == cudaSuccess;
    if (grad_a != nullptr)
        ok = ok && launch_pdl(grad_a_kernel, tiles(m.K, m.rows, m.E), dim3(kT, kT), 0, stream, m, dz, grad_a) == cudaSuccess;
    if (grad_w != nullptr)
        ok = ok && launch_pdl(grad_w_kernel, tiles(m.K, m.F, m.E), dim3(kT, kT), 0, stream, m, dz, grad_w) == cudaSuccess;
    return ok ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
