// The experts' product on MXFP4 rows: y[r, :] = A[r, :] W[e(r), :, :]^T, sums in
// binary32, BF16 out (format in mxfp4.cuh).
#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

// Rows [r0, r1) of expert e.  Offsets that run backwards or out of the buffer
// are clamped and reported.
__device__ __forceinline__ void expert_rows(const int32_t *off, int e, int64_t rows, int64_t cap, int64_t &r0,
                                            int64_t &r1, bool &bad) {
    if (off == nullptr) {
        r0 = 0;
        r1 = rows;
        return;
    }
    const int64_t a = __ldg(off + e), b = __ldg(off + e + 1);
    if (a < 0 || b < a) bad = true;
    if (cap > 0) {
        const int64_t c = b - a;
        r0 = e * cap;
        r1 = r0 + (c < 0 ? 0 : c > cap ? cap : c);
    } else {
        if (b > rows) bad = true;
        r0 = a < 0 ? 0 : a > rows ? rows : a;
        r1 = b < r0 ? r0 : b > rows ? rows : b;
    }
}

__global__ void __launch_bounds__(kThreads)
matmul_mxfp4_simple_kernel(const uint8_t *__restrict__ a, const uint8_t *__restrict__ sa, int64_t rows,
                           const uint8_t *__restrict__ w, const uint8_t *__restrict__ sw, int E, int F, int K,
                           const int32_t *__restrict__ off, int64_t cap, uint16_t *__restrict__ y, uint32_t *status) {
    __shared__ float ta[kTile][33], tw[kTile][33];
    __shared__ int64_t s_r0, s_r1;
    __shared__ int s_e;
    griddep_wait();
    if (threadIdx.x == 0) {
        int64_t left = blockIdx.y, r0, r1;
        bool bad = false;
        s_e = -1;
        for (int e = 0; e < E; ++e) {
            expert_rows(off, e, rows, cap, r0, r1, bad);
            const int64_t tiles = (r1 - r0 + kTile - 1) / kTile;
            if (s_e < 0 && left < tiles) {
                s_e = e;
                s_r0 = r0 + left * kTile;
                s_r1 = r1;
            }
            left -= tiles;
        }
        if (bad) report(status, kErrRange);
    }
    __syncthreads();
    const int e = s_e;
    if (e < 0) return;
    const int64_t r0 = s_r0, r1 = s_r1;
    const int f0 = blockIdx.x * kTile;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    const int per_row = K / 8;
    for (int k0 = 0; k0 < K; k0 += 32) {
        const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
        float v[8] = {};
        if (r0 + r < r1) {
            cvt_f32x8_e2m1(__ldg(reinterpret_cast<const uint32_t *>(a) + (r0 + r) * per_row + k0 / 8 + c), v);
            const float s = mx_scale(__ldg(sa + (r0 + r) * (K / 32) + k0 / 32));
            for (int j = 0; j < 8; ++j) v[j] *= s;
        }
        for (int j = 0; j < 8; ++j) ta[r][c * 8 + j] = v[j];
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (f0 + r < F) {
            const int64_t row = (int64_t)e * F + f0 + r;
            cvt_f32x8_e2m1(__ldg(reinterpret_cast<const uint32_t *>(w) + row * per_row + k0 / 8 + c), v);
            const float s = mx_scale(__ldg(sw + row * (K / 32) + k0 / 32));
            for (int j = 0; j < 8; ++j) v[j] *= s;
        }
        for (int j = 0; j < 8; ++j) tw[r][c * 8 + j] = v[j];
        __syncthreads();
#pragma unroll 8
        for (int kk = 0; kk < 32; ++kk) {
            float x[4], z[4];
            for (int i = 0; i < 4; ++i) x[i] = ta[ty + 16 * i][kk];
            for (int i = 0; i < 4; ++i) z[i] = tw[tx + 16 * i][kk];
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], z[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty + 16 * i;
            const int f = f0 + tx + 16 * j;
            if (r < r1 && f < F) y[r * F + f] = (uint16_t)cvt_bf16x2(acc[i][j], 0.0f);
        }
}

}  // namespace

cgl_status launch_matmul_mxfp4(const uint8_t *a, const uint8_t *sa, int64_t rows, const uint8_t *w, const uint8_t *sw,
                               int E, int F, int K, const int32_t *off, int64_t cap, uint16_t *y, int num_sms,
                               uint32_t *status, cudaStream_t stream) {
    (void)num_sms;
    if (rows == 0) return CGL_OK;
    const int64_t tiles = rows / kTile + E;
    if (tiles > 65535) return CGL_EINVAL;
    const dim3 grid((F + kTile - 1) / kTile, (unsigned)tiles);
    return launch_pdl(matmul_mxfp4_simple_kernel, grid, dim3(kThreads), 0, stream, a, sa, rows, w, sw, E, F, K, off, cap,
                      y, status) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
