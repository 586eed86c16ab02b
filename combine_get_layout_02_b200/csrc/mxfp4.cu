// MXFP4 rows: quantise, dequantise, and the dispatch that quantises each token
// once and writes its copies to the receive rows (format in mxfp4.cuh).
//
// All three are bound by the bytes they move.  One thread owns eight values of
// the flattened [rows, cols / 8] grid: 16-byte loads of 16-bit values (two of
// 32-bit ones), one 4-byte store of codes; a warp reads and writes contiguous
// bytes.  Four lanes share a block of 32 and its maximum.
#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_kernel(const void *__restrict__ x, int64_t chunks, uint32_t *__restrict__ codes,
                      uint8_t *__restrict__ scales) {
    griddep_wait();
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    // warp-uniform loop (chunks is a multiple of 4: blocks never straddle its end)
    for (int64_t base = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); base < chunks; base += stride) {
        const int64_t i = base + (threadIdx.x & 31);
        const bool active = i < chunks;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (active) {
            Vec8<DT> in;
            in.load(x, i);
            in.widen(v);
        }
        uint32_t byte;
        const uint32_t q = mx_quantize8(v, byte);
        if (active) {
            codes[i] = q;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
dequantize_mxfp4_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t chunks,
                        void *__restrict__ out) {
    griddep_wait();
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < chunks; i += stride) {
        float v[8];
        cvt_f32x8_e2m1(__ldg(codes + i), v);
        const float s = mx_scale(__ldg(scales + (i >> 2)));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], s);
        Vec8<DT>::store(out, i, v);
    }
}

__global__ void __launch_bounds__(kThreads)
dispatch_mxfp4_kernel(const uint16_t *__restrict__ x, int64_t n, int h, int k, const int32_t *__restrict__ dst_pos,
                      uint8_t *__restrict__ recv_x, uint8_t *__restrict__ recv_scale, int64_t recv_rows,
                      uint32_t *status) {
    griddep_wait();                   // dst_pos (and x) may come from the kernels just before
    const int per_row = h >> 3, nblk = h >> 5;
    const int64_t total = n * per_row;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    bool bad = false;
    for (int64_t base = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); base < total; base += stride) {
        const int64_t g = base + (threadIdx.x & 31);
        const bool active = g < total;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (active) {
            Vec8<CGL_BF16> in;
            in.load(x, g);
            in.widen(v);
        }
        uint32_t byte;
        const uint32_t q = mx_quantize8(v, byte);
        if (!active) continue;
        const int64_t t = g / per_row;
        const int c = (int)(g - t * per_row);
        const int32_t *dp = dst_pos + t * k;
        for (int j = 0; j < k; ++j) {
            const int32_t row = __ldg(dp + j);
            if (row < 0) continue;
            if (row >= recv_rows) { bad = true; continue; }
            reinterpret_cast<uint32_t *>(recv_x)[(int64_t)row * per_row + c] = q;
            if ((c & 3) == 0) recv_scale[(int64_t)row * nblk + (c >> 2)] = (uint8_t)byte;
        }
    }
    if (bad) report(status, kErrRange);
}

template <int DT>
cgl_status launch_q(const void *x, int64_t chunks, uint8_t *codes, uint8_t *scales, int num_sms, cudaStream_t stream) {
    const int grid = copy_grid((const void *)quantize_mxfp4_kernel<DT>, kThreads, (chunks + kThreads - 1) / kThreads,
                               num_sms);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(quantize_mxfp4_kernel<DT>, dim3(grid), dim3(kThreads), 0, stream, x, chunks,
                      reinterpret_cast<uint32_t *>(codes), scales) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

template <int DT>
cgl_status launch_dq(const uint8_t *codes, const uint8_t *scales, int64_t chunks, void *out, int num_sms,
                     cudaStream_t stream) {
    const int grid = copy_grid((const void *)dequantize_mxfp4_kernel<DT>, kThreads, (chunks + kThreads - 1) / kThreads,
                               num_sms);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(dequantize_mxfp4_kernel<DT>, dim3(grid), dim3(kThreads), 0, stream,
                      reinterpret_cast<const uint32_t *>(codes), scales, chunks, out) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace

cgl_status launch_quantize_mxfp4(const void *x, int dtype, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                                 int num_sms, cudaStream_t stream) {
    const int64_t chunks = rows * (cols / 8);
    if (chunks == 0) return CGL_OK;
    switch (dtype) {
        case CGL_BF16: return launch_q<CGL_BF16>(x, chunks, codes, scales, num_sms, stream);
        case CGL_F16: return launch_q<CGL_F16>(x, chunks, codes, scales, num_sms, stream);
        default: return launch_q<CGL_F32>(x, chunks, codes, scales, num_sms, stream);
    }
}

cgl_status launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                   int dtype, int num_sms, cudaStream_t stream) {
    const int64_t chunks = rows * (cols / 8);
    if (chunks == 0) return CGL_OK;
    switch (dtype) {
        case CGL_BF16: return launch_dq<CGL_BF16>(codes, scales, chunks, out, num_sms, stream);
        case CGL_F16: return launch_dq<CGL_F16>(codes, scales, chunks, out, num_sms, stream);
        default: return launch_dq<CGL_F32>(codes, scales, chunks, out, num_sms, stream);
    }
}

cgl_status launch_dispatch_mxfp4(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos, uint8_t *recv_x,
                                 uint8_t *recv_scale, int64_t recv_rows, int num_sms, uint32_t *status,
                                 cudaStream_t stream, unsigned long long *claim) {
    (void)claim;
    if (n == 0) return CGL_OK;
    const int64_t work = n * (h / 8);
    const int grid = copy_grid((const void *)dispatch_mxfp4_kernel, kThreads, (work + kThreads - 1) / kThreads, num_sms);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(dispatch_mxfp4_kernel, dim3(grid), dim3(kThreads), 0, stream, x, n, h, k, dst_pos, recv_x,
                      recv_scale, recv_rows, status) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
