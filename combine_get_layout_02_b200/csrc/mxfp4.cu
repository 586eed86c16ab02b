// MXFP4 rows: quantise and dequantise (format in mxfp4.cuh).
//
// Both are bound by the bytes they move.  One thread owns eight values of
// the flattened [rows, cols / 8] grid: 16-byte loads of 16-bit values (two of
// 32-bit ones), one 4-byte store of codes; a warp reads and writes contiguous
// bytes.  Four lanes share a block of 32 and its maximum.  Four chunks a thread
// are loaded before the first is used (16384 x 7168 BF16: quantise 51 us,
// dequantise 53 us, 88% and 85% of the measured copy rate).
#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // chunks of eight values a thread has in flight

template <int DT>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_kernel(const void *__restrict__ x, int64_t chunks, uint32_t *__restrict__ codes,
                      uint8_t *__restrict__ scales) {
    griddep_wait();
    const int64_t stride = (int64_t)gridDim.x * kThreads * kUnroll;
    // warp-uniform loop (chunks is a multiple of 4: blocks never straddle its end)
    for (int64_t base = (int64_t)blockIdx.x * kThreads * kUnroll + (threadIdx.x & ~31); base < chunks; base += stride) {
        const int64_t i0 = base + (threadIdx.x & 31);
        Vec8<DT> in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i0 + u * kThreads < chunks) in[u].load(x, i0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = i0 + u * kThreads;
            const bool active = i < chunks;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (active) in[u].widen(v);
            uint32_t byte;
            const uint32_t q = mx_quantize8(v, byte);
            if (active) {
                codes[i] = q;
                if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
            }
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
dequantize_mxfp4_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t chunks,
                        void *__restrict__ out) {
    griddep_wait();
    const int64_t stride = (int64_t)gridDim.x * kThreads * kUnroll;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; i0 < chunks; i0 += stride) {
        uint32_t q[kUnroll], byte[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = i0 + u * kThreads;
            q[u] = i < chunks ? __ldg(codes + i) : 0u;
            byte[u] = i < chunks ? __ldg(scales + (i >> 2)) : 0u;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= chunks) break;
            float v[8];
            cvt_f32x8_e2m1(q[u], v);
            const float s = mx_scale(byte[u]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], s);
            Vec8<DT>::store(out, i, v);
        }
    }
}

// Binary32 values in fours, so that a warp's store covers 512 bytes in a row
// (with eight a thread, two stores of every second 16 bytes: 135 us for
// 16384 x 7168 values, where this takes 95 us, 86% of the measured copy rate).
__global__ void __launch_bounds__(kThreads)
dequantize_mxfp4_f32_kernel(const uint16_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t quads,
                            float4 *__restrict__ out) {
    griddep_wait();
    const int64_t stride = (int64_t)gridDim.x * kThreads * kUnroll;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x; i0 < quads; i0 += stride) {
        uint16_t q[kUnroll];
        uint32_t byte[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = i0 + u * kThreads;
            q[u] = i < quads ? __ldg(codes + i) : (uint16_t)0;
            byte[u] = i < quads ? __ldg(scales + (i >> 3)) : 0u;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= quads) break;
            float v[4];
            cvt_f32x4_e2m1(q[u], v);
            const float s = mx_scale(byte[u]);
            st_cs_v4(out + i, make_uint4(__float_as_uint(__fmul_rn(v[0], s)), __float_as_uint(__fmul_rn(v[1], s)),
                                         __float_as_uint(__fmul_rn(v[2], s)), __float_as_uint(__fmul_rn(v[3], s))));
        }
    }
}

template <int DT>
cgl_status launch_q(const void *x, int64_t chunks, uint8_t *codes, uint8_t *scales, int num_sms, cudaStream_t stream) {
    const int grid = copy_grid((const void *)quantize_mxfp4_kernel<DT>, kThreads, (chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll),
                               num_sms);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(quantize_mxfp4_kernel<DT>, dim3(grid), dim3(kThreads), 0, stream, x, chunks,
                      reinterpret_cast<uint32_t *>(codes), scales) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

template <int DT>
cgl_status launch_dq(const uint8_t *codes, const uint8_t *scales, int64_t chunks, void *out, int num_sms,
                     cudaStream_t stream) {
    const int64_t units = DT == CGL_F32 ? 2 * chunks : chunks;
    const void *kernel = DT == CGL_F32 ? (const void *)dequantize_mxfp4_f32_kernel : (const void *)dequantize_mxfp4_kernel<DT>;
    const int grid = copy_grid(kernel, kThreads, (units + kThreads * kUnroll - 1) / (kThreads * kUnroll), num_sms);
    if (grid <= 0) return CGL_ECUDA;
    cudaError_t err;
    if (DT == CGL_F32)
        err = launch_pdl(dequantize_mxfp4_f32_kernel, dim3(grid), dim3(kThreads), 0, stream,
                         reinterpret_cast<const uint16_t *>(codes), scales, units, static_cast<float4 *>(out));
    else
        err = launch_pdl(dequantize_mxfp4_kernel<DT == CGL_F32 ? CGL_BF16 : DT>, dim3(grid), dim3(kThreads), 0, stream,
                         reinterpret_cast<const uint32_t *>(codes), scales, units, out);
    return err == cudaSuccess ? CGL_OK : CGL_ECUDA;
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

}  // namespace cgl
