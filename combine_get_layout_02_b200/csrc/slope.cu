// The gradient in front of the activation, dz = grad_y act'(z), for the two products
// of the BF16 product's backward pass, and the bias's gradient, its sum over an
// expert's rows.
//
// One pass over grad_y and z: a thread has eight neighbouring columns (a gated
// activation's gate and up) and every few rows of a piece of kPiece rows of one
// expert, keeps its columns' sums in registers and leaves the piece's in the
// workspace; a second kernel adds the pieces of each expert in their order.  dz goes
// out as BF16, which the tensor cores take; the bias's sums take it unrounded.
// Bound by bytes: 8192 x 7168, GELU, z in binary32, with the bias 98 us (470 MB, 72 us
// at the copy rate); 32768 x 2 x 2048 gated, sums alone 147 (671 MB, 102).
#include "matmul_bf16.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 64;

__host__ __device__ __forceinline__ int pieces_of(int rows) { return (int)(((uint32_t)rows + kPiece - 1) / kPiece); }

__device__ __forceinline__ void load8(const uint16_t *p, bool vec, int n, float v[8]) {
    if (vec) {
        const uint4 a = ld_nc_v4(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? widen16(__ldg(p + i)) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const float *p, bool vec, int n, float v[8]) {
    if (vec) {
        const uint4 a = ld_nc_l1_v4(p), b = ld_nc_l1_v4(p + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldg(p + i) : 0.0f;
    }
}
__device__ __forceinline__ void store8(uint16_t *p, bool vec, int n, const float v[8]) {
    if (vec) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)cvt_bf16x2(v[i], 0.0f);
    }
}

// g times the activation's derivative.  ReLU selects: a closed unit drops what comes in,
// infinities and NaN too, which a product by 0 would keep; where z is NaN so is dz.
__device__ __forceinline__ float through(float g, float z, int act) {
    if (act == CGL_ACT_RELU) return z > 0.0f ? g : z != z ? z : 0.0f;
    if (act == CGL_ACT_GELU) {
        float bell;
        const float cdf = normal_cdf(z, bell);
        return g * (cdf + 0.39894228f * bell * z);
    }
    const float s = sigmoid(z);
    return g * (s * (1.0f + z * (1.0f - s)));
}

struct Slope {
    const int32_t *off;
    int64_t rows, cap;
    int E, cols;             // cols: of grad_y
    int act;
    const uint16_t *g;
    const void *z;
    uint16_t *dz;            // null: the sums alone
    int64_t ld;
    float *part;             // [pieces][columns of dz], null: dz alone
    int vec;
    int across;              // threads side by side
    uint32_t *status;
};

// Gated: `Z` z's type.
template <bool GATED, typename Z>
__global__ void __launch_bounds__(kThreads)
slope_kernel(const Slope a) {
    extern __shared__ int32_t s_first[];   // pieces before each expert
    __shared__ float s_sum[(GATED ? 2 : 1) * kThreads * 8];
    griddep_wait();
    bool bad = false;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        int r0, m;
        expert_rows(a.off, a.rows, a.cap, e, r0, m, bad);
        s_first[e] = pieces_of(m);
    }
    const bool refused = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x + blockIdx.y == 0) report(a.status, kErrRange);
    if (refused) return;
    if (threadIdx.x < 32) {
        const int per = (a.E + 31) / 32, e0 = threadIdx.x * per, e1 = e0 + per < a.E ? e0 + per : a.E;
        int sum = 0;
        for (int e = e0; e < e1; ++e) sum += s_first[e];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if ((int)threadIdx.x >= o) before += v;
        }
        before -= sum;
        for (int e = e0; e < e1; ++e) {
            const int n = s_first[e];
            s_first[e] = before;
            before += n;
        }
        if (e0 < a.E && e1 == a.E) s_first[a.E] = before;
    }
    __syncthreads();
    const int pieces = s_first[a.E];
    const int cx = threadIdx.x % a.across, ry = threadIdx.x / a.across, down = kThreads / a.across;
    const int col = (blockIdx.x * a.across + cx) * 8, n = a.cols - col < 8 ? a.cols - col : 8;   // n: columns there
    const int F = GATED ? 2 * a.cols : a.cols;
    const Z *z = static_cast<const Z *>(a.z);
    for (int piece = blockIdx.y; piece < pieces; piece += gridDim.y) {
        int lo = 0, hi = a.E - 1;   // the last expert whose first piece is not behind this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_first[mid] <= piece) lo = mid;
            else hi = mid - 1;
        }
        int r0, m;
        expert_rows(a.off, a.rows, a.cap, lo, r0, m, bad);
        const int at = (piece - s_first[lo]) * kPiece, end = m - at < kPiece ? m - at : kPiece;
        float sum[8] = {}, up[8] = {};
        if (n > 0)
#pragma unroll 2
            for (int i = ry; i < end; i += down) {
                const int64_t r = (int64_t)r0 + at + i;
                float g[8], d[8];
                load8(a.g + r * a.cols + col, a.vec, n, g);
                if (GATED) {
                    float x[8], u[8], du[8];
                    load8(z + r * F + col, a.vec, n, x);
                    load8(z + r * F + a.cols + col, a.vec, n, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float s = sigmoid(x[j]);
                        d[j] = g[j] * u[j] * (s * (1.0f + x[j] * (1.0f - s)));
                        du[j] = g[j] * (x[j] * s);
                        sum[j] += d[j];
                        up[j] += du[j];
                    }
                    if (a.dz != nullptr) {
                        store8(a.dz + r * a.ld + col, a.vec, n, d);
                        store8(a.dz + r * a.ld + a.cols + col, a.vec, n, du);
                    }
                } else {
                    if (a.act == CGL_ACT_NONE) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[j] = g[j];
                    } else {
                        float x[8];
                        load8(z + r * F + col, a.vec, n, x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[j] = through(g[j], x[j], a.act);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += d[j];
                    if (a.dz != nullptr) store8(a.dz + r * a.ld + col, a.vec, n, d);
                }
            }
        if (a.part == nullptr) continue;
        const int wide = a.across * 8;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s_sum[ry * wide + cx * 8 + j] = sum[j];
            if (GATED) s_sum[kThreads * 8 + ry * wide + cx * 8 + j] = up[j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < (GATED ? 2 : 1) * wide; c += kThreads) {
            const int h = c / wide, to = blockIdx.x * wide + c % wide;
            float v = 0.0f;
            for (int i = 0; i < down; ++i) v += s_sum[h * kThreads * 8 + i * wide + c % wide];
            if (to < a.cols) a.part[(int64_t)piece * F + h * a.cols + to] = v;
        }
    }
}

// Block: 32 columns of one expert; each of its warps adds every eighth piece, then the warps' sums in order.
__global__ void __launch_bounds__(kThreads)
bias_kernel(const int32_t *off, int64_t rows, int64_t cap, int E, int F, const float *__restrict__ part, uint16_t *__restrict__ grad_bias,
            uint32_t *status) {
    __shared__ int s_first;
    __shared__ float s_sum[kThreads];
    griddep_wait();
    if (threadIdx.x == 0) s_first = 0;
    bool bad = false;
    int before = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int r0, m;
        expert_rows(off, rows, cap, e, r0, m, bad);
        if (e < (int)blockIdx.y) before += pieces_of(m);
    }
    const bool refused = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x + blockIdx.y == 0) report(status, kErrRange);
    if (refused) return;
    if (before > 0) atomicAdd(&s_first, before);
    __syncthreads();
    int r0, m;
    expert_rows(off, rows, cap, blockIdx.y, r0, m, bad);
    const int f = blockIdx.x * 32 + (threadIdx.x & 31), n = pieces_of(m);
    float v = 0.0f;
    if (f < F)
#pragma unroll 4
        for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) v += part[(int64_t)(s_first + i) * F + f];
    s_sum[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 32 && f < F) {
        v = 0.0f;
        for (int i = 0; i < kThreads / 32; ++i) v += s_sum[32 * i + threadIdx.x];
        grad_bias[(int64_t)blockIdx.y * F + f] = (uint16_t)cvt_bf16x2(v, 0.0f);
    }
}

size_t round16(size_t v) { return (v + 15) / 16 * 16; }

}  // namespace

bool grad_y_is_dz(int act, int F, const uint16_t *grad_y) {
    return act == CGL_ACT_NONE && F % 8 == 0 && (reinterpret_cast<uintptr_t>(grad_y) & 15) == 0;
}

// dz with rows of whole 16 bytes, then the pieces' sums.
size_t matmul_bf16_backward_workspace_bytes(int64_t rows, int E, int F) {
    return round16((size_t)rows * ((F + 7) / 8 * 8) * 2) + (size_t)(rows / kPiece + E) * F * 4 + 16;
}

cgl_status launch_slope(const MatmulArgs &m, const uint16_t *grad_y, const void *preact, bool preact_f32, bool products,
                        uint16_t *grad_bias, void *ws, const uint16_t **dz, int64_t *ld, cudaStream_t stream) {
    const bool gated = m.act == CGL_ACT_SWIGLU;
    Slope a = {};
    a.off = m.off, a.rows = m.rows, a.cap = m.cap, a.E = m.E, a.cols = gated ? m.F / 2 : m.F, a.act = m.act;
    a.g = grad_y, a.z = m.act == CGL_ACT_NONE ? nullptr : preact, a.status = m.status;   // not read without an activation
    a.vec = a.cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(grad_y) | reinterpret_cast<uintptr_t>(a.z)) & 15) == 0;
    a.ld = (m.F + 7) / 8 * 8;
    const bool as_is = grad_y_is_dz(m.act, m.F, grad_y);
    if (ws == nullptr && ((products && !as_is) || grad_bias != nullptr)) return CGL_EINVAL;
    a.dz = products && !as_is ? static_cast<uint16_t *>(ws) : nullptr;
    a.part = grad_bias == nullptr ? nullptr : reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round16((size_t)m.rows * a.ld * 2));
    *dz = as_is ? grad_y : a.dz;
    *ld = a.ld;
    if (m.rows > 0 && (a.dz != nullptr || a.part != nullptr)) {
        a.across = 1;
        while (a.across < 32 && a.across * 8 < a.cols) a.across *= 2;
        const int64_t most = m.rows / kPiece + m.E;   // no more pieces than this
        const int64_t blocks_x = (a.cols + a.across * 8 - 1) / (a.across * 8);
        const int sms = device_sm_count();
        if (sms <= 0) return CGL_ECUDA;
        int64_t blocks_y = (8 * (int64_t)sms + blocks_x - 1) / blocks_x;
        if (blocks_y > most) blocks_y = most;
        const auto kernel = gated ? (preact_f32 ? slope_kernel<true, float> : slope_kernel<true, uint16_t>)
                                  : (preact_f32 ? slope_kernel<false, float> : slope_kernel<false, uint16_t>);
        if (launch_pdl(kernel, dim3((unsigned)blocks_x, (unsigned)blocks_y), dim3(kThreads), (size_t)(m.E + 1) * 4, stream, a) != cudaSuccess)
            return CGL_ECUDA;
    }
    if (grad_bias != nullptr &&
        launch_pdl(bias_kernel, dim3((m.F + 31) / 32, m.E), dim3(kThreads), 0, stream, m.off, m.rows, m.cap, m.E, m.F, a.part, grad_bias,
                   m.status) != cudaSuccess)
        return CGL_ECUDA;
    return CGL_OK;
}

}  // namespace cgl
