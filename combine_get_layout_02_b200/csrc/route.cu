// Routing: top-k experts of every token and their weights, and the gradient of
// the weights for the logits (formulas at cgl_route in cgl.h).
//
// One warp a token.
#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

template <int DT>
__device__ __forceinline__ float logit(const void *p, int64_t i) {
    if (DT == CGL_F32) return __ldg(static_cast<const float *>(p) + i);
    const unsigned short b = __ldg(static_cast<const unsigned short *>(p) + i);
    return DT == CGL_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

template <int DT>
__device__ __forceinline__ void put(void *p, int64_t i, float v) {
    if (DT == CGL_F32) static_cast<float *>(p)[i] = v;
    else if (DT == CGL_BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)cvt_bf16x2(v, 0.0f);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// The lane with the largest v and, among equals, the smallest index; every lane gets both.
__device__ __forceinline__ void warp_best(double &v, int &i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double u = __shfl_xor_sync(kAll, v, o);
        const int j = __shfl_xor_sync(kAll, i, o);
        if (u > v || (u == v && j < i)) v = u, i = j;
    }
}

// The picks of one token in binary64: lane j < k gets the j-th expert, or -1.
// False (for all lanes) where a logit or a choice is not a number.
template <int DT>
__device__ __noinline__ bool pick_exact(const RouteArgs &a, const void *row, int &expert) {
    const int lane = threadIdx.x & 31, E = a.E;
    double c[kMaxExperts / 32];
    double m = -INFINITY, sum = 0.0;
    bool bad = false;
    if (a.score == CGL_SCORE_SOFTMAX) {
        for (int e = lane; e < E; e += 32) {
            const double l = (double)logit<DT>(row, e);
            bad = bad || l == INFINITY;
            m = fmax(m, l);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
        for (int e = lane; e < E; e += 32) {
            const double l = (double)logit<DT>(row, e);
            if (l > -INFINITY) sum += exp(l - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    const auto score = [&](double l) { return a.score == CGL_SCORE_SOFTMAX ? exp(l - m) / sum : 1.0 / (1.0 + exp(-l)); };
    const int per = E / a.groups;
    uint32_t open = kAll;
    for (int i = 0, e = lane; e < E; e += 32, ++i) {
        const double l = (double)logit<DT>(row, e);
        bad = bad || l != l;
        c[i] = l;
        if (l > -INFINITY && a.bias != nullptr) {
            c[i] = score(l) + (double)__ldg(a.bias + e);
            bad = bad || c[i] != c[i];
        }
    }
    if (__any_sync(kAll, bad)) return false;
    if (a.groups > 1) {
        double mine = -INFINITY;   // lane g: the value of group g
        for (int g = 0; g < a.groups; ++g) {
            double best[2];
            int taken = -1;
            for (int r = 0; r < (a.by == CGL_GROUP_TOP2 ? 2 : 1); ++r) {
                double v = -INFINITY;
                int at = E;
                for (int i = 0, e = lane; e < E; e += 32, ++i) {
                    if (e / per != g || e == taken) continue;
                    const double u = a.by == CGL_GROUP_TOP2 && a.bias == nullptr && c[i] > -INFINITY ? score(c[i]) : c[i];
                    if (u > v || (u == v && u > -INFINITY && e < at)) v = u, at = e;
                }
                warp_best(v, at);
                best[r] = v;
                taken = at;
            }
            if (lane == g) mine = a.by == CGL_GROUP_TOP2 && best[1] > -INFINITY ? best[0] + best[1] : best[0];
        }
        open = 0;
        for (int r = 0; r < a.keep; ++r) {
            double v = mine;
            int at = mine > -INFINITY ? lane : 32;
            warp_best(v, at);
            if (at == 32) break;
            open |= 1u << at;
            if (lane == at) mine = -INFINITY;
        }
    }
    expert = -1;
    for (int j = 0; j < a.k; ++j) {
        double v = -INFINITY;
        int at = E;
        for (int i = 0, e = lane; e < E; e += 32, ++i)
            if (c[i] > v && ((open >> (e / per)) & 1)) v = c[i], at = e;
        warp_best(v, at);
        if (at == E) break;
        if (lane == j) expert = at;
        if ((at & 31) == lane) c[at >> 5] = -INFINITY;
    }
    return true;
}

// What lane j's slot has of its token's weight (scale aside), slots without an
// expert 0; D over the slots where they are renormalised, `m` and `sum` the row's
// largest logit and sum of exponentials for the plain softmax.
__device__ __forceinline__ float share(int score, bool renorm, bool there, float l, float m, float sum) {
    float t;
    if (score == CGL_SCORE_SIGMOID) {
        // sigmoid(l) exp(-b), b = min(largest l, 0): a factor that all slots share keeps the quotient where every sigmoid underflows
        const float b = renorm ? fminf(warp_max(there ? l : -INFINITY), 0.0f) : 0.0f;
        const float z = expf(-fabsf(l));
        t = (l > 0.0f ? 1.0f : expf(l - b)) / (1.0f + z);
    } else {
        const float b = renorm ? warp_max(there ? l : -INFINITY) : m;
        t = expf(l - b);
        if (!renorm) return there && l > -INFINITY ? t / sum : there && l != l ? l : 0.0f;
    }
    if (!there || l == -INFINITY) t = 0.0f;
    if (!renorm) return t;
    const float d = warp_sum(t);
    return d == 0.0f ? 0.0f : t / d;
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
route_kernel(const RouteArgs a) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.n; t += step) {
        const char *row = static_cast<const char *>(a.logits) + t * a.E * (DT == CGL_F32 ? 4 : 2);
        int e = -1;
        const bool fine = pick_exact<DT>(a, row, e);
        const bool there = fine && e >= 0;
        const float l = there ? logit<DT>(row, e) : -INFINITY;
        float m = -INFINITY, sum = 0.0f;
        if (a.score == CGL_SCORE_SOFTMAX && !a.renorm && fine) {
            for (int i = lane; i < a.E; i += 32) m = fmaxf(m, logit<DT>(row, i));
            m = warp_max(m);
            for (int i = lane; i < a.E; i += 32) {
                const float x = logit<DT>(row, i);
                if (x > -INFINITY) sum += expf(x - m);
            }
            sum = warp_sum(sum);
        }
        const float w = share(a.score, a.renorm, there, l, m, sum);
        if (lane < a.k) {
            a.idx[t * a.k + lane] = there ? e : -1;
            a.weights[t * a.k + lane] = fine ? (there ? a.scale * w : 0.0f) : NAN;
        }
        if (!fine && lane == 0) report(a.status, kErrRange);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float *__restrict__ gw, const void *__restrict__ logits, const int32_t *__restrict__ idx, int64_t n,
                      int E, int k, int score, bool renorm, float scale, void *__restrict__ grad, uint32_t *status) {
    extern __shared__ float s_rows[];   // a row of E values a warp
    griddep_wait();
    const int lane = threadIdx.x & 31;
    float *s = s_rows + (threadIdx.x >> 5) * E;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n; t += step) {
        const char *row = static_cast<const char *>(logits) + t * E * (DT == CGL_F32 ? 4 : 2);
        const int e = lane < k ? __ldg(idx + t * k + lane) : -1;
        const bool there = e >= 0 && e < E;
        if (!there && e != -1) report(status, kErrRange);
        const bool any = __any_sync(kAll, there);
        const bool whole = score == CGL_SCORE_SOFTMAX && !renorm && any;
        float m = -INFINITY, sum = 0.0f;
        if (whole) {
            for (int i = lane; i < E; i += 32) m = fmaxf(m, logit<DT>(row, i));
            m = warp_max(m);
            for (int i = lane; i < E; i += 32) {
                const float x = logit<DT>(row, i);
                if (!(x == -INFINITY)) sum += expf(x - m);
            }
            sum = warp_sum(sum);
        }
        const float l = there ? logit<DT>(row, e) : -INFINITY;
        const float w = share(score, renorm, there, l, m, sum), g = there ? scale * __ldg(gw + t * k + lane) : 0.0f;
        const float dot = warp_sum(there ? g * w : 0.0f);
        float v = w * (renorm ? g - dot : g);
        if (score == CGL_SCORE_SIGMOID) {   // 1 - sigmoid(l)
            const float z = expf(-fabsf(l));
            v *= (l > 0.0f ? z : 1.0f) / (1.0f + z);
        }
        for (int i = lane; i < E; i += 32) {
            const float x = whole ? logit<DT>(row, i) : 0.0f;
            s[i] = whole && !(x == -INFINITY) ? -dot * (expf(x - m) / sum) : 0.0f;
        }
        __syncwarp();
        for (int j = 0; j < k; ++j) {   // in the slots' order: an expert may be in two
            if (lane == j && there) s[e] += v;
            __syncwarp();
        }
        for (int i = lane; i < E; i += 32) put<DT>(grad, t * E + i, s[i]);
        __syncwarp();
    }
}

}  // namespace

cgl_status launch_route(const RouteArgs &a, cudaStream_t stream) {
    if (a.n == 0) return CGL_OK;
    const auto kernel = a.dtype == CGL_BF16 ? route_kernel<CGL_BF16> : a.dtype == CGL_F16 ? route_kernel<CGL_F16> : route_kernel<CGL_F32>;
    const int grid = persistent_grid((const void *)kernel, kThreads, 0, 8, 0, (a.n + kWarps - 1) / kWarps);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, a) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

cgl_status launch_route_backward(const float *gw, const void *logits, int dtype, const int32_t *idx, int64_t n, int E, int k,
                                 int score, bool renorm, float scale, void *grad, uint32_t *status, cudaStream_t stream) {
    if (n == 0) return CGL_OK;
    const auto kernel = dtype == CGL_BF16 ? route_backward_kernel<CGL_BF16>
                        : dtype == CGL_F16 ? route_backward_kernel<CGL_F16> : route_backward_kernel<CGL_F32>;
    const size_t smem = (size_t)kWarps * E * 4;   // at most 32 KiB
    const int grid = persistent_grid((const void *)kernel, kThreads, smem, 8, 0, (n + kWarps - 1) / kWarps);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, gw, logits, idx, n, E, k, score, renorm, scale, grad,
                      status) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
