// Balance loss of the routing, per-expert counts, and the gradient for the
// router's logits.
//
// Sequence s of T tokens, T_s of them routed (some slot holds an id in range),
// c[e] its slots with id e, p[t, :] the token's probabilities:
//   loss = sum_s sum_t sum_e w[e] p[t, e],   w[e] = alpha E c[e] / (S k T_s^2)
//   dloss/dlogit[t, i] = p_i (w_i - sum_e p_e w_e) * (softmax: 1; sigmoid: 1 - sigmoid(l_i)).
// The counts carry no gradient, so once they are known one pass over the
// logits gives the loss and the gradient.  sum_e p_e = 1: w enters both less
// its mean, u (E c[e] - sum c) with u = alpha / (S k T_s^2), whose bracket is
// an exact integer, so near-equal counts lose nothing to cancellation.
//
// Kernels: histograms of id chunks (shared-memory integer atomics, order
// without effect) -> one warp per token, the chunks' counts summed by every
// block for itself -> the blocks' loss sums in a fixed order.
#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kCountThreads = 512;
constexpr int kMainThreads = 256;
constexpr int kMainWarps = kMainThreads / 32;
constexpr int64_t kMaxBlocks = 1184;   // 148 SMs x 8 blocks; a constant, so sums do not depend on the device

struct Shape {
    int64_t tokens;      // per sequence
    int64_t seqs;
    int k, E;
    int count_chunks;    // histogram blocks per sequence
    int64_t count_tokens;
    int main_chunks;     // blocks per sequence of the main pass
};

Shape shape(int64_t n, int k, int E, int64_t S) {
    Shape s;
    s.tokens = n / S;
    s.seqs = S;
    s.k = k;
    s.E = E;
    const int64_t want = (s.tokens * k + 8191) / 8192, fit = kMaxBlocks / S > 0 ? kMaxBlocks / S : 1;
    int64_t c = want < 32 ? want : 32;
    if (c > fit) c = fit;
    if (c < 1) c = 1;
    s.count_chunks = (int)c;
    s.count_tokens = (s.tokens + c - 1) / c;
    int64_t d = (s.tokens + kMainWarps - 1) / kMainWarps;
    if (d > fit) d = fit;
    s.main_chunks = d < 1 ? 1 : (int)d;
    return s;
}

__global__ void __launch_bounds__(kCountThreads)
balance_count_kernel(const int32_t *__restrict__ idx, int64_t tokens, int k, int E, int chunks, int64_t per_chunk,
                     int32_t *__restrict__ part, uint32_t *status) {
    extern __shared__ int32_t s_count[];   // [E + 1]: slots per expert, routed tokens
    griddep_wait();
    for (int e = threadIdx.x; e <= E; e += kCountThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t seq = blockIdx.x / chunks, c = blockIdx.x % chunks;
    const int64_t t0 = c * per_chunk, t1 = t0 + per_chunk < tokens ? t0 + per_chunk : tokens;
    bool bad = false;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kCountThreads) {
        const int32_t *p = idx + (seq * tokens + t) * k;
        bool any = false;
        for (int j = 0; j < k; ++j) {
            const int32_t e = __ldg(p + j);
            if (e >= 0 && e < E) {
                atomicAdd(&s_count[e], 1);
                any = true;
            } else if (e != -1) {
                bad = true;
            }
        }
        if (any) atomicAdd(&s_count[E], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kCountThreads) part[(int64_t)blockIdx.x * (E + 1) + e] = s_count[e];
    if (bad) report(status, kErrRange);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if (DT == CGL_F32) return __ldg(static_cast<const float *>(p) + i);
    const unsigned short b = __ldg(static_cast<const unsigned short *>(p) + i);
    return DT == CGL_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

template <int DT>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if (DT == CGL_F32) static_cast<float *>(p)[i] = v;
    else if (DT == CGL_BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)cvt_bf16x2(v, 0.0f);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// One warp per token, lane l holding experts l, l + 32, ...  part: the count
// kernel's chunks (chunks > 0), or counts / routed as the forward gave them.
template <int DT, int V>
__global__ void __launch_bounds__(kMainThreads)
balance_main_kernel(const void *__restrict__ logits, const int32_t *__restrict__ idx, int64_t tokens, int k, int E,
                    double scale, int sigmoid, const int32_t *__restrict__ part, int chunks,
                    int32_t *__restrict__ counts, int32_t *__restrict__ routed, const float *__restrict__ grad_loss,
                    void *__restrict__ grad, double *__restrict__ loss_part, int main_chunks) {
    extern __shared__ float s_w[];   // [E] weights less their mean
    __shared__ long long s_total;
    __shared__ int s_routed;
    __shared__ double s_loss[kMainWarps];
    griddep_wait();
    const int64_t seq = blockIdx.x / main_chunks;
    const int chunk = (int)(blockIdx.x % main_chunks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *s_c = reinterpret_cast<int32_t *>(s_w);
    if (threadIdx.x == 0) { s_total = 0; s_routed = 0; }
    __syncthreads();
    long long mine = 0;
    for (int e = threadIdx.x; e <= E; e += kMainThreads) {
        int32_t c = 0;
        if (chunks > 0)
            for (int i = 0; i < chunks; ++i) c += part[(seq * chunks + i) * (E + 1) + e];
        else
            c = e < E ? counts[seq * E + e] : routed[seq];
        if (e < E) {
            s_c[e] = c;
            mine += c;
            if (chunks > 0 && chunk == 0) counts[seq * E + e] = c;
        } else {
            s_routed = c;
            if (chunks > 0 && chunk == 0) routed[seq] = c;
        }
    }
    atomicAdd((unsigned long long *)&s_total, (unsigned long long)mine);
    __syncthreads();
    const long long total = s_total;
    const double t = (double)s_routed, unit = t > 0 ? scale / (t * t) : 0.0;   // scale = alpha / (S k)
    const float mean = (float)(unit * (double)total);
    for (int e = threadIdx.x; e < E; e += kMainThreads)
        s_w[e] = (float)(unit * (double)((long long)E * s_c[e] - total));
    __syncthreads();
    const float g = grad != nullptr ? (grad_loss != nullptr ? __ldg(grad_loss) : 1.0f) : 0.0f;
    double acc = 0.0;
    for (int64_t r = chunk * kMainWarps + warp; r < tokens; r += (int64_t)main_chunks * kMainWarps) {
        const int64_t tok = seq * tokens + r;
        bool any = false;
        if (lane < k) {
            const int32_t e = __ldg(idx + tok * k + lane);
            any = e >= 0 && e < E;
        }
        any = __any_sync(0xFFFFFFFFu, any);
        if (!any) {
            if (grad != nullptr)
                for (int e = lane; e < E; e += 32) store1<DT>(grad, tok * E + e, 0.0f);
            continue;
        }
        float l[V], p[V], gate[V];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < E ? load1<DT>(logits, tok * E + e) : -INFINITY;
            m = fmaxf(m, l[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float sum = 0.0f, dot = 0.0f;
        if (m == -INFINITY) m = 0.0f;        // nothing left (or NaN): exp(-inf) below, not exp(nan)
        if (sigmoid) m = fminf(m, 0.0f);     // common factor: keeps p where every sigmoid underflows
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (sigmoid) {
                const float z = expf(-fabsf(l[i])), d = 1.0f / (1.0f + z);
                p[i] = (l[i] > 0.0f ? 1.0f : expf(l[i] - m)) * d;
                gate[i] = (l[i] > 0.0f ? z : 1.0f) * d;
            } else {
                p[i] = expf(l[i] - m);
                gate[i] = 1.0f;
            }
            sum += p[i];
            const int e = lane + 32 * i;
            if (e < E) dot += p[i] * s_w[e];
        }
        sum = warp_sum(sum);
        dot = warp_sum(dot);
        const bool none = sum == 0.0f;       // every logit is -inf: p = 0
        const float inv = none ? 0.0f : 1.0f / sum;
        dot *= inv;
        if (!none) acc += (double)(mean + dot);
        if (grad != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (e < E) store1<DT>(grad, tok * E + e, g * (p[i] * inv) * (s_w[e] - dot) * gate[i]);
            }
        }
    }
    if (loss_part != nullptr) {
        if (lane == 0) s_loss[warp] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
            double v = 0.0;
            for (int i = 0; i < kMainWarps; ++i) v += s_loss[i];
            loss_part[blockIdx.x] = v;
        }
    }
}

__global__ void __launch_bounds__(256) balance_sum_kernel(const double *__restrict__ part, int64_t n,
                                                          float *__restrict__ loss) {
    __shared__ double s[256];
    griddep_wait();
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) v += part[i];
    s[threadIdx.x] = v;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) *loss = (float)s[0];
}

size_t round16(size_t v) { return (v + 15) / 16 * 16; }

template <int DT, int V>
cudaError_t launch_main(const Shape &s, const void *logits, const int32_t *idx, double scale, int sigmoid,
                        const int32_t *part, int chunks, int32_t *counts, int32_t *routed, const float *grad_loss,
                        void *grad, double *loss_part, cudaStream_t stream) {
    return launch_pdl(balance_main_kernel<DT, V>, dim3((unsigned)(s.seqs * s.main_chunks)), dim3(kMainThreads),
                      (size_t)s.E * 4, stream, logits, idx, s.tokens, s.k, s.E, scale, sigmoid, part, chunks, counts,
                      routed, grad_loss, grad, loss_part, s.main_chunks);
}

template <int DT, typename... A>
cudaError_t main_by_width(const Shape &s, A... a) {
    if (s.E <= 32) return launch_main<DT, 1>(s, a...);
    if (s.E <= 64) return launch_main<DT, 2>(s, a...);
    if (s.E <= 128) return launch_main<DT, 4>(s, a...);
    if (s.E <= 256) return launch_main<DT, 8>(s, a...);
    if (s.E <= 512) return launch_main<DT, 16>(s, a...);
    return launch_main<DT, 32>(s, a...);
}

template <typename... A>
cudaError_t main_by_type(int dtype, const Shape &s, A... a) {
    switch (dtype) {
        case CGL_BF16: return main_by_width<CGL_BF16>(s, a...);
        case CGL_F16: return main_by_width<CGL_F16>(s, a...);
        default: return main_by_width<CGL_F32>(s, a...);
    }
}

}  // namespace

size_t balance_workspace_bytes(int64_t n, int k, int E, int64_t S) {
    const Shape s = shape(n, k, E, S);
    return round16((size_t)S * s.count_chunks * (E + 1) * 4) + (size_t)S * s.main_chunks * 8;
}

cgl_status launch_balance_loss(const void *logits, int dtype, const int32_t *idx, int64_t n, int k, int E, int64_t S,
                               float alpha, int score, const float *grad_loss, float *loss, int32_t *counts,
                               int32_t *routed, void *grad, void *ws, uint32_t *status, cudaStream_t stream) {
    const Shape s = shape(n, k, E, S);
    int32_t *part = static_cast<int32_t *>(ws);
    double *loss_part =
        reinterpret_cast<double *>(static_cast<uint8_t *>(ws) + round16((size_t)S * s.count_chunks * (E + 1) * 4));
    if (launch_pdl(balance_count_kernel, dim3((unsigned)(S * s.count_chunks)), dim3(kCountThreads), (size_t)(E + 1) * 4,
                   stream, idx, s.tokens, k, E, s.count_chunks, s.count_tokens, part, status) != cudaSuccess)
        return CGL_ECUDA;
    if (main_by_type(dtype, s, logits, idx, (double)alpha / ((double)S * k), score, (const int32_t *)part,
                     s.count_chunks, counts, routed, grad_loss, grad, loss_part, stream) != cudaSuccess)
        return CGL_ECUDA;
    return launch_pdl(balance_sum_kernel, dim3(1), dim3(256), 0, stream, loss_part, S * s.main_chunks, loss) ==
                   cudaSuccess ? CGL_OK : CGL_ECUDA;
}

cgl_status launch_balance_loss_backward(const float *grad_loss, const void *logits, int dtype, const int32_t *idx,
                                        int64_t n, int k, int E, int64_t S, float alpha, int score,
                                        const int32_t *counts, const int32_t *routed, void *grad, cudaStream_t stream) {
    if (n == 0) return CGL_OK;
    const Shape s = shape(n, k, E, S);
    return main_by_type(dtype, s, logits, idx, (double)alpha / ((double)S * k), score, (const int32_t *)nullptr, 0,
                        const_cast<int32_t *>(counts), const_cast<int32_t *>(routed), grad_loss, grad,
                        (double *)nullptr, stream) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
