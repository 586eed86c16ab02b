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
// Two kernels: histograms of id chunks (shared-memory integer atomics, whose
// order has no effect; clusters of eight blocks add theirs up through distributed
// shared memory), then the pass over the logits, where every block first
// sums the clusters' counts for itself and the last block to finish adds up the
// blocks' loss sums in their order.  The grid goes by the sizes alone, so equal
// inputs give equal bits.
//
// The pass is bound by the bytes of the logits and the gradient, and close
// behind by its instructions: a lane holds 8 neighbouring experts (one 16-byte
// load of 16-bit logits) and their weights in registers, 2 to 32 lanes share a
// token, the exponential is one ex2, and the next token's logits are loaded
// ahead.  Where E % 8 != 0 or the rows are not 16-byte aligned a lane holds
// experts l, l + 32, ... instead.
#include "mxfp4.cuh"
#include "launch.h"

namespace cgl {

namespace {

constexpr int kCountThreads = 512;
constexpr int kMainThreads = 256;
constexpr int kMainWarps = kMainThreads / 32;
constexpr int64_t kMaxBlocks = 592;    // 148 SMs x 4 blocks; a constant, so sums do not depend on the device
constexpr int64_t kChunkIds = 4096;    // ids a histogram block
constexpr int kCluster = 8;            // histogram blocks a cluster, where a sequence has more than one
constexpr int kMaxParts = 16;          // clusters a sequence
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = 1048576.0f;     // 2^20, see the softmax

struct Shape {
    int64_t tokens;      // per sequence
    int64_t seqs;
    int k, E;
    int count_chunks;    // histogram blocks per sequence: 1, or a multiple of kCluster
    int parts;           // sums per sequence that they leave
    int64_t count_tokens;
    int main_chunks;     // blocks per sequence of the main pass
};

// The vector form: lanes that share a token, and groups of 8 experts a lane.
// 16-bit logits of many tokens take two groups a lane where there are over 8
// (half the lanes, one shuffle round less for two tokens at once).  BF16, 256
// experts, loss and gradient as two calls, one group and two: 4096 tokens 13.4 and
// 12.3 us, 8192 15.6 and 15.1, 12288 19.3 and 17.7, 65536 49.5 and 40.2; with 128
// experts 11.3 and 10.8, 13.5 and 12.3, 15.3 and 14.5, 29.6 and 25.0.  So the border is
// where the gain is sure, not where it begins; with the sigmoid 4096 tokens gain
// nothing (12.5 and 12.6).  Binary32 logits need the registers for occupancy (36 and 40).
constexpr int64_t kManyTokens = 12288;
struct Width { int lanes, groups; };
Width width_for(int64_t n, int E, int dtype) {
    const int groups = (E + 7) / 8;
    Width w = {1, 1};
    if (dtype != CGL_F32 && n >= kManyTokens && groups > 8) w.groups = 2;
    while (w.lanes < 32 && w.lanes * w.groups < groups) w.lanes *= 2;
    while (w.lanes * w.groups < groups) w.groups *= 2;
    return w;
}

Shape shape(int64_t n, int k, int E, int64_t S, int dtype) {
    Shape s;
    s.tokens = n / S;
    s.seqs = S;
    s.k = k;
    s.E = E;
    // fit: blocks of the main pass a sequence.  Just past a divisor of kMaxBlocks it
    // leaves some unused (65536 x 256 BF16, loss: 296 sequences 20.1 us, 297 26.2, 592
    // 21.8), just past kMaxBlocks there is a second wave (593: 25.4).
    const int64_t want = (s.tokens * k + kChunkIds - 1) / kChunkIds, fit = kMaxBlocks / S > 0 ? kMaxBlocks / S : 1;
    int64_t c = 1;
    if (want > 1 && S * kCluster <= 2 * kMaxBlocks) {   // 2: a block has little to do
        const int64_t most = 2 * fit / kCluster > 1 ? 2 * fit / kCluster : 1;
        c = (want + kCluster - 1) / kCluster;
        c = (c < most ? c : most) < kMaxParts ? (c < most ? c : most) : kMaxParts;
        s.parts = (int)c;
        c *= kCluster;
    } else {
        s.parts = 1;
    }
    s.count_chunks = (int)c;
    s.count_tokens = (s.tokens + c - 1) / c;
    const int64_t at_once = kMainWarps * (E % 8 == 0 ? 32 / width_for(n, E, dtype).lanes : 1);   // tokens a block has in hand
    int64_t d = (s.tokens + at_once - 1) / at_once;
    if (d > fit) d = fit;
    s.main_chunks = d < 1 ? 1 : (int)d;
    return s;
}

// part[cluster][E + 1]: slots per expert, routed tokens.  ticket: zeroed for the main kernel.
__global__ void __launch_bounds__(kCountThreads)
balance_count_kernel(const int32_t *__restrict__ idx, int64_t tokens, int k, int E, int chunks, int64_t per_chunk,
                     int32_t *__restrict__ part, uint32_t *__restrict__ ticket, uint32_t *status) {
    extern __shared__ int32_t s_count[];
    griddep_wait();
    // The main kernel's blocks may come now: what they read before their own
    // wait is the logits and ids, and those are there, since this block's wait is over.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
    for (int e = threadIdx.x; e <= E; e += kCountThreads) s_count[e] = 0;
    __syncthreads();
    const int64_t seq = blockIdx.x / chunks, c = blockIdx.x % chunks;
    const int64_t t0 = c * per_chunk, t1 = t0 + per_chunk < tokens ? t0 + per_chunk : tokens;
    const bool vec = (k & 3) == 0 && (reinterpret_cast<uintptr_t>(idx) & 15) == 0;
    bool bad = false;
    int routed = 0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kCountThreads) {
        const int32_t *p = idx + (seq * tokens + t) * k;
        bool any = false;
        for (int j = 0; j < k; j += 8) {   // the loads of 8 slots before the first of them is used
            int32_t id[8];
            if (vec) {
                const int4 a = __ldg(reinterpret_cast<const int4 *>(p + j));
                const int4 b = j + 4 < k ? __ldg(reinterpret_cast<const int4 *>(p + j) + 1) : make_int4(-1, -1, -1, -1);
                id[0] = a.x, id[1] = a.y, id[2] = a.z, id[3] = a.w, id[4] = b.x, id[5] = b.y, id[6] = b.z, id[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) id[i] = j + i < k ? __ldg(p + j + i) : -1;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (id[i] >= 0 && id[i] < E) {
                    atomicAdd(&s_count[id[i]], 1);
                    any = true;
                } else if (id[i] != -1) {
                    bad = true;
                }
            }
        }
        routed += any;
    }
    routed = __reduce_add_sync(0xFFFFFFFFu, routed);   // behind the loop, which lanes leave apart: all 32 are here
    if ((threadIdx.x & 31) == 0 && routed > 0) atomicAdd(&s_count[E], routed);
    if (chunks == 1) {
        __syncthreads();
        for (int e = threadIdx.x; e <= E; e += kCountThreads) part[(int64_t)blockIdx.x * (E + 1) + e] = s_count[e];
    } else {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int e = blockIdx.x % kCluster + threadIdx.x * kCluster; e <= E; e += kCountThreads * kCluster) {
            int32_t sum = 0;
#pragma unroll
            for (int r = 0; r < kCluster; ++r) {
                int32_t v;
                asm volatile(
                    "{\n.reg .b32 a;\n"
                    "mapa.shared::cluster.u32 a, %1, %2;\n"
                    "ld.shared::cluster.s32 %0, [a];\n}"
                    : "=r"(v)
                    : "r"((uint32_t)__cvta_generic_to_shared(s_count + e)), "r"(r)
                    : "memory");
                sum += v;
            }
            part[(int64_t)(blockIdx.x / kCluster) * (E + 1) + e] = sum;
        }
        __syncwarp();   // no block leaves while another reads its counts
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (bad) report(status, kErrRange);
}

// 2^x; with FTZ results below 2^-126 are 0, without it they are subnormal.
template <bool FTZ>
__device__ __forceinline__ float ex2(float x) {
    float r;
    if (FTZ) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    else asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / x for x in [1, 2], within one step.
__device__ __forceinline__ float rcp12(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// A token's logits in one lane: N groups of eight neighbours (VEC), or N single experts 32 apart.
template <int DT, int LANES, int N, bool VEC>
struct Row {
    static constexpr int V = VEC ? 8 * N : N;
    Vec8<DT> raw[VEC ? N : 1];
    float one[VEC ? 1 : N];

    static __device__ __forceinline__ int expert(int lane, int i) {
        return VEC ? ((i / 8) * LANES + lane) * 8 + i % 8 : lane + 32 * i;
    }
    // Where expert e's weight stands in shared memory: four of a lane's eight
    // side by side, the lanes' fours side by side, so that a 16-byte read of all
    // lanes meets each bank once a phase.
    static __device__ __forceinline__ int place(int e) {
        if (!VEC) return e;
        const int i = e & 7, g = e >> 3;
        return ((g / LANES * 2 + (i >> 2)) * LANES + g % LANES) * 4 + (i & 3);
    }
    static __device__ __forceinline__ void weights(const float *s_w, int lane, int c, float w[8]) {
        if (VEC) {
            *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(s_w + ((c * 2) * LANES + lane) * 4);
            *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(s_w + ((c * 2 + 1) * LANES + lane) * 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 8 * c + i < N ? s_w[lane + 32 * (8 * c + i)] : 0.0f;
        }
    }
    __device__ __forceinline__ void load(const void *p, int64_t tok, int E, int lane) {
        if (VEC) {
#pragma unroll
            for (int c = 0; c < N; ++c)
                if (expert(lane, 8 * c) < E) raw[c].load(p, (tok * E + expert(lane, 8 * c)) >> 3);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (expert(lane, i) < E) one[i] = load1<DT>(p, tok * E + expert(lane, i));
        }
    }
    __device__ __forceinline__ void widen(float l[V], int E, int lane) const {
        if (VEC) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
                raw[c].widen(l + 8 * c);
                if (expert(lane, 8 * c) >= E)
#pragma unroll
                    for (int i = 0; i < 8; ++i) l[8 * c + i] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = expert(lane, i) < E ? one[i] : -INFINITY;
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t tok, int E, int lane, const float v[V]) {
        if (VEC) {
#pragma unroll
            for (int c = 0; c < N; ++c)
                if (expert(lane, 8 * c) < E) Vec8<DT>::store(p, (tok * E + expert(lane, 8 * c)) >> 3, v + 8 * c);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (expert(lane, i) < E) store1<DT>(p, tok * E + expert(lane, i), v[i]);
        }
    }
};

// LANES lanes a token.  part: the count kernel's sums (chunks a sequence), or null,
// chunks 0, and counts / routed as the forward gave them (loss_part null then).
template <int DT, int LANES, int N, bool VEC, bool SIG>
__global__ void __launch_bounds__(kMainThreads, Row<DT, LANES, N, VEC>::V <= 16 ? 4 : 1)   // 4: the grid is one wave
balance_main_kernel(const void *__restrict__ logits, const int32_t *__restrict__ idx, int64_t tokens, int k, int E,
                    double scale, const int32_t *__restrict__ part, int chunks, int32_t *counts,
                    int32_t *routed, const float *__restrict__ grad_loss, void *__restrict__ grad, double *loss_part,
                    uint32_t *ticket, float *loss, int main_chunks) {
    using R = Row<DT, LANES, N, VEC>;
    constexpr int V = R::V, kTokens = 32 / LANES;   // tokens a warp has in hand
    extern __shared__ __align__(16) float s_w[];    // [V * LANES] weights less their mean, then [E] counts
    __shared__ unsigned long long s_total;
    __shared__ int s_routed;
    __shared__ double s_loss[kMainWarps];
    __shared__ bool s_last;
    if (chunks == 0) griddep_wait();
    const int64_t seq = blockIdx.x / main_chunks;
    const int chunk = (int)(blockIdx.x % main_chunks);
    const int lane = threadIdx.x % LANES, warp = threadIdx.x >> 5;
    const int64_t step = (int64_t)main_chunks * kMainWarps * kTokens;
    int64_t r = ((int64_t)chunk * kMainWarps + warp) * kTokens + (threadIdx.x & 31) / LANES;
    R row;
    int32_t id = -1;   // the lane's first slot, with the row
    if (r < tokens && lane < k) id = __ldg(idx + (seq * tokens + r) * k + lane);
    if (r < tokens) row.load(logits, seq * tokens + r, E, lane);   // in flight through the weights
    if (chunks > 0) griddep_wait();   // the counts (see balance_count_kernel on the logits)
    int32_t *s_c = reinterpret_cast<int32_t *>(s_w + V * LANES);
    if (threadIdx.x == 0) s_total = 0;
    __syncthreads();
    unsigned long long mine = 0;
    for (int e = threadIdx.x; e <= E; e += kMainThreads) {
        int32_t c = 0;
        if (chunks > 0) {
            const int32_t *q = part + seq * chunks * (E + 1) + e;
#pragma unroll 16
            for (int i = 0; i < chunks; ++i) c += q[(int64_t)i * (E + 1)];
        } else {
            c = e < E ? counts[seq * E + e] : routed[seq];
        }
        if (e < E) {
            s_c[e] = c;
            mine += c;
            if (chunks > 0 && chunk == 0) counts[seq * E + e] = c;
        } else {
            s_routed = c;
            if (chunks > 0 && chunk == 0) routed[seq] = c;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s_total, mine);
    __syncthreads();
    const long long total = (long long)s_total;
    const double t = (double)s_routed, unit = t > 0 ? scale / (t * t) : 0.0;   // scale = alpha / (S k)
    const float mean = (float)(unit * (double)total);
    for (int e = threadIdx.x; e < V * LANES; e += kMainThreads)
        s_w[R::place(e)] = e < E ? (float)(unit * (double)((long long)E * s_c[e] - total)) : 0.0f;
    __syncthreads();
    const float g = grad != nullptr && grad_loss != nullptr ? __ldg(grad_loss) : 1.0f;
    double acc = 0.0;
    for (; __any_sync(0xFFFFFFFFu, r < tokens); r += step) {
        const bool here = r < tokens;
        const int64_t tok = seq * tokens + r;
        float l[V], p[V];
        row.widen(l, here ? E : 0, lane);
        bool any = here && id >= 0 && id < E;
        if (r + step < tokens) {
            if (lane < k) id = __ldg(idx + (tok + step) * k + lane);
            row.load(logits, tok + step, E, lane);
        }
        for (int j = lane + LANES; here && j < k; j += LANES) {
            const int32_t e = __ldg(idx + tok * k + j);
            any = any || (e >= 0 && e < E);
        }
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, any);
        any = ((votes >> ((threadIdx.x & 31) / LANES * LANES)) & (LANES == 32 ? 0xFFFFFFFFu : (1u << (LANES & 31)) - 1u)) != 0;
        float m = -INFINITY, low = INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m = fmaxf(m, l[i]);
            low = fminf(low, SIG ? -fabsf(l[i]) : l[i]);
        }
        m = group_max<LANES>(m);
        if (m == -INFINITY) m = 0.0f;        // nothing left (or NaN): exp(-inf) below, not exp(nan)
        float sum = 0.0f, dot = 0.0f;
        if (!SIG) {
            // The shift's rounding is a factor that all p share: at most 2^(2^-4) up
            // to |m| = kFar.  Past it that factor would leave binary32's range, so
            // there the difference is taken first.
            const bool far = fabsf(m) > kFar;
            const float base = far ? m : 0.0f, shift = far ? 0.0f : -m * kLog2e;
            if (__any_sync(0xFFFFFFFFu, far || fmaf(low, kLog2e, shift) < -125.0f)) {
#pragma unroll
                for (int i = 0; i < V; ++i) p[i] = ex2<false>(fmaf(l[i] - base, kLog2e, shift));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) p[i] = ex2<true>(fmaf(l[i], kLog2e, shift));
            }
        } else {
            // sigmoid(l) exp(-m) with m = min(max l, 0): the common factor keeps p
            // where every sigmoid underflows.  l becomes the slope 1 - sigmoid(l).
            m = fminf(m, 0.0f);
            if (__any_sync(0xFFFFFFFFu, m < 0.0f || low < -86.0f)) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool up = l[i] > 0.0f;
                    const float z = ex2<false>(-fabsf(l[i]) * kLog2e), d = rcp12(1.0f + z);
                    p[i] = (up ? 1.0f : ex2<false>((l[i] - m) * kLog2e)) * d;
                    l[i] = (up ? z : 1.0f) * d;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool up = l[i] > 0.0f;
                    const float z = ex2<true>(-fabsf(l[i]) * kLog2e), d = rcp12(1.0f + z);
                    p[i] = (up ? 1.0f : z) * d;
                    l[i] = (up ? z : 1.0f) * d;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < (V + 7) / 8; ++c) {
            float w[8];
            R::weights(s_w, lane, c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (8 * c + i < V) {
                    sum += p[8 * c + i];
                    dot = fmaf(p[8 * c + i], w[i], dot);
                }
            }
        }
        sum = group_sum<LANES>(sum);
        dot = group_sum<LANES>(dot);
        // Every logit -inf (else the largest one's term is 0.4 or more), or a token without a copy.
        const bool none = sum == 0.0f || !any;
        const float inv = none ? 0.0f : __fdiv_rn(1.0f, sum);
        dot = none ? 0.0f : dot * inv;
        if (!none && lane == 0) acc += (double)(mean + dot);
        if (grad != nullptr && here) {
            const float gi = g * inv, gd = -gi * dot;
#pragma unroll
            for (int c = 0; c < (V + 7) / 8; ++c) {
                float w[8];
                R::weights(s_w, lane, c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (8 * c + i < V) {
                        const float q = p[8 * c + i] * fmaf(w[i], gi, gd);
                        p[8 * c + i] = none ? 0.0f : SIG ? q * l[8 * c + i] : q;   // 0 for NaN too where the token takes no part
                    }
                }
            }
            R::store(grad, tok, E, lane, p);
        }
    }
    if (loss_part == nullptr) return;
#pragma unroll
    for (int o = 16; o >= LANES && o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    if ((threadIdx.x & 31) == 0) s_loss[warp] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int i = 0; i < kMainWarps; ++i) v += s_loss[i];
        loss_part[blockIdx.x] = v;
        __threadfence();
        s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double v = 0.0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kMainThreads) v += *(volatile double *)(loss_part + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s_loss[warp] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
        for (int i = 0; i < kMainWarps; ++i) v += s_loss[i];
        *loss = (float)v;
    }
}

size_t round16(size_t v) { return (v + 15) / 16 * 16; }

struct Args {
    const void *logits;
    const int32_t *idx;
    double scale;
    int score;
    const int32_t *part;
    int chunks;
    int32_t *counts, *routed;
    const float *grad_loss;
    void *grad;
    double *loss_part;
    uint32_t *ticket;
    float *loss;
    cudaStream_t stream;
};

template <int DT, int LANES, int N, bool VEC>
cudaError_t launch_main(const Shape &s, const Args &a) {
    const size_t smem = (size_t)(LANES * N * (VEC ? 8 : 1) + s.E) * 4;
    const auto kernel = a.score == CGL_SCORE_SIGMOID ? balance_main_kernel<DT, LANES, N, VEC, true>
                                                     : balance_main_kernel<DT, LANES, N, VEC, false>;
    return launch_pdl(kernel, dim3((unsigned)(s.seqs * s.main_chunks)), dim3(kMainThreads), smem, a.stream, a.logits, a.idx,
                      s.tokens, s.k, s.E, a.scale, a.part, a.chunks, a.counts, a.routed, a.grad_loss, a.grad, a.loss_part,
                      a.ticket, a.loss, s.main_chunks);
}

template <int DT>
cudaError_t main_by_width(const Shape &s, const Args &a) {
    if (s.E % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.grad)) & 15) == 0) {
        const Width w = width_for(s.tokens * s.seqs, s.E, DT);
        switch (w.lanes * 8 + w.groups) {
            case 1 * 8 + 1: return launch_main<DT, 1, 1, true>(s, a);
            case 2 * 8 + 1: return launch_main<DT, 2, 1, true>(s, a);
            case 4 * 8 + 1: return launch_main<DT, 4, 1, true>(s, a);
            case 8 * 8 + 1: return launch_main<DT, 8, 1, true>(s, a);
            case 8 * 8 + 2: return launch_main<DT, 8, 2, true>(s, a);
            case 16 * 8 + 1: return launch_main<DT, 16, 1, true>(s, a);
            case 16 * 8 + 2: return launch_main<DT, 16, 2, true>(s, a);
            case 32 * 8 + 1: return launch_main<DT, 32, 1, true>(s, a);
            case 32 * 8 + 2: return launch_main<DT, 32, 2, true>(s, a);
            default: return launch_main<DT, 32, 4, true>(s, a);
        }
    }
    if (s.E <= 32) return launch_main<DT, 32, 1, false>(s, a);
    if (s.E <= 128) return launch_main<DT, 32, 4, false>(s, a);
    if (s.E <= 256) return launch_main<DT, 32, 8, false>(s, a);
    return launch_main<DT, 32, 32, false>(s, a);
}

cudaError_t main_by_type(int dtype, const Shape &s, const Args &a) {
    switch (dtype) {
        case CGL_BF16: return main_by_width<CGL_BF16>(s, a);
        case CGL_F16: return main_by_width<CGL_F16>(s, a);
        default: return main_by_width<CGL_F32>(s, a);
    }
}

}  // namespace

// The ticket (16 bytes), the blocks' loss sums, the chunks' counts.
size_t balance_workspace_bytes(int64_t n, int k, int E, int64_t S) {
    const Shape s = shape(n, k, E, S, CGL_F32), h = shape(n, k, E, S, CGL_BF16);   // types may differ in their blocks
    const int blocks = s.main_chunks > h.main_chunks ? s.main_chunks : h.main_chunks;
    return 16 + round16((size_t)S * blocks * 8) + (size_t)S * s.parts * (E + 1) * 4;
}

cgl_status launch_balance_loss(const void *logits, int dtype, const int32_t *idx, int64_t n, int k, int E, int64_t S,
                               float alpha, int score, const float *grad_loss, float *loss, int32_t *counts,
                               int32_t *routed, void *grad, void *ws, uint32_t *status, cudaStream_t stream) {
    const Shape s = shape(n, k, E, S, dtype);
    uint32_t *ticket = static_cast<uint32_t *>(ws);
    double *loss_part = reinterpret_cast<double *>(static_cast<uint8_t *>(ws) + 16);
    int32_t *part = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + 16 + round16((size_t)S * s.main_chunks * 8));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(S * s.count_chunks));
    cfg.blockDim = dim3(kCountThreads);
    cfg.dynamicSmemBytes = (size_t)(E + 1) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = s.count_chunks > 1 ? kCluster : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, balance_count_kernel, idx, s.tokens, k, E, s.count_chunks, s.count_tokens, part, ticket,
                           status) != cudaSuccess)
        return CGL_ECUDA;
    const Args a = {logits, idx, (double)alpha / ((double)S * k), score, part, s.parts, counts, routed,
                    grad_loss, grad, loss_part, ticket, loss, stream};
    return main_by_type(dtype, s, a) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

cgl_status launch_balance_loss_backward(const float *grad_loss, const void *logits, int dtype, const int32_t *idx,
                                        int64_t n, int k, int E, int64_t S, float alpha, int score,
                                        const int32_t *counts, const int32_t *routed, void *grad, cudaStream_t stream) {
    if (n == 0) return CGL_OK;
    const Shape s = shape(n, k, E, S, dtype);
    const Args a = {logits, idx, (double)alpha / ((double)S * k), score, nullptr, 0, const_cast<int32_t *>(counts),
                    const_cast<int32_t *>(routed), grad_loss, grad, nullptr, nullptr, nullptr, stream};
    return main_by_type(dtype, s, a) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
