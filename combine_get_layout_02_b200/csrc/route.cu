// Routing: top-k experts of every token and their weights, and the gradient of
// the weights for the logits (formulas at cgl_route in cgl.h).
//
// One warp a token.  A lane turns its eight neighbouring logits (up to 256 experts; one,
// four, 16 or 32 for other numbers) into 32-bit keys and sorts them by a network; k
// rounds of a warp maximum (redux) pick the experts, the winner's lane popping its
// list.  Four tokens share a warp's lanes for what only the picks need.  Choices that
// 32 bits cannot put in order are compared in binary64, so ids are the definition's.
//
// What bounds it (B200, replayed from a graph; 65536 x 256 BF16, top-8, 33.5 MB or 5.1 us
// of logits): instructions.  Forward 23.7 us, softmax as it is 29.5: 255 instructions a
// token, 163 of them on the integer pipe, which issues every other cycle (65% of cycles
// issue).  A warp takes a token whatever the experts: 64 or 128 of them 26 us.  With a
// bias and sigmoid 40 (480 instructions); binary32, bias, 8 groups by pairs 62 (739); 160
// experts in 8 groups, which do not fill lanes and go through shared memory, 57 (682); 16384
// x 512 25 (910: lists past eight a lane are scanned for every pick).  Backward 11.4 us
// renormalised (floor 6.4 with ids and gradients; 103 instructions, and 46% of an SM's
// warps at 64 registers), 19.4 for the whole softmax (11.5), where each logit's exponential
// is made twice for want of registers.  128 tokens 2.4 to 3.1 us.  16-bit logits with top-8
// and neither bias nor groups spill nothing; most other kernels up to 256 experts up to 104
// bytes a thread (64 or 80 registers for four or three blocks an SM), past 512 experts up
// to 432 at 128 registers.
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

// Sixteen bytes of neighbours: four binary32 or eight 16-bit values.
template <int DT>
__device__ __forceinline__ uint4 pack(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == CGL_F32) w[i] = __float_as_uint(v[i]);
        else if (DT == CGL_BF16) w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
        else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// Which groups stay, in binary64: a bit each.  Lanes share the groups out, a power of two of them a group.
template <int DT>
__device__ __noinline__ uint32_t groups_exact(const RouteArgs &a, const void *row) {
    const int lane = threadIdx.x & 31, E = a.E, per = E / a.groups;
    double m = -INFINITY, sum = 0.0;
    const bool softmax = a.score == CGL_SCORE_SOFTMAX, scored = a.bias != nullptr || a.by == CGL_GROUP_TOP2;
    if (softmax && scored) {
        for (int e = lane; e < E; e += 32) m = fmax(m, (double)logit<DT>(row, e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
#pragma unroll 2
        for (int e = lane; e < E; e += 32) {
            const double l = (double)logit<DT>(row, e);
            if (l > -INFINITY) sum += exp(l - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    int share = 32;
    while (share * a.groups > 32) share /= 2;
    const int g = lane / share;
    double first = -INFINITY, second = -INFINITY;
    if (g < a.groups)
#pragma unroll 2
        for (int i = lane % share; i < per; i += share) {
            const int e = g * per + i;
            double v = (double)logit<DT>(row, e);
            if (scored && v > -INFINITY) {
                v = softmax ? exp(v - m) / sum : 1.0 / (1.0 + exp(-v));
                if (a.bias != nullptr) v += (double)__ldg(a.bias + e);
            }
            second = fmax(second, fmin(first, v));
            first = fmax(first, v);
        }
    for (int o = 1; o < share; o <<= 1) {
        const double u = __shfl_xor_sync(kAll, first, o), v = __shfl_xor_sync(kAll, second, o);
        second = fmax(fmin(first, u), fmax(second, v));
        first = fmax(first, u);
    }
    const double value = a.by == CGL_GROUP_TOP2 && second > -INFINITY ? first + second : first;
    int rank = 0;
    for (int i = 0; i < a.groups; ++i) {
        const double v = __shfl_sync(kAll, value, i * share);
        rank += v > value || (v == value && i < g);
    }
    const bool kept = g < a.groups && value > -INFINITY && rank < a.keep;
    uint32_t open = 0;
    for (int i = 0; i < a.groups; ++i) open |= (uint32_t)__shfl_sync(kAll, (int)kept, i * share) << i;
    return open;
}

// Over the lanes of the picks: the first eight (size 4) or all (16).
__device__ __forceinline__ float picks_sum(float v, int size) {
    for (int o = size; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float picks_max(float v, int size) {
    for (int o = size; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// 1 / x, within a step.
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What lane j's slot has of its token's weight (scale aside), slots without an expert
// 0: the sigmoid, or with renorm the quotient by the picks' sum (softmax or sigmoid).
__device__ __forceinline__ float share(int score, bool renorm, bool there, float l, int size) {
    const float top = renorm ? picks_max(there ? l : -INFINITY, size) : 0.0f;
    float t;
    if (score == CGL_SCORE_SIGMOID) {
        // sigmoid(l) exp(-b), b = min(largest l, 0): a factor that all slots share keeps the quotient where every sigmoid underflows
        const float b = fminf(top, 0.0f), z = expf(-fabsf(l));
        t = l > 0.0f ? 1.0f : z;
        if (__any_sync(kAll, b < 0.0f)) t = l > 0.0f ? 1.0f : expf(l - b);
        t *= rcp(1.0f + z);
    } else {
        t = expf(l - top);
    }
    if (!there || l == -INFINITY) t = 0.0f;
    if (!renorm) return t;
    const float d = picks_sum(t, size);
    return d == 0.0f ? 0.0f : t * rcp(d);
}

// ---- the order in binary32, by keys ------------------------------------------------------------

// 32-bit keys in the order of floats: the sign flipped, negative values reversed.  The
// addition makes +0 of -0, which is equal to it and would stand below it by its bits.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two 16-bit values, -0 made +0; every other value as it is (a NaN's bits may change).
template <int DT>
__device__ __forceinline__ uint32_t one_zero(uint32_t w) {
    uint32_t r;
    if (DT == CGL_F16) asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0u));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0x3F803F80u), "r"(0u));   // w * 1 + 0
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// The same of a 16-bit value, which `f` holds.
template <int DT>
__device__ __forceinline__ uint32_t ordered16(float f) {
    f += 0.0f;
    const uint32_t u = DT == CGL_F16 ? __half_as_ushort(__float2half_rn(f)) : __float_as_uint(f) >> 16;
    return u ^ (u & 0x8000u ? 0xFFFFu : 0x8000u);
}

// A lane's V neighbouring logits, VEC in pieces of eight.
template <int DT, int V, bool VEC>
struct Row {
    uint4 raw[VEC ? V / 8 : 1][DT == CGL_F32 ? 2 : 1];
    float one[VEC ? 1 : V];
    __device__ __forceinline__ void load(const void *row, int E, int lane) {
        if (VEC) {
#pragma unroll
            for (int c = 0; c < V / 8; ++c)
                if (lane * V + 8 * c < E)
#pragma unroll
                    for (int h = 0; h < (DT == CGL_F32 ? 2 : 1); ++h)   // kept in L1: the picks' logits are read again
                        raw[c][h] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (lane * V + 8 * c) * (DT == CGL_F32 ? 4 : 2)) + h);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane * V + i < E) one[i] = logit<DT>(row, lane * V + i);
        }
    }
    // Whether one is not a number.
    __device__ __forceinline__ bool nan(int E, int lane) const {
        bool bad = false;
        if (VEC) {
            constexpr uint32_t kAbs = DT == CGL_F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu, kInf = DT == CGL_F16 ? 0x7C00u : 0x7F80u;
#pragma unroll
            for (int c = 0; c < V / 8; ++c) {
                uint32_t m = 0;
#pragma unroll
                for (int h = 0; h < (DT == CGL_F32 ? 2 : 1); ++h) {
                    const uint4 q = raw[c][h];
                    if (DT == CGL_F32) m = max(m, max(max(q.x & kAbs, q.y & kAbs), max(q.z & kAbs, q.w & kAbs)));
                    else m = __vmaxu2(__vmaxu2(q.x & kAbs, q.y & kAbs), __vmaxu2(q.z & kAbs, q.w & kAbs));
                }
                const bool hit = DT == CGL_F32 ? m > 0x7F800000u : (m >> 16) > kInf || (m & 0xFFFFu) > kInf;
                bad = bad || (hit && lane * V + 8 * c < E);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) bad = bad || (lane * V + i < E && one[i] != one[i]);
        }
        return bad;
    }
    // The keys of 16-bit logits: their order above, code - i below.
    __device__ __forceinline__ void keys(uint32_t key[V], int E, int lane, uint32_t code) const {
#pragma unroll
        for (int c = 0; c < (VEC ? V / 8 : 0); ++c) {
            const uint32_t w[4] = {one_zero<DT>(raw[c][0].x), one_zero<DT>(raw[c][0].y), one_zero<DT>(raw[c][0].z), one_zero<DT>(raw[c][0].w)};
            const bool there = lane * V + 8 * c < E;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t minus = ((w[i] >> 15) & 0x00010001u) * 0xFFFFu, x = there ? w[i] ^ (minus | 0x80008000u) : 0u;
                key[8 * c + 2 * i] = __byte_perm(x, code - 8 * c - 2 * i, 0x1054);       // the low half's
                key[8 * c + 2 * i + 1] = __byte_perm(x, code - 8 * c - 2 * i - 1, 0x3254);
            }
        }
    }
    __device__ __forceinline__ void widen(float l[V], int E, int lane) const {
        if (VEC) {
#pragma unroll
            for (int c = 0; c < V / 8; ++c) {
                const uint32_t w[8] = {raw[c][0].x, raw[c][0].y, raw[c][0].z, raw[c][0].w, raw[c][DT == CGL_F32].x,
                                       raw[c][DT == CGL_F32].y, raw[c][DT == CGL_F32].z, raw[c][DT == CGL_F32].w};
                const bool there = lane * V + 8 * c < E;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float f;
                    if (DT == CGL_F32) f = __uint_as_float(w[i]);
                    else if (DT == CGL_BF16) f = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
                    else f = __half2float(__ushort_as_half((unsigned short)((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu)));
                    l[8 * c + i] = there ? f : -INFINITY;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = lane * V + i < E ? one[i] : -INFINITY;
        }
    }
};

// Descending, by a network (V <= 8); beyond, lists stay as they are and pop() looks for the next.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t k[V]) {
    const auto at = [&](int i, int j) {
        const uint32_t x = max(k[i], k[j]), y = min(k[i], k[j]);
        k[i] = x, k[j] = y;
    };
    if (V == 4) {
        at(0, 1), at(2, 3), at(0, 2), at(1, 3), at(1, 2);
    } else if (V == 8) {
        at(0, 2), at(1, 3), at(4, 6), at(5, 7);
        at(0, 4), at(1, 5), at(2, 6), at(3, 7);
        at(0, 1), at(2, 3), at(4, 5), at(6, 7);
        at(2, 4), at(3, 5);
        at(1, 4), at(3, 6);
        at(1, 2), at(3, 4), at(5, 6);
    }
}
// The lane's largest key, and a list without it.
template <int V>
__device__ __forceinline__ uint32_t head(const uint32_t k[V]) {
    if (V <= 8) return k[0];
    uint32_t m = k[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, k[i]);
    return m;
}
template <int V>
__device__ __forceinline__ void pop(uint32_t k[V], uint32_t top, int deep) {   // keys are unique; deep: how many are still of use
    if (V <= 8) {
        if (k[0] == top) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < deep) k[i] = i + 1 < V ? k[i + 1] : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) k[i] = k[i] == top ? 0 : k[i];
    }
}

// Keys hold the choice's first bits and, below, B bits that put lower indexes first.
// 16-bit logits without a bias are whole in their keys, of binary32 ones 32 - B bits
// are.  Choices with a bias lie between the least bias and the largest plus 1: they
// are held as parts of that range, 2^-23 of it (2^-22 past 256 experts), which near 1
// is finer than as many bits of a binary32 number.  Where what is cut off, or the
// choice's own rounding, could change the order (`near`: between neighbours of the
// order down to the first that is not picked), the candidates are compared again in
// binary64, all of them in lanes: one value a lane and not a whole row.  A NaN is
// found by its bits.
enum Kind { kPlain, kBias, kGroups, kGroupsBias };

template <int DT, int V, bool VEC, int K, int KIND>
__global__ void __launch_bounds__(kThreads, V > 8 ? 2 : KIND >= kGroups ? 3 : 4)
route_kernel(const RouteArgs a) {
    constexpr int B = V <= 8 ? 8 : 10;
    constexpr uint32_t kLow = (1u << B) - 1;
    __shared__ uint32_t s_group[kWarps][2][32];   // groups that do not fill whole lanes: their two largest keys
    griddep_wait();
    const int lane = threadIdx.x & 31, E = a.E, k = K > 0 ? K : a.k, warp = threadIdx.x >> 5;
    constexpr bool biased = KIND == kBias || KIND == kGroupsBias, groups = KIND >= kGroups;
    const bool softmax = a.score == CGL_SCORE_SOFTMAX;
    const bool whole = softmax && (biased || (groups && a.by == CGL_GROUP_TOP2));   // the softmax's sum before the choice
    constexpr bool exact = DT != CGL_F32 && !biased;
    // biases: their range, +infinity or NaN among them (the whole order in binary64), -infinity (never picked)
    float bias[V], from = 0.0f, unit = 0.0f, scale = 0.0f, slack = 0.0f;
    bool odd_bias = false;
    if (biased) {
        float least = INFINITY, most = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = lane * V + i < E ? __ldg(a.bias + lane * V + i) : -INFINITY;
            odd_bias = odd_bias || !(bias[i] < INFINITY);
            if (fabsf(bias[i]) < INFINITY) least = fminf(least, bias[i]), most = fmaxf(most, bias[i]);
        }
        least = -warp_max(-least), most = warp_max(most);
        const float range = most - least + 1.125f;
        odd_bias = __any_sync(kAll, odd_bias) || !(range < 0x1p60f && range > 0.0f);
        from = least - 0.0625f * range, unit = 1.125f * range * 0x1p-23f, scale = 1.0f / unit;
        // what a choice may be off by: its score and sum (2^-21, and a half step of the sum), its place in the range
        slack = 0x1p-20f + 0x1p-22f * (fabsf(from) + range) + (B > 8 ? 2.0f : 1.0f) * unit;
    }
    const float cut = biased ? 0.0f : __uint_as_float((127 - 22 + B) << 23);   // binary32 logits: what is cut off, of their size
    const uint32_t code = kLow - lane * V;           // less i: the low bits of the lane's i-th key
    const uint32_t prefix = exact ? 0xFFFF0000u : ~kLow;
    const uint32_t least = biased ? 0u : exact && DT == CGL_F16 ? 0x03FF0000u : 0x007FFFFFu & prefix;   // of -infinity
    const auto live = [&](uint32_t key) { return (key & prefix) > least; };
    const auto value_of = [&](uint32_t key) {
        if (DT == CGL_F16 && exact) return __half2float(__ushort_as_half((unsigned short)((key >> 16) ^ (key >> 31 ? 0x8000u : 0xFFFFu))));
        const float f = unordered(key & prefix);   // exact: below 16 bits a negative value's are ones
        return biased ? fmaf((float)(key >> 9), unit, from) : exact ? __uint_as_float(__float_as_uint(f) & 0xFFFF0000u) : f;
    };
    const int per = groups ? E / a.groups : E, lanes = per / V;   // lanes a group
    const bool filled = per % V == 0 && (lanes & (lanes - 1)) == 0;
    const bool pairs = groups && a.by == CGL_GROUP_TOP2;
    const int group = filled && groups ? lane / lanes : lane;   // whose value this lane holds
    const int size = k <= 8 ? 4 : 16;                // shuffles over the picks
    uint32_t packed[(V + 3) / 4] = {};               // the groups of the lane's experts, a byte each
    if (groups && !filled)
#pragma unroll
        for (int i = 0; i < V; ++i) packed[i / 4] |= (uint32_t)((lane * V + i) / per & 31) << (8 * (i % 4));
    const auto group_of = [&](int i) { return (packed[i / 4] >> (8 * (i % 4))) & 31; };
    // A warp takes `batch` tokens after one another and then, eight lanes a token, their weights at once.
    // One with groups, whose registers leave no room: binary32, 8 groups by maxima, 8192 x 256 10.2 us and four at once
    // 11.4, 16384 16.1 and 18.3, 65536 52.4 and 52.7; with a bias, by pairs, 13.8 and 14.2, 19.8 and 19.5, 61.6 and 59.7.
    const int batch = groups ? 1 : a.batch;
    const int64_t step = (int64_t)gridDim.x * kWarps * batch;
    const size_t row_bytes = (size_t)E * (DT == CGL_F32 ? 4 : 2);
    const char *const logits = static_cast<const char *>(a.logits);
    int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * batch;
    Row<DT, V, VEC> ahead;
    if (t0 < a.n) ahead.load(logits + t0 * row_bytes, E, lane);
    for (; t0 < a.n; t0 += step) {
        int picked = -1, failed = 0;       // of this lane's slot; failed: a bit a token
        float row_top = 0.0f, row_sum = 1.0f;
#pragma unroll 1
        for (int q = 0; q < batch && t0 + q < a.n; ++q) {
            const char *row = logits + (t0 + q) * row_bytes;
            uint32_t key[V];
            float l[V], top = -INFINITY, sum = 1.0f;
            bool bad = ahead.nan(E, lane);
            if (VEC && DT != CGL_F32 && exact) ahead.keys(key, E, lane, code);
            else ahead.widen(l, E, lane);
            const int64_t then = q + 1 < batch && t0 + q + 1 < a.n ? t0 + q + 1 : t0 + step;
            if (then < a.n) ahead.load(logits + then * row_bytes, E, lane);
            bad = __any_sync(kAll, bad);
            if (whole) {
                if (VEC && DT != CGL_F32 && exact) {
#pragma unroll
                    for (int i = 0; i < V; ++i) l[i] = live(key[i]) ? value_of(key[i]) : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
                top = warp_max(top);
                top = top == -INFINITY ? 0.0f : top;
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) sum += ex2((l[i] - top) * kLog2e);
                sum = warp_sum(sum);
            }
            const float inv = rcp(sum);
            const auto score = [&](float x) { return softmax ? ex2((x - top) * kLog2e) * inv : rcp(1.0f + ex2(-x * kLog2e)); };
            if (biased) {   // 2^23 + a number below 2^23: its bits are the place in the range
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float c = fmaf(score(l[i]) + bias[i] - from, scale, 0x1p23f);
                    key[i] = l[i] > -INFINITY && bias[i] > -INFINITY ? ((__float_as_uint(c) << 9) & ~kLow) | (code - i) : 0u;
                }
            } else if (!(VEC && DT != CGL_F32 && exact)) {
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = exact ? (ordered16<DT>(l[i]) << 16) | (code - i) : (ordered(l[i]) & ~kLow) | (code - i);
            }
            bool again = odd_bias;     // the whole token in binary64
            if (groups) {
                uint32_t first, second = 0;   // a group's two largest keys, in its lanes, or in lane g that of group g
                if (filled) {
                    if (V <= 8) {
                        sort_keys<V>(key);
                        first = key[0];
                        second = V > 1 ? key[V > 1] : 0u;
                    } else {
                        first = 0;
#pragma unroll
                        for (int i = 0; i < V; ++i) second = max(second, min(first, key[i])), first = max(first, key[i]);
                    }
                    for (int o = 1; o < lanes; o <<= 1) {
                        const uint32_t u = __shfl_xor_sync(kAll, first, o);
                        if (pairs) second = max(min(first, u), max(second, __shfl_xor_sync(kAll, second, o)));
                        first = max(first, u);
                    }
                } else {
                    s_group[warp][0][lane] = s_group[warp][1][lane] = 0;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (live(key[i])) atomicMax(&s_group[warp][0][group_of(i)], key[i]);
                    __syncwarp();
                    if (pairs) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (live(key[i]) && key[i] != s_group[warp][0][group_of(i)]) atomicMax(&s_group[warp][1][group_of(i)], key[i]);
                        __syncwarp();
                    }
                    first = s_group[warp][0][lane], second = s_group[warp][1][lane];
                    __syncwarp();
                }
                const bool real = group < a.groups && live(first), two = live(second);
                // the group's value, and what it may be off by
                const float x = value_of(first), y = two ? value_of(second) : 0.0f;
                float value = x, off = slack + cut * fabsf(x);
                if (pairs && biased) {
                    value = x + y;
                    off = 2 * slack;
                } else if (pairs) {
                    value = score(x) + (two ? score(y) : 0.0f);
                    off = 0x1p-18f + cut * (fabsf(x) + fabsf(y));   // a score's slope is below 1
                }
                if (softmax && !whole) top = __any_sync(kAll, real && x == INFINITY) ? INFINITY : 0.0f;
                // the best by their values' keys, whose last five bits are the group's number
                const uint32_t mine = real ? (ordered(value) & ~31u) | (31 - group) : 0u;
                uint32_t left = mine, worst = 0;
                for (int r = 0; r < a.keep; ++r) {
                    const uint32_t m = __reduce_max_sync(kAll, left);
                    if (m != 0) worst = m;
                    if (left == m) left = 0;
                }
                bool kept = real && mine >= worst;
                const uint32_t best = __reduce_max_sync(kAll, left);   // of those that go
                if (best != 0 && !(exact && !pairs)) {   // 16-bit values are exact: equal ones stand in the order of their groups
                    const float p = unordered(worst & ~31u), q = unordered(best & ~31u);
                    const float far = 2.0f * __uint_as_float(__reduce_max_sync(kAll, real ? __float_as_uint(off) : 0u)) + 0x1p-17f * fmaxf(fabsf(p), fabsf(q));
                    if (!(p - q > far) && !bad) kept = (groups_exact<DT>(a, row) >> (group & 31)) & 1;
                }
                if (filled) {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = kept ? key[i] : 0u;
                } else {
                    const uint32_t open = __ballot_sync(kAll, kept);
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = (open >> group_of(i)) & 1 ? key[i] : 0u;
                    sort_keys<V>(key);
                }
            } else {
                sort_keys<V>(key);
            }
            uint32_t mine = 0;         // lane j: the j-th key
            if (K > 0 && exact) {      // lists as deep as the picks to come
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const uint32_t m = __reduce_max_sync(kAll, head<V>(key));
                    if (lane == j) mine = m;
                    if (j + 1 < K) pop<V>(key, m, K - 1 - j);
                }
            } else {
                uint32_t last = 0;     // the one behind the k-th
                int found = 0;
#pragma unroll
                for (int j = 0; j <= (K > 0 ? K : k); ++j, ++found) {
                    const uint32_t m = __reduce_max_sync(kAll, head<V>(key));
                    if (lane == j) mine = m;
                    last = m;
                    pop<V>(key, m, V);
                }
                uint32_t next = __shfl_down_sync(kAll, mine, 1);
                if (lane == 31) next = last;
                const float x = value_of(mine), y = value_of(next);
                const float margin = 2 * slack + cut * fmaxf(fabsf(x), fabsf(y));
                const bool near = !exact && lane < k && live(next) && (biased ? !(x - y > margin) : (mine & prefix) == (next & prefix));
                if (__any_sync(kAll, near) && !bad) {
                    // candidates: down to the first that is surely behind the k-th, at most 32
                    const uint32_t border = __shfl_sync(kAll, mine, k - 1);
                    const float kth = value_of(border);
                    found = k;
                    bool more = true;
                    while (true) {
                        const float z = value_of(last);
                        more = live(last) && (biased ? !(kth - z > 2 * slack + cut * fmaxf(fabsf(kth), fabsf(z))) : (last & prefix) == (border & prefix));
                        if (!more || found == 32) break;
                        if (lane == found) mine = last;
                        ++found;
                        last = __reduce_max_sync(kAll, head<V>(key));
                        pop<V>(key, last, V);
                    }
                    again = again || more;
                    if (!again) {
                        const bool there = lane < found && live(mine);
                        const int e = there ? (int)(kLow - (mine & kLow)) : E;
                        double v = -INFINITY, norm = 1.0;
                        if (biased && softmax) {
                            norm = 0.0;
#pragma unroll 1
                            for (int i = lane; i < E; i += 32) norm += exp((double)logit<DT>(row, i) - (double)top);
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) norm += __shfl_xor_sync(kAll, norm, o);
                        }
                        if (there) {
                            v = (double)logit<DT>(row, e);
                            if (biased) v = (softmax ? exp(v - (double)top) / norm : 1.0 / (1.0 + exp(-v))) + (double)__ldg(a.bias + e);
                        }
                        int rank = 0;
                        for (int i = 0; i < found; ++i) {
                            const double u = __shfl_sync(kAll, v, i);
                            const int j = __shfl_sync(kAll, e, i);
                            rank += u > v || (u == v && j < e);
                        }
                        const uint32_t key_of = there ? mine : 0;
                        mine = 0;
                        for (int i = 0; i < found; ++i) {
                            const int r = __shfl_sync(kAll, rank, i);
                            const uint32_t q = __shfl_sync(kAll, key_of, i);
                            if (lane == r && q != 0) mine = q;
                        }
                    }
                }
            }
            if (softmax) {
                if (!whole && !groups) top = value_of(__shfl_sync(kAll, mine, 0));
                bad = bad || top == INFINITY;
                if (!a.renorm && !whole) {
                    Row<DT, V, VEC> present;
                    present.load(row, E, lane);             // from L1
                    present.widen(l, E, lane);
                    top = l[0];
#pragma unroll
                    for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
                    top = warp_max(top);
                    top = top == -INFINITY ? 0.0f : top;
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += ex2((l[i] - top) * kLog2e);
                    sum = warp_sum(sum);
                }
            }
            int e = lane < k && live(mine) ? (int)(kLow - (mine & kLow)) : -1;
            if (again && !bad) bad = !pick_exact<DT>(a, row, e);
            failed |= (int)bad << q;
            const int other = batch > 1 ? __shfl_sync(kAll, e, lane & 7) : e;
            if (batch == 1 || lane >> 3 == q) picked = other, row_top = top, row_sum = sum;
        }
        const int q = batch > 1 ? lane >> 3 : 0, slot = batch > 1 ? lane & 7 : lane;
        const int64_t t = t0 + q;
        const bool bad = (failed >> q) & 1, there = !bad && picked >= 0;
        const float x = there ? logit<DT>(logits + t * row_bytes, picked) : -INFINITY;
        float w;
        if (softmax && !a.renorm) w = there ? expf(x - row_top) * rcp(row_sum) : 0.0f;
        else w = share(a.score, a.renorm, there, x, size);
        if (slot < k && q < batch && t < a.n) {
            a.idx[t * k + slot] = there ? picked : -1;
            a.weights[t * k + slot] = bad ? NAN : there ? a.scale * w : 0.0f;
        }
        if (failed != 0 && lane == 0) report(a.status, kErrRange);
    }
}

// ---- the gradient --------------------------------------------------------------------------------

// A warp takes four tokens of up to eight slots at once (T 4, up to 256 experts), eight
// lanes a token for what the slots need, or one token (T 1).  A lane writes 8 C experts,
// neighbours in pieces of 16 bytes with the lanes' pieces side by side (VEC), or experts
// lane, lane + 32, ...
template <int DT, int T, int C, bool VEC>
__global__ void __launch_bounds__(kThreads, C == 1 ? 4 : 2)
route_backward_kernel(const float *__restrict__ gw, const void *__restrict__ logits, const int32_t *__restrict__ idx, int64_t n,
                      int E, int k, int score, bool renorm, float scale, void *__restrict__ grad, uint32_t *status) {
    extern __shared__ __align__(16) float s_rows[];   // T rows of the picks' gradients a warp, zero between tokens
    griddep_wait();
    const int lane = threadIdx.x & 31, pitch = (E + 7) / 8 * 8, size = T > 1 || k <= 8 ? 4 : 16;
    const int q = T > 1 ? lane >> 3 : 0, slot = T > 1 ? lane & 7 : lane;   // this lane's token and slot
    float *const rows = s_rows + (threadIdx.x >> 5) * T * pitch, *const mine = rows + q * pitch;
    for (int i = lane; i < T * pitch; i += 32) rows[i] = 0.0f;
    __syncwarp();
    const int64_t step = (int64_t)gridDim.x * kWarps * T;
    const size_t row_bytes = (size_t)E * (DT == CGL_F32 ? 4 : 2);
    const char *const base = static_cast<const char *>(logits);
    const bool whole = score == CGL_SCORE_SOFTMAX && !renorm;
    constexpr int P = VEC ? (DT == CGL_F32 ? 4 : 8) : 1, N = 8 * C / P;   // experts a piece, pieces a lane
    const auto expert = [&](int piece) { return (piece * 32 + lane) * P; };
    int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * T;
    int id = -1;
    float g = 0.0f;
    if (slot < k && t0 + q < n) id = __ldg(idx + (t0 + q) * k + slot), g = __ldg(gw + (t0 + q) * k + slot);
    for (; t0 < n; t0 += step) {
        const int64_t t = t0 + q;
        const int e = id;
        const bool there = e >= 0 && e < E;
        const float x = there ? logit<DT>(base + t * row_bytes, e) : -INFINITY, gs = there ? scale * g : 0.0f;
        if (!there && e != -1) report(status, kErrRange);
        uint4 raw[T][VEC ? N : 1];
        float one[T][VEC ? 1 : N];
        if (whole) {
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (t0 + u < n && expert(c) < E) {
                        const char *row = base + (t0 + u) * row_bytes;
                        if (VEC) raw[u][VEC ? c : 0] = ld_nc_v4(row + expert(c) * (DT == CGL_F32 ? 4 : 2));
                        else one[u][VEC ? 0 : c] = logit<DT>(row, expert(c));
                    }
        }
        const int64_t then = t + step;
        id = -1;
        if (slot < k && then < n) id = __ldg(idx + then * k + slot), g = __ldg(gw + then * k + slot);
        const auto widen = [&](int u, float l[8 * C]) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
                const uint4 a = raw[u][VEC ? c : 0];
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float f;
                    if (!VEC) f = one[u][VEC ? 0 : c];
                    else if (DT == CGL_F32) f = __uint_as_float(w[i % 4]);
                    else if (DT == CGL_BF16) f = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
                    else f = __half2float(__ushort_as_half((unsigned short)((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu)));
                    l[P * c + i] = expert(c) < E ? f : -INFINITY;
                }
            }
        };
        float tops[T], sums[T], top = 0.0f, sum = 1.0f;   // of each row, and of this lane's token
        if (whole) {
#pragma unroll
            for (int u = 0; u < T; ++u) {
                float l[8 * C], m = -INFINITY, v = 0.0f;
                widen(u, l);
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) m = fmaxf(m, l[i]);
                m = warp_max(m);
                m = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) v += ex2((l[i] - m) * kLog2e);
                tops[u] = m, sums[u] = warp_sum(v);
                if (u == q) top = m, sum = sums[u];
            }
        }
        float w;
        if (whole) w = there && x != -INFINITY ? expf(x - top) / sum : 0.0f;   // a NaN stays
        else w = share(score, renorm, there, x, size);
        float dot = 0.0f, v = w * gs;
        if (whole) {
            dot = picks_sum(there ? v : 0.0f, size);
        } else if (renorm) {
            // g_j - sum_i g_i w_i as sum_i w_i (g_j - g_i): the weights' sum is 1, and where one is nearly all of it nothing cancels
            float d = 0.0f;
            for (int i = 0; i < k; ++i) {
                const int from = T > 1 ? (lane & ~7) + i : i;
                d = fmaf(__shfl_sync(kAll, w, from), gs - __shfl_sync(kAll, gs, from), d);
            }
            v = w * d;
        }
        if (score == CGL_SCORE_SIGMOID) {   // 1 - sigmoid
            const float z = expf(-fabsf(x));
            v *= (x > 0.0f ? z : 1.0f) * rcp(1.0f + z);
        }
        // into their places; an expert that is in two slots, which its slots' numbers show, gets its terms one by one
        if (there) mine[e] = __int_as_float(lane);
        __syncwarp();
        const bool twice = there && __float_as_int(mine[e]) != lane;
        if (__any_sync(kAll, twice)) {
            __syncwarp();
            if (there) mine[e] = 0.0f;
            __syncwarp();
            for (int j = 0; j < k; ++j) {
                if (slot == j && there) mine[e] += v;
                __syncwarp();
            }
        } else {
            __syncwarp();
            if (there) mine[e] = v;
        }
        __syncwarp();
        const uint32_t any = __ballot_sync(kAll, there);
#pragma unroll
        for (int u = 0; u < T; ++u) {
            if (t0 + u >= n) break;
            // a token without a slot gets 0, whatever its logits
            const bool spread = whole && (T > 1 ? (any >> (8 * u)) & 0xFFu : any) != 0 && sums[u] != 0.0f;
            const float least = -__shfl_sync(kAll, dot, 8 * u) / (whole ? sums[u] : 1.0f);
            float l[8 * C];
            if (whole) {
                widen(u, l);
#pragma unroll
                for (int i = 0; i < 8 * C; ++i) l[i] = least * ex2((l[i] - tops[u]) * kLog2e);
            }
            const float *s = rows + u * pitch;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                if (expert(c) >= E) break;
                float o[P];
#pragma unroll
                for (int i = 0; i < P; i += VEC ? 4 : 1) {
                    if (VEC) *reinterpret_cast<float4 *>(o + i) = *reinterpret_cast<const float4 *>(s + expert(c) + i);
                    else o[i] = s[expert(c)];
                }
                if (spread)
#pragma unroll
                    for (int i = 0; i < P; ++i) o[i] += l[P * c + i];
                void *to = static_cast<char *>(grad) + (t0 + u) * row_bytes + expert(c) * (DT == CGL_F32 ? 4 : 2);
                if (!VEC) put<DT>(to, 0, o[0]);
                else st_cs_v4(to, pack<DT>(o));
            }
        }
        __syncwarp();
        if (there) mine[e] = 0.0f;
        __syncwarp();
    }
}

template <int DT, int KIND>
void *route_by_width(int E, int k, bool vec) {
    if (E <= 32) return (void *)route_kernel<DT, 1, false, 0, KIND>;
    if (E <= 128) return k == 8 ? (void *)route_kernel<DT, 4, false, 8, KIND> : (void *)route_kernel<DT, 4, false, 0, KIND>;
    if (E <= 256 && vec) return k == 8 ? (void *)route_kernel<DT, 8, true, 8, KIND> : (void *)route_kernel<DT, 8, true, 0, KIND>;
    if (E <= 256) return (void *)route_kernel<DT, 8, false, 0, KIND>;
    if (E <= 512) return vec ? (void *)route_kernel<DT, 16, true, 0, KIND> : (void *)route_kernel<DT, 16, false, 0, KIND>;
    return vec ? (void *)route_kernel<DT, 32, true, 0, KIND> : (void *)route_kernel<DT, 32, false, 0, KIND>;
}
template <int DT>
void *route_by_kind(const RouteArgs &a, bool vec) {
    if (a.groups > 1) return a.bias != nullptr ? route_by_width<DT, kGroupsBias>(a.E, a.k, vec) : route_by_width<DT, kGroups>(a.E, a.k, vec);
    return a.bias != nullptr ? route_by_width<DT, kBias>(a.E, a.k, vec) : route_by_width<DT, kPlain>(a.E, a.k, vec);
}
template <int DT>
void *backward_by_width(int E, bool vec, bool four) {
    if (E <= 256 && vec) return four ? (void *)route_backward_kernel<DT, 4, 1, true> : (void *)route_backward_kernel<DT, 1, 1, true>;
    if (E <= 256) return four ? (void *)route_backward_kernel<DT, 4, 1, false> : (void *)route_backward_kernel<DT, 1, 1, false>;
    return vec ? (void *)route_backward_kernel<DT, 1, 4, true> : (void *)route_backward_kernel<DT, 1, 4, false>;
}

// From so many tokens on a warp takes four at once, up to eight slots each.  256 experts,
// one at once and four: forward of 4096 BF16 tokens 3.4 and 3.0 us (softmax as it is 3.5 and
// 3.9), 8192 5.8 and 4.3 (6.0 and 5.3), 65536 32.8 and 23.6; of binary32 ones with a bias 8192
// 11.3 and 8.8; backward 4096 3.2 and 2.7 (3.1 and 3.7), 8192 5.0 and 3.1 (4.8 and 4.4).
constexpr int64_t kFour = 8192;

}  // namespace

cgl_status launch_route(const RouteArgs &args, cudaStream_t stream) {
    RouteArgs a = args;
    if (a.n == 0) return CGL_OK;
    const bool vec = a.E % 8 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
    const auto kernel = reinterpret_cast<void (*)(RouteArgs)>(a.dtype == CGL_BF16  ? route_by_kind<CGL_BF16>(a, vec)
                                                              : a.dtype == CGL_F16 ? route_by_kind<CGL_F16>(a, vec)
                                                                                   : route_by_kind<CGL_F32>(a, vec));
    a.batch = a.k <= 8 && a.groups == 1 && a.n >= kFour ? 4 : 1;
    const int64_t warps = (a.n + a.batch - 1) / a.batch;
    const int grid = persistent_grid((const void *)kernel, kThreads, 0, 8, 0, (warps + kWarps - 1) / kWarps);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, a) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

cgl_status launch_route_backward(const float *gw, const void *logits, int dtype, const int32_t *idx, int64_t n, int E, int k,
                                 int score, bool renorm, float scale, void *grad, uint32_t *status, cudaStream_t stream) {
    if (n == 0) return CGL_OK;
    const bool vec = E % 8 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(grad)) & 15) == 0;
    const bool four = E <= 256 && k <= 8 && n >= kFour;
    const auto kernel = reinterpret_cast<void (*)(const float *, const void *, const int32_t *, int64_t, int, int, int, bool, float, void *, uint32_t *)>(
        dtype == CGL_BF16  ? backward_by_width<CGL_BF16>(E, vec, four)
        : dtype == CGL_F16 ? backward_by_width<CGL_F16>(E, vec, four)
                           : backward_by_width<CGL_F32>(E, vec, four));
    const size_t smem = (size_t)kWarps * (four ? 4 : 1) * ((E + 7) / 8 * 8) * 4;   // at most 32 KiB
    const int64_t warps = four ? (n + 3) / 4 : n;
    const int grid = persistent_grid((const void *)kernel, kThreads, smem, 8, 0, (warps + kWarps - 1) / kWarps);
    if (grid <= 0) return CGL_ECUDA;
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, gw, logits, idx, n, E, k, score, renorm, scale, grad,
                      status) == cudaSuccess ? CGL_OK : CGL_ECUDA;
}

}  // namespace cgl
