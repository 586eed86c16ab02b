// The exported C ABI (declared in include/cgl.h): argument checks, then one
// call into the launchers.  Host-visible errors return before any launch.
#include <initializer_list>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "launch.h"

namespace cgl {

namespace {

std::mutex g_mu;

struct KernelCache {
    const void *kernel;
    int device;
    size_t smem;         // dynamic shared memory limit set so far
    int ctas_per_sm;     // occupancy at kThreads, 0 = not computed
};
std::vector<KernelCache> g_kernels;
int g_sms[256] = {0};

KernelCache &entry(const void *kernel, int device) {
    for (auto &e : g_kernels)
        if (e.kernel == kernel && e.device == device) return e;
    g_kernels.push_back({kernel, device, 48 * 1024, 0});
    return g_kernels.back();
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int opt_sms(const cgl_opts *o) { return o ? o->num_sms : 0; }
int opt_cap(const cgl_opts *o) { return o ? o->capacity : 0; }
uint32_t opt_flags(const cgl_opts *o) { return o ? o->flags : 0u; }
bool flags_ok(const cgl_opts *o) { return (opt_flags(o) & ~CGL_OPT_UE8M0_SCALES) == 0; }
bool opt_pow2(const cgl_opts *o) { return (opt_flags(o) & CGL_OPT_UE8M0_SCALES) != 0; }
unsigned long long *opt_scratch(const cgl_opts *o) {
    return o ? static_cast<unsigned long long *>(o->scratch) : nullptr;
}

}  // namespace

int device_sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return 0;
    if (g_sms[dev] == 0) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        g_sms[dev] = v;
    }
    return g_sms[dev];
}

bool ensure_smem_attr(const void *kernel, size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lk(g_mu);
    KernelCache &e = entry(kernel, dev);
    if (bytes <= e.smem) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
        cudaSuccess)
        return false;
    e.smem = bytes;
    return true;
}

namespace {
struct OccEntry {
    const void *kernel;
    int device, threads;
    size_t smem;
    int ctas;
};
OccEntry g_occ[256];
int g_occ_n = 0;
}  // namespace

int persistent_grid(const void *kernel, int threads, size_t smem, int target_per_sm, int num_sms_cap,
                    int64_t work) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int sms = device_sm_count();
    if (sms <= 0) return 0;
    int fit = 0;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        for (int i = 0; i < g_occ_n; ++i)
            if (g_occ[i].kernel == kernel && g_occ[i].device == dev && g_occ[i].threads == threads &&
                g_occ[i].smem == smem)
                fit = g_occ[i].ctas;
        if (fit == 0) {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem) != cudaSuccess)
                return 0;
            if (fit < 1) fit = 1;
            if (g_occ_n < 256) g_occ[g_occ_n++] = {kernel, dev, threads, smem, fit};
        }
    }
    int per_sm = target_per_sm < fit ? target_per_sm : fit;
    if (per_sm < 1) per_sm = 1;
    const int use_sms = (num_sms_cap > 0 && num_sms_cap < sms) ? num_sms_cap : sms;
    const int64_t want = (int64_t)use_sms * per_sm;
    return (int)(work < want ? work : want);
}

int copy_grid(const void *kernel, int threads, int64_t work_ctas, int num_sms_cap) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int sms = device_sm_count();
    if (sms <= 0) return 0;
    int per_sm = 0;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        KernelCache &e = entry(kernel, dev);
        if (e.ctas_per_sm == 0) {
            int v = 0;
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, threads, 0) != cudaSuccess)
                return 0;
            e.ctas_per_sm = v > 0 ? v : 1;
        }
        per_sm = e.ctas_per_sm;
    }
    const int use_sms = (num_sms_cap > 0 && num_sms_cap < sms) ? num_sms_cap : sms;
    const int64_t cap = (int64_t)use_sms * per_sm;
    return (int)(work_ctas < cap ? work_ctas : cap);
}

}  // namespace cgl

using namespace cgl;

extern "C" {

int cgl_version(void) { return 500; }

const char *cgl_status_string(int s) {
    switch (s) {
        case CGL_OK: return "ok";
        case CGL_EINVAL: return "invalid argument";
        case CGL_EALIGN: return "misaligned pointer";
        case CGL_ERANGE: return "expert id or receive row out of range";
        case CGL_ECAPACITY: return "padded expert capacity exceeded";
        case CGL_ETIMEOUT: return "bounded wait timed out";
        case CGL_ECUDA: return "CUDA runtime error";
        case CGL_ENOTIMPL: return "not implemented";
        default: return "unknown status";
    }
}

// Tokens and slots in 32 bits; n by itself first, so that the product stays in 64.
static bool slots_ok(int64_t n, int k) {
    return n >= 0 && n < ((int64_t)1 << 31) && k >= 1 && k <= kMaxTopk && n * k < ((int64_t)1 << 31);
}

static bool layout_sizes_ok(int64_t n, int k, int E, int R) {
    return slots_ok(n, k) && E >= 1 && E <= kMaxExperts && R >= 1 && R <= E && E % R == 0;
}

size_t cgl_layout_workspace_bytes(int64_t n, int k, int E, int R) {
    if (!layout_sizes_ok(n, k, E, R)) return 0;
    return layout_workspace_bytes(n, k, E, R);
}

int cgl_layout_kernel_count(int64_t n, int k, int E, int R) {
    if (!layout_sizes_ok(n, k, E, R)) return -1;
    return layout_fused_fits(n, k, E, R) ? 1 : 2;
}

cgl_status cgl_get_layout(const int32_t *topk_idx, int64_t n, int k, int E, int R,
                          const cgl_opts *opts, int32_t *tokens_per_expert, int32_t *tokens_per_rank,
                          uint8_t *is_token_in_rank, int32_t *expert_offset, int32_t *max_count,
                          int32_t *dst_pos, int32_t *recv_src, void *workspace,
                          size_t workspace_bytes, uint32_t *status_dev, void *stream) {
    if (!layout_sizes_ok(n, k, E, R) || !flags_ok(opts)) return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || (int64_t)E * cap >= ((int64_t)1 << 31)) return CGL_EINVAL;
    const int64_t rows = cap > 0 ? (int64_t)E * cap : n * k;
    if (!tokens_per_expert || !tokens_per_rank || !expert_offset || !max_count || !workspace)
        return CGL_EINVAL;
    if (n > 0 && (!topk_idx || !dst_pos || !is_token_in_rank)) return CGL_EINVAL;
    if (rows > 0 && !recv_src) return CGL_EINVAL;
    if (workspace_bytes < layout_workspace_bytes(n, k, E, R)) return CGL_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(tokens_per_expert, 4) || !aligned(tokens_per_rank, 4) ||
        !aligned(expert_offset, 4) || !aligned(max_count, 4) || !aligned(dst_pos, 4) ||
        !aligned(recv_src, 4) || !aligned(status_dev, 4) || !aligned(is_token_in_rank, 16) ||
        !aligned(workspace, 16))
        return CGL_EALIGN;
    return launch_layout(topk_idx, n, k, E, R, cap, tokens_per_expert, tokens_per_rank,
                         is_token_in_rank, expert_offset, max_count, dst_pos, recv_src, workspace,
                         status_dev, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_get_rank_layout(const int32_t *topk_idx, int64_t n, int k, int E, int R,
                               const cgl_opts *opts, int32_t *tokens_per_rank, int32_t *rank_offset,
                               int32_t *max_count, int32_t *rank_dst, int32_t *recv_token,
                               void *workspace, size_t workspace_bytes, uint32_t *status_dev,
                               void *stream) {
    if (!layout_sizes_ok(n, k, E, R) || !flags_ok(opts)) return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || (int64_t)R * cap >= ((int64_t)1 << 31)) return CGL_EINVAL;
    const int64_t rows = cap > 0 ? (int64_t)R * cap : n * k;
    if (!tokens_per_rank || !rank_offset || !max_count || !workspace) return CGL_EINVAL;
    if (n > 0 && (!topk_idx || !rank_dst)) return CGL_EINVAL;
    if (rows > 0 && !recv_token) return CGL_EINVAL;
    if (workspace_bytes < layout_workspace_bytes(n, k, R, R)) return CGL_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(tokens_per_rank, 4) || !aligned(rank_offset, 4) ||
        !aligned(max_count, 4) || !aligned(rank_dst, 4) || !aligned(recv_token, 4) ||
        !aligned(status_dev, 4) || !aligned(workspace, 16))
        return CGL_EALIGN;
    return launch_rank_layout(topk_idx, n, k, E, R, cap, tokens_per_rank, rank_offset, max_count,
                              rank_dst, recv_token, workspace, status_dev,
                              static_cast<cudaStream_t>(stream));
}

cgl_status cgl_dispatch_fp8(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos,
                            uint8_t *recv_x, float *recv_scale, int64_t recv_rows,
                            const cgl_opts *opts, uint32_t *status_dev, void *stream) {
    if (n < 0 || h <= 0 || h % 128 != 0 || k < 1 || k > kMaxTopk || recv_rows < 0)
        return CGL_EINVAL;
    if (opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (n > 0 && (!x || !dst_pos)) return CGL_EINVAL;
    if (n > 0 && recv_rows > 0 && (!recv_x || !recv_scale)) return CGL_EINVAL;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || !aligned(dst_pos, 4) ||
        !aligned(recv_scale, 4) || !aligned(status_dev, 4) || !aligned(opt_scratch(opts), 8))
        return CGL_EALIGN;
    return launch_dispatch_fp8(x, n, h, k, dst_pos, recv_x, recv_scale, recv_rows, opt_sms(opts), opt_pow2(opts),
                               status_dev, static_cast<cudaStream_t>(stream), opt_scratch(opts));
}

cgl_status cgl_dispatch_bf16(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos,
                             uint16_t *recv_x, int64_t recv_rows, const cgl_opts *opts,
                             uint32_t *status_dev, void *stream) {
    if (n < 0 || h <= 0 || h % 8 != 0 || k < 1 || k > kMaxTopk || recv_rows < 0) return CGL_EINVAL;
    if (opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (n > 0 && (!x || !dst_pos)) return CGL_EINVAL;
    if (n > 0 && recv_rows > 0 && !recv_x) return CGL_EINVAL;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || !aligned(dst_pos, 4) || !aligned(status_dev, 4) ||
        !aligned(opt_scratch(opts), 8))
        return CGL_EALIGN;
    return launch_dispatch_bf16(x, n, h, k, dst_pos, recv_x, recv_rows, opt_sms(opts), status_dev,
                                static_cast<cudaStream_t>(stream), opt_scratch(opts));
}

cgl_status cgl_combine(const uint16_t *y, int64_t recv_rows, const int32_t *dst_pos,
                       const float *topk_weights, int64_t n, int h, int k, uint16_t *out,
                       const cgl_opts *opts, uint32_t *status_dev, void *stream) {
    if (n < 0 || h <= 0 || h % 8 != 0 || k < 1 || k > kMaxTopk || recv_rows < 0) return CGL_EINVAL;
    if (opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (n > 0 && (!dst_pos || !topk_weights || !out)) return CGL_EINVAL;
    if (n > 0 && recv_rows > 0 && !y) return CGL_EINVAL;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(dst_pos, 4) ||
        !aligned(topk_weights, 4) || !aligned(status_dev, 4))
        return CGL_EALIGN;
    return launch_combine(y, recv_rows, dst_pos, topk_weights, n, h, k, out, opt_sms(opts),
                          status_dev, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_combine_backward(const uint16_t *grad_out, const uint16_t *y, int64_t recv_rows,
                                const int32_t *dst_pos, const float *topk_weights, int64_t n, int h,
                                int k, uint16_t *grad_y, float *grad_w, const cgl_opts *opts,
                                uint32_t *status_dev, void *stream) {
    if (n < 0 || h <= 0 || h % 16 != 0 || h > 16384 || k < 1 || k > kMaxTopk || recv_rows < 0)
        return CGL_EINVAL;
    if (opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (n > 0 && (!grad_out || !dst_pos || !topk_weights || !grad_w)) return CGL_EINVAL;
    if (n > 0 && recv_rows > 0 && (!y || !grad_y)) return CGL_EINVAL;
    if (!aligned(grad_out, 16) || !aligned(y, 16) || !aligned(grad_y, 16) || !aligned(dst_pos, 4) ||
        !aligned(topk_weights, 4) || !aligned(grad_w, 4) || !aligned(status_dev, 4))
        return CGL_EALIGN;
    return launch_combine_backward(grad_out, y, recv_rows, dst_pos, topk_weights, n, h, k, grad_y, grad_w,
                                   opt_sms(opts), status_dev, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_decode_dispatch_fp8(const int32_t *topk_idx, int64_t n, int k, int E, int R,
                                   const cgl_opts *opts, const uint16_t *x, int h,
                                   int32_t *tokens_per_expert, int32_t *tokens_per_rank,
                                   uint8_t *is_token_in_rank, int32_t *expert_offset, int32_t *max_count,
                                   int32_t *dst_pos, int32_t *recv_src, uint8_t *recv_x,
                                   float *recv_scale, uint32_t *status_dev, void *stream) {
    if (!layout_sizes_ok(n, k, E, R) || h <= 0 || h % 128 != 0 || !flags_ok(opts)) return CGL_EINVAL;
    const int per_block = 1024 / k < 256 ? 1024 / k : 256;   // tokens one layout block holds
    if (n > per_block) return CGL_EINVAL;
    if (decode_fused_smem_bytes(n, k, E, R) > 47 * 1024) return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || (int64_t)E * cap >= ((int64_t)1 << 31) || opt_sms(opts) < 0) return CGL_EINVAL;
    const int64_t rows = cap > 0 ? (int64_t)E * cap : n * k;
    if (!tokens_per_expert || !tokens_per_rank || !expert_offset || !max_count) return CGL_EINVAL;
    if (n > 0 && (!topk_idx || !x || !dst_pos || !is_token_in_rank)) return CGL_EINVAL;
    if (rows > 0 && (!recv_src || !recv_x || !recv_scale)) return CGL_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(x, 16) || !aligned(tokens_per_expert, 4) ||
        !aligned(tokens_per_rank, 4) || !aligned(is_token_in_rank, 16) || !aligned(expert_offset, 4) ||
        !aligned(max_count, 4) || !aligned(dst_pos, 4) || !aligned(recv_src, 4) ||
        !aligned(recv_x, 16) || !aligned(recv_scale, 4) || !aligned(status_dev, 4))
        return CGL_EALIGN;
    return launch_decode_dispatch_fp8(topk_idx, n, k, E, R, cap, x, h, tokens_per_expert, tokens_per_rank,
                                      is_token_in_rank, expert_offset, max_count, dst_pos, recv_src, recv_x,
                                      recv_scale, opt_sms(opts), opt_pow2(opts), status_dev,
                                      static_cast<cudaStream_t>(stream));
}

size_t cgl_layout_dispatch_workspace_bytes(int64_t n, int k, int E, int R) {
    if (!layout_sizes_ok(n, k, E, R)) return 0;
    return layout_dispatch_workspace_bytes(n, k, E, R);
}

int cgl_layout_dispatch_kernel_count(int64_t n, int k, int E, int R, int h, const cgl_opts *opts) {
    if (!layout_sizes_ok(n, k, E, R) || h <= 0 || h % 128 != 0 || opt_sms(opts) < 0) return -1;
    if (layout_dispatch_fused_fits(n, k, E, R, h, opt_sms(opts))) return 1;
    return (layout_fused_fits(n, k, E, R) ? 1 : 2) + 1;
}

cgl_status cgl_layout_dispatch_fp8(const int32_t *topk_idx, int64_t n, int k, int E, int R,
                                   const cgl_opts *opts, const uint16_t *x, int h,
                                   int32_t *tokens_per_expert, int32_t *tokens_per_rank,
                                   uint8_t *is_token_in_rank, int32_t *expert_offset, int32_t *max_count,
                                   int32_t *dst_pos, int32_t *recv_src, uint8_t *recv_x, float *recv_scale,
                                   void *workspace, size_t workspace_bytes, uint32_t *status_dev,
                                   void *stream) {
    if (!layout_sizes_ok(n, k, E, R) || h <= 0 || h % 128 != 0 || !flags_ok(opts)) return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || (int64_t)E * cap >= ((int64_t)1 << 31) || opt_sms(opts) < 0) return CGL_EINVAL;
    const int64_t rows = cap > 0 ? (int64_t)E * cap : n * k;
    if (!tokens_per_expert || !tokens_per_rank || !expert_offset || !max_count || !workspace)
        return CGL_EINVAL;
    if (n > 0 && (!topk_idx || !x || !dst_pos || !is_token_in_rank)) return CGL_EINVAL;
    if (rows > 0 && (!recv_src || !recv_x || !recv_scale)) return CGL_EINVAL;
    if (workspace_bytes < layout_dispatch_workspace_bytes(n, k, E, R)) return CGL_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(x, 16) || !aligned(tokens_per_expert, 4) ||
        !aligned(tokens_per_rank, 4) || !aligned(is_token_in_rank, 16) || !aligned(expert_offset, 4) ||
        !aligned(max_count, 4) || !aligned(dst_pos, 4) || !aligned(recv_src, 4) ||
        !aligned(recv_x, 16) || !aligned(recv_scale, 4) || !aligned(status_dev, 4) || !aligned(workspace, 16))
        return CGL_EALIGN;
    return launch_layout_dispatch_fp8(topk_idx, n, k, E, R, cap, x, h, tokens_per_expert, tokens_per_rank,
                                      is_token_in_rank, expert_offset, max_count, dst_pos, recv_src, recv_x,
                                      recv_scale, workspace, opt_sms(opts), opt_pow2(opts), status_dev,
                                      static_cast<cudaStream_t>(stream));
}

cgl_status cgl_selftest_bounded_wait(uint64_t *workspace, int nflags, uint32_t *status_dev, void *stream) {
    if (!workspace || !status_dev || nflags < 1 || nflags > 4096) return CGL_EINVAL;
    if (!aligned(workspace, 8) || !aligned(status_dev, 4)) return CGL_EALIGN;
    return launch_wait_probe(workspace, nflags, status_dev, static_cast<cudaStream_t>(stream));
}

static bool dtype_ok(int dtype) { return dtype == CGL_BF16 || dtype == CGL_F16 || dtype == CGL_F32; }

// Rows of MXFP4: codes (cols / 2 bytes a row), at most 2^48 values in all.
static bool mx_sizes_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols > 0 && cols % 32 == 0 && cols <= ((int64_t)1 << 30) && rows <= ((int64_t)1 << 32) &&
           rows <= ((int64_t)1 << 48) / cols;
}

cgl_status cgl_quantize_mxfp4(const void *x, int dtype, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                              const cgl_opts *opts, void *stream) {
    if (!mx_sizes_ok(rows, cols) || !dtype_ok(dtype) || opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (rows > 0 && (!x || !codes || !scales)) return CGL_EINVAL;
    if (!aligned(x, 16) || !aligned(codes, 16)) return CGL_EALIGN;
    return launch_quantize_mxfp4(x, dtype, rows, cols, codes, scales, opt_sms(opts), static_cast<cudaStream_t>(stream));
}

cgl_status cgl_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                int dtype, const cgl_opts *opts, void *stream) {
    if (!mx_sizes_ok(rows, cols) || !dtype_ok(dtype) || opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (rows > 0 && (!out || !codes || !scales)) return CGL_EINVAL;
    if (!aligned(out, 16) || !aligned(codes, 16)) return CGL_EALIGN;
    return launch_dequantize_mxfp4(codes, scales, rows, cols, out, dtype, opt_sms(opts),
                                   static_cast<cudaStream_t>(stream));
}

cgl_status cgl_dispatch_mxfp4(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos, uint8_t *recv_x,
                              uint8_t *recv_scale, int64_t recv_rows, const cgl_opts *opts, uint32_t *status_dev,
                              void *stream) {
    if (!mx_sizes_ok(n, h) || !slots_ok(n, k) || recv_rows < 0)
        return CGL_EINVAL;
    if (opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (n > 0 && (!x || !dst_pos)) return CGL_EINVAL;
    if (n > 0 && recv_rows > 0 && (!recv_x || !recv_scale)) return CGL_EINVAL;
    if (!aligned(x, 16) || !aligned(recv_x, 16) || !aligned(dst_pos, 4) || !aligned(status_dev, 4) ||
        !aligned(opt_scratch(opts), 8))
        return CGL_EALIGN;
    return launch_dispatch_mxfp4(x, n, h, k, dst_pos, recv_x, recv_scale, recv_rows, opt_sms(opts), status_dev,
                                 static_cast<cudaStream_t>(stream), opt_scratch(opts));
}

cgl_status cgl_matmul_mxfp4(const uint8_t *a, const uint8_t *a_scale, int64_t num_rows, const uint8_t *w,
                            const uint8_t *w_scale, int E, int F, int K, const int32_t *expert_offset, uint16_t *y,
                            const cgl_opts *opts, uint32_t *status_dev, void *stream) {
    if (E < 1 || E > kMaxExperts || F < 1 || F > (1 << 20) || K < 32 || K % 32 != 0 || K > (1 << 20) || num_rows < 0 ||
        num_rows > ((int64_t)1 << 31) - 4096)
        return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (!expert_offset && (E != 1 || cap != 0)) return CGL_EINVAL;
    if (cap > 0 && num_rows < (int64_t)E * cap) return CGL_EINVAL;
    if (!w || !w_scale) return CGL_EINVAL;
    if (num_rows > 0 && (!a || !a_scale || !y)) return CGL_EINVAL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(y, 2) || !aligned(expert_offset, 4) || !aligned(status_dev, 4))
        return CGL_EALIGN;
    return launch_matmul_mxfp4(a, a_scale, num_rows, w, w_scale, E, F, K, expert_offset, cap, y, opt_sms(opts),
                               status_dev, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_selftest_matmul_timeout(const uint8_t *a, const uint8_t *a_scale, int64_t num_rows, const uint8_t *w,
                                       const uint8_t *w_scale, int F, int K, uint16_t *y, int64_t wait_cycles,
                                       uint32_t *status_dev, void *stream) {
    if (F < 1 || F > (1 << 20) || K < 32 || K % 32 != 0 || K > (1 << 20) || num_rows < 1 || num_rows > (1 << 20) ||
        wait_cycles < 0)
        return CGL_EINVAL;
    if (!a || !a_scale || !w || !w_scale || !y || !status_dev) return CGL_EINVAL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(y, 2) || !aligned(status_dev, 4)) return CGL_EALIGN;
    return launch_matmul_mxfp4(a, a_scale, num_rows, w, w_scale, 1, F, K, nullptr, 0, y, 0, status_dev,
                               static_cast<cudaStream_t>(stream), wait_cycles);
}

static bool balance_sizes_ok(int64_t n, int k, int E, int64_t S) {
    return slots_ok(n, k) && E >= 1 && E <= kMaxExperts && S >= 1 && S <= ((int64_t)1 << 24) && n % S == 0;
}

size_t cgl_balance_loss_workspace_bytes(int64_t n, int k, int E, int64_t S) {
    return balance_sizes_ok(n, k, E, S) ? balance_workspace_bytes(n, k, E, S) : 0;
}

cgl_status cgl_balance_loss(const void *logits, int dtype, const int32_t *topk_idx, int64_t n, int k, int E, int64_t S,
                            float alpha, int score, const float *grad_loss, float *loss, int32_t *counts,
                            int32_t *num_routed, void *grad_logits, void *workspace, size_t workspace_bytes,
                            uint32_t *status_dev, void *stream) {
    if (!balance_sizes_ok(n, k, E, S) || !dtype_ok(dtype)) return CGL_EINVAL;
    if (score != CGL_SCORE_SOFTMAX && score != CGL_SCORE_SIGMOID) return CGL_EINVAL;
    if (!loss || !counts || !num_routed || !workspace) return CGL_EINVAL;
    if (n > 0 && (!logits || !topk_idx)) return CGL_EINVAL;
    if (workspace_bytes < balance_workspace_bytes(n, k, E, S)) return CGL_EINVAL;
    const size_t item = dtype == CGL_F32 ? 4 : 2;
    if (!aligned(logits, item) || !aligned(grad_logits, item) || !aligned(topk_idx, 4) || !aligned(grad_loss, 4) ||
        !aligned(loss, 4) || !aligned(counts, 4) || !aligned(num_routed, 4) || !aligned(workspace, 16) ||
        !aligned(status_dev, 4))
        return CGL_EALIGN;
    return launch_balance_loss(logits, dtype, topk_idx, n, k, E, S, alpha, score, grad_loss, loss, counts, num_routed,
                               grad_logits, workspace, status_dev, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_balance_loss_backward(const float *grad_loss, const void *logits, int dtype, const int32_t *topk_idx,
                                     int64_t n, int k, int E, int64_t S, float alpha, int score, const int32_t *counts,
                                     const int32_t *num_routed, void *grad_logits, void *stream) {
    if (!balance_sizes_ok(n, k, E, S) || !dtype_ok(dtype)) return CGL_EINVAL;
    if (score != CGL_SCORE_SOFTMAX && score != CGL_SCORE_SIGMOID) return CGL_EINVAL;
    if (!counts || !num_routed) return CGL_EINVAL;
    if (n > 0 && (!logits || !topk_idx || !grad_logits)) return CGL_EINVAL;
    const size_t item = dtype == CGL_F32 ? 4 : 2;
    if (!aligned(logits, item) || !aligned(grad_logits, item) || !aligned(topk_idx, 4) || !aligned(grad_loss, 4) ||
        !aligned(counts, 4) || !aligned(num_routed, 4))
        return CGL_EALIGN;
    return launch_balance_loss_backward(grad_loss, logits, dtype, topk_idx, n, k, E, S, alpha, score, counts,
                                        num_routed, grad_logits, static_cast<cudaStream_t>(stream));
}

// Arrays of a call, to find those that have bytes in common.
struct Bytes {
    const void *p;
    size_t n;
};
static bool meet(Bytes a, std::initializer_list<Bytes> others) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p);
    for (const Bytes &b : others) {
        const uintptr_t y = reinterpret_cast<uintptr_t>(b.p);
        if (a.p && b.p && a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n) return true;
    }
    return false;
}

static bool route_sizes_ok(int64_t n, int E, int k) {
    return slots_ok(n, k) && E >= 1 && E <= kMaxExperts && k <= E;
}

cgl_status cgl_route(const void *logits, int dtype, int64_t n, int E, int k, const float *bias, int groups, int keep,
                     int by, int score, int renorm, float scale, int32_t *topk_idx, float *topk_weights,
                     uint32_t *status_dev, void *stream) {
    if (!route_sizes_ok(n, E, k) || !dtype_ok(dtype)) return CGL_EINVAL;
    if (groups < 1 || groups > 32 || E % groups != 0 || keep < 1 || keep > groups) return CGL_EINVAL;
    if (by != CGL_GROUP_MAX && by != CGL_GROUP_TOP2) return CGL_EINVAL;
    if (score != CGL_SCORE_SOFTMAX && score != CGL_SCORE_SIGMOID) return CGL_EINVAL;
    if (n > 0 && (!logits || !topk_idx || !topk_weights)) return CGL_EINVAL;
    if (!aligned(logits, dtype == CGL_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
        !aligned(topk_weights, 4) || !aligned(status_dev, 4))
        return CGL_EALIGN;
    const size_t slots = (size_t)n * k * 4;
    const Bytes in = {logits, (size_t)n * E * (dtype == CGL_F32 ? 4 : 2)}, steer = {bias, (size_t)E * 4}, ids = {topk_idx, slots}, ws = {topk_weights, slots};
    if (meet(ids, {in, steer, ws}) || meet(ws, {in, steer})) return CGL_EINVAL;
    const RouteArgs a = {logits, dtype, n, E, k, bias, groups, keep, by, score, renorm != 0, scale, topk_idx, topk_weights,
                         status_dev};
    return launch_route(a, static_cast<cudaStream_t>(stream));
}

cgl_status cgl_route_backward(const float *grad_weights, const void *logits, int dtype, const int32_t *topk_idx,
                              int64_t n, int E, int k, int score, int renorm, float scale, void *grad_logits,
                              uint32_t *status_dev, void *stream) {
    if (!slots_ok(n, k) || E < 1 || E > kMaxExperts || !dtype_ok(dtype))
        return CGL_EINVAL;
    if (score != CGL_SCORE_SOFTMAX && score != CGL_SCORE_SIGMOID) return CGL_EINVAL;
    if (n > 0 && (!grad_weights || !logits || !topk_idx || !grad_logits)) return CGL_EINVAL;
    const size_t item = dtype == CGL_F32 ? 4 : 2;
    if (!aligned(logits, item) || !aligned(grad_logits, item) || !aligned(topk_idx, 4) || !aligned(grad_weights, 4) ||
        !aligned(status_dev, 4))
        return CGL_EALIGN;
    const size_t rows = (size_t)n * E * item, slots = (size_t)n * k * 4;
    if (meet({grad_logits, rows}, {{logits, rows}, {grad_weights, slots}, {topk_idx, slots}})) return CGL_EINVAL;
    return launch_route_backward(grad_weights, logits, dtype, topk_idx, n, E, k, score, renorm != 0, scale, grad_logits,
                                 status_dev, static_cast<cudaStream_t>(stream));
}

static bool bf16_product_sizes_ok(int64_t rows, int E, int F, int K) {
    return E >= 1 && E <= kMaxExperts && F >= 1 && F <= (1 << 20) && K >= 8 && K % 8 == 0 && K <= (1 << 20) && rows >= 0 &&
           rows <= ((int64_t)1 << 31) - 4096;
}

static bool preact_ok(const void *preact, int dtype) { return preact == nullptr || dtype == CGL_BF16 || dtype == CGL_F32; }

static cgl_status bf16_product_ok(const uint16_t *a, int64_t rows, const uint16_t *w, int E, int F, int K,
                                  const int32_t *expert_offset, int act, const cgl_opts *opts, uint32_t *status_dev) {
    if (!bf16_product_sizes_ok(rows, E, F, K) || act < CGL_ACT_NONE || act > CGL_ACT_SWIGLU) return CGL_EINVAL;
    if (act == CGL_ACT_SWIGLU && F % 2 != 0) return CGL_EINVAL;
    const int cap = opt_cap(opts);
    if (cap < 0 || opt_sms(opts) < 0 || !flags_ok(opts)) return CGL_EINVAL;
    if (!expert_offset && (E != 1 || cap != 0)) return CGL_EINVAL;
    if (cap > 0 && rows < (int64_t)E * cap) return CGL_EINVAL;
    if (!w || (rows > 0 && !a)) return CGL_EINVAL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(expert_offset, 4) || !aligned(status_dev, 4)) return CGL_EALIGN;
    return CGL_OK;
}

cgl_status cgl_matmul_bf16(const uint16_t *a, int64_t rows, const uint16_t *w, int E, int F, int K,
                           const int32_t *expert_offset, const uint16_t *bias, int act, const uint16_t *residual,
                           uint16_t *y, void *preact, int preact_dtype, const cgl_opts *opts, uint32_t *status_dev, void *stream) {
    const cgl_status ok = bf16_product_ok(a, rows, w, E, F, K, expert_offset, act, opts, status_dev);
    if (ok != CGL_OK) return ok;
    if (rows > 0 && !y) return CGL_EINVAL;
    if (!preact_ok(preact, preact_dtype)) return CGL_EINVAL;
    if (!aligned(bias, 2) || !aligned(residual, 2) || !aligned(y, 2) || !aligned(preact, preact_dtype == CGL_F32 ? 4 : 2)) return CGL_EALIGN;
    // Blocks read their operands while others write; each reads its own part of the residual, which y may therefore be.
    const Bytes out = {y, (size_t)rows * (act == CGL_ACT_SWIGLU ? F / 2 : F) * 2}, z = {preact, (size_t)rows * F * (preact_dtype == CGL_F32 ? 4 : 2)},
                rest = {residual, out.n}, x = {a, (size_t)rows * K * 2}, weights = {w, (size_t)E * F * K * 2}, b = {bias, (size_t)E * F * 2},
                off = {expert_offset, (size_t)(E + 1) * 4};
    if (meet(out, {x, weights, b, off, z}) || meet(z, {x, weights, b, off, rest}) || (y != residual && meet(out, {rest}))) return CGL_EINVAL;
    const MatmulArgs m = {a, rows, w, E, F, K, expert_offset, opt_cap(opts), act, opt_sms(opts), status_dev};
    return launch_matmul_bf16(m, bias, residual, y, preact, preact_dtype == CGL_F32, static_cast<cudaStream_t>(stream));
}

size_t cgl_matmul_bf16_backward_workspace_bytes(int64_t rows, int E, int F, int K) {
    return bf16_product_sizes_ok(rows, E, F, K) ? matmul_bf16_backward_workspace_bytes(rows, E, F) : 0;
}

cgl_status cgl_matmul_bf16_backward(const uint16_t *grad_y, const uint16_t *a, int64_t rows, const uint16_t *w, int E,
                                    int F, int K, const int32_t *expert_offset, int act, const void *preact,
                                    int preact_dtype, uint16_t *grad_a, uint16_t *grad_w, uint16_t *grad_bias, void *workspace,
                                    size_t workspace_bytes, const cgl_opts *opts, uint32_t *status_dev, void *stream) {
    const cgl_status ok = bf16_product_ok(a, rows, w, E, F, K, expert_offset, act, opts, status_dev);
    if (ok != CGL_OK) return ok;
    if (rows > 0 && (!grad_y || (act != CGL_ACT_NONE && !preact))) return CGL_EINVAL;
    if (!preact_ok(preact, preact_dtype)) return CGL_EINVAL;
    if (workspace ? workspace_bytes < matmul_bf16_backward_workspace_bytes(rows, E, F) : grad_bias || !grad_y_is_dz(act, F, grad_y))
        return CGL_EINVAL;
    if (!aligned(grad_y, 2) || !aligned(preact, preact_dtype == CGL_F32 ? 4 : 2) || !aligned(grad_a, 16) || !aligned(grad_w, 16) || !aligned(grad_bias, 2) ||
        !aligned(workspace, 16))
        return CGL_EALIGN;
    // dz, the bias's gradient, grad_a and grad_w are made in this order.  grad_y and preact are done with after dz, but for a grad_y that is dz.
    const bool as_is = grad_y_is_dz(act, F, grad_y);
    const Bytes g = {grad_y, (size_t)rows * (act == CGL_ACT_SWIGLU ? F / 2 : F) * 2}, dz = {grad_y, as_is ? g.n : 0}, x = {a, (size_t)rows * K * 2},
                weights = {w, (size_t)E * F * K * 2}, z = {preact, act == CGL_ACT_NONE ? 0 : (size_t)rows * F * (preact_dtype == CGL_F32 ? 4 : 2)},
                off = {expert_offset, (size_t)(E + 1) * 4}, da = {grad_a, x.n}, dw = {grad_w, weights.n}, db = {grad_bias, (size_t)E * F * 2},
                scratch = {workspace, as_is && !grad_bias ? 0 : matmul_bf16_backward_workspace_bytes(rows, E, F)};
    if (meet(da, {weights, dz, dw, off}) || (grad_w && meet(da, {x})) || meet(dw, {x, dz, off}) || meet(db, {x, weights, dz, da, dw, off}) ||
        meet(scratch, {g, z, x, weights, off, da, dw, db}))
        return CGL_EINVAL;
    const MatmulArgs m = {a, rows, w, E, F, K, expert_offset, opt_cap(opts), act, opt_sms(opts), status_dev};
    return launch_matmul_bf16_backward(m, grad_y, preact, preact_dtype == CGL_F32, grad_a, grad_w, grad_bias, workspace,
                                       static_cast<cudaStream_t>(stream));
}

cgl_status cgl_selftest_matmul_bf16_timeout(int what, const uint16_t *x, int64_t rows, const uint16_t *y_or_w, int F, int K,
                                            uint16_t *result, int64_t wait_cycles, uint32_t *status_dev, void *stream) {
    if (what < 0 || what > 2 || F < 8 || F % 8 != 0 || F > (1 << 20) || K < 8 || K % 8 != 0 || K > (1 << 20) || rows < 1 ||
        rows > (1 << 20) || wait_cycles < 0)
        return CGL_EINVAL;
    if (!x || !y_or_w || !result || !status_dev) return CGL_EINVAL;
    if (!aligned(x, 16) || !aligned(y_or_w, 16) || !aligned(result, 16) || !aligned(status_dev, 4)) return CGL_EALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MatmulArgs m = {what == 1 ? nullptr : x, rows, what == 2 ? nullptr : y_or_w, 1, F, K, nullptr, 0, CGL_ACT_NONE, 0, status_dev, wait_cycles};
    if (what == 0) return launch_matmul_bf16(m, nullptr, nullptr, result, nullptr, false, s);
    // without an activation and a bias's gradient the products read grad_y itself: no workspace
    return launch_matmul_bf16_backward(m, what == 1 ? x : y_or_w, nullptr, false, what == 1 ? result : nullptr,
                                       what == 2 ? result : nullptr, nullptr, nullptr, s);
}

}  // extern "C"
