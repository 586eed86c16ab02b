// Internal launchers behind the C ABI (not exported).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "cgl.h"

namespace cgl {

// Raise a kernel's dynamic shared-memory limit once per device; false on error.
bool ensure_smem_attr(const void *kernel, size_t bytes);

// SMs on the current device (cached per device); 0 on error.
int device_sm_count();

// Grid for a persistent kernel (CTAs loop over `work` items): SMs in use x
// min(target CTAs per SM, CTAs per SM that fit), at most `work`; 0 on error.
int persistent_grid(const void *kernel, int threads, size_t smem, int target_per_sm, int num_sms_cap,
                    int64_t work);

// Grid for a grid-stride copy kernel: enough CTAs for `work_ctas`, capped at
// (SMs in use) x (resident CTAs per SM).
int copy_grid(const void *kernel, int threads, int64_t work_ctas, int num_sms_cap);

// Launch `kernel` with programmatic stream serialisation: it may start while
// the previous kernel in the stream is finishing, and must griddep_wait()
// before reading anything that kernel (or an earlier one) wrote.  One exception:
// balance_main_kernel, always launched right behind balance_count_kernel, reads
// before its wait what the kernels ahead of that one wrote, because that one's
// blocks trigger it only behind their own waits.  No kernel may come between the
// two, and that trigger must stay behind the wait.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

size_t layout_workspace_bytes(int64_t n, int k, int E, int R);

// True if some layout kernel for these sizes needs more shared memory than a
// kernel gets without raising its attribute (host-side bookkeeping on first use).
bool layout_needs_smem_optin(int E, int R, int k);

// True if the layout for these sizes runs as one cooperative kernel on the current device.
bool layout_fused_fits(int64_t n, int k, int E, int R);

cgl_status launch_layout(const int32_t *idx, int64_t n, int k, int E, int R, int cap,
                         int32_t *tokens_per_expert, int32_t *tokens_per_rank, uint8_t *in_rank,
                         int32_t *expert_offset, int32_t *max_count, int32_t *dst_pos,
                         int32_t *recv_src, void *ws, uint32_t *status, cudaStream_t stream);

// Per-rank layout: keys are destination ranks (one row per token and rank).
cgl_status launch_rank_layout(const int32_t *idx, int64_t n, int k, int E, int R, int cap,
                              int32_t *tokens_per_rank, int32_t *rank_offset, int32_t *max_count,
                              int32_t *rank_dst, int32_t *recv_token, void *ws, uint32_t *status,
                              cudaStream_t stream);

// pow2: power-of-two (UE8M0) scales instead of amax_c / 448 (cgl_opts.flags).
// claim: null (static token order), or two 64-bit words that are zero when
// the kernel starts (a token counter the CTAs claim from, and a count of
// finished CTAs); the last CTA to finish zeroes both again.
cgl_status launch_dispatch_fp8(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos,
                               uint8_t *recv_x, float *recv_scale, int64_t recv_rows,
                               int num_sms, bool pow2, uint32_t *status, cudaStream_t stream,
                               unsigned long long *claim = nullptr);

cgl_status launch_dispatch_bf16(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos,
                                uint16_t *recv_x, int64_t recv_rows, int num_sms, uint32_t *status,
                                cudaStream_t stream, unsigned long long *claim = nullptr);

cgl_status launch_combine(const uint16_t *y, int64_t recv_rows, const int32_t *dst_pos,
                          const float *w, int64_t n, int h, int k, uint16_t *out, int num_sms,
                          uint32_t *status, cudaStream_t stream);

// One block running the layout's bounded inter-block wait, with its exit path
// (generation advance), on a workspace header whose flags hold no tag it waits for.
cgl_status launch_wait_probe(uint64_t *ws, int nflags, uint32_t *status, cudaStream_t stream);

// Dynamic shared memory of the fused decode kernel (bytes).
size_t decode_fused_smem_bytes(int64_t n, int k, int E, int R);

cgl_status launch_decode_dispatch_fp8(const int32_t *idx, int64_t n, int k, int E, int R, int cap,
                                      const uint16_t *x, int h, int32_t *tokens_per_expert,
                                      int32_t *tokens_per_rank, uint8_t *in_rank, int32_t *expert_offset,
                                      int32_t *max_count, int32_t *dst_pos, int32_t *recv_src,
                                      uint8_t *recv_x, float *recv_scale, int num_sms, bool pow2,
                                      uint32_t *status, cudaStream_t stream);

// Fused layout + FP8 dispatch (one cooperative launch when it applies, else
// the layout and the dispatch kernels in turn).
size_t layout_dispatch_workspace_bytes(int64_t n, int k, int E, int R);
bool layout_dispatch_fused_fits(int64_t n, int k, int E, int R, int h, int num_sms);
cgl_status launch_layout_dispatch_fp8(const int32_t *idx, int64_t n, int k, int E, int R, int cap,
                                      const uint16_t *x, int h, int32_t *tokens_per_expert,
                                      int32_t *tokens_per_rank, uint8_t *in_rank, int32_t *expert_offset,
                                      int32_t *max_count, int32_t *dst_pos, int32_t *recv_src, uint8_t *recv_x,
                                      float *recv_scale, void *ws, int num_sms, bool pow2, uint32_t *status,
                                      cudaStream_t stream);

cgl_status launch_combine_backward(const uint16_t *g, const uint16_t *y, int64_t recv_rows,
                                   const int32_t *dst_pos, const float *w, int64_t n, int h, int k,
                                   uint16_t *grad_y, float *grad_w, int num_sms, uint32_t *status,
                                   cudaStream_t stream);

// MXFP4 rows (dtype: a cgl_dtype; cols a multiple of 32).
cgl_status launch_quantize_mxfp4(const void *x, int dtype, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                                 int num_sms, cudaStream_t stream);
cgl_status launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                   int dtype, int num_sms, cudaStream_t stream);
cgl_status launch_dispatch_mxfp4(const uint16_t *x, int64_t n, int h, int k, const int32_t *dst_pos, uint8_t *recv_x,
                                 uint8_t *recv_scale, int64_t recv_rows, int num_sms, uint32_t *status,
                                 cudaStream_t stream, unsigned long long *claim);

// The experts' product on MXFP4 rows (off null: one expert, all rows; wait_cycles: a wait's limit, < 0: about a second).
cgl_status launch_matmul_mxfp4(const uint8_t *a, const uint8_t *sa, int64_t rows, const uint8_t *w, const uint8_t *sw,
                               int E, int F, int K, const int32_t *off, int64_t cap, uint16_t *y, int num_sms,
                               uint32_t *status, cudaStream_t stream, int64_t wait_cycles = -1);

// Balance loss (score: 0 softmax, 1 normalised sigmoid; grad null: loss and counts only).
size_t balance_workspace_bytes(int64_t n, int k, int E, int64_t S);
cgl_status launch_balance_loss(const void *logits, int dtype, const int32_t *idx, int64_t n, int k, int E, int64_t S,
                               float alpha, int score, const float *grad_loss, float *loss, int32_t *counts,
                               int32_t *routed, void *grad, void *ws, uint32_t *status, cudaStream_t stream);
cgl_status launch_balance_loss_backward(const float *grad_loss, const void *logits, int dtype, const int32_t *idx,
                                        int64_t n, int k, int E, int64_t S, float alpha, int score,
                                        const int32_t *counts, const int32_t *routed, void *grad, cudaStream_t stream);

// Routing (groups: experts in neighbouring equal groups, the best `keep` stay).
struct RouteArgs {
    const void *logits;
    int dtype;
    int64_t n;
    int E, k;
    const float *bias;
    int groups, keep, by, score;
    bool renorm;
    float scale;
    int32_t *idx;
    float *weights;
    uint32_t *status;
    int batch = 1;   // tokens a warp takes together (set by launch_route)
};
cgl_status launch_route(const RouteArgs &a, cudaStream_t stream);
cgl_status launch_route_backward(const float *grad_weights, const void *logits, int dtype, const int32_t *idx, int64_t n,
                                 int E, int k, int score, bool renorm, float scale, void *grad, uint32_t *status,
                                 cudaStream_t stream);

// The experts' BF16 product and its gradients (off null: one expert, all rows; wait_cycles: a wait's limit, < 0: about a second).
struct MatmulArgs {
    const uint16_t *a;
    int64_t rows;
    const uint16_t *w;
    int E, F, K;   // F: rows of w (both halves of a gated one)
    const int32_t *off;
    int64_t cap;
    int act;
    int num_sms;
    uint32_t *status;
    int64_t wait_cycles = -1;
};
// preact: BF16, or binary32 (preact_f32).
cgl_status launch_matmul_bf16(const MatmulArgs &m, const uint16_t *bias, const uint16_t *residual, uint16_t *y, void *preact,
                              bool preact_f32, cudaStream_t stream);
size_t matmul_bf16_backward_workspace_bytes(int64_t rows, int E, int F);
cgl_status launch_matmul_bf16_backward(const MatmulArgs &m, const uint16_t *grad_y, const void *preact, bool preact_f32, uint16_t *grad_a,
                                       uint16_t *grad_w, uint16_t *grad_bias, void *ws, cudaStream_t stream);
// Whether the products of the backward pass read grad_y itself, as dz: then only a bias's gradient needs the workspace.
bool grad_y_is_dz(int act, int F, const uint16_t *grad_y);
// Its first step: dz for the products (BF16, rows of *ld values; grad_y itself where it serves) and grad_bias, where wanted.
cgl_status launch_slope(const MatmulArgs &m, const uint16_t *grad_y, const void *preact, bool preact_f32, bool products,
                        uint16_t *grad_bias, void *ws, const uint16_t **dz, int64_t *ld, cudaStream_t stream);

}  // namespace cgl
