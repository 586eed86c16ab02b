"""Single-GPU MoE layout / dispatch / combine for B200 (sm_100a), over the C ABI in include/cgl.h.

Python binding only: this module allocates outputs with torch (device memory),
picks the current CUDA stream, and passes raw pointers to libcgl.so.  Every
step of the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and every call raises if the library is missing or the
tensors are not on a CUDA device.

    lay = get_layout(topk_idx, num_experts=256, num_ranks=64)
    recv_x, recv_scale = dispatch_fp8(x, lay.dst_pos, lay.num_recv_rows)
    out = combine(y, lay.dst_pos, topk_weights)

The operations are the dispatch ("send each token to its gated experts") and
combine ("merge the expert outputs back, accumulating") of the DeepEP pages
(GitHub-issue mirror "Technical Overview of DeepEP"; brainleap "Day2 DeepEP",
"DeepEP是什么" and "All-to-All通信"), with FP8 dispatch and BF16 combine as in
their benchmark settings, run inside one GPU with ranks as expert partitions.

Between the two, with rows and weights in MXFP4 (four bits a value, one
power-of-two scale per 32), and for training the loss that keeps the routing even:

    wq, ws = quantize_mxfp4(w)                       # once; w [E, out, H]
    recv_x, recv_scale = dispatch_mxfp4(x, lay.dst_pos, lay.num_recv_rows)
    y = matmul_mxfp4(recv_x, recv_scale, wq, ws, lay.expert_offset, lay.capacity)
    aux = balance_loss(logits, topk_idx, alpha=1e-3, grad_loss=g)   # .loss, .counts, .grad_logits

In front of the layout the gate, and between dispatch and combine the same product on BF16 rows, with
bias, activation and residual; both have a backward pass:

    r = route(logits, 8, score="sigmoid", bias=b, num_groups=8, topk_groups=4)      # .topk_idx, .topk_weights
    h = matmul_bf16(recv_x, w1, lay.expert_offset, activation="swiglu")
"""

from __future__ import annotations

import ctypes as C
import os
from typing import NamedTuple, Optional

import torch

__all__ = [
    "CglError", "Layout", "RankLayout", "lib", "get_layout", "get_rank_layout", "dispatch_fp8", "dispatch_bf16", "combine",
    "combine_backward", "decode_dispatch_fp8", "layout_workspace_bytes", "layout_kernel_count", "status_bits", "check_status", "new_status",
    "quantize_mxfp4", "dequantize_mxfp4", "dispatch_mxfp4", "matmul_mxfp4", "BalanceLoss", "balance_loss",
    "balance_loss_backward", "balance_loss_workspace_bytes",
    "Routing", "route", "route_backward", "matmul_bf16", "MatmulGrads", "matmul_bf16_backward",
    "matmul_bf16_backward_workspace_bytes",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcgl.so")

OK, EINVAL, EALIGN, ERANGE, ECAPACITY, ETIMEOUT, ECUDA, ENOTIMPL = range(8)
_NAMES = {OK: "CGL_OK", EINVAL: "CGL_EINVAL", EALIGN: "CGL_EALIGN", ERANGE: "CGL_ERANGE",
          ECAPACITY: "CGL_ECAPACITY", ETIMEOUT: "CGL_ETIMEOUT", ECUDA: "CGL_ECUDA",
          ENOTIMPL: "CGL_ENOTIMPL"}


class CglError(RuntimeError):
    """A non-OK status from the library (host-side) or a device error bit."""

    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        super().__init__(f"{where}: {_NAMES.get(code, code)} ({detail or _status_string(code)})")


class Opts(C.Structure):
    _fields_ = [("num_sms", C.c_int32), ("capacity", C.c_int32), ("flags", C.c_uint32), ("scratch", C.c_void_p)]


OPT_UE8M0_SCALES = 1   # cgl_opts.flags: power-of-two (UE8M0) FP8 scales


_lib = None


def lib():
    """The loaded libcgl.so (ctypes), with argument types declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libcgl.so is not built ({LIB_PATH}); run "
                               "`python -m combine_get_layout_02_b200.build`")
        L = C.CDLL(LIB_PATH)
        P, I64, I = C.c_void_p, C.c_int64, C.c_int
        OP = C.POINTER(Opts)
        L.cgl_version.argtypes = []
        L.cgl_version.restype = I
        L.cgl_status_string.argtypes = [I]
        L.cgl_status_string.restype = C.c_char_p
        L.cgl_layout_workspace_bytes.argtypes = [I64, I, I, I]
        L.cgl_layout_workspace_bytes.restype = C.c_size_t
        L.cgl_layout_kernel_count.argtypes = [I64, I, I, I]
        L.cgl_layout_kernel_count.restype = I
        L.cgl_get_layout.argtypes = [P, I64, I, I, I, OP, P, P, P, P, P, P, P, P, C.c_size_t, P, P]
        L.cgl_get_layout.restype = I
        L.cgl_get_rank_layout.argtypes = [P, I64, I, I, I, OP, P, P, P, P, P, P, C.c_size_t, P, P]
        L.cgl_get_rank_layout.restype = I
        L.cgl_dispatch_fp8.argtypes = [P, I64, I, I, P, P, P, I64, OP, P, P]
        L.cgl_dispatch_fp8.restype = I
        L.cgl_dispatch_bf16.argtypes = [P, I64, I, I, P, P, I64, OP, P, P]
        L.cgl_dispatch_bf16.restype = I
        L.cgl_combine.argtypes = [P, I64, P, P, I64, I, I, P, OP, P, P]
        L.cgl_combine.restype = I
        L.cgl_decode_dispatch_fp8.argtypes = [P, I64, I, I, I, OP, P, I, P, P, P, P, P, P, P, P, P, P, P]
        L.cgl_decode_dispatch_fp8.restype = I
        L.cgl_layout_dispatch_workspace_bytes.argtypes = [I64, I, I, I]
        L.cgl_layout_dispatch_workspace_bytes.restype = C.c_size_t
        L.cgl_layout_dispatch_kernel_count.argtypes = [I64, I, I, I, I, OP]
        L.cgl_layout_dispatch_kernel_count.restype = I
        L.cgl_layout_dispatch_fp8.argtypes = [P, I64, I, I, I, OP, P, I, P, P, P, P, P, P, P, P, P, P,
                                              C.c_size_t, P, P]
        L.cgl_layout_dispatch_fp8.restype = I
        L.cgl_combine_backward.argtypes = [P, P, I64, P, P, I64, I, I, P, P, OP, P, P]
        L.cgl_combine_backward.restype = I
        L.cgl_quantize_mxfp4.argtypes = [P, I, I64, I64, P, P, OP, P]
        L.cgl_quantize_mxfp4.restype = I
        L.cgl_dequantize_mxfp4.argtypes = [P, P, I64, I64, P, I, OP, P]
        L.cgl_dequantize_mxfp4.restype = I
        L.cgl_dispatch_mxfp4.argtypes = [P, I64, I, I, P, P, P, I64, OP, P, P]
        L.cgl_dispatch_mxfp4.restype = I
        L.cgl_matmul_mxfp4.argtypes = [P, P, I64, P, P, I, I, I, P, P, OP, P, P]
        L.cgl_matmul_mxfp4.restype = I
        L.cgl_balance_loss_workspace_bytes.argtypes = [I64, I, I, I64]
        L.cgl_balance_loss_workspace_bytes.restype = C.c_size_t
        L.cgl_balance_loss.argtypes = [P, I, P, I64, I, I, I64, C.c_float, I, P, P, P, P, P, P, C.c_size_t, P, P]
        L.cgl_balance_loss.restype = I
        L.cgl_balance_loss_backward.argtypes = [P, P, I, P, I64, I, I, I64, C.c_float, I, P, P, P, P]
        L.cgl_balance_loss_backward.restype = I
        F = C.c_float
        L.cgl_route.argtypes = [P, I, I64, I, I, P, I, I, I, I, I, F, P, P, P, P]
        L.cgl_route.restype = I
        L.cgl_route_backward.argtypes = [P, P, I, P, I64, I, I, I, I, F, P, P, P]
        L.cgl_route_backward.restype = I
        L.cgl_matmul_bf16.argtypes = [P, I64, P, I, I, I, P, P, I, P, P, P, I, OP, P, P]
        L.cgl_matmul_bf16.restype = I
        L.cgl_matmul_bf16_backward_workspace_bytes.argtypes = [I64, I, I, I]
        L.cgl_matmul_bf16_backward_workspace_bytes.restype = C.c_size_t
        L.cgl_matmul_bf16_backward.argtypes = [P, P, I64, P, I, I, I, P, I, P, I, P, P, P, P, C.c_size_t, OP, P, P]
        L.cgl_matmul_bf16_backward.restype = I
        _lib = L
    return _lib


def _status_string(code: int) -> str:
    try:
        return lib().cgl_status_string(int(code)).decode()
    except RuntimeError:
        return "status"


def _check(code: int, where: str):
    if code != OK:
        raise CglError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _opts(num_sms: int = 0, capacity: int = 0, pow2_scales: bool = False, scratch: Optional[torch.Tensor] = None):
    if scratch is None and num_sms == 0 and capacity == 0 and not pow2_scales:
        return None   # NULL: all fields zero
    sp = None
    if scratch is not None:
        if not scratch.is_cuda or scratch.numel() * scratch.element_size() < 16 or not scratch.is_contiguous():
            raise CglError(EINVAL, "scratch", "a contiguous device tensor of at least 16 bytes")
        sp = scratch.data_ptr()
    return C.byref(Opts(int(num_sms), int(capacity), OPT_UE8M0_SCALES if pow2_scales else 0, sp))


def new_scratch(device=None) -> torch.Tensor:
    """Zeroed 16-byte device scratch (cgl_opts.scratch) for dispatch_fp8 / dispatch_bf16: with it the
    dispatch kernel hands tokens out dynamically; each call leaves it zero.  Calls that may run at the
    same time need their own."""
    return torch.zeros(2, dtype=torch.int64, device=device or "cuda")


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status word (uint32 stored as int32[1])."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def status_bits(status: torch.Tensor) -> list:
    """Names of the device error bits set in a status word (reads it: synchronises)."""
    v = int(status.item()) & 0xFFFFFFFF
    return [_NAMES[c] for c in range(1, 8) if v & (1 << c)]


def check_status(status: torch.Tensor, where: str = "device"):
    v = int(status.item()) & 0xFFFFFFFF
    for c in range(1, 8):
        if v & (1 << c):
            raise CglError(c, where, "device-reported")


def layout_workspace_bytes(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int) -> int:
    return int(lib().cgl_layout_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks))


def layout_kernel_count(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int) -> int:
    """Kernels one get_layout call launches for these sizes on the current device (1 or 2)."""
    return int(lib().cgl_layout_kernel_count(num_tokens, num_topk, num_experts, num_ranks))


class Layout(NamedTuple):
    tokens_per_expert: torch.Tensor   # int32 [E]
    tokens_per_rank: torch.Tensor     # int32 [R]
    is_token_in_rank: torch.Tensor    # uint8 [N, R]
    expert_offset: torch.Tensor       # int32 [E + 1]
    max_count: torch.Tensor           # int32 [1]
    dst_pos: torch.Tensor             # int32 [N, k]
    recv_src: torch.Tensor            # int32 [num_recv_rows]
    num_recv_rows: int                # N*k (compact) or E*capacity (padded)
    capacity: int


def get_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, capacity: int = 0, *,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               out: Optional[Layout] = None, stream=None) -> Layout:
    """Counts, prefix sums and stable receive rows for top-k routing (cgl_get_layout)."""
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    n, k = idx.shape
    E, R = int(num_experts), int(num_ranks)
    dev = idx.device
    rows = E * capacity if capacity > 0 else n * k
    ws_bytes = layout_workspace_bytes(n, k, E, R)
    if ws_bytes == 0:
        raise CglError(EINVAL, "get_layout", "invalid sizes")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if out is None:
        out = Layout(
            torch.empty(E, dtype=torch.int32, device=dev),
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((n, R), dtype=torch.uint8, device=dev),
            torch.empty(E + 1, dtype=torch.int32, device=dev),
            torch.empty(1, dtype=torch.int32, device=dev),
            torch.empty((n, k), dtype=torch.int32, device=dev),
            torch.empty(rows, dtype=torch.int32, device=dev),
            rows, int(capacity))
    code = lib().cgl_get_layout(
        _ptr(idx), n, k, E, R, _opts(0, capacity), _ptr(out.tokens_per_expert),
        _ptr(out.tokens_per_rank), _ptr(out.is_token_in_rank), _ptr(out.expert_offset),
        _ptr(out.max_count), _ptr(out.dst_pos), _ptr(out.recv_src), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    _check(code, "cgl_get_layout")
    return out


class RankLayout(NamedTuple):
    tokens_per_rank: torch.Tensor     # int32 [R]
    rank_offset: torch.Tensor         # int32 [R + 1]
    max_count: torch.Tensor           # int32 [1]
    rank_dst: torch.Tensor            # int32 [N, k]  (row per first slot on each rank, else -1)
    recv_token: torch.Tensor          # int32 [num_recv_rows]
    num_recv_rows: int                # N*k (compact) or R*capacity (padded)
    capacity: int


def get_rank_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, capacity: int = 0, *,
                    status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    out: Optional[RankLayout] = None, stream=None) -> RankLayout:
    """One copy per (token, destination rank): the deduplicated layout (cgl_get_rank_layout)."""
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    n, k = idx.shape
    E, R = int(num_experts), int(num_ranks)
    dev = idx.device
    rows = R * capacity if capacity > 0 else n * k
    ws_bytes = layout_workspace_bytes(n, k, R, R)
    if ws_bytes == 0 or E % R:
        raise CglError(EINVAL, "get_rank_layout", "invalid sizes")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if out is None:
        out = RankLayout(
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty(R + 1, dtype=torch.int32, device=dev),
            torch.empty(1, dtype=torch.int32, device=dev),
            torch.empty((n, k), dtype=torch.int32, device=dev),
            torch.empty(rows, dtype=torch.int32, device=dev),
            rows, int(capacity))
    code = lib().cgl_get_rank_layout(
        _ptr(idx), n, k, E, R, _opts(0, capacity), _ptr(out.tokens_per_rank), _ptr(out.rank_offset),
        _ptr(out.max_count), _ptr(out.rank_dst), _ptr(out.recv_token), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    _check(code, "cgl_get_rank_layout")
    return out


def dispatch_fp8(x: torch.Tensor, dst_pos: torch.Tensor, num_recv_rows: int, *,
                 recv_x: Optional[torch.Tensor] = None, recv_scale: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, num_sms: int = 0, pow2_scales: bool = False,
                 scratch: Optional[torch.Tensor] = None, stream=None):
    """FP8 E4M3 dispatch with per-token 1x128 fp32 scales (cgl_dispatch_fp8).

    pow2_scales: power-of-two (UE8M0) scales (CGL_OPT_UE8M0_SCALES).
    scratch: new_scratch() (cgl_opts.scratch): tokens handed out dynamically, same results.
    Returns (recv_x uint8 [rows, H], recv_scale fp32 [rows, H/128]); rows that
    receive no copy are left as they were (uninitialised when allocated here)."""
    x = _dev(x, "x", torch.bfloat16, 2)
    dst = _dev(dst_pos, "dst_pos", torch.int32, 2)
    n, h = x.shape
    k = dst.shape[1]
    if recv_x is None:
        recv_x = torch.empty((num_recv_rows, h), dtype=torch.uint8, device=x.device)
    if recv_scale is None:
        recv_scale = torch.empty((num_recv_rows, h // 128), dtype=torch.float32, device=x.device)
    code = lib().cgl_dispatch_fp8(_ptr(x), n, h, k, _ptr(dst), _ptr(recv_x), _ptr(recv_scale),
                                  int(num_recv_rows), _opts(num_sms, 0, pow2_scales, scratch), _ptr(status),
                                  _stream(stream))
    _check(code, "cgl_dispatch_fp8")
    return recv_x, recv_scale


def dispatch_bf16(x: torch.Tensor, dst_pos: torch.Tensor, num_recv_rows: int, *,
                  recv_x: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  num_sms: int = 0, scratch: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """BF16 row dispatch (cgl_dispatch_bf16); also the combine-backward re-dispatch of grads.

    scratch: new_scratch() (cgl_opts.scratch): tokens handed out dynamically, same results."""
    x = _dev(x, "x", torch.bfloat16, 2)
    dst = _dev(dst_pos, "dst_pos", torch.int32, 2)
    n, h = x.shape
    k = dst.shape[1]
    if recv_x is None:
        recv_x = torch.empty((num_recv_rows, h), dtype=torch.bfloat16, device=x.device)
    code = lib().cgl_dispatch_bf16(_ptr(x), n, h, k, _ptr(dst), _ptr(recv_x), int(num_recv_rows),
                                   _opts(num_sms, 0, False, scratch), _ptr(status), _stream(stream))
    _check(code, "cgl_dispatch_bf16")
    return recv_x


def combine(y: torch.Tensor, dst_pos: torch.Tensor, topk_weights: torch.Tensor, *,
            out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            num_sms: int = 0, stream=None) -> torch.Tensor:
    """Top-k weighted BF16 combine with an fp32 fixed-order accumulator (cgl_combine)."""
    y = _dev(y, "y", torch.bfloat16, 2)
    dst = _dev(dst_pos, "dst_pos", torch.int32, 2)
    w = _dev(topk_weights, "topk_weights", torch.float32, 2)
    n, k = dst.shape
    h = y.shape[1]
    if out is None:
        out = torch.empty((n, h), dtype=torch.bfloat16, device=y.device)
    code = lib().cgl_combine(_ptr(y), y.shape[0], _ptr(dst), _ptr(w), n, h, k, _ptr(out),
                             _opts(num_sms), _ptr(status), _stream(stream))
    _check(code, "cgl_combine")
    return out


def combine_backward(grad_out: torch.Tensor, y: torch.Tensor, dst_pos: torch.Tensor,
                     topk_weights: torch.Tensor, *, grad_y: Optional[torch.Tensor] = None,
                     grad_w: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     num_sms: int = 0, stream=None):
    """Gradient of combine: (grad_y BF16 [rows, H], grad_w fp32 [N, k]) (cgl_combine_backward)."""
    g = _dev(grad_out, "grad_out", torch.bfloat16, 2)
    y = _dev(y, "y", torch.bfloat16, 2)
    dst = _dev(dst_pos, "dst_pos", torch.int32, 2)
    w = _dev(topk_weights, "topk_weights", torch.float32, 2)
    n, k = dst.shape
    h = g.shape[1]
    if grad_y is None:
        grad_y = torch.empty_like(y)
    if grad_w is None:
        grad_w = torch.empty((n, k), dtype=torch.float32, device=g.device)
    code = lib().cgl_combine_backward(_ptr(g), _ptr(y), y.shape[0], _ptr(dst), _ptr(w), n, h, k,
                                      _ptr(grad_y), _ptr(grad_w), _opts(num_sms), _ptr(status),
                                      _stream(stream))
    _check(code, "cgl_combine_backward")
    return grad_y, grad_w


def decode_dispatch_fp8(topk_idx: torch.Tensor, x: torch.Tensor, num_experts: int, num_ranks: int,
                        capacity: int = 0, *, out: Optional[Layout] = None,
                        recv_x: Optional[torch.Tensor] = None, recv_scale: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, num_sms: int = 0, pow2_scales: bool = False,
                        stream=None):
    """Layout + FP8 dispatch of a small (decode) batch in one launch (cgl_decode_dispatch_fp8).

    Returns (Layout, recv_x uint8 [rows, H], recv_scale fp32 [rows, H/128])."""
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    x = _dev(x, "x", torch.bfloat16, 2)
    n, k = idx.shape
    h = x.shape[1]
    E, R = int(num_experts), int(num_ranks)
    dev = idx.device
    rows = E * capacity if capacity > 0 else n * k
    if out is None:
        out = Layout(
            torch.empty(E, dtype=torch.int32, device=dev),
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((n, R), dtype=torch.uint8, device=dev),
            torch.empty(E + 1, dtype=torch.int32, device=dev),
            torch.empty(1, dtype=torch.int32, device=dev),
            torch.empty((n, k), dtype=torch.int32, device=dev),
            torch.empty(rows, dtype=torch.int32, device=dev),
            rows, int(capacity))
    if recv_x is None:
        recv_x = torch.empty((rows, h), dtype=torch.uint8, device=dev)
    if recv_scale is None:
        recv_scale = torch.empty((rows, h // 128), dtype=torch.float32, device=dev)
    code = lib().cgl_decode_dispatch_fp8(
        _ptr(idx), n, k, E, R, _opts(num_sms, capacity, pow2_scales), _ptr(x), h, _ptr(out.tokens_per_expert),
        _ptr(out.tokens_per_rank), _ptr(out.is_token_in_rank), _ptr(out.expert_offset), _ptr(out.max_count),
        _ptr(out.dst_pos), _ptr(out.recv_src), _ptr(recv_x), _ptr(recv_scale), _ptr(status), _stream(stream))
    _check(code, "cgl_decode_dispatch_fp8")
    return out, recv_x, recv_scale


def layout_dispatch_workspace_bytes(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int) -> int:
    return int(lib().cgl_layout_dispatch_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks))


def layout_dispatch_kernel_count(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int,
                                 hidden: int, num_sms: int = 0) -> int:
    return int(lib().cgl_layout_dispatch_kernel_count(num_tokens, num_topk, num_experts, num_ranks, hidden,
                                                      _opts(num_sms, 0)))


def layout_dispatch_fp8(topk_idx: torch.Tensor, x: torch.Tensor, num_experts: int, num_ranks: int,
                        capacity: int = 0, *, out: Optional[Layout] = None,
                        recv_x: Optional[torch.Tensor] = None, recv_scale: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        num_sms: int = 0, pow2_scales: bool = False, stream=None):
    """Layout + FP8 dispatch of any batch in one call (cgl_layout_dispatch_fp8).

    Returns (Layout, recv_x uint8 [rows, H], recv_scale fp32 [rows, H/128])."""
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    x = _dev(x, "x", torch.bfloat16, 2)
    n, k = idx.shape
    h = x.shape[1]
    E, R = int(num_experts), int(num_ranks)
    dev = idx.device
    rows = E * capacity if capacity > 0 else n * k
    ws_bytes = layout_dispatch_workspace_bytes(n, k, E, R)
    if ws_bytes == 0:
        raise CglError(EINVAL, "layout_dispatch_fp8", "invalid sizes")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if out is None:
        out = Layout(
            torch.empty(E, dtype=torch.int32, device=dev),
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((n, R), dtype=torch.uint8, device=dev),
            torch.empty(E + 1, dtype=torch.int32, device=dev),
            torch.empty(1, dtype=torch.int32, device=dev),
            torch.empty((n, k), dtype=torch.int32, device=dev),
            torch.empty(rows, dtype=torch.int32, device=dev),
            rows, int(capacity))
    if recv_x is None:
        recv_x = torch.empty((rows, h), dtype=torch.uint8, device=dev)
    if recv_scale is None:
        recv_scale = torch.empty((rows, h // 128), dtype=torch.float32, device=dev)
    code = lib().cgl_layout_dispatch_fp8(
        _ptr(idx), n, k, E, R, _opts(num_sms, capacity, pow2_scales), _ptr(x), h, _ptr(out.tokens_per_expert),
        _ptr(out.tokens_per_rank), _ptr(out.is_token_in_rank), _ptr(out.expert_offset), _ptr(out.max_count),
        _ptr(out.dst_pos), _ptr(out.recv_src), _ptr(recv_x), _ptr(recv_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    _check(code, "cgl_layout_dispatch_fp8")
    return out, recv_x, recv_scale


# ---- MXFP4 rows, the experts' product, the balance loss ----------------------------------------

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # cgl_dtype
_SCORES = {"softmax": 0, "sigmoid": 1}                              # cgl_score


def _on(stream, t: torch.Tensor, name: str):
    """Makes `stream` (a torch stream or a handle) current on t's device, so that what a call allocates belongs to it as well."""
    device = _dev(t, name).device
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)   # without a device: the current one's
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, {name} on {device}")
    return torch.cuda.stream(stream)


def _launch(where: str, fn, device, *args):
    """fn(*args, stream) with `device` current and on its current stream."""
    # the raw stream: torch.cuda.current_stream() makes a Stream object, 4 us of a small call's 15
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            code = fn(*args, raw)
    else:
        code = fn(*args, raw)
    if code != OK:
        raise CglError(code, where)


def _buf(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    """An output the caller may have passed: checked, or allocated on `like`'s device."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)   # 0.5 us less than torch.empty
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != like.device:
        raise TypeError(f"{name} must be {dtype} on {like.device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t


def _same(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _float_type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return _DTYPES[t.dtype]


def quantize_mxfp4(x: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, num_sms: int = 0, stream=None):
    """MXFP4 codes and scales of x [..., C], C % 32 == 0 (cgl_quantize_mxfp4).

    Returns (codes uint8 [..., C/2], two codes a byte with the lower index in the low half;
    scales uint8 [..., C/32], 2^(byte - 127)).  Blocks with an infinity or NaN get scale byte 255 (NaN)."""
    if stream is not None:
        with _on(stream, x, "x"):
            return quantize_mxfp4(x, codes=codes, scales=scales, num_sms=num_sms)
    x = _dev(x, "x")
    dt = _float_type(x, "x")
    *lead, c = x.shape or (0,)
    if c == 0 or c % 32:
        raise ValueError(f"x must have a last dimension that is a multiple of 32, got {tuple(x.shape)}")
    codes = _buf(codes, "codes", (*lead, c // 2), torch.uint8, x)
    scales = _buf(scales, "scales", (*lead, c // 32), torch.uint8, x)
    _launch("cgl_quantize_mxfp4", lib().cgl_quantize_mxfp4, x.device, _ptr(x), dt, x.numel() // c, c,
            _ptr(codes), _ptr(scales), _opts(num_sms))
    return codes, scales


def dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16, *,
                     out: Optional[torch.Tensor] = None, num_sms: int = 0, stream=None) -> torch.Tensor:
    """The values MXFP4 codes [..., C/2] and scales [..., C/32] stand for, [..., C] (cgl_dequantize_mxfp4)."""
    if stream is not None:
        with _on(stream, codes, "codes"):
            return dequantize_mxfp4(codes, scales, dtype, out=out, num_sms=num_sms)
    codes = _dev(codes, "codes", torch.uint8)
    scales = _dev(scales, "scales", torch.uint8)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    _same(codes.device, scales=scales)
    *lead, half = codes.shape or (0,)
    c = 2 * half
    if c == 0 or c % 32 or scales.shape != (*lead, c // 32):
        raise ValueError(f"codes [..., C/2] and scales [..., C/32] expected, got {tuple(codes.shape)}, {tuple(scales.shape)}")
    out = _buf(out, "out", (*lead, c), dtype, codes)
    _launch("cgl_dequantize_mxfp4", lib().cgl_dequantize_mxfp4, codes.device, _ptr(codes), _ptr(scales),
            out.numel() // c, c, _ptr(out), _DTYPES[dtype], _opts(num_sms))
    return out


def dispatch_mxfp4(x: torch.Tensor, dst_pos: torch.Tensor, num_recv_rows: int, *,
                   recv_x: Optional[torch.Tensor] = None, recv_scale: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, num_sms: int = 0,
                   scratch: Optional[torch.Tensor] = None, stream=None):
    """MXFP4 dispatch: each token quantised once, its row written to its receive rows (cgl_dispatch_mxfp4).

    scratch: new_scratch() (cgl_opts.scratch): tokens handed out dynamically, same results.
    Returns (recv_x uint8 [rows, H/2], recv_scale uint8 [rows, H/32]); rows that receive no copy
    are left as they were (uninitialised when allocated here)."""
    if stream is not None:
        with _on(stream, x, "x"):
            return dispatch_mxfp4(x, dst_pos, num_recv_rows, recv_x=recv_x, recv_scale=recv_scale, status=status,
                                  num_sms=num_sms, scratch=scratch)
    x = _dev(x, "x", torch.bfloat16, 2)
    dst = _dev(dst_pos, "dst_pos", torch.int32, 2)
    n, h = x.shape
    if dst.shape[0] != n:
        raise ValueError(f"dst_pos must have {n} rows, got {dst.shape[0]}")
    _same(x.device, dst_pos=dst, status=status, scratch=scratch)
    if h == 0 or h % 32 or num_recv_rows < 0:
        raise CglError(EINVAL, "dispatch_mxfp4", "hidden must be a multiple of 32")
    recv_x = _buf(recv_x, "recv_x", (num_recv_rows, h // 2), torch.uint8, x)
    recv_scale = _buf(recv_scale, "recv_scale", (num_recv_rows, h // 32), torch.uint8, x)
    _launch("cgl_dispatch_mxfp4", lib().cgl_dispatch_mxfp4, x.device, _ptr(x), n, h, dst.shape[1], _ptr(dst),
            _ptr(recv_x), _ptr(recv_scale), int(num_recv_rows), _opts(num_sms, 0, False, scratch), _ptr(status))
    return recv_x, recv_scale


def matmul_mxfp4(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                 expert_offset: Optional[torch.Tensor] = None, capacity: int = 0, *,
                 y: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 num_sms: int = 0, stream=None) -> torch.Tensor:
    """The experts' product on MXFP4 rows, y[r] = a[r] @ w[expert of r].T in BF16 (cgl_matmul_mxfp4).

    a uint8 [rows, in/2], a_scale uint8 [rows, in/32] (dispatch_mxfp4 or quantize_mxfp4);
    w uint8 [E, out, in/2], w_scale uint8 [E, out, in/32].  expert_offset int32 [E + 1] and
    capacity as get_layout gives them; without expert_offset w has one expert (or is [out, in/2])
    and takes every row.  Rows of no expert are left as they were."""
    if stream is not None:
        with _on(stream, a, "a"):
            return matmul_mxfp4(a, a_scale, w, w_scale, expert_offset, capacity, y=y, status=status, num_sms=num_sms)
    a = _dev(a, "a", torch.uint8, 2)
    a_scale = _dev(a_scale, "a_scale", torch.uint8, 2)
    w = _dev(w, "w", torch.uint8)
    w_scale = _dev(w_scale, "w_scale", torch.uint8)
    if expert_offset is None and w.dim() == 2 and w_scale.dim() == 2:
        w, w_scale = w.unsqueeze(0), w_scale.unsqueeze(0)
    if w.dim() != 3:
        raise ValueError(f"w must have 3 dims, got {w.dim()}")
    (rows, kb), (E, F, wb) = a.shape, w.shape
    K = 2 * kb
    if wb != kb or K == 0 or K % 32 or a_scale.shape != (rows, K // 32) or w_scale.shape != (E, F, K // 32):
        raise ValueError(f"a [rows, in/2], a_scale [rows, in/32], w [E, out, in/2], w_scale [E, out, in/32] expected, got "
                         f"{tuple(a.shape)}, {tuple(a_scale.shape)}, {tuple(w.shape)}, {tuple(w_scale.shape)}")
    if expert_offset is not None:
        _dev(expert_offset, "expert_offset", torch.int32, 1)
        if expert_offset.shape[0] != E + 1:
            raise ValueError(f"expert_offset must have {E + 1} entries, got {expert_offset.shape[0]}")
    _same(a.device, a_scale=a_scale, w=w, w_scale=w_scale, expert_offset=expert_offset, status=status)
    y = _buf(y, "y", (rows, F), torch.bfloat16, a)
    _launch("cgl_matmul_mxfp4", lib().cgl_matmul_mxfp4, a.device, _ptr(a), _ptr(a_scale), rows, _ptr(w),
            _ptr(w_scale), E, F, K, _ptr(expert_offset), _ptr(y), _opts(num_sms, capacity), _ptr(status))
    return y


class BalanceLoss(NamedTuple):
    loss: torch.Tensor                    # fp32 [1]
    counts: torch.Tensor                  # int32 [S, E]: slots per expert of each sequence
    num_routed: torch.Tensor              # int32 [S]: tokens of each sequence with a copy somewhere
    grad_logits: Optional[torch.Tensor]   # [N, E] in the logits' type, if grad_loss was given


def balance_loss_workspace_bytes(num_tokens: int, num_topk: int, num_experts: int, num_sequences: int = 1) -> int:
    return int(lib().cgl_balance_loss_workspace_bytes(num_tokens, num_topk, num_experts, num_sequences))


def _balance_args(logits, topk_idx, score, num_sequences, where):
    logits = _dev(logits, "logits", None, 2)
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    dt = _float_type(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if idx.shape[0] != logits.shape[0]:
        raise ValueError(f"topk_idx must have {logits.shape[0]} rows, got {idx.shape[0]}")
    _same(logits.device, topk_idx=idx)
    (n, E), k = logits.shape, idx.shape[1]
    ws_bytes = int(lib().cgl_balance_loss_workspace_bytes(n, k, E, num_sequences))
    if ws_bytes == 0:
        raise CglError(EINVAL, where, "invalid sizes")
    return logits, idx, dt, n, k, E, ws_bytes


def balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, *, num_sequences: int = 1, alpha: float = 1.0,
                 score: str = "softmax", grad_loss: Optional[torch.Tensor] = None,
                 loss: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                 num_routed: Optional[torch.Tensor] = None, grad_logits: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None) -> BalanceLoss:
    """Balance loss of a routing, its per-expert counts and, with grad_loss, its gradient (cgl_balance_loss).

    logits [N, E] (bfloat16, float16 or float32), topk_idx int32 [N, k] (-1 = no copy; a token with no copy
    takes no part).  score: "softmax", or "sigmoid" (normalised over the experts).  grad_loss: fp32 [1] on the
    device, the gradient that arrives at the loss; without it, balance_loss_backward gives grad_logits later."""
    if stream is not None:
        with _on(stream, logits, "logits"):
            return balance_loss(logits, topk_idx, num_sequences=num_sequences, alpha=alpha, score=score,
                                grad_loss=grad_loss, loss=loss, counts=counts, num_routed=num_routed,
                                grad_logits=grad_logits, workspace=workspace, status=status)
    logits, idx, dt, n, k, E, ws_bytes = _balance_args(logits, topk_idx, score, num_sequences, "balance_loss")
    dev = logits.device
    if grad_loss is not None:
        _buf(_dev(grad_loss, "grad_loss", torch.float32), "grad_loss", (1,), torch.float32, logits)
    elif grad_logits is not None:
        raise ValueError("grad_logits needs grad_loss")
    _same(dev, status=status)
    S = num_sequences
    loss = _buf(loss, "loss", (1,), torch.float32, logits)
    if grad_loss is not None:
        grad_logits = torch.empty_like(logits) if grad_logits is None else \
            _buf(grad_logits, "grad_logits", (n, E), logits.dtype, logits)
    if counts is None and num_routed is None and workspace is None:   # one allocation for the three, workspace first
        ints = ws_bytes // 4
        small = logits.new_empty(ints + S * (E + 1), dtype=torch.int32)
        counts, num_routed = small.as_strided((S, E), (E, 1), ints), small.as_strided((S,), (1,), ints + S * E)
        ws = small.data_ptr()
    else:
        counts = _buf(counts, "counts", (S, E), torch.int32, logits)
        num_routed = _buf(num_routed, "num_routed", (S,), torch.int32, logits)
        if workspace is None:
            workspace = logits.new_empty(ws_bytes, dtype=torch.uint8)
        else:
            _same(dev, workspace=_dev(workspace, "workspace"))
            ws_bytes = workspace.numel() * workspace.element_size()
        ws = workspace.data_ptr()
    _launch("cgl_balance_loss", lib().cgl_balance_loss, dev, _ptr(logits), dt, _ptr(idx), n, k, E, S, float(alpha),
            _SCORES[score], _ptr(grad_loss), _ptr(loss), _ptr(counts), _ptr(num_routed), _ptr(grad_logits), ws, ws_bytes,
            _ptr(status))
    return BalanceLoss(loss, counts, num_routed, grad_logits)


def balance_loss_backward(grad_loss: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                          counts: torch.Tensor, num_routed: torch.Tensor, *, num_sequences: int = 1,
                          alpha: float = 1.0, score: str = "softmax", grad_logits: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Gradient of balance_loss for the logits, from the forward's counts and num_routed (cgl_balance_loss_backward)."""
    if stream is not None:
        with _on(stream, logits, "logits"):
            return balance_loss_backward(grad_loss, logits, topk_idx, counts, num_routed, num_sequences=num_sequences,
                                         alpha=alpha, score=score, grad_logits=grad_logits)
    logits, idx, dt, n, k, E, _ = _balance_args(logits, topk_idx, score, num_sequences, "balance_loss_backward")
    dev = logits.device
    _buf(_dev(grad_loss, "grad_loss", torch.float32), "grad_loss", (1,), torch.float32, logits)
    _buf(_dev(counts, "counts", torch.int32), "counts", (num_sequences, E), torch.int32, logits)
    _buf(_dev(num_routed, "num_routed", torch.int32), "num_routed", (num_sequences,), torch.int32, logits)
    grad_logits = _buf(grad_logits, "grad_logits", (n, E), logits.dtype, logits)
    _launch("cgl_balance_loss_backward", lib().cgl_balance_loss_backward, dev, _ptr(grad_loss), _ptr(logits),
            dt, _ptr(idx), n, k, E, num_sequences, float(alpha), _SCORES[score], _ptr(counts), _ptr(num_routed),
            _ptr(grad_logits))
    return grad_logits


# ---- routing, the experts' BF16 product --------------------------------------------------------

_GROUP_SCORES = {"max": 0, "top2": 1}                                              # cgl_group_score
_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}           # cgl_activation


def _choice(value, names, what: str) -> int:
    if value not in names:
        raise ValueError(f"{what} must be one of {sorted(names)}, got {value!r}")
    return names[value]


try:   # 0.8 us of a small call's 10; torch.empty_strided takes 1.5, new_empty 2, torch.empty 2.4
    from torch._C._dynamo.guards import _empty_strided_cuda as _short_empty
except ImportError:
    _short_empty = None


def _public_empty(shape, strides, dtype):
    """A tensor on the current device."""
    return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _first_empty(shape, strides, dtype):
    """Like _public_empty; chooses what later calls take.  The short path is private to torch: it has to give what the public one gives."""
    global _empty
    try:
        t = _short_empty((2, 3), (3, 1), torch.int32)
        same = (t.shape, t.stride(), t.dtype, t.device.type, t.device.index) == ((2, 3), (3, 1), torch.int32, "cuda", torch.cuda.current_device())
    except Exception:
        same = False
    _empty = _short_empty if same else _public_empty
    return _empty(shape, strides, dtype)


_empty = _first_empty


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    """_buf, with the short path to the allocator (not where new memory is to be filled, as in torch's deterministic mode)."""
    if t is not None:
        return _buf(t, name, shape, dtype, like)
    strides = (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1) if len(shape) == 3 else (1,)
    device = like.device
    if device.index != torch._C._cuda_getDevice() or torch.are_deterministic_algorithms_enabled():
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    return _empty(shape, strides, dtype)


class Routing(NamedTuple):
    topk_idx: torch.Tensor       # int32 [N, k], best first; -1: no expert left
    topk_weights: torch.Tensor   # fp32 [N, k]


def route(logits: torch.Tensor, num_topk: int, *, bias: Optional[torch.Tensor] = None, num_groups: int = 1,
          topk_groups: int = 1, group_score: str = "max", score: str = "softmax", renormalize: bool = True,
          scale: float = 1.0, topk_idx: Optional[torch.Tensor] = None, topk_weights: Optional[torch.Tensor] = None,
          status: Optional[torch.Tensor] = None, stream=None) -> Routing:
    """Top-k experts of every token and their weights, for get_layout and combine (cgl_route).

    logits [N, E] (bfloat16, float16 or float32; -inf: the token may not take that expert).  score: "softmax" or
    "sigmoid".  bias: fp32 [E], added to the scores for the choice alone.  The best topk_groups of num_groups groups
    stay, by their best choice (group_score "max") or the sum of their two best ("top2").  renormalize: the picked
    scores are divided by their sum; scale multiplies the weights."""
    if stream is not None:
        with _on(stream, logits, "logits"):
            return route(logits, num_topk, bias=bias, num_groups=num_groups, topk_groups=topk_groups, group_score=group_score,
                         score=score, renormalize=renormalize, scale=scale, topk_idx=topk_idx, topk_weights=topk_weights,
                         status=status)
    logits = _dev(logits, "logits", None, 2)
    dt = _float_type(logits, "logits")
    n, E = logits.shape
    if bias is not None:
        _buf(_dev(bias, "bias", torch.float32), "bias", (E,), torch.float32, logits)
    if status is not None:
        _same(logits.device, status=status)
    kind, by = _choice(score, _SCORES, "score"), _choice(group_score, _GROUP_SCORES, "group_score")
    if not 1 <= num_topk <= min(E, 32):
        raise CglError(EINVAL, "route", "num_topk must be in [1, min(E, 32)]")
    topk_idx = _out(topk_idx, "topk_idx", (n, num_topk), torch.int32, logits)
    topk_weights = _out(topk_weights, "topk_weights", (n, num_topk), torch.float32, logits)
    _launch("cgl_route", lib().cgl_route, logits.device, logits.data_ptr(), dt, n, E, num_topk, _ptr(bias), num_groups, topk_groups,
            by, kind, bool(renormalize), scale, topk_idx.data_ptr(), topk_weights.data_ptr(), _ptr(status))
    return Routing(topk_idx, topk_weights)


def route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0, grad_logits: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of route's weights for the logits, from grad_weights fp32 [N, k] and route's topk_idx (cgl_route_backward)."""
    if stream is not None:
        with _on(stream, logits, "logits"):
            return route_backward(grad_weights, logits, topk_idx, score=score, renormalize=renormalize, scale=scale,
                                  grad_logits=grad_logits, status=status)
    logits = _dev(logits, "logits", None, 2)
    idx = _dev(topk_idx, "topk_idx", torch.int32, 2)
    g = _dev(grad_weights, "grad_weights", torch.float32, 2)
    dt = _float_type(logits, "logits")
    n, E = logits.shape
    if idx.shape[0] != n or g.shape != idx.shape:
        raise ValueError(f"topk_idx and grad_weights [{n}, k] expected, got {tuple(idx.shape)}, {tuple(g.shape)}")
    _same(logits.device, topk_idx=idx, grad_weights=g, status=status)
    kind = _choice(score, _SCORES, "score")
    grad_logits = _out(grad_logits, "grad_logits", (n, E), logits.dtype, logits)
    _launch("cgl_route_backward", lib().cgl_route_backward, logits.device, g.data_ptr(), logits.data_ptr(), dt, idx.data_ptr(), n, E,
            idx.shape[1], kind, bool(renormalize), scale, grad_logits.data_ptr(), _ptr(status))
    return grad_logits


def matmul_bf16_backward_workspace_bytes(num_rows: int, num_experts: int, out_features: int, in_features: int) -> int:
    return int(lib().cgl_matmul_bf16_backward_workspace_bytes(num_rows, num_experts, out_features, in_features))


def _matmul_args(a, w, expert_offset, activation, status):
    """Checked a [rows, in], w [E, out, in] and offsets; returns them with the sizes and the output's columns."""
    a = _dev(a, "a", torch.bfloat16, 2)
    w = _dev(w, "w", torch.bfloat16)
    if expert_offset is None and w.dim() == 2:
        w = w.unsqueeze(0)
    if w.dim() != 3:
        raise ValueError(f"w must have 3 dims, got {w.dim()}")
    (rows, K), (E, out, wk) = a.shape, w.shape
    act = _choice(activation, _ACTIVATIONS, "activation")
    if wk != K or K == 0 or K % 8:
        raise ValueError(f"a [rows, in] and w [E, out, in] with in % 8 == 0 expected, got {tuple(a.shape)}, {tuple(w.shape)}")
    if act == 4 and out % 2:
        raise ValueError(f"swiglu needs an even number of rows in w, got {out}")
    if expert_offset is not None:
        _dev(expert_offset, "expert_offset", torch.int32, 1)
        if expert_offset.shape[0] != E + 1:
            raise ValueError(f"expert_offset must have {E + 1} entries, got {expert_offset.shape[0]}")
    device = a.device
    if w.device != device or (expert_offset is not None and expert_offset.device != device) or status is not None:
        _same(device, w=w, expert_offset=expert_offset, status=status)
    return a, w, act, rows, E, out, K, out // 2 if act == 4 else out


def _preact(t, shape, like):
    """A preact buffer, binary32 or BF16, and its cgl_dtype."""
    dtype = t.dtype if isinstance(t, torch.Tensor) else torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"preact must be float32 or bfloat16, got {dtype}")
    return _out(t, "preact", shape, dtype, like), _DTYPES[dtype]


def _given(t, name: str, shape, dtype, like):
    """An input that may be None: checked."""
    if t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == like.device and t.is_contiguous()):
        return t
    return _buf(_dev(t, name, dtype), name, shape, dtype, like)   # names what is wrong


def matmul_bf16(a: torch.Tensor, w: torch.Tensor, expert_offset: Optional[torch.Tensor] = None, capacity: int = 0, *,
                bias: Optional[torch.Tensor] = None, activation: str = "none", residual: Optional[torch.Tensor] = None,
                with_preact: bool = False, y: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, num_sms: int = 0, stream=None):
    """The experts' product on BF16 rows, y[r] = act(a[r] @ w[expert of r].T + bias) + residual[r] (cgl_matmul_bf16).

    a [rows, in] (dispatch_bf16's rows), w [E, out, in], bias [E, out], residual and y [rows, out], all bfloat16.
    expert_offset int32 [E + 1] and capacity as get_layout gives them; without expert_offset w has one expert (or is
    [out, in], bias then [out]) and takes every row.  activation: "none", "relu", "gelu", "silu", or "swiglu": the
    first half of w's rows is the gate, the second the up projection, and y and residual have out / 2 columns.
    Rows of no expert are left as they were.  y may be the residual itself; other overlaps are refused.  with_preact: returns (y, preact), the sums with bias in fp32
    [rows, out], which matmul_bf16_backward takes; otherwise y alone.  preact: a buffer for them, fp32, or bfloat16,
    which halves its bytes and costs the gradients a rounding."""
    if stream is not None:
        with _on(stream, a, "a"):
            return matmul_bf16(a, w, expert_offset, capacity, bias=bias, activation=activation, residual=residual,
                               with_preact=with_preact, y=y, preact=preact, status=status, num_sms=num_sms)
    flat = isinstance(w, torch.Tensor) and w.dim() == 2
    a, w, act, rows, E, out, K, cols = _matmul_args(a, w, expert_offset, activation, status)
    if bias is not None:
        _given(bias, "bias", (out,) if flat else (E, out), torch.bfloat16, a)
    _given(residual, "residual", (rows, cols), torch.bfloat16, a)
    y = _out(y, "y", (rows, cols), torch.bfloat16, a)
    keep = with_preact or preact is not None
    preact, kind = _preact(preact, (rows, out), a) if keep else (None, 0)
    _launch("cgl_matmul_bf16", lib().cgl_matmul_bf16, a.device, _ptr(a), rows, _ptr(w), E, out, K, _ptr(expert_offset), _ptr(bias),
            act, _ptr(residual), _ptr(y), _ptr(preact), kind, _opts(num_sms, capacity), _ptr(status))
    return (y, preact) if keep else y


class MatmulGrads(NamedTuple):
    grad_a: Optional[torch.Tensor]      # bf16 [rows, in]
    grad_w: Optional[torch.Tensor]      # bf16 [E, out, in]
    grad_bias: Optional[torch.Tensor]   # bf16 [E, out]


def matmul_bf16_backward(grad_y: torch.Tensor, a: torch.Tensor, w: torch.Tensor, expert_offset: Optional[torch.Tensor] = None,
                         capacity: int = 0, *, activation: str = "none", preact: Optional[torch.Tensor] = None,
                         want_a: bool = True, want_w: bool = True, want_bias: bool = False,
                         grad_a: Optional[torch.Tensor] = None, grad_w: Optional[torch.Tensor] = None,
                         grad_bias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, num_sms: int = 0, stream=None) -> MatmulGrads:
    """Gradients of matmul_bf16 for its rows, weights and bias (cgl_matmul_bf16_backward); the residual's is grad_y itself.

    preact: what matmul_bf16(..., with_preact=True) gave (not needed without an activation).  Rows of grad_a of no
    expert are left as they were (uninitialised when allocated here); grad_w and grad_bias of an expert without rows are 0.
    Gradients may be written over preact and what else cgl_matmul_bf16_backward is done with; other overlaps are refused."""
    if stream is not None:
        with _on(stream, a, "a"):
            return matmul_bf16_backward(grad_y, a, w, expert_offset, capacity, activation=activation, preact=preact, want_a=want_a,
                                        want_w=want_w, want_bias=want_bias, grad_a=grad_a, grad_w=grad_w, grad_bias=grad_bias,
                                        workspace=workspace, status=status, num_sms=num_sms)
    flat = isinstance(w, torch.Tensor) and w.dim() == 2
    a, w, act, rows, E, out, K, cols = _matmul_args(a, w, expert_offset, activation, status)
    bf16, lead = torch.bfloat16, () if flat else (E,)
    if _given(grad_y, "grad_y", (rows, cols), bf16, a) is None:
        raise TypeError("grad_y must be a CUDA tensor")
    if act != 0 and preact is None:
        raise ValueError(f"activation {activation!r} needs preact")
    kind = 0 if preact is None else _preact(_dev(preact, "preact"), (rows, out), a)[1]
    for name, t, want in (("grad_a", grad_a, want_a), ("grad_w", grad_w, want_w), ("grad_bias", grad_bias, want_bias)):
        if t is not None and not want:
            raise ValueError(f"{name} was given but is not wanted")
    grad_a = _out(grad_a, "grad_a", (rows, K), bf16, a) if want_a else None
    grad_w = _out(grad_w, "grad_w", (*lead, out, K), bf16, a) if want_w else None
    grad_bias = _out(grad_bias, "grad_bias", (*lead, out), bf16, a) if want_bias else None
    ws_bytes = 0
    if workspace is not None:
        _same(a.device, workspace=_dev(workspace, "workspace"))
        ws_bytes = workspace.numel() * workspace.element_size()
    elif act != 0 or want_bias or out % 8 or grad_y.data_ptr() % 16:   # else the products read grad_y itself
        ws_bytes = matmul_bf16_backward_workspace_bytes(rows, E, out, K)
        if ws_bytes == 0:
            raise CglError(EINVAL, "matmul_bf16_backward", "invalid sizes")
        workspace = _out(None, "workspace", (ws_bytes,), torch.uint8, a)
    _launch("cgl_matmul_bf16_backward", lib().cgl_matmul_bf16_backward, a.device, _ptr(grad_y), _ptr(a), rows, _ptr(w), E, out, K,
            _ptr(expert_offset), act, _ptr(preact), kind, _ptr(grad_a), _ptr(grad_w), _ptr(grad_bias), _ptr(workspace), ws_bytes,
            _opts(num_sms, capacity), _ptr(status))
    return MatmulGrads(grad_a, grad_w, grad_bias)
