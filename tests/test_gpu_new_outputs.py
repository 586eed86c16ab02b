"""Outputs that a call allocates for itself are ordinary tensors, and in torch's deterministic mode, which fills new memory,
rows that no expert has read as NaN."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


def _padded():
    a = torch.ones(40, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(4, 24, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 3, 3, 13, 20], dtype=torch.int32, device="cuda")
    has = torch.zeros(40, dtype=torch.bool, device="cuda")
    for i, n in enumerate((3, 0, 10, 7)):
        has[10 * i:10 * i + n] = True
    return a, w, off, has


def test_rows_of_no_expert_are_filled_in_deterministic_mode():
    a, w, off, has = _padded()
    junk = torch.zeros(1 << 20, dtype=torch.bfloat16, device="cuda")
    del junk                                     # what the outputs may be cut from
    torch.use_deterministic_algorithms(True)
    try:
        y, z = cgl.matmul_bf16(a, w, off, 10, with_preact=True)
        d = cgl.matmul_bf16_backward(y, a, w, off, 10, want_w=False)
    finally:
        torch.use_deterministic_algorithms(False)
    for t in (y, z, d.grad_a):
        assert t[~has].isnan().all() and not t[has].isnan().any()


def test_shapes_and_types():
    a, w, off, has = _padded()
    r = cgl.route(torch.zeros(6, 32, device="cuda"), 4)
    y, z = cgl.matmul_bf16(a, w, off, 10, with_preact=True, activation="swiglu")
    d = cgl.matmul_bf16_backward(torch.ones_like(y), a, w, off, 10, preact=z, activation="swiglu", want_bias=True)
    for t, shape, dtype in ((r.topk_idx, (6, 4), torch.int32), (r.topk_weights, (6, 4), torch.float32), (y, (40, 12), torch.bfloat16),
                            (z, (40, 24), torch.float32), (d.grad_a, (40, 16), torch.bfloat16), (d.grad_w, (4, 24, 16), torch.bfloat16),
                            (d.grad_bias, (4, 24), torch.bfloat16)):
        assert type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == a.device and not t.requires_grad
