"""Logits of -0 and +0: equal values, so the lower index goes first, in every path that puts logits in order."""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
from test_gpu_route import TYPES, _check, _grad

pytestmark = pytest.mark.gpu


def _zeros(n, e, seed, dtype, values=(-1.0, -0.0, 0.0, 0.5)):
    gen = torch.Generator().manual_seed(seed)
    return torch.tensor(values)[torch.randint(0, len(values), (n, e), generator=gen)].to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("dtype", TYPES)
def test_two_zeros(dtype):
    l = torch.tensor([[-0.0, 0.0], [0.0, -0.0]], dtype=TYPES[dtype], device="cuda")
    assert cgl.route(l, 1).topk_idx.tolist() == [[0], [0]]
    assert cgl.route(l, 2, score="sigmoid").topk_idx.tolist() == [[0, 1], [0, 1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("e,k", [(8, 3), (32, 8), (64, 6), (100, 8), (128, 8), (250, 8), (256, 6), (256, 8), (400, 8), (512, 8), (1000, 12), (1021, 5)])
def test_zeros_in_the_order(e, k, dtype, score):
    """Among few values, and among zeros and negative values alone, so that zeros are the best."""
    for values in ((-1.0, -0.0, 0.0, 0.5), (-0.0, 0.0), (-2.0, -0.0, -1.0, 0.0, -torch.inf)):
        _check(_zeros(40, e, e + k, dtype, values), k, _grad(40, k), score=score)


@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("e,k,groups,keep", [(16, 4, 4, 2), (24, 3, 3, 1), (64, 8, 8, 3), (160, 6, 8, 3), (256, 8, 8, 4), (512, 8, 16, 5), (1000, 8, 20, 7)])
def test_zeros_in_groups(e, k, groups, keep, dtype, biased, by):
    """Groups whose best values are zeros of either sign; with the biases a group's value is a sum of equal choices."""
    bias = torch.zeros(e, device="cuda") if biased else None
    for score in ("softmax", "sigmoid"):
        for values in ((-1.0, -0.0, 0.0), (-0.0, 0.0)):
            _check(_zeros(40, e, e + groups, dtype, values), k, None, bias, groups, keep, by, score)


@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_where_rows_are_not_aligned_and_tokens_are_many(dtype):
    l = _zeros(9001, 256, 3, dtype, (-0.0, 0.0, -1.0))
    buf = torch.empty(l.numel() + 1, dtype=l.dtype, device="cuda")
    shifted = buf[1:].view(l.shape)
    shifted.copy_(l)
    r = cgl.route(l, 8, score="sigmoid")
    for part in (cgl.route(shifted, 8, score="sigmoid"), cgl.route(l[:4000].contiguous(), 8, score="sigmoid")):
        assert torch.equal(part.topk_idx, r.topk_idx[:len(part.topk_idx)])
    _check(l[:200].contiguous(), 8, None, score="sigmoid")
    masked = (torch.randn(200, 256, generator=torch.Generator().manual_seed(1)).cuda() * (l[:200] == 0)).to(TYPES[dtype])   # a 0 / 1 mask leaves both zeros
    _check(masked, 8, None, score="sigmoid")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("e,k", [(1024, 32), (256, 8), (256, 5), (128, 8), (32, 4)])
def test_every_16_bit_value(e, k, dtype):
    """All bit patterns but NaN, 65536 / e rows: keys are in the order of the values, subnormal ones and infinities too."""
    bits = np.random.default_rng(e).permutation(65536).astype(np.uint16).view(np.int16)
    l = torch.from_numpy(bits).view(TYPES[dtype]).view(-1, e)
    l = torch.where(l.isnan(), torch.tensor(-0.0, dtype=l.dtype), l)
    _check(l.cuda().contiguous(), k, None, score="sigmoid")
    small = torch.where(l.abs().float() < torch.finfo(l.dtype).smallest_normal * 4, l, torch.tensor(-1.0, dtype=l.dtype))
    _check(small.cuda().contiguous(), k, None, score="sigmoid")
