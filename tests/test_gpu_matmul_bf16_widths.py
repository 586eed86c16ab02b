"""The product and its gradients where the width of a tile is a close choice: experts of one size, at and around whole
tiles, and experts of very different sizes.  Whole numbers, so results are exact."""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


def _check(counts, k, f, seed, cap=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ends = np.cumsum(counts)
    off = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32, device="cuda")
    rows = len(counts) * cap if cap else int(ends[-1])

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device="cuda").bfloat16()

    a, w, g = whole(rows, k), whole(len(counts), f, k), whole(rows, f)
    st = cgl.new_status()
    y = cgl.matmul_bf16(a, w, off, cap, status=st)
    d = cgl.matmul_bf16_backward(g, a, w, off, cap, status=st)
    assert cgl.status_bits(st) == []
    for i, n in enumerate(counts):
        r0 = i * cap if cap else int(ends[i]) - n
        r = slice(r0, r0 + (min(n, cap) if cap else n))
        x, m, q = a[r].float(), w[i].float(), g[r].float()
        assert torch.equal(y[r], (x @ m.T).bfloat16()) and torch.equal(d.grad_a[r], (q @ m).bfloat16()) and torch.equal(d.grad_w[i], (q.T @ x).bfloat16())


@pytest.mark.parametrize("rows", [1, 31, 33, 128, 176, 207, 208, 209, 224, 240, 241, 255, 256, 257, 320, 511, 512, 513, 768])
@pytest.mark.parametrize("e,k,f", [(16, 192, 520), (5, 520, 192), (64, 64, 256)])
def test_experts_of_one_size(e, k, f, rows):
    _check([rows] * e, k, f, rows)


@pytest.mark.parametrize("e,k,f,mean", [(16, 256, 512, 256), (16, 256, 512, 512), (32, 128, 768, 100), (8, 512, 264, 700)])
@pytest.mark.parametrize("seed", range(4))
def test_experts_of_many_sizes(seed, e, k, f, mean):
    gen = np.random.default_rng(seed)
    p = (np.arange(e) + 1.0) ** (-0.4 * seed)
    _check(gen.multinomial(mean * e, p / p.sum()).tolist(), k, f, seed)


@pytest.mark.parametrize("cap", [200, 256, 272, 520])
def test_padded(cap):
    _check([cap, 0, cap - 3, cap + 9, 1, 16], 256, 272, cap, cap)
