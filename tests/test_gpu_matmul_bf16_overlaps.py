"""Gradients of the BF16 product written over what it has done with, and a forward onto its residual: the same bits as
into buffers of their own.  (Overlaps that would be wrong are refused.)"""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


def _case(rows, k, f, act):
    gen = torch.Generator(device="cuda").manual_seed(rows + f)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    return normal(rows, k), normal(3, f, k), off, normal(rows, f // 2 if act == "swiglu" else f), torch.randn(rows, f, generator=gen, device="cuda")


def _same(got, want):
    return all((p is None) == (q is None) and (p is None or torch.equal(p.view(torch.int16), q.view(torch.int16))) for p, q in zip(got, want))


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("rows,k,f", [(700, 264, 528), (90, 64, 128)])
def test_over_what_is_done_with(rows, k, f, act):
    a, w, off, g, z = _case(rows, k, f, act)

    def run(g=g, w=w, z=z, **kw):
        return cgl.matmul_bf16_backward(g, a, w, off, activation=act, preact=z, **kw)

    want = run(want_bias=True)
    zc = z.clone()
    assert _same(run(z=zc, want_bias=True, grad_a=zc.view(torch.bfloat16).flatten()[:rows * k].view(rows, k)), want)          # pre-activations
    zc = z.clone()
    if 3 * f * k <= 2 * rows * f:
        assert _same(run(z=zc, want_bias=True, grad_w=zc.view(torch.bfloat16).flatten()[:3 * f * k].view(3, f, k)), want)
    wc = w.clone()
    assert _same(run(w=wc, want_bias=True, grad_w=wc), want)                                                                 # the weights, by their gradient
    if g.numel() >= rows * k:
        gc = g.clone()
        assert _same(run(g=gc, want_bias=True, grad_a=gc.flatten()[:rows * k].view(rows, k)), want)
    ac = a.clone()
    only = cgl.matmul_bf16_backward(g, ac, w, off, activation=act, preact=z, want_w=False, grad_a=ac)                        # the rows, where grad_w is not wanted
    assert _same(only, (want.grad_a, None, None))


def test_refused_from_python():
    a, w, off, g, z = _case(90, 64, 64, "none")
    with pytest.raises(cgl.CglError, match="CGL_EINVAL"):
        cgl.matmul_bf16(a, w, off, y=a)
    with pytest.raises(cgl.CglError, match="CGL_EINVAL"):
        cgl.matmul_bf16_backward(g, a, w, off, grad_a=a)
    with pytest.raises(cgl.CglError, match="CGL_EINVAL"):
        cgl.matmul_bf16_backward(g, a, w, off, want_w=False, grad_a=g)
    r = g.clone()
    assert cgl.matmul_bf16(a, w, off, residual=r, y=r) is r
    assert torch.equal(r, cgl.matmul_bf16(a, w, off, residual=g))
    l = torch.randn(16, 8, device="cuda")
    with pytest.raises(cgl.CglError, match="CGL_EINVAL"):
        cgl.route(l, 8, topk_weights=l)
