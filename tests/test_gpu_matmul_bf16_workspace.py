"""The BF16 product's gradients without an activation: what is handed over as preact is not read, whatever its alignment,
and changes neither the results nor what needs a workspace."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


def _shifted(t, by):
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("f", [64, 40, 33])
@pytest.mark.parametrize("shift_g", [0, 1])
@pytest.mark.parametrize("shift_z", [0, 1])
def test_preact_is_not_read_without_an_activation(shift_z, shift_g, f, dtype):
    rows, k = 75, 72
    gen = torch.Generator(device="cuda").manual_seed(f)
    a, w, g = (torch.randint(-4, 5, s, generator=gen, device="cuda").bfloat16() for s in ((rows, k), (f, k), (rows, f)))
    g = _shifted(g, shift_g)
    z = _shifted(torch.full((rows, f), torch.nan, dtype=dtype, device="cuda"), shift_z)
    dz = g.double()
    refs = dz @ w.double(), dz.T @ a.double(), dz.sum(0)
    for bias in (False, True):
        for want_a, want_w in ((True, True), (True, False), (False, True)):
            st = cgl.new_status()
            d = cgl.matmul_bf16_backward(g, a, w, preact=z, want_a=want_a, want_w=want_w, want_bias=bias, status=st)
            assert cgl.status_bits(st) == []
            for got, ref, want in zip(d, refs, (want_a, want_w, bias)):
                assert (got is None) != want and (got is None or torch.equal(got, ref.float().bfloat16()))
