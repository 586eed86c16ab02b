"""ReLU's gradient selects: a closed unit (z <= 0) gives 0 whatever gradient comes in, an open one passes it on, and where
z is NaN the gradient is NaN, as the forward keeps it.  Whole numbers otherwise, so results are exact."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("rows,k,f", [(70, 64, 40), (130, 72, 33), (5, 8, 8)])
def test_what_comes_in_at_closed_units_is_dropped(rows, k, f, wide):
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device="cuda").bfloat16()

    a, w, g, z = whole(rows, k), whole(f, k), whole(rows, f), whole(rows, f)
    z[1], z[2, :4] = -1.0, 0.0
    z[2, 1] = -0.0
    z[3, 2] = -torch.inf
    open_ = z > 0
    clean = torch.where(open_, g, 0)
    g[~open_ & (whole(rows, f) > 0)] = torch.inf
    g[~open_ & (whole(rows, f) > 1)] = torch.nan
    g[1, 0], g[2, 0], g[2, 1], g[3, 2] = -torch.inf, torch.inf, torch.nan, torch.inf
    pre = z.float() if wide else z
    d = cgl.matmul_bf16_backward(g, a, w, activation="relu", preact=pre, want_bias=True)
    want = cgl.matmul_bf16_backward(clean, a, w, activation="relu", preact=pre, want_bias=True)
    dz = clean.double()
    for got, same, ref in zip(d, want, (dz @ w.double(), dz.T @ a.double(), dz.sum(0))):
        assert torch.equal(got, same) and torch.equal(got, ref.float().bfloat16())


@pytest.mark.parametrize("wide", [True, False])
def test_a_pre_activation_that_is_not_a_number_shows(wide):
    rows, k, f = 20, 16, 24
    a, w, g = (torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in ((rows, k), (f, k), (rows, f)))
    z = torch.ones(rows, f, device="cuda", dtype=torch.float32 if wide else torch.bfloat16)
    z[7, 5] = torch.nan
    d = cgl.matmul_bf16_backward(g, a, w, activation="relu", preact=z, want_bias=True)
    for got, hit in zip(d, ((7, slice(None)), (5, slice(None)), (5,))):
        bad = torch.zeros_like(got, dtype=torch.bool)
        bad[hit] = True
        assert torch.equal(got.isnan(), bad)
    g[7, 5] = 0.0
    assert cgl.matmul_bf16_backward(g, a, w, activation="relu", preact=z, want_bias=True).grad_bias[5].isnan()


@pytest.mark.parametrize("bad", [torch.inf, torch.nan])
def test_an_open_unit_passes_it_on(bad):
    rows, k, f = 20, 16, 24
    a, w, g = (torch.ones(s, device="cuda", dtype=torch.bfloat16) for s in ((rows, k), (f, k), (rows, f)))
    g[7, 5] = bad
    z = torch.ones(rows, f, device="cuda")
    d = cgl.matmul_bf16_backward(g, a, w, activation="relu", preact=z, want_bias=True)
    assert not d.grad_a[7].isfinite().any() and not d.grad_w[5].isfinite().any() and not d.grad_bias[5].isfinite()
    assert d.grad_bias[:5].isfinite().all() and d.grad_a[:7].isfinite().all()
