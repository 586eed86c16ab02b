"""Routing and its gradient against the definition in 64 bits.

Ids have to be equal: choices nearer than binary32 resolves are part of the cases.  Tolerances, u = 2^-24: a share is
an exponential (its argument l - b is rounded once and scaled once, 2 D u with D the row's spread; the exponential 4u),
a sigmoid adds a sum and a quotient (4u), the sum over E terms E / 16 + 10 additions, one division and one product
(2u): off by tp = (2 D + E / 16 + 24) u of its value at most.  A gradient is share * gate * (g - dot): each factor is
off by at most tp, the dot by tp + 40 u of sum |g| share, so tol = 4 tp times the sum of the terms' sizes, half a step
of the output's type, and one step where that is subnormal.  Below 2^-126 no relative bound holds: a subnormal
exponential and its quotient are each off by a step of 2^-149, which a divisor of at least 1/2 (the largest term of a
renormalised sum is 1/2 to 1) at most doubles, so a share is off by less than 2^-146 more; it is multiplied by
|g - dot| <= 2 max |g|, here below 32, so that a gradient is off by less than 2^-140 more.
"""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
import routeref
from combine_get_layout_02_b200 import workloads as W

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _spread(l):
    x = l.double().cpu().numpy()
    f = np.where(np.isfinite(x), x, 0.0)
    return np.minimum(np.abs(f).max(axis=1, keepdims=True) * 2, 2.0 ** 20)


def _check(l, k, g=None, bias=None, groups=1, keep=1, by="max", score="softmax", renorm=True, scale=1.0):
    assert g is None or scale * g.abs().max() < 16
    n, e = l.shape
    host = l.float().cpu().numpy()
    st = cgl.new_status()
    idx = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), -7.0, device="cuda")
    r = cgl.route(l, k, bias=bias, num_groups=groups, topk_groups=keep, group_score=by, score=score, renormalize=renorm,
                  scale=scale, topk_idx=idx, topk_weights=w, status=st)
    assert r.topk_idx is idx and r.topk_weights is w
    ri, rw, bad = routeref.route(host, k, None if bias is None else bias.cpu().numpy(), groups, keep, by, score, renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), ri)
    got = w.double().cpu().numpy()
    assert cgl.status_bits(st) == (["CGL_ERANGE"] if bad.any() else [])
    assert np.isnan(got[bad]).all()
    tp = (2 * _spread(l) + e / 16 + 24) * U
    assert (np.abs(got - rw)[~bad] <= (tp * np.abs(rw) + 2.0 ** -126)[~bad]).all()
    if g is not None:
        d = cgl.route_backward(g, l, idx, score=score, renormalize=renorm, scale=scale, status=st)
        ref, size = routeref.backward(g.cpu().numpy(), host, ri, score, renorm, scale)
        fi = torch.finfo(l.dtype)
        tol = 4 * (tp + 40 * U) * size + fi.eps / 2 * np.abs(ref) + fi.smallest_normal * fi.eps + 2.0 ** -140
        diff = np.abs(d.double().cpu().numpy() - ref)
        assert d.dtype == l.dtype and (diff[~bad] <= tol[~bad]).all()
        assert (d[torch.tensor(bad)] == 0).all()      # no expert was picked
    return r


def _logits(n, e, seed, dtype="f32", spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(n, e, generator=g)).to(TYPES[dtype]).cuda()


def _grad(n, k, seed=1):
    return torch.randn(n, k, generator=torch.Generator().manual_seed(seed)).cuda()


def _bias(e, seed=2, step=0.001):
    return (torch.round(100 * torch.randn(e, generator=torch.Generator().manual_seed(seed))) * step).float().cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (3, 8, 8), (128, 16, 4), (65, 33, 3), (77, 64, 6), (50, 100, 32), (200, 128, 8),
                                   (150, 256, 8), (40, 250, 9), (30, 300, 5), (20, 512, 16), (10, 1024, 32), (9, 1000, 31)])
def test_plain(n, e, k, dtype, renorm, score):
    _check(_logits(n, e, n + e, dtype), k, _grad(n, k), score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,e,k,groups,keep", [(100, 16, 4, 4, 2), (130, 256, 8, 8, 4), (60, 256, 8, 32, 5), (60, 160, 6, 8, 3), (40, 64, 8, 32, 20),
                                               (50, 24, 3, 3, 1), (33, 512, 10, 16, 4), (20, 1024, 32, 4, 2), (64, 32, 4, 32, 7), (30, 96, 24, 2, 1),
                                               (40, 256, 8, 2, 2)])
def test_groups(n, e, k, groups, keep, dtype, biased, by, score):
    k = min(k, e)
    _check(_logits(n, e, n + groups, dtype), k, None, _bias(e) if biased else None, groups, keep, by, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("e", [16, 256, 1024])
def test_bias(e, dtype, score):
    l = _logits(120, e, 5, dtype)
    for b in (torch.zeros(e, device="cuda"), _bias(e), _bias(e, step=1.0), torch.full((e,), -3.0, device="cuda")):
        _check(l, 8, _grad(120, 8), b, score=score, renorm=False)
        _check(l, 8, None, b, score=score, scale=0.5)


def test_more_slots_than_the_groups_hold():
    """Two groups of four stay for six... the other slots have no expert."""
    for by in ("max", "top2"):
        r = _check(_logits(50, 16, 3), 10, _grad(50, 10), groups=4, keep=2, by=by)
        assert (r.topk_idx[:, 8:] == -1).all() and (r.topk_weights[:, 8:] == 0).all() and (r.topk_idx[:, :8] >= 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_masks(dtype, biased, renorm, score):
    """Masked experts, tokens with fewer experts than slots, with one, with none; masks of the type's lowest value."""
    n, e, k = 90, 40, 6
    l = _logits(n, e, 8, dtype)
    gen = torch.Generator().manual_seed(3)
    l[torch.rand(n, e, generator=gen).cuda() < torch.linspace(0, 1, n).cuda()[:, None]] = -torch.inf
    l[3] = -torch.inf
    l[4] = -torch.inf
    l[4, 17] = 1.5
    l[5, 5:] = torch.finfo(l.dtype).min
    l[6] = torch.finfo(l.dtype).min
    l[7, :] = torch.finfo(l.dtype).min
    l[7, 9] = -torch.inf
    b = _bias(e) if biased else None
    for groups, keep, by in ((1, 1, "max"), (8, 3, "max"), (8, 3, "top2"), (10, 9, "top2")):
        r = _check(l, k, _grad(n, k), b, groups, keep, by, score, renorm, 1.5)
        assert (r.topk_idx[3] == -1).all() and (r.topk_weights[3] == 0).all()
        assert r.topk_idx[4].tolist() == [17, -1, -1, -1, -1, -1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [20, 256, 1000])
def test_ties_go_to_the_lower_index(e, score):
    """Five values of logits, no two of whose pairs have scores of equal sum."""
    gen = torch.Generator().manual_seed(1)
    l = (0.3 + 0.7 * torch.randint(0, 5, (200, e), generator=gen).float()).cuda()
    few = (torch.randint(0, 3, (e,), generator=gen) * 0.25).float().cuda()
    for b in (None, torch.zeros(e, device="cuda"), few):
        _check(l, min(e, 12), None, b, score=score)
        _check(l, 5, None, b, groups=4, keep=3, by="max", score=score)
        if b is not few:     # sums of two choices with swapped biases are equal only to the reals
            _check(l, 5, None, b, groups=e // 5 if e == 20 else 4, keep=2, by="top2", score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 64, 256, 700])
def test_choices_nearer_than_binary32_tells(e, score):
    """Logits in [2, 4) up to three steps apart (sums of two scores then differ by 2^-48 or more where they do), and biases
    that bring different scores to within a step of each other."""
    gen = torch.Generator().manual_seed(2)
    base = 2 + 1.99 * torch.rand(300, 1, generator=gen)
    steps = torch.randint(0, 4, (300, e), generator=gen, dtype=torch.int32)
    l = (base.view(torch.int32) + steps).view(torch.float32).cuda()
    k = min(e, 8)
    zeros = torch.zeros(e, device="cuda")
    _check(l, k, None, score=score)
    _check(l, k, None, zeros, score=score)
    for b in (None, zeros):
        _check(l, k, None, b, groups=4, keep=2, by="max", score=score)
        _check(l, k, None, b, groups=4, keep=2, by="top2", score=score)
    x = torch.randn(1, e, generator=gen)
    s = torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())
    b = (1 - s[0]).float().cuda()                 # every choice is 1 to binary32
    steps = torch.randint(-1, 2, (300, e), generator=gen, dtype=torch.int32)
    l = (x.expand(300, e).contiguous().view(torch.int32) + steps).view(torch.float32).cuda()
    _check(l, k, None, b, score=score)
    _check(l, k, None, b, groups=4, keep=3, by="max", score=score)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_not_numbers(score, dtype):
    l = _logits(30, 64, 4, dtype)
    l[2, 7] = torch.nan
    l[9, 3] = torch.inf
    l[9, 5] = torch.inf
    l[11, 0] = torch.inf
    l[11, 1:] = -torch.inf
    for renorm in (True, False):
        for b in (None, _bias(64)):
            _check(l, 4, _grad(30, 4), b, score=score, renorm=renorm)
    b = _bias(64)
    b[5] = torch.inf
    b[6] = -torch.inf
    r = _check(l, 4, None, b, score=score)
    assert (r.topk_idx[0] != 6).all() and r.topk_idx[0, 0] == 5
    b[20] = torch.nan
    r = _check(l, 4, None, b, score=score)
    assert (r.topk_idx[:9] == -1).all() and r.topk_weights[:9].isnan().all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", [-3.0e38, -1.0e4, -200.0, -80.0, 0.0, 60.0, 3.0e4, 1.0e30])
def test_logits_of_any_size(at, score):
    """Renormalised weights are the quotient of the true scores, also where every score underflows or all are 1."""
    l = at + torch.randn(64, 48, generator=torch.Generator().manual_seed(1)).cuda() * max(1.0, abs(at) * 1e-6)
    for renorm in (True, False):
        _check(l, 6, _grad(64, 6), score=score, renorm=renorm)
    l = torch.randn(64, 48, generator=torch.Generator().manual_seed(2)).cuda() * 90
    _check(l, 6, _grad(64, 6), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("e", [7, 256])
def test_gradient_of_any_ids(e, renorm, score):
    """Slots that repeat an expert, without one, or out of range; against the formula, slot by slot."""
    n, k = 80, 6
    l, g = _logits(n, e, 3), _grad(n, k)
    gen = torch.Generator().manual_seed(6)
    idx = torch.randint(-1, min(e, 5), (n, k), generator=gen).int().cuda()
    idx[0] = 2
    idx[1] = -1
    st = cgl.new_status()
    d = cgl.route_backward(g, l, idx, score=score, renormalize=renorm, scale=0.7, status=st)
    assert cgl.status_bits(st) == []
    ref, size = routeref.backward(g.cpu().numpy(), l.cpu().numpy(), idx.cpu().numpy(), score, renorm, 0.7)
    tol = 4 * (2 * _spread(l) + e / 16 + 64) * U * size + 2.0 ** -126
    assert (np.abs(d.double().cpu().numpy() - ref) <= tol).all() and (d[1] == 0).all()
    idx[4, 2], idx[5, 1] = e, -2
    again = cgl.route_backward(g, l, idx, score=score, renormalize=renorm, scale=0.7, status=st)
    assert cgl.status_bits(st) == ["CGL_ERANGE"]
    idx[4, 2], idx[5, 1] = -1, -1
    assert torch.equal(again, cgl.route_backward(g, l, idx, score=score, renormalize=renorm, scale=0.7))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm, score):
    """Central differences of the 64-bit weights (step 2^-12: off by its square times a third derivative, below 2^-20 of
    the weights' scale here), the choice held fixed."""
    n, e, k = 6, 10, 4
    l, g = _logits(n, e, 12), _grad(n, k)
    r = cgl.route(l, k, score=score, renormalize=renorm, scale=1.3)
    d = cgl.route_backward(g, l, r.topk_idx, score=score, renormalize=renorm, scale=1.3).double().cpu().numpy()
    idx = r.topk_idx.long().cpu()

    def loss(x):
        s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
        w = s.gather(1, idx)
        w = w / w.sum(1, keepdim=True) if renorm else w
        return (1.3 * w * g.double().cpu()).sum(1).numpy()

    h = 2.0 ** -12
    for i in range(e):
        x = l.double().cpu()
        up, down = x.clone(), x.clone()
        up[:, i] += h
        down[:, i] -= h
        assert np.abs((loss(up) - loss(down)) / (2 * h) - d[:, i]).max() < 2.0 ** -18


@pytest.mark.parametrize("name", ["tiny", "decode", "prefill", "skewed"])
def test_workload_routing(name):
    """The named workloads' own routing: their scores, taken as logits, have the same order."""
    wl = W.WORKLOADS[name]
    inp = W.make_inputs(name, 0, num_tokens=300)
    s = torch.from_numpy(inp.scores).cuda()
    r = cgl.route(s, wl.topk, num_groups=wl.num_groups, topk_groups=wl.topk_group)
    assert np.array_equal(r.topk_idx.cpu().numpy(), inp.topk_idx)


@pytest.mark.parametrize("n", [0, 1, 3, 5000])
def test_rows_and_tails(n):
    """Nothing behind the last token is written; unaligned rows."""
    e, k = 256, 8
    for shift in (0, 1):
        l = torch.empty(n * e + shift, dtype=torch.bfloat16, device="cuda")[shift:].view(n, e)
        l.copy_(_logits(n, e, 2, "bf16"))
        idx = torch.full((n + 2, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((n + 2, k), -7.0, device="cuda")
        buf = torch.full((n * e + 64 + shift,), -7.0, dtype=torch.bfloat16, device="cuda")
        d = buf[shift:shift + n * e].view(n, e)
        r = cgl.route(l, k, score="sigmoid", topk_idx=idx[:n], topk_weights=w[:n])
        g = _grad(n, k)
        cgl.route_backward(g, l, r.topk_idx, score="sigmoid", grad_logits=d)
        assert (idx[n:] == -7).all() and (w[n:] == -7).all() and (buf[shift + n * e:] == -7).all()
        if 0 < n < 100:
            _check(l, k, g, score="sigmoid")
        if n:
            whole = cgl.route(l.clone(), k, score="sigmoid")
            assert torch.equal(whole.topk_idx, r.topk_idx) and torch.equal(whole.topk_weights, r.topk_weights)
            assert torch.equal(cgl.route_backward(g, l.clone(), r.topk_idx, score="sigmoid"), d)


@pytest.mark.parametrize("e", [16, 100, 248, 256])
@pytest.mark.parametrize("kind", ["plain", "bias", "groups"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_many_tokens(score, renorm, kind, e):
    """Batches in which a warp takes several tokens at once give what the tokens give in small batches, bit for bit."""
    for n, k, dtype in ((20_003, 8, "bf16"), (19_001, 5, "f32"), (18_950, 1, "f16")):
        l, g = _logits(n, e, 7, dtype), _grad(n, k)
        l[-9:-5] = -torch.inf
        l[11, 3:] = -torch.inf
        l[12, 2] = torch.nan
        how = dict(score=score, renormalize=renorm, scale=1.5)
        pick = dict(bias=_bias(e) if kind != "plain" else None, **(dict(num_groups=4, topk_groups=2, group_score="top2") if kind == "groups" else {}))
        st = cgl.new_status()
        r = cgl.route(l, k, status=st, **pick, **how)
        assert cgl.status_bits(st) == ["CGL_ERANGE"]
        idx = r.topk_idx.clone()
        idx[30, k - 1] = idx[30, 0]               # an expert twice
        d = cgl.route_backward(g, l, idx, **how)
        for a, b in ((0, 6000), (6000, 15_000), (15_000, n)):
            part = cgl.route(l[a:b].contiguous(), k, **pick, **how)
            assert torch.equal(part.topk_idx, r.topk_idx[a:b])
            assert torch.equal(part.topk_weights.view(torch.int32), r.topk_weights[a:b].view(torch.int32))
            dp = cgl.route_backward(g[a:b].contiguous(), l[a:b].contiguous(), idx[a:b].contiguous(), **how)
            assert torch.equal(dp.view(torch.int16), d[a:b].view(torch.int16))


def test_offsets_past_32_bits():
    n, e = 4_300_000, 512                         # 2.2e9 logits
    l = torch.zeros(n, e, dtype=torch.bfloat16, device="cuda")
    tail = _logits(64, e, 3, "bf16")
    l[-64:] = tail
    r = cgl.route(l, 2, renormalize=False)
    want = cgl.route(tail, 2, renormalize=False)
    assert torch.equal(r.topk_idx[-64:], want.topk_idx) and torch.equal(r.topk_weights[-64:], want.topk_weights)
    assert (r.topk_idx[:-64] == torch.tensor([0, 1], device="cuda")).all()
    g = _grad(64, 2)
    big = torch.zeros(n, 2, device="cuda")
    big[-64:] = g
    d = cgl.route_backward(big, l, r.topk_idx, renormalize=False)
    assert torch.equal(d[-64:], cgl.route_backward(g, tail, want.topk_idx, renormalize=False)) and (d[:-64] == 0).all()


def test_refusals():
    l, g = _logits(8, 32, 1), _grad(8, 4)
    idx = cgl.route(l, 4).topk_idx
    bad = [
        (TypeError, lambda: cgl.route(l.double(), 4)), (TypeError, lambda: cgl.route(l.cpu(), 4)), (ValueError, lambda: cgl.route(l[0], 4)),
        (ValueError, lambda: cgl.route(l[:, ::2], 4)), (cgl.CglError, lambda: cgl.route(l, 0)), (cgl.CglError, lambda: cgl.route(l, 33)),
        (cgl.CglError, lambda: cgl.route(l[:, :3].contiguous(), 4)), (ValueError, lambda: cgl.route(l, 4, score="tanh")),
        (ValueError, lambda: cgl.route(l, 4, group_score="sum")), (cgl.CglError, lambda: cgl.route(l, 4, num_groups=5)),
        (cgl.CglError, lambda: cgl.route(l, 4, num_groups=4, topk_groups=5)), (cgl.CglError, lambda: cgl.route(l, 4, num_groups=4, topk_groups=0)),
        (cgl.CglError, lambda: cgl.route(l, 4, num_groups=0)), (TypeError, lambda: cgl.route(l, 4, bias=torch.zeros(32))),
        (TypeError, lambda: cgl.route(l, 4, bias=torch.zeros(32, device="cuda").bfloat16())),
        (ValueError, lambda: cgl.route(l, 4, bias=torch.zeros(31, device="cuda"))),
        (ValueError, lambda: cgl.route(l, 4, topk_idx=torch.zeros(8, 5, dtype=torch.int32, device="cuda"))),
        (TypeError, lambda: cgl.route(l, 4, topk_weights=torch.zeros(8, 4, dtype=torch.float16, device="cuda"))),
        (ValueError, lambda: cgl.route_backward(g[:7].contiguous(), l, idx)), (TypeError, lambda: cgl.route_backward(g.half(), l, idx)),
        (TypeError, lambda: cgl.route_backward(g, l, idx.long())), (ValueError, lambda: cgl.route_backward(g, l, idx[:4].contiguous())),
        (ValueError, lambda: cgl.route_backward(g, l, idx, score="tanh")), (ValueError, lambda: cgl.route_backward(g, l, idx, grad_logits=l[:4])),
        (TypeError, lambda: cgl.route_backward(g, l, idx, grad_logits=l.bfloat16())),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was not refused")
