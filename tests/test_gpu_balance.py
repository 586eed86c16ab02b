"""The balance loss, its counts and its gradient against the definition in 64 bits.

Tolerances, u = 2^-24 (binary32's half step).  A probability is an exponential (2 steps = 4u, and D u from its
rounded argument, D the row's spread), divided by a sum of E such terms in lane order (E / 32 + 5 additions) and a
few single operations (6u): p is off by tp = (D + E / 32 + 15) u at most, a weight by u.  So the centred bracket
w_i - sum p w is off by at most 2 tp (|w_i| + sum p |w|), p times it by as much again, and the gradient by
p gate |g| 4 tp (|w_i| + sum p |w|) + half a step of the output type (+ its smallest subnormal).
"""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def definition(logits, idx, S, alpha, score, g=1.0):
    """Loss, counts, routed, grad and the tolerances of loss and grad, float64 on the host."""
    l = logits.double().cpu()
    idx = idx.cpu().long()
    n, E = l.shape
    k, T = idx.shape[1], n // S
    ok = (idx >= 0) & (idx < E)
    loss, tol_loss = 0.0, 0.0
    counts = torch.zeros(S, E, dtype=torch.int64)
    routed = torch.zeros(S, dtype=torch.int64)
    grad, tol = torch.zeros(n, E, dtype=torch.float64), torch.zeros(n, E, dtype=torch.float64)
    for s in range(S):
        r = slice(s * T, (s + 1) * T)
        counts[s] = torch.bincount(idx[r][ok[r]], minlength=E)
        here = ok[r].any(1)
        routed[s] = here.sum()
        t = int(routed[s])
        if t == 0:
            continue
        x = l[r]
        dead = torch.isneginf(x).all(1)
        if score == "softmax":
            p = torch.softmax(x, 1)
            gate = torch.ones_like(p)
        else:
            m = x.amax(1, keepdim=True).clamp(max=0)
            q = torch.where(x > 0, 1.0, torch.exp(x - m)) / (1 + torch.exp(-x.abs()))   # sigmoid(x) exp(-m)
            p = q / q.sum(1, keepdim=True)
            gate = torch.sigmoid(-x)
        p[dead] = 0
        p = p * here[:, None]
        w = alpha * E * counts[s].double() / (S * k * t * t)
        c = alpha * (E * counts[s] - counts[s].sum()).double() / (S * k * t * t)
        loss += (p * w).sum()
        size = (p * c.abs()).sum(1, keepdim=True)
        dot = (p * c).sum(1, keepdim=True)
        grad[r] = g * p * gate * (c - dot)
        spread = torch.where(torch.isfinite(x), (x - x.amax(1, keepdim=True)).abs(), 0.0).amax(1, keepdim=True).nan_to_num(0)
        tp = (spread + E / 32 + 15) * U
        tol[r] = abs(g) * p * gate * 4 * tp * (c.abs() + size)
        tol_loss += (p.sum(1) * (w.mean() * 3 * U) + 4 * (tp * size)[:, 0]).sum()
    half = torch.finfo(logits.dtype)
    tol = tol + half.eps / 2 * grad.abs() * (1 + 1e-3) + half.tiny * half.eps
    return float(loss), counts.int(), routed.int(), grad, float(tol_loss + U * abs(loss)) + 1e-45, tol


def _inputs(n, E, k, dtype, seed, pad=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(n, E, generator=g) * spread).to(dtype)
    idx = torch.argsort(torch.rand(n, E, generator=g), dim=1)[:, :k].int() if k <= E else \
        torch.randint(0, E, (n, k), generator=g, dtype=torch.int32)
    if pad:
        idx[torch.rand(n, k, generator=g) < pad / 2] = -1
        idx[torch.rand(n, generator=g) < pad] = -1
    return logits.cuda(), idx.contiguous().cuda()


def _check(logits, idx, S=1, alpha=0.02, score="softmax", g=1.0, status=None):
    loss, counts, routed, grad, tol_loss, tol = definition(logits, idx, S, alpha, score, g)
    gl = torch.full((1,), g, device="cuda")
    kw = dict(num_sequences=S, alpha=alpha, score=score)
    b = cgl.balance_loss(logits, idx, grad_loss=gl, status=status, **kw)
    assert torch.equal(b.counts.cpu(), counts) and torch.equal(b.num_routed.cpu(), routed)
    assert abs(float(b.loss) - loss) <= tol_loss
    assert ((b.grad_logits.cpu().double() - grad).abs() <= tol).all()
    f = cgl.balance_loss(logits, idx, status=status, **kw)
    assert f.grad_logits is None and torch.equal(f.loss, b.loss) and torch.equal(f.counts, b.counts)
    assert torch.equal(cgl.balance_loss_backward(gl, logits, idx, f.counts, f.num_routed, **kw), b.grad_logits)
    return b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,E,k,S,pad", [(1, 1, 1, 1, 0), (1, 16, 4, 1, 0), (128, 16, 4, 1, 0), (7, 5, 2, 7, 0.3), (96, 33, 3, 4, 0.2),
                                         (300, 64, 6, 3, 0.5), (1000, 256, 8, 1, 0.1), (515, 100, 32, 5, 0.1),
                                         (64, 1024, 8, 2, 0), (40, 1000, 1, 1, 0.2), (3000, 128, 2, 10, 0),
                                         (30, 130, 4, 1, 0.1), (50, 701, 5, 2, 0.1), (33, 512, 8, 1, 0.1)])
def test_against_definition(n, E, k, S, pad, score, dtype):
    logits, idx = _inputs(n, E, k, dtype, n + E, pad)
    _check(logits, idx, S, 0.02, score, g=256.0 if dtype == torch.float16 else 0.75)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(256, 8), (128, 3), (72, 2)])
def test_large_batch(E, k, score, dtype):
    """Past the size at which 16-bit logits take two groups of experts a lane."""
    logits, idx = _inputs(20000, E, k, dtype, 5, 0.05)
    _check(logits, idx, 4, 1e-3, score, g=0.75 * 2 ** 10)


def test_repeated_ids_and_unaligned_rows():
    """A token may name an expert twice; rows off the 16-byte grid take the other loads, with equal values."""
    g = torch.Generator().manual_seed(3)
    idx = torch.randint(0, 64, (200, 6), generator=g, dtype=torch.int32).cuda()
    idx[:, 1] = idx[:, 0]
    logits = _inputs(200, 64, 6, torch.float32, 4)[0]
    b = _check(logits, idx, 2)
    off = torch.empty(200 * 64 + 1, device="cuda")[1:].view(200, 64)
    off.copy_(logits)
    u = _check(off, idx, 2)
    assert torch.equal(u.counts, b.counts)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Spreads past the exponential's range, rows far below zero (every sigmoid underflows), far above it."""
    logits, idx = _inputs(64, 32, 4, torch.float32, 9, spread=1.0)
    logits[0:16] *= 60
    logits[16:32] -= 500
    logits[32:48] += 500
    _check(logits, idx, 1, 0.5, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_logits(score):
    """-inf experts get no probability; a row of nothing but -inf has none at all, and no gradient."""
    logits, idx = _inputs(50, 40, 4, torch.float32, 11)
    logits[:, ::3] = -torch.inf
    logits[7] = -torch.inf
    b = _check(logits, idx, 1, 0.5, score)
    assert (b.grad_logits[7] == 0).all() and (b.grad_logits[:, ::3] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_logit_spoils_its_row_and_the_loss(score):
    logits, idx = _inputs(20, 40, 4, torch.float32, 12)
    clean = cgl.balance_loss(logits, idx, grad_loss=torch.ones(1, device="cuda"), score=score)
    logits[3, 5] = torch.nan
    logits[4] = -torch.inf
    logits[4, 0] = torch.nan
    b = cgl.balance_loss(logits, idx, grad_loss=torch.ones(1, device="cuda"), score=score)
    assert b.loss.isnan().all() and b.grad_logits[3:5].isnan().all()
    rest = [i for i in range(20) if i not in (3, 4)]
    assert torch.equal(b.grad_logits[rest], clean.grad_logits[rest])


def test_nothing_routed_and_padded_sequences():
    logits, idx = _inputs(12, 8, 2, torch.float32, 13)
    idx[:] = -1
    b = _check(logits, idx, 3)
    assert float(b.loss) == 0 and (b.grad_logits == 0).all() and (b.num_routed == 0).all()
    logits[0, 0] = torch.nan            # tokens that take no part may hold anything
    assert float(_loss(logits, idx)) == 0
    logits, idx = _inputs(12, 8, 2, torch.float32, 14)
    idx[4:8] = -1
    _check(logits, idx, 3)


def _loss(logits, idx, **kw):
    return cgl.balance_loss(logits, idx, **kw).loss


def test_empty_batch():
    b = cgl.balance_loss(torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"),
                         num_sequences=2, grad_loss=torch.ones(1, device="cuda"))
    assert float(b.loss) == 0 and (b.counts == 0).all() and (b.num_routed == 0).all() and b.grad_logits.shape == (0, 8)


def test_bad_ids_are_reported_and_not_counted():
    logits, idx = _inputs(30, 8, 3, torch.float32, 15)
    idx[2, 1], idx[9] = 8, -2
    st = cgl.new_status()
    b = _check(logits, idx, 1, status=st)
    assert cgl.status_bits(st) == ["CGL_ERANGE"] and int(b.num_routed) == 29 and int(b.counts.sum()) == 30 * 3 - 4


def test_counts_are_the_layouts():
    logits, idx = _inputs(500, 64, 4, torch.float32, 16, 0.2)
    lay = cgl.get_layout(idx, 64, 8)
    assert torch.equal(cgl.balance_loss(logits, idx).counts[0], lay.tokens_per_expert)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """Central differences of the 64-bit loss (step 1e-4: truncation 1e-8 of the third derivative, at most a few times
    the first's size at these spreads; rounding 1e-12), so 1e-6 of the largest entry beside the kernel's own tolerance."""
    logits, idx = _inputs(6, 7, 2, torch.float32, 17, 0.2, spread=1.0)
    _, _, _, grad, _, tol = definition(logits, idx, 2, 1.0, score)
    got = cgl.balance_loss(logits, idx, num_sequences=2, score=score, grad_loss=torch.ones(1, device="cuda")).grad_logits.cpu()
    x, h = logits.double().cpu(), 1e-4
    diff = torch.zeros_like(x)
    for i in range(6):
        for j in range(7):
            up, dn = x.clone(), x.clone()
            up[i, j] += h
            dn[i, j] -= h
            # the definition takes its logits as given, float64 included
            diff[i, j] = (_loss64(up, idx, score) - _loss64(dn, idx, score)) / (2 * h)
    assert ((got.double() - diff).abs() <= tol + 1e-6 * diff.abs().max()).all()


def _loss64(x, idx, score):
    return definition(x, idx, 2, 1.0, score)[0]
