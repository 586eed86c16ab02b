"""The balance loss on finite logits of any size: rows masked with the type's lowest value, rows far from zero.

Tolerances, u = 2^-24.  The exponent (l - m) log2(e) is off by a rounding of the difference, of the product and of the
constant: 3 D u, D the largest l - m among the terms that binary32 can hold (exp(-104) is below half its smallest
subnormal; a term past that may be one such step, 2^-149).  Exponential 4u, the sum of E terms in lane order
(E / 32 + 5) u, single operations 10u: a probability is off by tp = (3 D + E / 32 + 19) u, a centred weight by u, so the
bracket c_i - sum p c by 2 tp (|c_i| + sum p |c|), p times it by as much again; then half a step of the output type.
"""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA = 0.5


def definition(logits, idx, score):
    """Loss and gradient in 64 bits (one sequence, every token routed), and their tolerances."""
    x, idx = logits.double().cpu(), idx.cpu().long()
    (n, e), k = x.shape, idx.shape[1]
    m = x.amax(1, keepdim=True)
    gate = torch.ones_like(x)
    if score == "sigmoid":
        m = m.clamp(max=0)
        gate = torch.sigmoid(-x)
    alive = ~torch.isneginf(x).all(1, keepdim=True)
    d = torch.where(alive, x - torch.where(alive, m, 0.0), -torch.inf)
    q = torch.exp(d if score == "softmax" else torch.where(x > 0, 0.0, d))
    if score == "sigmoid":
        q = q / (1 + torch.exp(-x.abs()))
    p = torch.where(alive, q / q.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(idx.flatten(), minlength=e)
    unit = ALPHA / (k * n * n)
    w, c = unit * e * counts.double(), unit * (e * counts - counts.sum()).double()
    dot, size = (p * c).sum(1, keepdim=True), (p * c.abs()).sum(1, keepdim=True)
    grad = p * gate * (c - dot)
    spread = torch.where(d > -104, d.abs(), 0.0).amax(1, keepdim=True)
    tp = (3 * spread + e / 32 + 19) * U
    half = torch.finfo(logits.dtype)
    tol = p * gate * 4 * tp * (c.abs() + size) + 2.0 ** -149 * (c.abs() + c.abs().amax()) + half.eps / 2 * grad.abs() * (1 + 1e-3) \
        + half.tiny * half.eps
    loss = (p * w).sum()
    tol_loss = (p.sum(1) * w.mean() * 3 * U).sum() + (4 * tp * (size + e * 2.0 ** -149)).sum() + U * loss.abs()
    return float(loss), grad, float(tol_loss) + 1e-45, tol


FAR = {
    "lowest": lambda x, e: torch.full_like(x, torch.finfo(x.dtype).min),
    "highest": lambda x, e: torch.full_like(x, torch.finfo(x.dtype).max),
    "-1e10": lambda x, e: torch.full_like(x, -1e10),
    "+1e10": lambda x, e: torch.full_like(x, 1e10),
    "-1e30": lambda x, e: torch.full_like(x, -1e30),
    "around -1e10": lambda x, e: (x.float() * 2000 - 1e10).to(x.dtype),
    "around +1e10": lambda x, e: (x.float() * 2000 + 1e10).to(x.dtype),
    "around -3e6": lambda x, e: (x.float() - 3e6).to(x.dtype),
    "around +1e6": lambda x, e: (x.float() + 1e6).to(x.dtype),
    "half masked with the lowest": lambda x, e: torch.where(torch.arange(e) % 2 == 0, x, torch.finfo(x.dtype).min),
    "one high": lambda x, e: torch.where(torch.arange(e) == 3, torch.tensor(3e38, dtype=x.dtype), x),
    "one high, the rest lowest": lambda x, e: torch.where(torch.arange(e) == e - 1, torch.tensor(3e38, dtype=x.dtype),
                                                          torch.finfo(x.dtype).min),
    "lowest among -inf": lambda x, e: torch.where(torch.arange(e) % 3 == 1, torch.tensor(torch.finfo(x.dtype).min, dtype=x.dtype),
                                                  -torch.inf),
    "-inf": lambda x, e: torch.full_like(x, -torch.inf),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,n", [(8, 60), (16, 60), (32, 64), (256, 64), (33, 40), (130, 40), (1024, 20), (256, 12500),
                                 (8, 61), (16, 61), (32, 61), (33, 41), (130, 43), (1024, 21)])
def test_finite_logits_of_any_size(e, n, score, dtype):
    """Rows of each kind among ordinary ones (several rows share a warp, which must not notice)."""
    g = torch.Generator().manual_seed(e)
    plain = torch.randn(n, e, generator=g).to(dtype)
    idx = torch.randint(0, max(e // 2, 1), (n, 4), generator=g, dtype=torch.int32).cuda()
    one = torch.ones(1, device="cuda")
    before = cgl.balance_loss(plain.cuda(), idx, alpha=ALPHA, score=score, grad_loss=one)
    logits, rows = plain.clone(), {}
    for i, (name, make) in enumerate(FAR.items()):
        if i >= n:
            break
        r = (5 * i + 1) % n
        rows[r] = name
        logits[r] = make(plain[r], e).to(dtype)
    dev = logits.cuda()
    b = cgl.balance_loss(dev, idx, alpha=ALPHA, score=score, grad_loss=one)
    loss, grad, tol_loss, tol = definition(logits, idx, score)
    got = b.grad_logits.cpu().double()
    wrong = [rows.get(r, "plain") for r in torch.nonzero(~((got - grad).abs() <= tol).all(1))[:, 0].tolist()]
    assert wrong == []
    assert abs(float(b.loss) - loss) <= tol_loss
    rest = torch.tensor([r for r in range(n) if r not in rows])
    assert torch.equal(b.grad_logits.cpu()[rest], before.grad_logits.cpu()[rest])
    f = cgl.balance_loss(dev, idx, alpha=ALPHA, score=score)
    assert torch.equal(f.loss, b.loss)
    back = cgl.balance_loss_backward(one, dev, idx, f.counts, f.num_routed, alpha=ALPHA, score=score)
    assert torch.equal(back, b.grad_logits)


@pytest.mark.parametrize("fill", ["lowest", "-1e10", "+1e10", "highest"])
def test_a_batch_of_one_far_row(fill):
    """One routed token with equal logits: uniform probabilities, whatever their size: the loss is alpha exactly."""
    logits = FAR[fill](torch.zeros(1, 32), 32).cuda()
    idx = torch.tensor([[1, 7, 9, 20]], dtype=torch.int32, device="cuda")
    b = cgl.balance_loss(logits, idx, alpha=ALPHA, grad_loss=torch.ones(1, device="cuda"))
    assert float(b.loss) == ALPHA and int(b.num_routed) == 1
    w = torch.full((32,), -0.5 * 4 / 4, device="cuda")     # alpha (E c - k) / k: 3.5 where chosen, -0.5 elsewhere
    w[idx[0].long()] = 3.5
    assert torch.equal(b.grad_logits[0], w / 32)
