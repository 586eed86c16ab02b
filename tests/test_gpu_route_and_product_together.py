"""The routing and the BF16 product as a layer uses them, forward and backward: with layout, dispatch and combine,
captured and replayed, on other streams, two at once, past 32-bit offsets."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu

HOW = dict(score="sigmoid", scale=1.5)
PICK = dict(num_groups=4, topk_groups=2, group_score="top2")


def _layer(n=300, h=256, f=192, e=16, seed=0):
    """x, logits, bias, first weights [E, 2 f, h] (gated), second [E, h, f], gradient of the output."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return [r(n, h).bfloat16().cuda(), r(n, e).cuda(), (0.1 * r(e)).cuda(), (r(e, 2 * f, h) / h ** 0.5).bfloat16().cuda(),
            (r(e, h, f) / f ** 0.5).bfloat16().cuda(), r(n, h).bfloat16().cuda()]


def _step(x, logits, bias, w1, w2, g, cap=0, k=4, stream=None, st=None):
    """A training step of the layer: output, and the gradients of x, logits and weights."""
    e, kw = w1.shape[0], dict(stream=stream, status=st)
    r = cgl.route(logits, k, bias=bias, **PICK, **HOW, **kw)
    lay = cgl.get_layout(r.topk_idx, e, e // 4, cap, **kw)
    rx = cgl.dispatch_bf16(x, lay.dst_pos, lay.num_recv_rows, **kw)
    hid, z = cgl.matmul_bf16(rx, w1, lay.expert_offset, cap, activation="swiglu", with_preact=True, **kw)
    y = cgl.matmul_bf16(hid, w2, lay.expert_offset, cap, **kw)
    out = cgl.combine(y, lay.dst_pos, r.topk_weights, **kw)
    gy, gw = cgl.combine_backward(g, y, lay.dst_pos, r.topk_weights, **kw)
    d2 = cgl.matmul_bf16_backward(gy, hid, w2, lay.expert_offset, cap, **kw)
    d1 = cgl.matmul_bf16_backward(d2.grad_a, rx, w1, lay.expert_offset, cap, activation="swiglu", preact=z, **kw)
    dl = cgl.route_backward(gw, logits, r.topk_idx, **HOW, **kw)
    dx = cgl.combine(d1.grad_a, lay.dst_pos, torch.ones_like(r.topk_weights), **kw)
    return out, dx, dl, d1.grad_w, d2.grad_w, r.topk_idx, r.topk_weights


@pytest.mark.parametrize("cap", [0, 300])
def test_step_against_64_bits(cap):
    """Every result within a few BF16 roundings of autograd's in 64 bits, the choice given: a result passes at most six (x is exact;
    z, hid, y or their gradients, dz, the result), each 2^-8 of its value, measured by the results' root mean square over all
    entries, since a rounded term's error is of the size of the terms and not of a cancelled sum."""
    args = _layer()
    st = cgl.new_status()
    out, dx, dl, dw1, dw2, idx, wt = _step(*args, cap=cap, st=st)
    assert cgl.status_bits(st) == []
    x, logits, bias, w1, w2, g = [t.double().cpu() for t in args]
    x, logits, w1, w2 = (t.requires_grad_() for t in (x, logits, w1, w2))
    s = torch.sigmoid(logits)
    at = idx.long().cpu()
    w = s.gather(1, at)
    w = 1.5 * w / w.sum(1, keepdim=True)
    ref = 0
    for j in range(idx.shape[1]):
        h = torch.einsum("th,tfh->tf", x, w1[at[:, j]])
        a, b = h.chunk(2, 1)
        ref = ref + w[:, j, None] * torch.einsum("tf,thf->th", torch.nn.functional.silu(a) * b, w2[at[:, j]])
    ref.backward(g)
    for got, want in ((out, ref.detach()), (dx, x.grad), (dl, logits.grad), (dw1, w1.grad), (dw2, w2.grad)):
        off = (got.double().cpu() - want).pow(2).mean().sqrt()
        assert off <= 6 * 2.0 ** -8 * want.pow(2).mean().sqrt()
    assert ((wt.double().cpu() - w.detach()).abs() <= 2.0 ** -18 * w.detach()).all()


def test_captured_step_replays_on_new_inputs():
    args = _layer()
    st = cgl.new_status()
    _step(*args, st=st)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                     # two graphs of the same step, each with its own buffers
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_step(*args, st=st))
        graphs.append(gr)
    for seed in (1, 2, 3):
        for a, b in zip(args, _layer(seed=seed)):
            a.copy_(b)
        for gr in graphs + graphs[::-1]:
            gr.replay()
        torch.cuda.synchronize()
        want = _step(*args, st=st)
        for got in outs:
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert cgl.status_bits(st) == []


def test_other_streams_and_two_calls_at_once():
    args = _layer(n=1500, h=512, f=384)
    want = _step(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):      # the current stream, or given
            got.append(_step(*args, stream=streams[i % 2] if i > 2 else None))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_given_stream_owns_what_the_calls_allocate(as_handle):
    """The given stream is behind; the caller's stream meanwhile reuses whatever memory it may."""
    x, logits, bias, w1, w2, g = _layer(n=600)
    r = cgl.route(logits, 4, bias=bias, **PICK, **HOW)
    lay = cgl.get_layout(r.topk_idx, 16, 4)
    rx = cgl.dispatch_bf16(x, lay.dst_pos, lay.num_recv_rows)
    how = dict(activation="swiglu")
    hid, z = cgl.matmul_bf16(rx, w1, lay.expert_offset, with_preact=True, **how)
    d = cgl.matmul_bf16_backward(hid, rx, w1, lay.expert_offset, preact=z, want_bias=True, **how)
    gw = torch.ones_like(r.topk_weights)
    dl = cgl.route_backward(gw, logits, r.topk_idx, **HOW)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                # about 10 ms
    kw = dict(stream=s.cuda_stream if as_handle else s)
    r2 = cgl.route(logits, 4, bias=bias, **PICK, **HOW, **kw)
    hid2, z2 = cgl.matmul_bf16(rx, w1, lay.expert_offset, with_preact=True, **how, **kw)
    d2 = cgl.matmul_bf16_backward(hid, rx, w1, lay.expert_offset, preact=z, want_bias=True, **how, **kw)
    dl2 = cgl.route_backward(gw, logits, r.topk_idx, **HOW, **kw)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 70_000, 300_000, 1 << 20) for _ in range(8)]
    torch.cuda.synchronize()
    for p, q in zip((*r, hid, z, *d, dl), (*r2, hid2, z2, *d2, dl2)):
        assert torch.equal(p, q)
    assert len(junk) == 40


def test_product_past_32_bit_offsets():
    """Rows, results, and their gradients past 2^32 bytes."""
    rows, k, f = 320_000, 64, 7168                # y: 2.3e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda", dtype=torch.int8).bfloat16()
    a, w = new(rows, k), new(f, k)
    y = cgl.matmul_bf16(a, w)
    for r in (slice(0, 300), slice(rows - 300, rows)):
        assert torch.equal(y[r], (a[r].double() @ w.double().T).float().bfloat16())
    grad = new(rows, f)
    d = cgl.matmul_bf16_backward(grad, a, w, want_bias=True)
    for r in (slice(0, 300), slice(rows - 300, rows)):
        assert torch.equal(d.grad_a[r], (grad[r].double() @ w.double()).float().bfloat16())
    want = sum(grad[i:i + 40_000].double().T @ a[i:i + 40_000].double() for i in range(0, rows, 40_000))
    assert want.abs().max() < 2 ** 24             # 320000 products of at most 16, partial sums far below
    assert torch.equal(d.grad_w, want.float().bfloat16())
    want = sum(grad[i:i + 40_000].double().sum(0) for i in range(0, rows, 40_000))
    assert torch.equal(d.grad_bias, want.float().bfloat16())


def test_weights_past_32_bit_offsets():
    e, f, k = 64, 8192, 4608                      # 2.4e9 values
    w = torch.zeros(e, f, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w[-1] = torch.randint(-4, 5, (f, k), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    a = torch.randint(-4, 5, (70, k), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    off = torch.full((e + 1,), 30, dtype=torch.int32, device="cuda")
    off[0], off[-1] = 0, 70
    y = cgl.matmul_bf16(a, w, off)
    assert (y[:30] == 0).all() and torch.equal(y[30:], (a[30:].double() @ w[-1].double().T).float().bfloat16())
    grad = torch.randint(-4, 5, (70, f), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    d = cgl.matmul_bf16_backward(grad, a, w, off)
    assert torch.equal(d.grad_a[30:], (grad[30:].double() @ w[-1].double()).float().bfloat16()) and (d.grad_a[:30] == 0).all()
    assert torch.equal(d.grad_w[-1], (grad[30:].double().T @ a[30:].double()).float().bfloat16())
    assert torch.equal(d.grad_w[0], (grad[:30].double().T @ a[:30].double()).float().bfloat16()) and (d.grad_w[1:-1] == 0).all()
