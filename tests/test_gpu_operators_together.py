"""The MXFP4 calls and the balance loss as a layer uses them: together with layout and combine, captured and
replayed, on other streams, two at once, with unaligned buffers and past 32-bit offsets."""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
import mxref
from combine_get_layout_02_b200 import workloads as W

pytestmark = pytest.mark.gpu


def _layer(n=300, h=512, f=256, e=16, k=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=g).bfloat16().cuda()
    logits = torch.randn(n, e, generator=g).cuda()
    idx = torch.topk(logits, k, dim=1).indices.int().contiguous()
    wt = torch.softmax(torch.randn(n, k, generator=g), 1).cuda()
    w = torch.randn(e, f, h, generator=g).cuda() / 32
    wq, ws = cgl.quantize_mxfp4(w)
    return x, logits, idx, wt, wq, ws


def _forward(x, idx, wt, wq, ws, cap=0, stream=None, **kw):
    e = wq.shape[0]
    lay = cgl.get_layout(idx, e, e // 4, cap, stream=stream, **kw)
    rx, rs = cgl.dispatch_mxfp4(x, lay.dst_pos, lay.num_recv_rows, stream=stream, **kw)
    y = cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset, cap, stream=stream, **kw)
    return lay, rx, rs, y, cgl.combine(y, lay.dst_pos, wt, stream=stream, **kw)


@pytest.mark.parametrize("cap", [0, 200, 40])
def test_layer_against_64_bits(cap):
    """Every stage against its definition; with 40 rows an expert some copies are dropped."""
    x, _, idx, wt, wq, ws = _layer()
    st = cgl.new_status()
    lay, rx, rs, y, out = _forward(x, idx, wt, wq, ws, cap, status=st)
    assert cgl.status_bits(st) == (["CGL_ECAPACITY"] if cap == 40 else [])
    vx = torch.tensor(mxref.values(*mxref.quantize(x.double().cpu().numpy()))).cuda()
    vw = mxref.values_t(wq, ws)
    dst = lay.dst_pos.long()
    # a copy's row: values are multiples of 2^-(...) far inside 24 bits, so the sum in binary32 is near exact; K = 512
    for j in range(idx.shape[1]):
        t = torch.nonzero(dst[:, j] >= 0)[:, 0]
        ref = torch.einsum("th,tfh->tf", vx[t], vw[idx[t, j].long()])
        s = torch.einsum("th,tfh->tf", vx[t].abs(), vw[idx[t, j].long()].abs())
        got = y[dst[t, j]].double()
        assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 512 * 2.0 ** -23 * s).all()
    # combine of these rows: fixed order, one rounding a product and a sum, then BF16
    acc = torch.zeros(out.shape, device="cuda")
    for j in range(idx.shape[1]):
        use = dst[:, j] >= 0
        acc[use] = acc[use] + wt[use, j, None] * y[dst[use, j]].float()
    assert torch.equal(out, acc.bfloat16())


def test_captured_layer_replays_on_new_inputs():
    x, logits, idx, wt, wq, ws = _layer()
    gl = torch.full((1,), 0.5, device="cuda")
    st = cgl.new_status()

    def step():
        *_, out = _forward(x, idx, wt, wq, ws, status=st)
        b = cgl.balance_loss(logits, idx, alpha=0.1, status=st)
        g = cgl.balance_loss_backward(gl, logits, idx, b.counts, b.num_routed, alpha=0.1)
        return out, b.loss, b.counts, g

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                     # two graphs of the same step, each with its own buffers
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    for seed in (1, 2, 3):
        x2, logits2, idx2, wt2, _, _ = _layer(seed=seed)
        for a, b in ((x, x2), (logits, logits2), (idx, idx2), (wt, wt2)):
            a.copy_(b)
        for gr in graphs + graphs[::-1]:
            gr.replay()
        torch.cuda.synchronize()
        want = step()
        for got in outs:
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert cgl.status_bits(st) == []


def test_other_streams_and_two_calls_at_once():
    x, logits, idx, wt, wq, ws = _layer(n=2000, h=1024, f=768)
    want = _forward(x, idx, wt, wq, ws)[-1]
    lw = cgl.balance_loss(logits, idx, grad_loss=torch.ones(1, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, loss = [], []
    for i in range(6):
        s = streams[i % 2]
        if i < 3:                          # the current stream, or given
            with torch.cuda.stream(s):
                got.append(_forward(x, idx, wt, wq, ws)[-1])
                loss.append(cgl.balance_loss(logits, idx, grad_loss=torch.ones(1, device="cuda")))
        else:
            with torch.cuda.stream(s):     # temporaries belong to s
                got.append(_forward(x, idx, wt, wq, ws, stream=s)[-1])
                loss.append(cgl.balance_loss(logits, idx, grad_loss=torch.ones(1, device="cuda"), stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert all(torch.equal(b.loss, lw.loss) and torch.equal(b.grad_logits, lw.grad_logits) for b in loss)


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_given_stream_owns_what_the_call_allocates(as_handle):
    """The given stream is behind; the caller's stream meanwhile reuses whatever memory it may."""
    x, logits, idx, wt, wq, ws = _layer(n=600)
    lay = cgl.get_layout(idx, 16, 4)
    one = torch.ones(1, device="cuda")
    want = cgl.balance_loss(logits, idx, grad_loss=one)
    rx, rs = cgl.dispatch_mxfp4(x, lay.dst_pos, lay.num_recv_rows)
    y = cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                # about 10 ms
    arg = s.cuda_stream if as_handle else s
    b = cgl.balance_loss(logits, idx, grad_loss=one, stream=arg)
    px, ps = cgl.dispatch_mxfp4(x, lay.dst_pos, lay.num_recv_rows, stream=arg)
    py = cgl.matmul_mxfp4(px, ps, wq, ws, lay.expert_offset, stream=arg)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 70_000, 300_000, 1 << 20) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(b.loss, want.loss) and torch.equal(b.counts, want.counts) and torch.equal(b.grad_logits, want.grad_logits)
    assert torch.equal(px, rx) and torch.equal(ps, rs) and torch.equal(py, y) and len(junk) == 40


def test_unaligned_buffers():
    """y and the scales at any address they may have; dispatch's scale rows too."""
    x, _, idx, wt, wq, ws = _layer(n=100, h=512, f=264)
    lay, rx, rs, y, _ = _forward(x, idx, wt, wq, ws)
    rows, f = y.shape
    y1 = torch.zeros(rows * f + 3, dtype=torch.bfloat16, device="cuda")[3:].view(rows, f)
    rs1 = torch.empty(rs.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(rs)
    ws1 = torch.empty(ws.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view_as(ws)
    ws1.copy_(ws)
    cgl.dispatch_mxfp4(x, lay.dst_pos, rows, recv_x=rx, recv_scale=rs1)
    assert torch.equal(rs1, rs)
    cgl.matmul_mxfp4(rx, rs1, wq, ws1, lay.expert_offset, y=y1)
    assert torch.equal(y1, y)
    s1 = torch.empty(rows * 16 + 5, dtype=torch.uint8, device="cuda")[5:].view(rows, 16)
    v = cgl.dequantize_mxfp4(rx, rs)
    c2, s2 = cgl.quantize_mxfp4(v, scales=s1)     # its values hold themselves
    assert torch.equal(cgl.dequantize_mxfp4(c2, s2), v)


def test_rows_past_32_bit_offsets():
    rows, c = 310_000, 7168                       # 2.2e9 values: byte offsets of x and out past 2^32
    x = torch.empty(rows, c, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    x[-3:] = torch.randn(3, c, device="cuda").bfloat16()
    codes, scales = cgl.quantize_mxfp4(x)
    tail = cgl.quantize_mxfp4(x[-3:].clone())
    assert torch.equal(codes[-3:], tail[0]) and torch.equal(scales[-3:], tail[1])
    out = cgl.dequantize_mxfp4(codes, scales, out=x)
    assert torch.equal(out[-3:], cgl.dequantize_mxfp4(*tail)) and (out[-1000:-3] == 1.0).all()


def test_product_past_32_bit_offsets():
    rows, k, f = 320_000, 64, 7168                # y: 2.3e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    a, sa = mxref.codes_like(rows, k, g, "cuda", 127, 127)
    w, sw = mxref.codes_like(f, k, g, "cuda", 127, 127)
    y = cgl.matmul_mxfp4(a, sa, w, sw)
    for r in (slice(0, 300), slice(rows - 300, rows)):
        ref, _ = mxref.product(a[r], sa[r], w[None], sw[None], [(0, 300)])
        assert torch.equal(y[r], ref.float().bfloat16())


def test_dispatch_past_32_bit_offsets():
    n, h, k = 40_000, 16384, 8                    # rows of 8192 bytes: 2.6e9 bytes of codes
    x = torch.randn(n, h, device="cuda").bfloat16()
    dst = (torch.arange(n * k, device="cuda", dtype=torch.int32).flip(0)).view(n, k).contiguous()
    rx, rs = cgl.dispatch_mxfp4(x, dst, n * k, scratch=cgl.new_scratch())
    for t in (0, 1, n - 1):
        codes, scales = cgl.quantize_mxfp4(x[t:t + 1])
        for j in (0, k - 1):
            assert torch.equal(rx[dst[t, j]], codes[0]) and torch.equal(rs[dst[t, j]], scales[0])


def test_workload_counts_and_offsets_feed_the_calls():
    """A named workload's routing through layout, counts and product, group-limited top-k."""
    inp = W.make_inputs("tiny", 0)
    idx = torch.from_numpy(inp.topk_idx).cuda()
    e = inp.workload.num_experts
    lay = cgl.get_layout(idx, e, inp.workload.num_ranks)
    scores = torch.from_numpy(inp.scores).cuda()
    b = cgl.balance_loss(torch.logit(scores.double()).float(), idx, score="sigmoid")
    assert torch.equal(b.counts[0], lay.tokens_per_expert) and int(b.num_routed) == idx.shape[0]
    assert float(b.loss) > 0


def test_python_refusals():
    x, logits, idx, wt, wq, ws = _layer(n=16, h=64, f=32, e=4, k=2)
    lay, rx, rs, y, _ = _forward(x, idx, wt, wq, ws)
    bad = [
        (TypeError, lambda: cgl.quantize_mxfp4(x.double())),
        (ValueError, lambda: cgl.quantize_mxfp4(x[:, :40].contiguous())),
        (ValueError, lambda: cgl.quantize_mxfp4(x.t())),
        (ValueError, lambda: cgl.quantize_mxfp4(x, codes=torch.empty(16, 31, dtype=torch.uint8, device="cuda"))),
        (TypeError, lambda: cgl.quantize_mxfp4(x, scales=torch.empty(16, 2, device="cuda"))),
        (TypeError, lambda: cgl.dequantize_mxfp4(rx, rs, torch.float64)),
        (ValueError, lambda: cgl.dequantize_mxfp4(rx, rs[:, :1].contiguous())),
        (TypeError, lambda: cgl.dequantize_mxfp4(rx, rs.int())),
        (TypeError, lambda: cgl.dispatch_mxfp4(x.float(), lay.dst_pos, 32)),
        (ValueError, lambda: cgl.dispatch_mxfp4(x, lay.dst_pos[:8], 32)),
        (cgl.CglError, lambda: cgl.dispatch_mxfp4(x[:, :40].contiguous(), lay.dst_pos, 32)),
        (ValueError, lambda: cgl.dispatch_mxfp4(x, lay.dst_pos, 32, recv_x=torch.empty(31, 32, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: cgl.matmul_mxfp4(rx, rs, wq[:, :, :16].contiguous(), ws, lay.expert_offset)),
        (ValueError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset[:4].contiguous())),
        (TypeError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset.long())),
        (cgl.CglError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws)),                           # four experts need offsets
        (cgl.CglError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset, 9)),     # 4 * 9 rows > 32
        (cgl.CglError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset, -1)),
        (ValueError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset, y=y[:4])),
        (TypeError, lambda: cgl.matmul_mxfp4(rx, rs, wq, ws, lay.expert_offset, y=y.float())),
        (ValueError, lambda: cgl.balance_loss(logits, idx, score="top")),
        (ValueError, lambda: cgl.balance_loss(logits, idx[:3].contiguous())),
        (cgl.CglError, lambda: cgl.balance_loss(logits, idx, num_sequences=3)),
        (TypeError, lambda: cgl.balance_loss(logits.double(), idx)),
        (TypeError, lambda: cgl.balance_loss(logits, idx.long())),
        (ValueError, lambda: cgl.balance_loss(logits, idx, grad_logits=torch.empty_like(logits))),
        (ValueError, lambda: cgl.balance_loss(logits, idx, grad_loss=torch.ones((), device="cuda"))),
        (cgl.CglError, lambda: cgl.balance_loss(logits, idx, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was not refused")
