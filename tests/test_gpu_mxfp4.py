"""MXFP4 rows on the GPU: quantise, dequantise and dispatch, bit for bit against a 64-bit search."""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
import mxref

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _rows(rows, c, dtype, seed):
    """Rows over the type's whole range of magnitudes, with zeros, exact borders and ties."""
    g = np.random.Generator(np.random.PCG64(seed))
    span = 12 if dtype == torch.float16 else 120
    x = g.standard_normal((rows, c)) * np.exp2(g.integers(-span, span, (rows, 1)))
    x[g.random((rows, c)) < 0.05] = 0
    if rows > 2:
        x[0] = 0
        x[1] = np.resize(np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5, -0.0, 5.0001, 1e-3]), c)   # ties at scale 1
        x[2] = np.resize(np.array([1.5, 1.5, -1.5, .75]), c)                                                  # amax on the border
    return torch.tensor(x).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c", [(1, 32), (3, 64), (5, 96), (33, 7168), (129, 224), (1000, 2080)])
def test_quantize_and_back(rows, c, dtype):
    x = _rows(rows, c, dtype, rows * c)
    ref_c, ref_s = mxref.quantize(x.double().numpy())
    codes, scales = cgl.quantize_mxfp4(x.cuda())
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    assert np.array_equal(codes.cpu().numpy(), ref_c)
    for out in TYPES:
        back = cgl.dequantize_mxfp4(codes, scales, dtype=out)
        want = torch.tensor(mxref.values(ref_c, ref_s)).to(torch.float32).to(out)
        assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_extremes(dtype):
    """Infinities and NaN spoil their own block only; the largest and smallest values of the type."""
    x = torch.ones(8, 64, dtype=dtype)
    x[0, 3], x[1, 40], x[2, 0] = torch.inf, -torch.inf, torch.nan
    x[3] = torch.finfo(dtype).max
    x[4] = -torch.finfo(dtype).tiny
    x[5] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps      # the smallest subnormal
    x[6, :32] = 0
    x[7] = torch.linspace(-1, 1, 64).to(dtype)
    ref_c, ref_s = mxref.quantize(x.double().numpy())
    codes, scales = cgl.quantize_mxfp4(x.cuda())
    assert np.array_equal(scales.cpu().numpy(), ref_s) and np.array_equal(codes.cpu().numpy(), ref_c)
    assert (ref_s == 255).sum() == 3
    back = cgl.dequantize_mxfp4(codes, scales, dtype=torch.float32).cpu()
    want = torch.tensor(mxref.values(ref_c, ref_s)).float()
    assert torch.equal(back.isnan(), want.isnan()) and torch.equal(back.nan_to_num(), want.nan_to_num())


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :256].contiguous()     # 512 values a row
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 16).contiguous()
    want = torch.tensor(mxref.values(codes.numpy(), scales.numpy()))
    for out in TYPES:
        got = cgl.dequantize_mxfp4(codes.cuda(), scales.cuda(), dtype=out).cpu()
        ref = want.float().to(out)        # binary32 holds every value below 2^128; past it, an infinity
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.nan_to_num(nan=0.0), ref.nan_to_num(nan=0.0))


def test_quantize_three_dims_and_given_outputs():
    x = torch.randn(3, 5, 160, device="cuda").bfloat16()
    codes = torch.empty(3, 5, 80, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 5, 5, dtype=torch.uint8, device="cuda")
    got = cgl.quantize_mxfp4(x, codes=codes, scales=scales, num_sms=1)
    assert got[0] is codes and got[1] is scales
    flat = cgl.quantize_mxfp4(x.view(15, 160))
    assert torch.equal(flat[0], codes.view(15, 80)) and torch.equal(flat[1], scales.view(15, 5))
    assert cgl.quantize_mxfp4(x[:0])[0].shape == (0, 5, 80)


def _place(n, k, rows, seed, skip=0.2):
    """A random injective placement of some (token, slot) copies into receive rows."""
    g = np.random.Generator(np.random.PCG64(seed))
    dst = g.permutation(rows)[: n * k].astype(np.int32).reshape(n, k)
    dst[g.random((n, k)) < skip] = -1
    return dst


@pytest.mark.parametrize("scratch", [False, True])
@pytest.mark.parametrize("n,h,k,extra", [(1, 32, 1, 0), (3, 64, 2, 5), (128, 256, 4, 0), (300, 7168, 8, 17),
                                         (1200, 2080, 3, 1), (513, 512, 32, 4), (40, 16416, 2, 0), (2500, 4096, 2, 9)])
def test_dispatch(n, h, k, extra, scratch):
    x = _rows(n, h, torch.bfloat16, n + h)
    dst = _place(n, k, n * k + extra, h)
    rows = n * k + extra
    rx = torch.full((rows, h // 2), 0xA5, dtype=torch.uint8, device="cuda")
    rs = torch.full((rows, h // 32), 0x5A, dtype=torch.uint8, device="cuda")
    st, sc = cgl.new_status(), cgl.new_scratch() if scratch else None
    cgl.dispatch_mxfp4(x.cuda(), torch.tensor(dst).cuda(), rows, recv_x=rx, recv_scale=rs, status=st, scratch=sc)
    assert cgl.status_bits(st) == []
    if scratch:
        assert torch.count_nonzero(sc).item() == 0
    codes, scales = cgl.quantize_mxfp4(x.cuda())       # checked against the search above
    want_x = torch.full_like(rx, 0xA5)
    want_s = torch.full_like(rs, 0x5A)
    tok, slot = np.nonzero(dst >= 0)
    at = torch.tensor(dst[tok, slot].astype(np.int64)).cuda()
    want_x[at], want_s[at] = codes[torch.tensor(tok).cuda()], scales[torch.tensor(tok).cuda()]
    assert torch.equal(rx, want_x) and torch.equal(rs, want_s)


def test_dispatch_reports_rows_past_the_buffer():
    x = torch.randn(4, 64, device="cuda").bfloat16()
    dst = torch.tensor([[0, 9], [1, -1], [2, 3], [4, -5]], dtype=torch.int32, device="cuda")
    st = cgl.new_status()
    rx = torch.zeros(5, 32, dtype=torch.uint8, device="cuda")
    rs = torch.zeros(5, 2, dtype=torch.uint8, device="cuda")
    cgl.dispatch_mxfp4(x, dst, 5, recv_x=rx, recv_scale=rs, status=st)
    assert cgl.status_bits(st) == ["CGL_ERANGE"]
    codes, scales = cgl.quantize_mxfp4(x)
    assert torch.equal(rx, codes[[0, 1, 2, 2, 3]]) and torch.equal(rs, scales[[0, 1, 2, 2, 3]])


def test_dispatch_empty_batches():
    dst = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    rx, rs = cgl.dispatch_mxfp4(torch.zeros(0, 64, device="cuda").bfloat16(), dst, 3)
    assert rx.shape == (3, 32) and rs.shape == (3, 2)
    x = torch.zeros(2, 64, device="cuda").bfloat16()
    rx, rs = cgl.dispatch_mxfp4(x, torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), 0)
    assert rx.shape == (0, 32)
