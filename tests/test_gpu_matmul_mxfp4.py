"""The experts' MXFP4 product against 64-bit sums.

Where every product is a multiple of 2^-q and every partial sum stays below 2^(24 - q), binary32 sums are exact in
any order and y must equal the exact sum rounded once.  Elsewhere |y - exact| <= 2^-8 |exact| (BF16's half step) +
K 2^-23 sum |a w| (K additions, each off by at most one binary32 step of a partial sum, which sum |a w| bounds).
"""

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
import mxref

pytestmark = pytest.mark.gpu


def _case(counts, k, f, seed, cap=0, lo=125, hi=128):
    e = len(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    rows = e * cap if cap else int(sum(counts))
    a, sa = mxref.codes_like(rows, k, g, "cuda", lo, hi)
    w, sw = mxref.codes_like(e * f, k, g, "cuda", lo, hi)
    return a, sa, w.view(e, f, -1), sw.view(e, f, -1), off, cap


def _check(a, sa, w, sw, off, cap, exact=True, tail=3):
    rows, (e, f, kb) = a.shape[0], w.shape
    where = mxref.spans(off, cap, rows) if off is not None else [(0, rows)]
    # rows behind the last expert's stay as they were
    a = torch.cat([a, a.new_full((tail, kb), 0x77)]) if not cap and off is not None else a
    sa = torch.cat([sa, sa.new_full((tail, sa.shape[1]), 255)]) if not cap and off is not None else sa
    y = torch.full((a.shape[0], f), -7.0, dtype=torch.bfloat16, device="cuda")
    st = cgl.new_status()
    got = cgl.matmul_mxfp4(a, sa, w, sw, off, cap, y=y, status=st)
    assert got is y and cgl.status_bits(st) == []
    ref, s = mxref.product(a, sa, w, sw, where)
    covered = torch.zeros(a.shape[0], dtype=torch.bool, device="cuda")
    for r0, r1 in where:
        covered[r0:r1] = True
    assert (y[~covered] == -7.0).all()
    y, ref, s = y[covered], ref[covered], s[covered]
    if exact:
        assert torch.equal(y, ref.float().bfloat16())
    else:
        tol = 2.0 ** -8 * ref.abs() + 2 * kb * 2.0 ** -23 * s
        assert ((y.double() - ref).abs() <= tol).all()


# scales 2^-2 .. 2^1 on both sides: products are multiples of 2^-6 and at most 36 * 4, so sums of K <= 1024 terms
# stay below 2^18 = 2^(24 - 6); larger K take scales of 1 only (multiples of 2^-2 below 36 * 7168 < 2^22)
@pytest.mark.parametrize("k,f", [(32, 1), (32, 8), (64, 130), (96, 128), (160, 257), (256, 512), (288, 96), (1024, 640)])
@pytest.mark.parametrize("counts", [[1], [0, 5, 0], [3, 128, 1, 64], [200, 0, 33, 129, 1], [300]])
def test_compact(counts, k, f):
    _check(*_case(counts, k, f, k * f + len(counts)))


@pytest.mark.parametrize("counts,k,f", [([1], 7168, 4096), ([4, 0, 130, 17], 7168, 264), ([513], 4096, 384),
                                        ([700, 1, 0, 260], 2048, 1111), ([2], 2080, 7168), ([40] * 64, 512, 256)])
def test_long_rows(counts, k, f):
    _check(*_case(counts, k, f, k, lo=127, hi=127))


@pytest.mark.parametrize("counts,cap", [([0, 3, 9, 4], 4), ([10, 0, 50, 64, 65, 200], 64), ([1, 1], 1), ([0, 0], 5),
                                        ([130, 129, 500], 300)])
def test_padded(counts, cap):
    _check(*_case(counts, 320, 192, cap, cap=cap))


@pytest.mark.parametrize("k", [1056, 1088, 1120, 1152, 1184, 7200])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_scale_rows_of_every_alignment(k, shift):
    """Rows of k / 32 scale bytes start at any byte; the arrays lie between NaN scales, which must not be read into them."""
    a, sa, w, sw, off, _ = _case([3, 0, 70], k, 130, k + shift, lo=127, hi=127)

    def place(s):
        buf = torch.full((s.numel() + 16,), 255, dtype=torch.uint8, device="cuda")
        t = buf[4 + shift:4 + shift + s.numel()].view(s.shape)
        t.copy_(s)
        return t

    _check(a, place(sa), w, place(sw), off, 0, tail=0)


def test_one_expert_without_offsets():
    a, sa, w, sw, _, _ = _case([77], 512, 200, 1)
    _check(a, sa, w, sw, None, 0)
    y = cgl.matmul_mxfp4(a, sa, w[0], sw[0])
    assert torch.equal(y, cgl.matmul_mxfp4(a, sa, w, sw))


@pytest.mark.parametrize("k", [96, 512, 7168])
def test_scales_over_a_wide_range(k):
    _check(*_case([100, 3, 64], k, 200, k, lo=90, hi=164), exact=False)


@pytest.mark.parametrize("counts,k,f,cap", [([40] * 20, 7168, 512, 0), ([150, 0, 3] * 8, 2048, 768, 0), ([9] * 60, 4096, 256, 16)])
def test_many_tiles_a_pair(counts, k, f, cap):
    """One pair of blocks walks every tile: rings and accumulators wrap many times."""
    a, sa, w, sw, off, cap = _case(counts, k, f, k, cap=cap, lo=127, hi=127)
    st = cgl.new_status()
    y = torch.full((a.shape[0], f), -7.0, dtype=torch.bfloat16, device="cuda")
    cgl.matmul_mxfp4(a, sa, w, sw, off, cap, y=y, status=st, num_sms=2)
    assert cgl.status_bits(st) == []
    ref, _ = mxref.product(a, sa, w, sw, mxref.spans(off, cap, a.shape[0]))
    assert torch.equal(y, torch.where(ref.isnan(), -7.0, ref).float().bfloat16())


def test_random_sizes():
    g = np.random.Generator(np.random.PCG64(7))
    for i in range(25):
        e = int(g.integers(1, 40))
        counts = (g.integers(0, 2, e) * np.exp2(g.uniform(0, 8.5, e))).astype(int).tolist()
        k, f = 32 * int(g.integers(1, 30)), int(g.integers(1, 500))
        cap = int(g.integers(1, 200)) if i % 3 == 0 else 0
        _check(*_case(counts, k, f, i, cap=cap, lo=126, hi=128))


def test_nan_scales_stay_in_their_rows_and_columns():
    a, sa, w, sw, off, _ = _case([40, 30], 256, 160, 3)
    sa[5, 2] = 255
    sw[1, 17, 0] = 255
    a[5, 32:48] = 0x22                  # finite codes under the NaN scale
    y = cgl.matmul_mxfp4(a, sa, w, sw, off)
    ref, _ = mxref.product(a, sa, w, sw, mxref.spans(off, 0, 70))
    assert torch.equal(y.isnan(), ref.isnan())
    assert y[5].isnan().all() and y[40:, 17].isnan().all() and y.isnan().sum() == 160 + 30
    ok = ~ref.isnan()
    assert torch.equal(y[ok], ref[ok].float().bfloat16())


def test_extreme_scales():
    """The smallest and largest scales: products below binary32's range vanish, above it become infinite."""
    a, sa, w, sw, off, _ = _case([16], 64, 128, 4)
    sa[:8], sa[8:] = 0, 254
    sw[0, :64], sw[0, 64:] = 0, 254
    a[:], w[:] = 0x22, 0x22             # every value 1.0
    y = cgl.matmul_mxfp4(a, sa, w, sw, off)
    assert (y[:8, :64] == 0).all()                 # 64 * 2^-254
    assert (y[:8, 64:] == 64.0).all()              # 64 * 2^(127 - 127)
    assert (y[8:, :64] == 64.0).all()
    assert torch.isinf(y[8:, 64:]).all()           # 64 * 2^254


@pytest.mark.parametrize("k", [64, 4096])       # 4096: pairs share a tile
def test_bad_offsets_are_reported_and_nothing_is_computed(k):
    a, sa, w, sw, off, _ = _case([8, 8, 0], k, 32, 5)
    for bad in ([0, 9, 4, 16], [0, 8, 17, 17], [-3, 8, 16, 16], [0, 16, 0, 16], [16, 0, 16, 0], [0, 8, 2 ** 31 - 1, 16]):
        st = cgl.new_status()
        y = torch.full((18, 32), -7.0, dtype=torch.bfloat16, device="cuda")
        cgl.matmul_mxfp4(a, sa, w, sw, torch.tensor(bad, dtype=torch.int32, device="cuda"), y=y[:16], status=st)
        assert cgl.status_bits(st) == ["CGL_ERANGE"]
        assert (y == -7.0).all()
    # padded rows: only offsets that run backwards are wrong, more copies than rows are the layout's overflow
    st = cgl.new_status()
    y = torch.full((15, 32), -7.0, dtype=torch.bfloat16, device="cuda")
    for offs, bits in (([0, 9, 4, 16], ["CGL_ERANGE"]), ([0, 900, 900, 2000], [])):
        st = cgl.new_status()
        cgl.matmul_mxfp4(a[:15], sa[:15], w, sw, torch.tensor(offs, dtype=torch.int32, device="cuda"), 5, y=y, status=st)
        assert cgl.status_bits(st) == bits
        assert ((y == -7.0).all() if bits else (y[5:10] == -7.0).all() and (y[:5] != -7.0).any())


def test_same_answer_every_time_and_on_one_sm():
    a, sa, w, sw, off, _ = _case([33, 200, 7, 0, 90], 1056, 300, 6, lo=100, hi=150)
    y = cgl.matmul_mxfp4(a, sa, w, sw, off)
    for _ in range(3):
        assert torch.equal(y, cgl.matmul_mxfp4(a, sa, w, sw, off))
    _check(a, sa, w, sw, off, 0, exact=False)
    one = cgl.matmul_mxfp4(a, sa, w, sw, off, num_sms=1)
    ref, s = mxref.product(a, sa, w, sw, mxref.spans(off, 0, 330))
    assert ((one.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1056 * 2.0 ** -23 * s).all()


def test_empty():
    a, sa, w, sw, off, _ = _case([0, 0], 64, 32, 8)
    assert cgl.matmul_mxfp4(a, sa, w, sw, off).shape == (0, 32)
    a, sa, w, sw, _, _ = _case([4], 64, 32, 8)
    y = torch.full((4, 32), -7.0, dtype=torch.bfloat16, device="cuda")
    cgl.matmul_mxfp4(a, sa, w, sw, torch.zeros(2, dtype=torch.int32, device="cuda"), y=y)
    assert (y == -7.0).all()
