"""The experts' BF16 product and its gradients against 64-bit sums.

With whole numbers of at most 4 in size every partial sum is a whole number below 2^24, exact in binary32 in any order:
without an activation, or with relu, results must equal the exact ones rounded once.  Elsewhere a sum of K terms is off
by dz = K 2^-23 sum |a w| at most (and the bias's addition by 2^-23 of its result); the activations are Lipschitz below
1.13 and evaluated within 2^-18 |z|; a gate multiplies what its partner is off by; then BF16's half step, 2^-8.
"""

import math

import numpy as np
import pytest
import torch

import combine_get_layout_02_b200 as cgl
import mxref

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "silu", "swiglu"]
HALF = 2.0 ** -8


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z


def slope64(z, g, act):
    if act == "relu":
        return g * (z > 0)
    if act == "gelu":
        return g * (torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if act in ("silu", "swiglu"):
        x, u = (z, 1.0) if act == "silu" else z.chunk(2, -1)
        s = torch.sigmoid(x)
        d = g * u * s * (1 + x * (1 - s))
        return d if act == "silu" else torch.cat((d, g * x * s), -1)
    return g


class Case:
    def __init__(self, counts, k, f, seed, cap=0, act="none", whole=True, tail=3, bias=True, residual=True):
        e = len(counts)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.act, self.cap, self.k, self.f, self.e, self.whole = act, cap, k, f, e, whole
        self.cols = f // 2 if act == "swiglu" else f
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        self.rows = e * cap if cap else int(sum(counts)) + tail       # rows behind the last expert's
        self.spans = mxref.spans(self.off, cap, self.rows)
        self.covered = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for r0, r1 in self.spans:
            self.covered[r0:r1] = True
        self.a, self.g, self.residual = self.new(self.rows, k), self.new(self.rows, self.cols), self.new(self.rows, self.cols)
        for t in (self.a, self.g, self.residual):
            t[~self.covered] = torch.nan                              # rows of no expert may hold anything
        self.w = self.new(e, f, k, scale=1.0 if whole else k ** -0.5)
        self.bias = self.new(e, f) if bias else None
        if not residual:
            self.residual = None

    def new(self, *shape, scale=1.0):
        if self.whole:
            return torch.randint(-4, 5, shape, generator=self.gen, device="cuda", dtype=torch.int8).bfloat16()
        return (scale * torch.randn(shape, generator=self.gen, device="cuda")).bfloat16()

    def forward(self, wide=False, **kw):
        st = cgl.new_status()
        y = torch.full((self.rows, self.cols), -7.0, dtype=torch.bfloat16, device="cuda")
        z = torch.full((self.rows, self.f), -7.0, dtype=torch.float32 if wide else torch.bfloat16, device="cuda")
        how = dict(bias=self.bias, activation=self.act, residual=self.residual, status=st, **kw)
        got = cgl.matmul_bf16(self.a, self.w, self.off, self.cap, y=y, preact=z, **how)
        assert got[0] is y and got[1] is z
        alone = torch.full_like(y, -7.0)
        assert cgl.matmul_bf16(self.a, self.w, self.off, self.cap, y=alone, **how) is alone
        assert cgl.status_bits(st) == [] and torch.equal(alone.view(torch.int16), y.view(torch.int16))   # NaN too
        return y, z

    def check_forward(self, **kw):
        y, z = self.forward(**kw)
        assert (y[~self.covered] == -7.0).all() and (z[~self.covered] == -7.0).all()
        for i, (r0, r1) in enumerate(self.spans):
            if r1 <= r0:
                continue
            a, w = self.a[r0:r1].double(), self.w[i].double()
            ref = a @ w.T
            off = 0.0 if self.whole else self.k * 2.0 ** -23 * (a.abs() @ w.abs().T)
            if self.bias is not None:
                ref = ref + self.bias[i].double()
                off = off + 2.0 ** -23 * ref.abs()
            v = act64(ref, self.act)
            more = self.residual[r0:r1].double() if self.residual is not None else 0.0
            if self.whole:
                assert torch.equal(z[r0:r1], ref.float().to(z.dtype))
            else:
                half = HALF if z.dtype == torch.bfloat16 else 2.0 ** -24
                assert ((z[r0:r1].double() - ref).abs() <= half * ref.abs() + off).all()
            if self.whole and self.act in ("none", "relu"):
                assert torch.equal(y[r0:r1], (v + more).float().bfloat16())
                continue
            off = off + torch.zeros_like(ref)
            if self.act == "swiglu":
                (g, u), (og, ou) = ref.chunk(2, -1), off.chunk(2, -1)
                err = (u.abs() + ou) * (1.13 * og + 2.0 ** -18 * g.abs()) + (g.abs() + og) * ou
            else:
                err = 1.13 * off + 2.0 ** -18 * ref.abs()
            v = v + more
            assert ((y[r0:r1].double() - v).abs() <= HALF * v.abs() + 1.01 * err + 2.0 ** -23 * v.abs()).all()
        return y, z

    def backward(self, z, **kw):
        st = cgl.new_status()
        self.da = torch.full((self.rows, self.k), -7.0, dtype=torch.bfloat16, device="cuda")
        d = cgl.matmul_bf16_backward(self.g, self.a, self.w, self.off, self.cap, activation=self.act,
                                     preact=None if self.act == "none" else z, want_bias=True, grad_a=self.da, status=st, **kw)
        assert cgl.status_bits(st) == [] and d.grad_a is self.da
        return d

    def check_backward(self, z, **kw):
        d = self.backward(z, **kw)
        assert (d.grad_a[~self.covered] == -7.0).all()
        exact = self.whole and self.act in ("none", "relu")
        for i, (r0, r1) in enumerate(self.spans):
            a, w = self.a[r0:r1].double(), self.w[i].double()
            x, g = z[r0:r1].double(), self.g[r0:r1].double()
            dz = slope64(x, g, self.act)
            refs = dz @ w, dz.T @ a, dz.sum(0)
            got = d.grad_a[r0:r1], d.grad_w[i], d.grad_bias[i]
            if exact:
                assert all(torch.equal(p, q.float().bfloat16()) for p, q in zip(got, refs))
                continue
            # dz: its evaluation, and for the products its rounding
            if self.act == "swiglu":
                e0 = 2.0 ** -18 * torch.cat((g * x.chunk(2, -1)[1], g), -1).abs() * (1 + x.abs())
            else:
                e0 = 2.0 ** -18 * g.abs() * (1 + x.abs())
            e1 = e0 + HALF * dz.abs()
            n = r1 - r0
            sizes = (e1 @ w.abs() + self.f * 2.0 ** -23 * (dz.abs() @ w.abs()), e1.T @ a.abs() + n * 2.0 ** -23 * (dz.abs().T @ a.abs()),
                     e0.sum(0) + n * 2.0 ** -23 * dz.abs().sum(0))
            for p, q, s in zip(got, refs, sizes):
                assert ((p.double() - q).abs() <= HALF * q.abs() + 1.01 * s + 2.0 ** -133).all()
        return d


SIZES = [(8, 2), (16, 8), (64, 16), (72, 130), (160, 258), (256, 512), (520, 96), (1024, 640)]
COUNTS = [[1], [0, 5, 0], [3, 128, 1, 64], [200, 0, 33, 257, 1], [300]]


@pytest.mark.parametrize("k,f", SIZES)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("act", ["none", "relu", "swiglu"])
def test_compact(act, counts, k, f):
    c = Case(counts, k, f, k * f + len(counts), act=act)
    for wide in (False, True):
        _, z = c.check_forward(wide=wide)
        c.check_backward(z)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,k,f", [([1], 7168, 512), ([4, 0, 130, 17], 1000, 264), ([513, 65], 512, 384), ([40] * 24, 136, 64)])
def test_normal_values(act, counts, k, f):
    c = Case(counts, k, f, k, act=act, whole=False)
    for wide in (False, True):
        _, z = c.check_forward(wide=wide)
        c.check_backward(z)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("counts,k,f", [([1], 7168, 4096), ([2], 2048, 7168), ([700, 1, 0, 260], 2048, 1112), ([4, 3, 0, 9], 7168, 1024)])
def test_long_rows(act, counts, k, f):
    c = Case(counts, k, f, k + f, act=act)
    _, z = c.check_forward()
    c.check_backward(z)


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("counts,cap", [([0, 3, 9, 4], 4), ([10, 0, 50, 64, 65, 200], 64), ([1, 1], 1), ([0, 0], 5), ([130, 129, 500], 300)])
def test_padded(counts, cap, act):
    c = Case(counts, 320, 192, cap, cap=cap, act=act)
    _, z = c.check_forward()
    c.check_backward(z)


@pytest.mark.parametrize("f", [1, 7, 9, 33, 255])
def test_odd_features(f):
    for act in ("none", "relu", "swiglu"):
        c = Case([5, 0, 70], 88, 2 * f if act == "swiglu" else f, f, act=act)
        for wide in (False, True):
            _, z = c.check_forward(wide=wide)
            c.check_backward(z)


def test_without_bias_and_residual():
    for act in ("none", "relu", "swiglu"):
        c = Case([9, 33], 72, 48, 1, act=act, bias=False, residual=False)
        _, z = c.check_forward()
        c.check_backward(z)


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_one_expert_without_offsets(act):
    c = Case([77], 512, 200, 1, act=act, tail=0)
    y, z = c.check_forward()
    d = c.check_backward(z)
    kw = dict(activation=act, residual=c.residual)
    pre = None if act == "none" else z
    assert torch.equal(y, cgl.matmul_bf16(c.a, c.w, bias=c.bias, **kw))
    assert torch.equal(y, cgl.matmul_bf16(c.a, c.w[0], bias=c.bias[0], **kw))
    flat = cgl.matmul_bf16_backward(c.g, c.a, c.w[0], activation=act, preact=pre, want_bias=True)
    assert flat.grad_w.shape == (200, 512) and flat.grad_bias.shape == (200,)
    assert torch.equal(flat.grad_a, d.grad_a) and torch.equal(flat.grad_w, d.grad_w[0]) and torch.equal(flat.grad_bias, d.grad_bias[0])


def test_wanted_gradients_alone():
    c = Case([30, 0, 66], 256, 96, 2, act="silu", whole=False)
    _, z = c.forward()
    d = c.backward(z)
    for want in ("a", "w", "bias"):
        one = cgl.matmul_bf16_backward(c.g, c.a, c.w, c.off, activation="silu", preact=z, want_a=want == "a", want_w=want == "w",
                                       want_bias=want == "bias")
        for name in ("a", "w", "bias"):
            got, ref = getattr(one, "grad_" + name), getattr(d, "grad_" + name)
            assert (got is None) == (name != want)
            if got is not None:
                rows = c.covered if name == "a" else slice(None)
                assert torch.equal(got[rows], ref[rows])
    none = cgl.matmul_bf16_backward(c.g, c.a, c.w, c.off, activation="silu", preact=z, want_a=False, want_w=False)
    assert none == (None, None, None)


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_residual_in_place(act):
    c = Case([20, 0, 140], 264, 130, 2, act=act)
    y, _ = c.forward()
    r = c.residual.clone()
    got = cgl.matmul_bf16(c.a, c.w, c.off, bias=c.bias, activation=act, residual=r, y=r)
    assert got is r and torch.equal(r[c.covered], y[c.covered]) and r[~c.covered].isnan().all()


@pytest.mark.parametrize("counts,k,f,cap", [([40] * 20, 2048, 512, 0), ([150, 0, 3] * 8, 512, 768, 0), ([9] * 60, 1024, 256, 16)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_many_tiles_a_pair(counts, k, f, cap, act):
    """One pair of blocks walks every tile: rings and accumulators wrap many times."""
    c = Case(counts, k, f, k, cap=cap, act=act)
    _, z = c.check_forward(num_sms=2)
    c.check_backward(z, num_sms=2)


def test_random_sizes():
    g = np.random.Generator(np.random.PCG64(7))
    for i in range(30):
        e = int(g.integers(1, 40))
        counts = (g.integers(0, 2, e) * np.exp2(g.uniform(0, 8.5, e))).astype(int).tolist()
        act = ["none", "relu", "swiglu"][i % 3]
        k, f = 8 * int(g.integers(1, 60)), 2 * int(g.integers(1, 250))
        c = Case(counts, k, f, i, cap=int(g.integers(1, 200)) if i % 4 == 0 else 0, act=act)
        _, z = c.check_forward()
        c.check_backward(z)


@pytest.mark.parametrize("rows,f,k", [(5000, 264, 72), (20_000, 64, 16), (70_000, 24, 200)])
def test_long_sums_over_rows(rows, f, k):
    """Few weights and many rows: the sum over the rows is the long one."""
    c = Case([rows, 0, 3], k, f, rows, act="none")
    _, z = c.check_forward()
    c.check_backward(z)


def test_nan_and_infinity_stay_in_their_rows_and_experts():
    for act in ("none", "relu", "silu", "swiglu"):
        c = Case([40, 30, 25], 256, 160, 3, act=act, whole=False)
        y0, z0 = c.forward()
        d0 = c.backward(z0)
        c.a[5, 7] = torch.nan                       # a row of the first expert
        c.a[69, 1] = torch.inf                      # the last row of the second
        c.w[2, 3, 4] = torch.nan                    # a feature of the third
        y, z = c.forward()
        d = c.backward(z)
        hurt = torch.zeros_like(c.covered)
        hurt[5], hurt[69], hurt[70:95] = True, True, True
        fine = c.covered & ~hurt
        assert torch.equal(y[fine], y0[fine]) and torch.equal(z[fine], z0[fine]) and torch.equal(d.grad_a[fine], d0.grad_a[fine])
        assert y[5].isnan().all() and z[70:95, 3].isnan().all() and d.grad_w[0][:, 7].isnan().any()
        others = [i for i in range(c.cols) if i != 3]
        assert torch.equal(y[70:95][:, others], y0[70:95][:, others])
        if act == "none":                           # dz has no NaN: the weights' gradients see their own expert's rows alone
            assert torch.equal(d.grad_w[2], d0.grad_w[2]) and torch.equal(d.grad_bias, d0.grad_bias)
            keep = [i for i in range(256) if i != 7]
            assert torch.equal(d.grad_w[0][:, keep], d0.grad_w[0][:, keep])
            keep = [i for i in range(256) if i != 1]
            assert torch.equal(d.grad_w[1][:, keep], d0.grad_w[1][:, keep])


def test_activations_of_large_sums():
    """Sums far out: the activations saturate, none gives NaN."""
    x = torch.tensor([-3e38, -1e30, -1000.0, -100.0, -50.0, -9.0, -1.0, -0.0, 0.0, 1.0, 9.0, 50.0, 100.0, 1000.0, 1e18], device="cuda").bfloat16()
    n = len(x)
    a = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    a[:, 0] = x
    w = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    g = torch.ones(n, 2, dtype=torch.bfloat16, device="cuda")
    for act in ACTS[:4]:
        y, z = cgl.matmul_bf16(a, w, activation=act, with_preact=True)
        ref = act64(x.double(), act)
        assert z.dtype == torch.float32 and torch.equal(z, torch.stack((x, x), 1).float())
        assert ((y.double() - ref[:, None]).abs() <= HALF * ref.abs()[:, None] + 2.0 ** -18 * ref.abs()[:, None] + 1e-30).all()
        d = cgl.matmul_bf16_backward(g, a, w, activation=act, preact=z, want_bias=True)
        dz = slope64(x.double(), torch.ones(n, device="cuda", dtype=torch.float64), act)
        assert ((d.grad_a[:, 0].double() - 2 * dz).abs() <= 2 * HALF * (2 * dz.abs()) + 2.0 ** -17).all()
    w = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    w[0, 0], w[1, 1] = 1.0, 1.0
    a[:, 1] = 2.0
    y, z = cgl.matmul_bf16(a, w, activation="swiglu", with_preact=True)
    ref = 2 * act64(x.double(), "silu")
    assert ((y[:, 0].double() - ref).abs() <= HALF * ref.abs() + 2.0 ** -18 * ref.abs() + 1e-30).all()
    d = cgl.matmul_bf16_backward(g[:, :1].contiguous(), a, w, activation="swiglu", preact=z)
    assert not d.grad_a.isnan().any()


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu"])
def test_gradient_against_differences(act):
    """Central differences of the 64-bit forward (step 2^-8: off by 2^-16 / 6 of the third derivative, which stays below 2 for each
    of these times its factors of order 4).  Sums are small enough that z is BF16 itself, so the gradient is that at z; then dz's
    rounding (2^-8 of the sum of the terms' sizes) and the result's."""
    gen = torch.Generator().manual_seed(4)
    n, k, f = 6, 8, 4
    a = torch.randint(-1, 2, (n, k), generator=gen).bfloat16().cuda()
    w = (torch.randint(-4, 5, (f, k), generator=gen) / 8).bfloat16().cuda()
    cols = f // 2 if act == "swiglu" else f
    g = (torch.randint(-3, 4, (n, cols), generator=gen) / 2).bfloat16().cuda()
    y, z = cgl.matmul_bf16(a, w, activation=act, with_preact=True)
    assert torch.equal(z.double(), a.double() @ w.double().T)
    d = cgl.matmul_bf16_backward(g, a, w, activation=act, preact=z, want_bias=True)

    def loss(a, w, b):
        return (act64(a @ w.T + b, act) * g.double()).sum()

    args = [a.double(), w.double(), torch.zeros(f, dtype=torch.float64, device="cuda")]
    h = 2.0 ** -8
    for i, got in enumerate((d.grad_a, d.grad_w, d.grad_bias)):
        for j in range(args[i].numel()):
            side = []
            for s in (h, -h):
                moved = [t.clone() for t in args]
                moved[i].view(-1)[j] += s
                side.append(loss(*moved))
            ref = float((side[0] - side[1]) / (2 * h))
            terms = f * 4.0 if i == 0 else n * 8.0          # |dz| stays below 8, |w| at most 1 / 2, |a| at most 1
            assert abs(float(got.reshape(-1)[j]) - ref) <= HALF * (abs(ref) + terms) + 2.0 ** -16 * terms


@pytest.mark.parametrize("k", [64, 4096])       # 4096: pairs share a tile
def test_bad_offsets_are_reported_and_nothing_is_computed(k):
    c = Case([8, 8, 0], k, 32, 5, tail=0)
    for bad in ([0, 9, 4, 16], [0, 8, 17, 17], [-3, 8, 16, 16], [0, 16, 0, 16], [16, 0, 16, 0], [0, 8, 2 ** 31 - 1, 16]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        st = cgl.new_status()
        y = torch.full((18, 32), -7.0, dtype=torch.bfloat16, device="cuda")
        cgl.matmul_bf16(c.a, c.w, off, y=y[:16], status=st)
        assert cgl.status_bits(st) == ["CGL_ERANGE"] and (y == -7.0).all()
        st = cgl.new_status()
        da = torch.full((18, k), -7.0, dtype=torch.bfloat16, device="cuda")
        dw, db = torch.full_like(c.w, -7.0), torch.full_like(c.bias, -7.0)
        cgl.matmul_bf16_backward(c.g, c.a, c.w, off, want_bias=True, grad_a=da[:16], grad_w=dw, grad_bias=db, status=st)
        assert cgl.status_bits(st) == ["CGL_ERANGE"] and (da == -7.0).all() and (dw == -7.0).all() and (db == -7.0).all()


def test_more_copies_than_a_padded_expert_has_rows():
    c = Case([0, 0, 0], 64, 32, 5, cap=5)
    c.a[:], c.bias = 1.0, None
    y = torch.full((15, 32), -7.0, dtype=torch.bfloat16, device="cuda")
    st = cgl.new_status()
    cgl.matmul_bf16(c.a, c.w, torch.tensor([0, 900, 900, 2000], dtype=torch.int32, device="cuda"), 5, y=y, status=st)
    assert cgl.status_bits(st) == [] and (y[5:10] == -7.0).all()
    assert torch.equal(y[:5], (c.a[:5].double() @ c.w[0].double().T).bfloat16())


def test_same_answer_every_time_and_on_one_sm():
    c = Case([33, 200, 7, 0, 90], 1056, 300, 6, act="swiglu", whole=False)
    y, z = c.forward()
    d = c.backward(z)
    for _ in range(3):
        y2, z2 = c.forward()
        d2 = c.backward(z)
        assert torch.equal(y2, y) and torch.equal(z2, z) and torch.equal(d2.grad_a, d.grad_a)
        assert torch.equal(d2.grad_w, d.grad_w) and torch.equal(d2.grad_bias, d.grad_bias)
    c.check_forward(num_sms=1)
    c.check_backward(z, num_sms=1)


def test_empty():
    c = Case([0, 0], 64, 32, 8, tail=0)
    y, z = c.forward()
    assert y.shape == (0, 32)
    d = c.backward(z)
    assert (d.grad_w == 0).all() and (d.grad_bias == 0).all()
    c = Case([0, 0], 64, 32, 8, tail=4)
    y, z = c.forward()
    d = c.backward(z)
    assert (y == -7.0).all() and (d.grad_a == -7.0).all() and (d.grad_w == 0).all() and (d.grad_bias == 0).all()


def test_unaligned_rows():
    """bias, residual, y, preact and grad_y at any 2-byte address."""
    for act, f in (("none", 40), ("swiglu", 80), ("gelu", 44)):
        c = Case([9, 0, 130], 136, f, 3, act=act, whole=False)
        y, z = c.forward()
        d = c.backward(z)
        _, z32 = c.forward(wide=True)
        d32 = c.backward(z32)

        def moved(t, shift=1):
            m = torch.full((t.numel() + shift + 8,), -7.0, dtype=t.dtype, device="cuda")
            v = m[shift:shift + t.numel()].view(t.shape)
            v.copy_(t)
            return v

        my, mz = moved(torch.full_like(y, -7.0)), moved(torch.full_like(z, -7.0))
        cgl.matmul_bf16(c.a, c.w, c.off, bias=moved(c.bias), activation=act, residual=moved(c.residual), y=my, preact=mz)
        assert torch.equal(my, y) and torch.equal(mz, z)
        pre = None if act == "none" else moved(z)
        d2 = cgl.matmul_bf16_backward(moved(c.g), c.a, c.w, c.off, activation=act, preact=pre, want_bias=True,
                                      grad_bias=moved(torch.zeros_like(c.bias)))
        rows = c.covered
        assert torch.equal(d2.grad_a[rows], d.grad_a[rows]) and torch.equal(d2.grad_w, d.grad_w) and torch.equal(d2.grad_bias, d.grad_bias)
        mz = moved(torch.full_like(z32, -7.0))
        cgl.matmul_bf16(c.a, c.w, c.off, bias=c.bias, activation=act, residual=c.residual, preact=mz)
        d2 = cgl.matmul_bf16_backward(c.g, c.a, c.w, c.off, activation=act, preact=None if act == "none" else mz, want_bias=True)
        assert torch.equal(mz, z32) and torch.equal(d2.grad_a[rows], d32.grad_a[rows]) and torch.equal(d2.grad_w, d32.grad_w)


def test_refusals():
    c = Case([9, 7], 64, 32, 3, tail=0)
    a, w, off, g = c.a, c.w, c.off, c.g
    bad = [
        (TypeError, lambda: cgl.matmul_bf16(a.float(), w, off)), (TypeError, lambda: cgl.matmul_bf16(a, w.half(), off)),
        (TypeError, lambda: cgl.matmul_bf16(a, w, off.long())), (ValueError, lambda: cgl.matmul_bf16(a, w[0], off)),
        (ValueError, lambda: cgl.matmul_bf16(a[:, :60].contiguous(), w[:, :, :60].contiguous(), off)),
        (ValueError, lambda: cgl.matmul_bf16(a[:, :56].contiguous(), w, off)), (ValueError, lambda: cgl.matmul_bf16(a, w, off[:2].contiguous())),
        (ValueError, lambda: cgl.matmul_bf16(a, w.transpose(1, 2), off)), (cgl.CglError, lambda: cgl.matmul_bf16(a, w)),
        (cgl.CglError, lambda: cgl.matmul_bf16(a, w, off, 9)), (cgl.CglError, lambda: cgl.matmul_bf16(a, w, off, -1)),
        (ValueError, lambda: cgl.matmul_bf16(a, w, off, activation="tanh")),
        (ValueError, lambda: cgl.matmul_bf16(a, w[:, :31].contiguous(), off, activation="swiglu")),
        (ValueError, lambda: cgl.matmul_bf16(a, w, off, bias=c.bias[0])), (TypeError, lambda: cgl.matmul_bf16(a, w, off, bias=c.bias.float())),
        (ValueError, lambda: cgl.matmul_bf16(a, w, off, activation="swiglu", residual=c.residual)),
        (ValueError, lambda: cgl.matmul_bf16(a, w, off, y=c.residual[:4])), (TypeError, lambda: cgl.matmul_bf16(a, w, off, preact=c.residual.half())),
        (ValueError, lambda: cgl.matmul_bf16_backward(g[:4], a, w, off)), (TypeError, lambda: cgl.matmul_bf16_backward(g.float(), a, w, off)),
        (ValueError, lambda: cgl.matmul_bf16_backward(g, a, w, off, activation="silu")),
        (ValueError, lambda: cgl.matmul_bf16_backward(g, a, w, off, activation="silu", preact=g[:3])),
        (ValueError, lambda: cgl.matmul_bf16_backward(g, a, w, off, grad_bias=c.bias)),
        (ValueError, lambda: cgl.matmul_bf16_backward(g, a, w, off, grad_w=w[:1])),
        (cgl.CglError, lambda: cgl.matmul_bf16_backward(g, a, w, off, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (cgl.CglError, lambda: cgl.matmul_bf16(a, w, off, num_sms=-1)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was not refused")
