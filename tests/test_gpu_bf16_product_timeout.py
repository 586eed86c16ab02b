"""Failure detection in the BF16 product without a fault: waits with a limit shorter than the work run out while copies
and MMAs are under way.  The call sets CGL_ETIMEOUT, returns soon, and the next calls are right."""

import ctypes as C
import time

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


def _selftest(what, x, other, out, f, k, wait, status):
    fn = cgl.lib().cgl_selftest_matmul_bf16_timeout
    p, i, q = C.c_void_p, C.c_int, C.c_int64
    fn.argtypes, fn.restype = [i, p, q, p, i, i, p, q, p, p], C.c_int
    return fn(what, x.data_ptr(), x.shape[0], other.data_ptr(), f, k, out.data_ptr(), wait, status.data_ptr(),
              torch.cuda.current_stream().cuda_stream)


def _whole(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()


def _case(what, rows, f, k):
    """Operands, the result's buffer with rows behind it, and the exact result (whole numbers)."""
    a, w, g = _whole(rows, k, seed=1), _whole(f, k, seed=2), _whole(rows, f, seed=3)
    x, other, shape = ((a, w, (rows, f)), (g, w, (rows, k)), (a, g, (f, k)))[what]
    out = torch.full((shape[0] + 8, shape[1]), -7.0, dtype=torch.bfloat16, device="cuda")
    return x, other, out, (lambda: (a.float() @ w.float().T, g.float() @ w.float(), g.float().T @ a.float())[what].bfloat16())


@pytest.mark.parametrize("what", [0, 1, 2])
def test_the_usual_limit_gives_the_usual_result(what):
    x, other, out, want = _case(what, 70, 200, 520)
    st = cgl.new_status()
    assert _selftest(what, x, other, out, 200, 520, 2 ** 31, st) == cgl.OK
    assert cgl.status_bits(st) == [] and torch.equal(out[:-8], want()) and (out[-8:] == -7.0).all()


# few tiles over several pairs; tiles enough for many pairs; long sums (the waits for a whole tile are the longest)
@pytest.mark.parametrize("what", [0, 1, 2])
@pytest.mark.parametrize("rows,f,k", [(1, 256, 2 ** 17), (300, 2560, 2 ** 14), (70_001, 264, 520)])
@pytest.mark.parametrize("wait", [1000, 0])
def test_waits_that_run_out(what, rows, f, k, wait):
    x, other, out, _ = _case(what, rows, f, k)
    st = cgl.new_status()
    torch.cuda.synchronize()
    t = time.perf_counter()
    assert _selftest(what, x, other, out, f, k, wait, st) == cgl.OK
    torch.cuda.synchronize()
    assert time.perf_counter() - t < 2.0
    assert cgl.status_bits(st) in (["CGL_ETIMEOUT"], [])       # a short sum may be done in time
    if wait == 0 and (what, rows) != (2, 1):
        assert cgl.status_bits(st) == ["CGL_ETIMEOUT"]
    assert (out[-8:] == -7.0).all()          # the result is undefined, what lies behind it is not
    x, other, out, want = _case(what, 300, 640, 2048)
    st = cgl.new_status()
    assert _selftest(what, x, other, out, 640, 2048, 2 ** 31, st) == cgl.OK
    assert cgl.status_bits(st) == [] and torch.equal(out[:-8], want())
