"""Failure detection in the experts' product without a fault: waits with a limit shorter than the work run out while copies
and MMAs are under way.  The call sets CGL_ETIMEOUT, returns soon, and the next calls are right."""

import ctypes as C
import time

import pytest
import torch

import combine_get_layout_02_b200 as cgl
import mxref

pytestmark = pytest.mark.gpu


def _selftest(a, sa, w, sw, y, wait, status):
    f = cgl.lib().cgl_selftest_matmul_timeout
    p, i, q = C.c_void_p, C.c_int, C.c_int64
    f.argtypes, f.restype = [p, p, q, p, p, i, i, p, q, p, p], C.c_int
    return f(a.data_ptr(), sa.data_ptr(), a.shape[0], w.data_ptr(), sw.data_ptr(), w.shape[0], 2 * a.shape[1], y.data_ptr(), wait,
             status.data_ptr(), torch.cuda.current_stream().cuda_stream)


def _case(rows, f, k):
    g = torch.Generator(device="cuda").manual_seed(rows + f)
    return *mxref.codes_like(rows, k, g, "cuda", 127, 127), *mxref.codes_like(f, k, g, "cuda", 127, 127)


def _next_call_is_right():
    a, sa, w, sw = _case(300, 640, 2048)
    st = cgl.new_status()
    y = cgl.matmul_mxfp4(a, sa, w, sw, status=st)
    ref, _ = mxref.product(a, sa, w[None], sw[None], [(0, 300)])
    assert cgl.status_bits(st) == [] and torch.equal(y, ref.float().bfloat16())


def test_the_usual_limit_gives_the_usual_result():
    a, sa, w, sw = _case(70, 200, 512)
    st = cgl.new_status()
    y = torch.empty(70, 200, dtype=torch.bfloat16, device="cuda")
    assert _selftest(a, sa, w, sw, y, 2 ** 31, st) == cgl.OK
    assert cgl.status_bits(st) == [] and torch.equal(y, cgl.matmul_mxfp4(a, sa, w, sw))


# one tile over 4 pairs; tiles enough for many pairs; K as long as it may be (the waits for a whole tile are the longest)
@pytest.mark.parametrize("rows,f,k", [(1, 128, 2 ** 20), (200, 256, 2 ** 20), (300, 2560, 2 ** 16)])
@pytest.mark.parametrize("wait", [1000, 0])
def test_waits_that_run_out(rows, f, k, wait):
    a, sa, w, sw = _case(rows, f, k)
    st = cgl.new_status()
    y = torch.full((rows + 8, f), -7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    assert _selftest(a, sa, w, sw, y, wait, st) == cgl.OK
    torch.cuda.synchronize()
    assert time.perf_counter() - t < 2.0
    assert cgl.status_bits(st) == ["CGL_ETIMEOUT"]
    assert (y[rows:] == -7.0).all()          # y itself is undefined, what lies behind it is not
    _next_call_is_right()
