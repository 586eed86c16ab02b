"""Refusals of the product's timeout self-test, without a GPU: nothing is launched."""

import ctypes as C

import pytest

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild

P = 0x10000


@pytest.mark.parametrize("bad,code", [
    (dict(K=40), cgl.EINVAL), (dict(K=2 ** 20 + 32), cgl.EINVAL), (dict(F=0), cgl.EINVAL), (dict(F=2 ** 20 + 1), cgl.EINVAL),
    (dict(rows=0), cgl.EINVAL), (dict(rows=2 ** 20 + 1), cgl.EINVAL), (dict(wait=-1), cgl.EINVAL), (dict(a=None), cgl.EINVAL),
    (dict(sa=None), cgl.EINVAL), (dict(w=None), cgl.EINVAL), (dict(sw=None), cgl.EINVAL), (dict(y=None), cgl.EINVAL),
    (dict(st=None), cgl.EINVAL), (dict(a=P + 8), cgl.EALIGN), (dict(w=P + 4), cgl.EALIGN), (dict(y=P + 1), cgl.EALIGN),
    (dict(st=P + 2), cgl.EALIGN)])
def test_refusals(bad, code):
    cbuild.build()
    f = cgl.lib().cgl_selftest_matmul_timeout
    p, i, q = C.c_void_p, C.c_int, C.c_int64
    f.argtypes, f.restype = [p, p, q, p, p, i, i, p, q, p, p], C.c_int
    a = dict(dict(a=P, sa=P, rows=2, w=P, sw=P, F=64, K=64, y=P, wait=0, st=P), **bad)
    assert f(a["a"], a["sa"], a["rows"], a["w"], a["sw"], a["F"], a["K"], a["y"], a["wait"], a["st"], None) == code
