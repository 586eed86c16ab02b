"""Refusals of the MXFP4 calls and the balance loss, on a machine without a GPU: nothing is launched."""

import ctypes as C

import pytest
import torch

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild

P = 0x10000   # 64 KiB-aligned, never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def L():
    cbuild.build()
    return cgl.lib()


def _opts(cap=0, sms=0, flags=0):
    return C.byref(cgl.Opts(sms, cap, flags, None))


@pytest.mark.parametrize("bad,code", [
    (dict(cols=33), cgl.EINVAL), (dict(cols=0), cgl.EINVAL), (dict(cols=-32), cgl.EINVAL), (dict(rows=-1), cgl.EINVAL),
    (dict(rows=2 ** 33), cgl.EINVAL), (dict(rows=2 ** 30, cols=2 ** 20), cgl.EINVAL), (dict(dtype=3), cgl.EINVAL), (dict(dtype=-1), cgl.EINVAL),
    (dict(x=None), cgl.EINVAL), (dict(codes=None), cgl.EINVAL), (dict(scales=None), cgl.EINVAL),
    (dict(opts=_opts(sms=-1)), cgl.EINVAL), (dict(opts=_opts(flags=2)), cgl.EINVAL),
    (dict(x=P + 8), cgl.EALIGN), (dict(codes=P + 4), cgl.EALIGN)])
def test_quantize_and_dequantize(L, bad, code):
    a = dict(dict(x=P, dtype=0, rows=4, cols=64, codes=P, scales=P, opts=None), **bad)
    assert L.cgl_quantize_mxfp4(a["x"], a["dtype"], a["rows"], a["cols"], a["codes"], a["scales"], a["opts"], None) == code
    assert L.cgl_dequantize_mxfp4(a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["dtype"], a["opts"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(h=48), cgl.EINVAL), (dict(h=0), cgl.EINVAL), (dict(k=0), cgl.EINVAL), (dict(k=33), cgl.EINVAL), (dict(n=-1), cgl.EINVAL),
    (dict(n=2 ** 30, k=4), cgl.EINVAL), (dict(rows=-1), cgl.EINVAL), (dict(x=None), cgl.EINVAL), (dict(dst=None), cgl.EINVAL),
    (dict(rx=None), cgl.EINVAL), (dict(rs=None), cgl.EINVAL), (dict(opts=_opts(sms=-2)), cgl.EINVAL),
    (dict(x=P + 2), cgl.EALIGN), (dict(rx=P + 8), cgl.EALIGN), (dict(dst=P + 2), cgl.EALIGN), (dict(st=P + 1), cgl.EALIGN)])
def test_dispatch(L, bad, code):
    a = dict(dict(x=P, n=4, h=64, k=2, dst=P, rx=P, rs=P, rows=8, opts=None, st=P), **bad)
    assert L.cgl_dispatch_mxfp4(a["x"], a["n"], a["h"], a["k"], a["dst"], a["rx"], a["rs"], a["rows"], a["opts"], a["st"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(K=40), cgl.EINVAL), (dict(K=0), cgl.EINVAL), (dict(F=0), cgl.EINVAL), (dict(E=0), cgl.EINVAL), (dict(E=1025), cgl.EINVAL),
    (dict(F=2 ** 20 + 1), cgl.EINVAL), (dict(K=2 ** 20 + 32), cgl.EINVAL), (dict(rows=-1), cgl.EINVAL), (dict(rows=2 ** 31), cgl.EINVAL),
    (dict(off=None), cgl.EINVAL), (dict(off=None, E=1, opts=_opts(cap=4)), cgl.EINVAL), (dict(opts=_opts(cap=5)), cgl.EINVAL),
    (dict(opts=_opts(cap=-1)), cgl.EINVAL), (dict(opts=_opts(sms=-1)), cgl.EINVAL), (dict(w=None), cgl.EINVAL), (dict(sw=None), cgl.EINVAL),
    (dict(a=None), cgl.EINVAL), (dict(sa=None), cgl.EINVAL), (dict(y=None), cgl.EINVAL),
    (dict(a=P + 8), cgl.EALIGN), (dict(w=P + 4), cgl.EALIGN), (dict(y=P + 1), cgl.EALIGN), (dict(off=P + 2), cgl.EALIGN), (dict(st=P + 2), cgl.EALIGN)])
def test_matmul(L, bad, code):
    a = dict(dict(a=P, sa=P, rows=16, w=P, sw=P, E=4, F=32, K=64, off=P, y=P, opts=None, st=P), **bad)
    assert L.cgl_matmul_mxfp4(a["a"], a["sa"], a["rows"], a["w"], a["sw"], a["E"], a["F"], a["K"], a["off"], a["y"], a["opts"], a["st"],
                              None) == code


def test_balance_workspace(L):
    assert L.cgl_balance_loss_workspace_bytes(4096, 8, 256, 1) > 0
    assert L.cgl_balance_loss_workspace_bytes(0, 8, 256, 4) > 0
    for bad in ((-1, 8, 256, 1), (10, 0, 256, 1), (10, 33, 256, 1), (10, 8, 0, 1), (10, 8, 1025, 1), (10, 8, 256, 0), (10, 8, 256, 3),
                (2 ** 28, 8, 256, 1), (0, 8, 256, 2 ** 24 + 1)):
        assert L.cgl_balance_loss_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(n=-2), cgl.EINVAL), (dict(k=0), cgl.EINVAL), (dict(E=1025), cgl.EINVAL), (dict(S=3), cgl.EINVAL), (dict(S=0), cgl.EINVAL),
    (dict(dtype=7), cgl.EINVAL), (dict(score=2), cgl.EINVAL), (dict(logits=None), cgl.EINVAL), (dict(idx=None), cgl.EINVAL),
    (dict(counts=None), cgl.EINVAL), (dict(routed=None), cgl.EINVAL), (dict(logits=P + 2), cgl.EALIGN), (dict(grad=P + 2), cgl.EALIGN),
    (dict(dtype=0, logits=P + 1), cgl.EALIGN), (dict(idx=P + 1), cgl.EALIGN), (dict(gl=P + 2), cgl.EALIGN), (dict(counts=P + 2), cgl.EALIGN)])
def test_balance(L, bad, code):
    a = dict(dict(logits=P, dtype=2, idx=P, n=8, k=2, E=16, S=2, score=0, gl=P, loss=P, counts=P, routed=P, grad=P, ws=P, wsb=1 << 20, st=P), **bad)

    def forward(a):
        return L.cgl_balance_loss(a["logits"], a["dtype"], a["idx"], a["n"], a["k"], a["E"], a["S"], 1.0, a["score"], a["gl"], a["loss"],
                                  a["counts"], a["routed"], a["grad"], a["ws"], a["wsb"], a["st"], None)

    assert forward(a) == code
    assert L.cgl_balance_loss_backward(a["gl"], a["logits"], a["dtype"], a["idx"], a["n"], a["k"], a["E"], a["S"], 1.0, a["score"],
                                       a["counts"], a["routed"], a["grad"], None) == code


@pytest.mark.parametrize("bad,code", [(dict(loss=None), cgl.EINVAL), (dict(ws=None), cgl.EINVAL), (dict(wsb=8), cgl.EINVAL),
                                      (dict(ws=P + 8), cgl.EALIGN), (dict(loss=P + 2), cgl.EALIGN), (dict(st=P + 2), cgl.EALIGN)])
def test_balance_forward_buffers(L, bad, code):
    a = dict(dict(loss=P, ws=P, wsb=1 << 20, st=P), **bad)
    assert L.cgl_balance_loss(P, 2, P, 8, 2, 16, 2, 1.0, 0, None, a["loss"], P, P, None, a["ws"], a["wsb"], a["st"], None) == code


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(TypeError):
        cgl.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        cgl.dequantize_mxfp4(u8, u8)
    with pytest.raises(TypeError):
        cgl.dispatch_mxfp4(x.bfloat16(), torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(TypeError):
        cgl.matmul_mxfp4(u8, u8, u8, u8)
    with pytest.raises(TypeError):
        cgl.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32))
