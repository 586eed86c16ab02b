"""Refusals of the routing and the BF16 product, on a machine without a GPU: nothing is launched."""

import contextlib
import ctypes as C

import pytest
import torch

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild

P = 0x10000   # 64 KiB-aligned, never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def L():
    cbuild.build()
    assert cgl.lib().cgl_version() >= 500
    return cgl.lib()


def _opts(cap=0, sms=0, flags=0):
    return C.byref(cgl.Opts(sms, cap, flags, None))


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), cgl.EINVAL), (dict(E=0), cgl.EINVAL), (dict(E=1025), cgl.EINVAL), (dict(k=0), cgl.EINVAL), (dict(k=33), cgl.EINVAL),
    (dict(E=4, k=5, G=1, keep=1), cgl.EINVAL), (dict(n=2 ** 30), cgl.EINVAL), (dict(dtype=3), cgl.EINVAL), (dict(dtype=-1), cgl.EINVAL),
    (dict(G=0), cgl.EINVAL), (dict(G=5), cgl.EINVAL), (dict(G=64), cgl.EINVAL), (dict(keep=0), cgl.EINVAL), (dict(keep=5), cgl.EINVAL),
    (dict(by=2), cgl.EINVAL), (dict(by=-1), cgl.EINVAL), (dict(score=2), cgl.EINVAL), (dict(logits=None), cgl.EINVAL), (dict(idx=None), cgl.EINVAL),
    (dict(w=None), cgl.EINVAL), (dict(logits=P + 2), cgl.EALIGN), (dict(dtype=0, logits=P + 1), cgl.EALIGN), (dict(bias=P + 2), cgl.EALIGN),
    (dict(idx=P + 2), cgl.EALIGN), (dict(w=P + 1), cgl.EALIGN), (dict(st=P + 2), cgl.EALIGN)])
def test_route(L, bad, code):
    a = dict(dict(logits=P, dtype=2, n=8, E=64, k=4, bias=P, G=4, keep=2, by=0, score=0, idx=P, w=P, st=P), **bad)
    assert L.cgl_route(a["logits"], a["dtype"], a["n"], a["E"], a["k"], a["bias"], a["G"], a["keep"], a["by"], a["score"], 1, 1.0, a["idx"],
                       a["w"], a["st"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), cgl.EINVAL), (dict(E=0), cgl.EINVAL), (dict(E=1025), cgl.EINVAL), (dict(k=0), cgl.EINVAL), (dict(k=33), cgl.EINVAL),
    (dict(n=2 ** 30), cgl.EINVAL), (dict(dtype=3), cgl.EINVAL), (dict(score=-1), cgl.EINVAL), (dict(g=None), cgl.EINVAL),
    (dict(logits=None), cgl.EINVAL), (dict(idx=None), cgl.EINVAL), (dict(grad=None), cgl.EINVAL), (dict(g=P + 2), cgl.EALIGN),
    (dict(logits=P + 2), cgl.EALIGN), (dict(idx=P + 1), cgl.EALIGN), (dict(grad=P + 2), cgl.EALIGN), (dict(st=P + 2), cgl.EALIGN)])
def test_route_backward(L, bad, code):
    a = dict(dict(g=P, logits=P, dtype=2, idx=P, n=8, E=64, k=4, score=0, grad=P, st=P), **bad)
    assert L.cgl_route_backward(a["g"], a["logits"], a["dtype"], a["idx"], a["n"], a["E"], a["k"], a["score"], 1, 1.0, a["grad"], a["st"],
                                None) == code


SHARED = [
    (dict(K=0), cgl.EINVAL), (dict(K=12), cgl.EINVAL), (dict(K=2 ** 20 + 8), cgl.EINVAL), (dict(F=0), cgl.EINVAL), (dict(F=2 ** 20 + 2), cgl.EINVAL),
    (dict(F=33, act=4), cgl.EINVAL), (dict(act=5), cgl.EINVAL), (dict(act=-1), cgl.EINVAL), (dict(E=0), cgl.EINVAL), (dict(E=1025), cgl.EINVAL),
    (dict(rows=-1), cgl.EINVAL), (dict(rows=2 ** 31), cgl.EINVAL), (dict(off=None), cgl.EINVAL), (dict(off=None, E=1, opts=_opts(cap=4)), cgl.EINVAL),
    (dict(opts=_opts(cap=5)), cgl.EINVAL), (dict(opts=_opts(cap=-1)), cgl.EINVAL), (dict(opts=_opts(sms=-1)), cgl.EINVAL),
    (dict(opts=_opts(flags=2)), cgl.EINVAL), (dict(w=None), cgl.EINVAL), (dict(a=None), cgl.EINVAL), (dict(a=P + 8), cgl.EALIGN),
    (dict(w=P + 8), cgl.EALIGN), (dict(off=P + 2), cgl.EALIGN), (dict(st=P + 2), cgl.EALIGN)]


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(y=None), cgl.EINVAL), (dict(y=P + 1), cgl.EALIGN), (dict(bias=P + 1), cgl.EALIGN), (dict(res=P + 1), cgl.EALIGN), (dict(z=P + 1), cgl.EALIGN),
    (dict(zt=1), cgl.EINVAL), (dict(zt=3), cgl.EINVAL), (dict(zt=2, z=P + 2), cgl.EALIGN)])
def test_matmul(L, bad, code):
    a = dict(dict(a=P, rows=16, w=P, E=4, F=32, K=64, off=P, bias=P, act=3, res=P, y=P, z=P, zt=0, opts=None, st=P), **bad)
    assert L.cgl_matmul_bf16(a["a"], a["rows"], a["w"], a["E"], a["F"], a["K"], a["off"], a["bias"], a["act"], a["res"], a["y"], a["z"], a["zt"],
                             a["opts"], a["st"], None) == code


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(g=None), cgl.EINVAL), (dict(z=None), cgl.EINVAL), (dict(ws=None), cgl.EINVAL), (dict(wsb=100), cgl.EINVAL), (dict(g=P + 1), cgl.EALIGN),
    (dict(z=P + 2), cgl.EALIGN), (dict(zt=0, z=P + 1), cgl.EALIGN), (dict(zt=1), cgl.EINVAL), (dict(da=P + 8), cgl.EALIGN), (dict(dw=P + 8), cgl.EALIGN), (dict(db=P + 1), cgl.EALIGN), (dict(ws=P + 8), cgl.EALIGN)])
def test_matmul_backward(L, bad, code):
    a = dict(dict(g=P, a=P, rows=16, w=P, E=4, F=32, K=64, off=P, act=3, z=P, zt=2, da=P, dw=P, db=P, ws=P, wsb=1 << 24, opts=None, st=P), **bad)
    assert L.cgl_matmul_bf16_backward(a["g"], a["a"], a["rows"], a["w"], a["E"], a["F"], a["K"], a["off"], a["act"], a["z"], a["zt"], a["da"], a["dw"],
                                      a["db"], a["ws"], a["wsb"], a["opts"], a["st"], None) == code


def test_workspace(L):
    f = L.cgl_matmul_bf16_backward_workspace_bytes
    assert f(0, 1, 8, 8) > 0 and f(1000, 4, 33, 64) >= 1000 * 33 * 2
    assert f(2 ** 31 - 4096, 1, 2 ** 20, 8) >= (2 ** 31 - 4096) * 2 ** 21
    for bad in ((-1, 1, 8, 8), (2 ** 31, 1, 8, 8), (8, 0, 8, 8), (8, 1025, 8, 8), (8, 1, 0, 8), (8, 1, 8, 0), (8, 1, 8, 12), (8, 1, 2 ** 20 + 1, 8)):
        assert f(*bad) == 0


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


CALLS = {
    "route": lambda **k: cgl.route(torch.zeros(2, 8), 2, **k),
    "route_backward": lambda **k: cgl.route_backward(torch.zeros(2, 2), torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32), **k),
    "matmul_bf16": lambda **k: cgl.matmul_bf16(_bf(2, 16), _bf(4, 16), **k),
    "matmul_bf16_backward": lambda **k: cgl.matmul_bf16_backward(_bf(2, 4), _bf(2, 16), _bf(4, 16), **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_are_refused(name):
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        CALLS[name]()
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        CALLS[name](stream=0x1234)


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_belongs_to_the_tensors_device(name, monkeypatch):
    class Stop(Exception):
        pass

    made = []

    class External:
        def __init__(self, handle, device=None):
            made.append((handle, device))

    @contextlib.contextmanager
    def current(stream):
        raise Stop
        yield

    class Elsewhere:
        cuda_stream, device = 0x1234, torch.device("cuda", 1)

    monkeypatch.setattr(cgl, "_dev", lambda t, *a, **k: t)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", current)
    with pytest.raises(Stop):
        CALLS[name](stream=0x1234)
    assert made == [(0x1234, torch.device("cpu"))]
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](stream=Elsewhere())
