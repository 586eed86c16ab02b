"""Outputs that overlap what a call still reads are refused, on the host: nothing is launched and no pointer read."""

import pytest

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild


@pytest.fixture(scope="module")
def L():
    cbuild.build()
    return cgl.lib()


def _arrays(**sizes):
    """A place of its own for each array, and where it ends."""
    at, out = 0x100000, {}
    for name, size in sizes.items():
        out[name] = at
        at += (size + 0xFFF) // 0x1000 * 0x1000 + 0x1000
    return out


def _onto(arrays, sizes, what, where, how):
    """`what` moved so that it meets `where` in its first bytes, its last bytes, or wholly."""
    at = {"same": arrays[where], "front": arrays[where] - sizes[what] + 16, "back": arrays[where] + sizes[where] - 16}[how]
    return dict(arrays, **{what: at // 16 * 16})


HOW = ["same", "front", "back"]
N, E, K = 64, 32, 8
ROUTE = dict(logits=N * E * 2, bias=E * 4, idx=N * K * 4, weights=N * K * 4)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("what,where", [("idx", "logits"), ("idx", "bias"), ("idx", "weights"), ("weights", "logits"), ("weights", "bias")])
def test_route(L, what, where, how):
    a = _onto(_arrays(**ROUTE), ROUTE, what, where, how)
    assert L.cgl_route(a["logits"], 0, N, E, K, a["bias"], 1, 1, 0, 0, 1, 1.0, a["idx"], a["weights"], None, None) == cgl.EINVAL


BACK = dict(g=N * K * 4, logits=N * E * 4, idx=N * K * 4, grad=N * E * 4)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("where", ["g", "logits", "idx"])
def test_route_backward(L, where, how):
    a = _onto(_arrays(**BACK), BACK, "grad", where, how)
    assert L.cgl_route_backward(a["g"], a["logits"], 2, a["idx"], N, E, K, 0, 1, 1.0, a["grad"], None, None) == cgl.EINVAL


R, X, F, C = 64, 3, 48, 40
MATMUL = dict(a=R * C * 2, w=X * F * C * 2, off=(X + 1) * 4, bias=X * F * 2, residual=R * F * 2, y=R * F * 2, preact=R * F * 4)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("what,where", [("y", i) for i in ("a", "w", "off", "bias", "residual", "preact")] +
                         [("preact", i) for i in ("a", "w", "off", "bias", "residual")])
def test_matmul(L, what, where, how):
    if (what, where, how) == ("y", "residual", "same"):
        pytest.skip("y may be the residual")
    a = _onto(_arrays(**MATMUL), MATMUL, what, where, how)
    assert L.cgl_matmul_bf16(a["a"], R, a["w"], X, F, C, a["off"], a["bias"], 3, a["residual"], a["y"], a["preact"], 2, None, None, None) == cgl.EINVAL


GRADS = dict(g=R * F * 2, a=R * C * 2, w=X * F * C * 2, off=(X + 1) * 4, preact=R * F * 4, da=R * C * 2, dw=X * F * C * 2, db=X * F * 2, ws=0)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("act", [0, 3])
@pytest.mark.parametrize("what,where", [("da", i) for i in ("a", "w", "off", "dw")] + [("dw", i) for i in ("a", "off")] +
                         [("db", i) for i in ("a", "w", "off", "da", "dw")] + [("ws", i) for i in ("g", "a", "w", "off", "da", "dw", "db")])
def test_matmul_backward(L, what, where, act, how):
    sizes = dict(GRADS, ws=cgl.matmul_bf16_backward_workspace_bytes(R, X, F, C))
    a = _onto(_arrays(**sizes), sizes, what, where, how)
    assert L.cgl_matmul_bf16_backward(a["g"], a["a"], R, a["w"], X, F, C, a["off"], act, a["preact"] if act else None, 2, a["da"], a["dw"], a["db"], a["ws"],
                                      sizes["ws"], None, None, None) == cgl.EINVAL


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("what", ["da", "dw", "db"])
def test_matmul_backward_that_reads_grad_y_to_the_end(L, what, how):
    sizes = dict(GRADS, ws=cgl.matmul_bf16_backward_workspace_bytes(R, X, F, C))
    a = _onto(_arrays(**sizes), sizes, what, "g", how)
    bias = what == "db"
    assert L.cgl_matmul_bf16_backward(a["g"], a["a"], R, a["w"], X, F, C, a["off"], 0, None, 0, a["da"], a["dw"], a["db"] if bias else None,
                                      a["ws"] if bias else None, sizes["ws"], None, None, None) == cgl.EINVAL


@pytest.mark.parametrize("how", HOW)
def test_workspace_on_preact(L, how):
    sizes = dict(GRADS, ws=cgl.matmul_bf16_backward_workspace_bytes(R, X, F, C))
    a = _onto(_arrays(**sizes), sizes, "ws", "preact", how)
    assert L.cgl_matmul_bf16_backward(a["g"], a["a"], R, a["w"], X, F, C, a["off"], 3, a["preact"], 2, a["da"], a["dw"], a["db"], a["ws"], sizes["ws"], None,
                                      None, None) == cgl.EINVAL
