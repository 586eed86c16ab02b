"""Token counts whose product with the slots leaves 64 bits are refused like any other that is too large; on the host,
nothing is launched."""

import pytest

import combine_get_layout_02_b200 as cgl
from combine_get_layout_02_b200 import build as cbuild

P = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def L():
    cbuild.build()
    return cgl.lib()


# n * k is 0, or small and positive, in 64 bits
COUNTS = [(2 ** 59, 32), (2 ** 60, 16), (2 ** 61, 8), (2 ** 61 + 3, 8), (2 ** 63 - 1, 2), (2 ** 31, 1)]


@pytest.mark.parametrize("n,k", COUNTS)
def test_refused(L, n, k):
    assert L.cgl_route(P, 2, n, 64, k, None, 1, 1, 0, 0, 1, 1.0, P, P, P, None) == cgl.EINVAL
    assert L.cgl_route_backward(P, P, 2, P, n, 64, k, 0, 1, 1.0, P, P, None) == cgl.EINVAL
    assert L.cgl_dispatch_mxfp4(P, n, 64, k, P, P, P, 8, None, P, None) == cgl.EINVAL
    assert L.cgl_get_layout(P, n, k, 64, 8, None, P, P, P, P, P, P, P, P, 1 << 62, P, None) == cgl.EINVAL
    assert L.cgl_get_rank_layout(P, n, k, 64, 8, None, P, P, P, P, P, P, 1 << 62, P, None) == cgl.EINVAL
    assert L.cgl_balance_loss(P, 2, P, n, k, 64, 1, 1.0, 0, P, P, P, P, P, P, 1 << 62, P, None) == cgl.EINVAL
    assert L.cgl_balance_loss_backward(P, P, 2, P, n, k, 64, 1, 1.0, 0, P, P, P, None) == cgl.EINVAL


@pytest.mark.parametrize("n,k", COUNTS)
def test_no_workspace_for_them(L, n, k):
    assert cgl.layout_workspace_bytes(n, k, 64, 8) == 0
    assert cgl.layout_kernel_count(n, k, 64, 8) == -1
    assert L.cgl_layout_dispatch_workspace_bytes(n, k, 64, 8) == 0
    assert cgl.balance_loss_workspace_bytes(n, k, 64, 1) == 0
