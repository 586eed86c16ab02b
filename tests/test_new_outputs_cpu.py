"""Outputs that a call allocates for itself: torch's short path to the allocator is taken only where it gives what the
public one gives, and never where torch is asked to fill new memory.  Without a GPU: both paths are stood in for."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl


class Like:
    device = torch.device("cuda", 0)


class Made:
    def __init__(self, shape=(2, 3), strides=(3, 1), dtype=torch.int32, device=torch.device("cuda", 0)):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self.stride = lambda: tuple(strides)


def _fails(error):
    def short(*args):
        raise error
    return short


@pytest.fixture
def public(monkeypatch):
    calls = []
    monkeypatch.setattr(torch, "empty_strided", lambda *a, **k: calls.append((a, k)) or "public")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(cgl, "_empty", cgl._first_empty)
    return calls


def test_a_short_path_that_gives_the_same_is_taken(public, monkeypatch):
    monkeypatch.setattr(cgl, "_short_empty", Made)
    for _ in range(2):
        t = cgl._out(None, "y", (5, 7), torch.bfloat16, Like)
        assert (t.shape, t.stride(), t.dtype) == ((5, 7), (7, 1), torch.bfloat16) and not public


@pytest.mark.parametrize("short", [
    None, _fails(TypeError()), _fails(RuntimeError()), lambda s, t, d: None, lambda s, t, d: Made(s, t, torch.float32),
    lambda s, t, d: Made(s, t, d, torch.device("cpu")), lambda s, t, d: Made(s, t, d, torch.device("cuda", 1)), lambda s, t, d: Made(s, (1, 2), d),
    lambda s, t, d: Made((3, 2), t, d)])
def test_any_other_is_not(short, public, monkeypatch):
    monkeypatch.setattr(cgl, "_short_empty", short)
    for shape, strides in (((5, 7), (7, 1)), ((2, 5, 7), (35, 7, 1)), ((9,), (1,))):
        assert cgl._out(None, "y", shape, torch.bfloat16, Like) == "public"
        args, how = public.pop()
        assert args == (shape, strides) and how["dtype"] is torch.bfloat16 and torch.device(how["device"]).type == "cuda"


def test_another_device_and_deterministic_mode_take_the_public_path(public, monkeypatch):
    monkeypatch.setattr(cgl, "_short_empty", Made)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    assert cgl._out(None, "y", (5, 7), torch.bfloat16, Like) == "public" and public.pop()[1]["device"] == Like.device
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    torch.use_deterministic_algorithms(True)
    try:
        assert cgl._out(None, "y", (5, 7), torch.bfloat16, Like) == "public"
    finally:
        torch.use_deterministic_algorithms(False)
