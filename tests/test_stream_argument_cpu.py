"""The stream argument of the MXFP4 calls and the balance loss, without a GPU: a stream belongs to a device, the
tensors', whichever is current."""

import contextlib

import pytest
import torch

import combine_get_layout_02_b200 as cgl


class Stop(Exception):
    pass


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


CALLS = {
    "quantize_mxfp4": lambda **k: cgl.quantize_mxfp4(torch.zeros(2, 32), **k),
    "dequantize_mxfp4": lambda **k: cgl.dequantize_mxfp4(_u8(2, 16), _u8(2, 1), **k),
    "dispatch_mxfp4": lambda **k: cgl.dispatch_mxfp4(torch.zeros(2, 32).bfloat16(), torch.zeros(2, 1, dtype=torch.int32), 2, **k),
    "matmul_mxfp4": lambda **k: cgl.matmul_mxfp4(_u8(2, 16), _u8(2, 1), _u8(4, 16), _u8(4, 1), **k),
    "balance_loss": lambda **k: cgl.balance_loss(torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32), **k),
    "balance_loss_backward": lambda **k: cgl.balance_loss_backward(
        torch.ones(1), torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32),
        torch.ones(1, dtype=torch.int32), **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_handle_is_taken_on_the_tensors_device(name, monkeypatch):
    made = []

    class External:
        def __init__(self, handle, device=None):
            made.append((handle, device))

    @contextlib.contextmanager
    def current(stream):
        assert isinstance(stream, External)
        raise Stop
        yield

    monkeypatch.setattr(cgl, "_dev", lambda t, *a, **k: t)      # stands for tensors on a device that is not current
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", current)
    with pytest.raises(Stop):
        CALLS[name](stream=0x1234)
    assert made == [(0x1234, torch.device("cpu"))]


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    class Elsewhere:
        cuda_stream, device = 0x1234, torch.device("cuda", 1)

    monkeypatch.setattr(cgl, "_dev", lambda t, *a, **k: t)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("another device's stream was made current"))
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](stream=Elsewhere())


@pytest.mark.parametrize("name", CALLS)
def test_tensors_off_the_gpu_are_refused_with_a_stream_too(name):
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        CALLS[name](stream=0x1234)
