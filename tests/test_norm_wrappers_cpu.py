"""Host-only tests of what the Python wrappers of the norm, SwiGLU and
checkpoint operators do before a launch: the stream they take a handle for,
the devices they refuse."""
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8


class PoolStream:
    """torch.cuda.ExternalStream as it behaves: a handle of 0 is none given, and
    a stream of torch's pool comes back, which does not wait for the default."""

    def __init__(self, handle):
        self.cuda_stream = handle if handle else 0x5EED


class DefaultStream:
    cuda_stream = 0


@pytest.mark.parametrize("handle", [0, 0x1230])
def test_a_handle_is_the_stream_it_names(handle, monkeypatch):
    monkeypatch.setattr(torch.cuda, "ExternalStream", PoolStream)
    monkeypatch.setattr(torch.cuda, "default_stream", DefaultStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: stream)
    assert fp8._on(handle).cuda_stream == handle


class OnDevice:
    """A CUDA tensor as the wrappers' checks see it."""
    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.device_index, self.shape, self.dtype, self.device = device, shape, dtype, f"cuda:{device}"

    def get_device(self):
        return self.device_index

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self):
        return (self.shape[-1], 1)[2 - len(self.shape):]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the call went past its checks")


@pytest.mark.parametrize("current", [0, 1])
def test_tensors_of_another_device_are_refused(current, monkeypatch):
    """Every tensor of every call, one at a time on the device that is not the
    current one; outputs are given, so that nothing is allocated."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    F32, U8 = torch.float32, torch.uint8

    def refused(shapes, call):
        for odd in shapes:
            t = {k: OnDevice(1 - current if k == odd else current, *v[0], dtype=v[1]) for k, v in shapes.items()}
            with pytest.raises(fp8.Fp8Error, match=f"on cuda:{1 - current}, the current device is {current}"):
                call(t)

    B = torch.bfloat16
    x, vec, rows = ((4, 64), B), ((64,), B), ((4,), F32)
    codes, scales = ((4, 64), U8), ((4, 2), U8)
    keep = lambda t, parts=1: fp8.Checkpoint(t["q"], t["s"], 0, 64 // parts, parts)  # noqa: E731
    refused(dict(x=x, w=vec, b=vec, y=x), lambda t: fp8.norm_forward(t["x"], t["w"], t["b"], out=t["y"]))
    refused(dict(dy=x, x=x, mean=rows, rstd=rows, w=vec, dx=x),
            lambda t: fp8.norm_backward(t["dy"], t["x"], t["mean"], t["rstd"], t["w"], out=t["dx"]))
    refused(dict(dy=x, q=codes, s=scales, rstd=rows, dx=x),
            lambda t: fp8.norm_backward(t["dy"], keep(t), None, t["rstd"], out=t["dx"]))
    refused(dict(x=x), lambda t: fp8.checkpoint(t["x"]))
    refused(dict(q=codes, s=scales, x=x),
            lambda t: fp8.checkpoint_restore(keep(t), out=t["x"]))
    refused(dict(x=x, h=((4, 32), B)), lambda t: fp8.swiglu_checkpoint(t["x"], h_out=t["h"]))
    refused(dict(dh=((4, 32), B), x=x, d=x),
            lambda t: fp8.swiglu_backward(t["dh"], t["x"], out=t["d"]))
    refused(dict(dh=((4, 32), B), q=codes, s=scales, d=x),
            lambda t: fp8.swiglu_backward(t["dh"], keep(t, 2), out=t["d"]))
