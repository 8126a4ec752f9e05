"""Host-only tests of what the wrappers of the norms into 8 bits and of the SwiGLU
products refuse before anything is allocated or launched."""
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
from test_norm_wrappers_cpu import OnDevice

B, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.mark.parametrize("current", [0, 1])
def test_tensors_of_another_device_are_refused(current, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)

    def refused(shapes, call):
        for odd in shapes:
            t = {k: OnDevice(1 - current if k == odd else current, *v[0], dtype=v[1]) for k, v in shapes.items()}
            with pytest.raises(fp8.Fp8Error, match=f"on cuda:{1 - current}, the current device is {current}"):
                call(t)

    x, vec, one = ((32, 64), B), ((64,), B), ((1,), F32)
    refused(dict(x=x, r=x, w=vec, b=vec, o=x),
            lambda t: fp8.norm_quantize(t["x"], t["r"], t["w"], t["b"], out=t["o"]))
    refused(dict(x=x, r=x, w=vec, b=vec, o=x),
            lambda t: fp8.mx_norm_quantize(t["x"], t["r"], t["w"], t["b"], out=t["o"]))
    delayed = fp8.Recipe(kind=fp8.DELAYED)
    refused(dict(scale=one, amax=one), lambda t: fp8.norm_quantize(
        OnDevice(current, 32, 64), recipe=delayed, scale_in=t["scale"], amax_out=t["amax"]))
    refused(dict(dy=x, x=x, rstd=((32,), F32), w=vec, ds=x), lambda t: fp8.norm_backward(
        t["dy"], t["x"], None, t["rstd"], t["w"], kind=fp8.RMS_NORM, dsum=t["ds"]))
    q, s, w, sw = ((32, 64), U8), ((512,), U8), ((256, 64), U8), ((1024,), U8)
    refused(dict(q=q, s=s, w=w, sw=sw),
            lambda t: fp8.mx_swiglu_gemm(t["q"], 0, t["s"], t["w"], 0, t["sw"], h=True))
    refused(dict(q=q, s=s, w=w, sw=sw, gu=((32, 512), B)), lambda t: fp8.mx_swiglu_gemm_backward(
        t["q"], 0, t["s"], t["w"], 0, t["sw"], t["gu"], d_gate_up=True))
    refused(dict(q=q, s=s, w=w, sw=sw, cq=((32, 512), U8), cs=((32, 16), U8)),
            lambda t: fp8.mx_swiglu_gemm_backward(t["q"], 0, t["s"], t["w"], 0, t["sw"],
                                                  fp8.Checkpoint(t["cq"], t["cs"], 0, 256, 2), d_gate_up=True))
    refused(dict(q=q, w=w, s=one, sw=one, scale=one, amax=one), lambda t: fp8.swiglu_gemm(
        t["q"], 0, t["w"], 0, t["s"], t["sw"], fmt=0, scale_in=t["scale"], amax_out=t["amax"]))
    refused(dict(q=q, w=w, s=one, sw=one, gu=((32, 512), B), scale=one, amax=one), lambda t: fp8.swiglu_gemm_backward(
        t["q"], 0, t["w"], 0, t["s"], t["sw"], t["gu"], fmt=0, scale_in=t["scale"], amax_out=t["amax"]))


def test_scales_that_are_too_few_are_refused(monkeypatch):
    """A kernel would read the scales of whole 128-row blocks and K tiles."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    on = lambda *shape, dtype=U8: OnDevice(0, *shape, dtype=dtype)  # noqa: E731
    for sA, sW in ((511, 2048), (512, 2047)):  # 32 rows pad to 128; F = 160 pads each half to 256
        with pytest.raises(fp8.Fp8Error, match="are needed"):
            fp8.mx_swiglu_gemm(on(32, 96), 0, on(sA), on(320, 96), 0, on(sW), h=True)
    with pytest.raises(fp8.Fp8Error, match="vector of"):
        fp8.swiglu_gemm(on(32, 96), 0, on(320, 96), 0, on(31, dtype=F32), on(1, dtype=F32), h=True)
