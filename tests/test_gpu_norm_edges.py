"""GPU tests of the norm, SwiGLU and checkpoint operators where callers and
values leave the usual: the default stream by its handle."""
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


def test_default_stream_by_its_handle():
    """stream=0 is torch's default stream: a call on it comes after what was
    put there before, and before what is put there next."""
    with fp8._on(torch.cuda.default_stream().cuda_stream):
        assert torch.cuda.current_stream().cuda_stream == 0
    x, w = torch.randn((3000, 4096), device=DEV).to(BF16), torch.ones(4096, dtype=BF16, device=DEV)
    want = fp8.norm_forward(x, w, checkpoint_fmt=0)
    dy = want.y * 0.1
    back = fp8.norm_backward(dy, want.checkpoint, want.mean, want.rstd, w)
    gate_up, kept = fp8.checkpoint(x), fp8.checkpoint(x, parts=2)
    h, _ = fp8.swiglu_checkpoint(x)
    grad = fp8.swiglu_backward(h, kept)
    for _ in range(5):
        late = torch.zeros_like(x)
        for _ in range(20):
            late.add_(0.0)
        late.copy_(x)   # after 20 passes over it
        f = fp8.norm_forward(late, w, checkpoint_fmt=0, stream=0)
        b = fp8.norm_backward(dy, f.checkpoint, f.mean, f.rstd, w, stream=0)
        c = fp8.checkpoint(late, stream=0)
        h2, _ = fp8.swiglu_checkpoint(late, stream=0)
        d = fp8.swiglu_backward(h2, kept, stream=0)
        r = fp8.checkpoint_restore(c, stream=0)
        assert torch.equal(f.y, want.y) and torch.equal(b.dx, back.dx) and torch.equal(b.dweight, back.dweight)
        assert torch.equal(c.q, gate_up.q) and torch.equal(h2, h) and torch.equal(d, grad)
        assert torch.equal(r, fp8.checkpoint_restore(gate_up))
