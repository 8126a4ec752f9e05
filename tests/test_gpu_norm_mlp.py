"""GPU test of the example block: RMS norm, MXFP8 linears, SwiGLU and their
backward, with every kept activation in 8 bits, against float64 autograd.

Bound: each conversion to 8 bits moves a tensor by a relative 2-norm of about
0.027 (E4M3) or 0.053 (E5M2): half a step of 2^-3 or 2^-2 of a binade's start,
uniform, over values spread evenly inside a binade.  A gradient passes at most
two E5M2 and five E4M3 conversions (the x gradient: dout, d gate|up; both
weights, h's inputs, gate|up and the normalized rows in their checkpoints),
0.096 in all if independent; twice that is allowed.  Kept in bf16 instead, the
same gradients must differ from these by no more than the two checkpoints'
share, 0.027 each through slopes of at most about 1.1, again doubled: 0.12."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import fp8_mixed_precision_scale_gb300 as fp8  # noqa: E402

pytestmark = pytest.mark.gpu


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("shape", [(256, 256, 512), (128, 1024, 704), (96, 160, 96)])
def test_block_against_autograd(shape):
    import norm_mlp
    tokens, hidden, ffn = shape
    x, d_out, weight, w_gate_up, w_down = norm_mlp.problem(tokens, hidden, ffn)
    block = norm_mlp.NormMLP(weight, w_gate_up, w_down)
    out, saved = block.forward(x)
    got = block.backward(d_out, saved)
    assert fp8.fp8_sync_status() == 0

    leaves = [t.double().requires_grad_() for t in (x, weight, w_gate_up, w_down)]
    xx, w, wgu, wd = leaves
    y = xx * torch.rsqrt((xx * xx).mean(1, keepdim=True) + 1e-5) * w
    gate, up = (y @ wgu.T).chunk(2, 1)
    ref = xx + (torch.nn.functional.silu(gate) * up) @ wd.T
    ref.backward(d_out.double())
    assert off(out, ref.detach()) < 0.1
    for name, g, leaf in zip(("x", "weight", "w_gate_up", "w_down"), got, leaves):
        assert off(g, leaf.grad) < 0.2, name

    plain = norm_mlp.NormMLP(weight, w_gate_up, w_down, keep_8_bits=False)
    out2, saved2 = plain.forward(x)
    assert torch.equal(out, out2)   # what is kept changes no forward value
    for name, g, b in zip(("x", "weight", "w_gate_up", "w_down"), got, plain.backward(d_out, saved2)):
        assert off(g, b) < 0.12, name
    assert saved.bytes() < 0.7 * saved2.bytes()
