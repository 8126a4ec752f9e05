"""A pre-norm SwiGLU MLP block, forward and backward in MXFP8, that keeps every
activation its backward needs in 8 bits.

    out = x + down( silu(gate) * up ),   gate | up = rms_norm(x) W_gate_up^T

The linear layers run on the block-scaled tensor-core GEMMs.  Between the
forward and the backward the block holds:

  * the normalized rows and gate|up as 8-bit checkpoints (norm_forward's
    checkpoint_fmt and swiglu_checkpoint), which norm_backward and
    swiglu_backward read;
  * the transposed MXFP8 operands of the two weight gradients.

    python examples/norm_mlp.py [--tokens 8192 --hidden 4096 --ffn 14336]

prints the time of a step, the bytes kept against bf16 activations, and how far
the gradients lie from those of the same block with gate|up and x kept in bf16.

The library forms h in bf16 in the kernel that also stores the codes.  The bf16
block calls it too and drops them, so its step has a write of 2.06 bytes an element
of h too many: about 36 us at the sizes above, to be taken off its time.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mixed_precision_scale_gb300 as fp8  # noqa: E402

E4M3, E5M2 = fp8.E4M3FN, fp8.E5M2  # activations and weights, gradients


@dataclass
class Saved:
    """What the backward needs of one forward."""
    rstd: torch.Tensor
    norm: object            # checkpoint of the normalized rows (or x itself)
    gate_up: object         # checkpoint of gate|up (or gate|up itself)
    y_t: tuple              # transposed MXFP8 operand of the norm's output
    h_t: tuple              # ... and of the SwiGLU's

    def bytes(self) -> int:
        tensors = [self.rstd, *self.y_t, *self.h_t]
        for c in (self.norm, self.gate_up):
            tensors += [c.q, c.s] if isinstance(c, fp8.Checkpoint) else [c]
        return sum(t.numel() * t.element_size() for t in tensors)


class NormMLP:
    """weight bf16 [hidden]; w_gate_up bf16 [2 ffn, hidden]; w_down bf16
    [hidden, ffn]; tokens, hidden and ffn multiples of 32."""

    def __init__(self, weight, w_gate_up, w_down, keep_8_bits=True):
        self.weight, self.keep = weight, keep_8_bits
        self.gate_up = fp8.mx_quantize(w_gate_up, E4M3)
        self.down = fp8.mx_quantize(w_down, E4M3)

    def forward(self, x):
        n = fp8.norm_forward(x, self.weight, kind=fp8.RMS_NORM, checkpoint_fmt=E4M3 if self.keep else None)
        y = fp8.mx_quantize(n.y, E4M3)
        gate_up = fp8.mx_gemm(y.q_row, E4M3, y.s_row, self.gate_up.q_row, E4M3, self.gate_up.s_row)
        if self.keep:
            h, kept = fp8.swiglu_checkpoint(gate_up, E4M3)
        else:
            h, kept = fp8.swiglu_checkpoint(gate_up, E4M3)[0], gate_up   # the codes are dropped
        q = fp8.mx_quantize(h, E4M3)
        out = fp8.mx_gemm(q.q_row, E4M3, q.s_row, self.down.q_row, E4M3, self.down.s_row)
        saved = Saved(n.rstd, n.checkpoint if self.keep else x, kept, (y.q_colT, y.s_col), (q.q_colT, q.s_col))
        return out.add_(x), saved

    def backward(self, d_out, saved):
        """Gradients of x, weight, w_gate_up and w_down."""
        tokens = d_out.shape[0]
        d = fp8.mx_quantize(d_out, E5M2)
        dw_down = fp8.mx_gemm(d.q_colT, E5M2, d.s_col, saved.h_t[0], E4M3, saved.h_t[1], K=tokens)
        dh = fp8.mx_gemm(d.q_row, E5M2, d.s_row, self.down.q_colT, E4M3, self.down.s_col, K=d_out.shape[1])
        g = fp8.mx_quantize(fp8.swiglu_backward(dh, saved.gate_up), E5M2)
        dw_gate_up = fp8.mx_gemm(g.q_colT, E5M2, g.s_col, saved.y_t[0], E4M3, saved.y_t[1], K=tokens)
        dy = fp8.mx_gemm(g.q_row, E5M2, g.s_row, self.gate_up.q_colT, E4M3, self.gate_up.s_col, K=g.q_row.shape[1])
        n = fp8.norm_backward(dy, saved.norm, None, saved.rstd, self.weight, kind=fp8.RMS_NORM)
        return n.dx.add_(d_out), n.dweight, dw_gate_up, dw_down


def problem(tokens, hidden, ffn, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    weight = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(torch.bfloat16)
    return (r((tokens, hidden), 1.0), r((tokens, hidden), 1e-2), weight, r((2 * ffn, hidden), hidden ** -0.5),
            r((hidden, ffn), ffn ** -0.5))


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=8192)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--ffn", type=int, default=14336)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    x, d_out, weight, w_gate_up, w_down = problem(a.tokens, a.hidden, a.ffn)
    grads = {}
    for keep in (False, True):
        block = NormMLP(weight, w_gate_up, w_down, keep_8_bits=keep)
        out, saved = block.forward(x)
        grads[keep] = block.backward(d_out, saved)
        kept = saved.bytes()
        del out, saved
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for i in range(a.steps + 3):
            if i == 3:
                start.record()
            out, saved = block.forward(x)
            block.backward(d_out, saved)
        end.record()
        torch.cuda.synchronize()
        print(f"activations kept in {'8 bits' if keep else 'bf16  '}: {kept / 2 ** 20:8.1f} MiB a layer, "
              f"{start.elapsed_time(end) / a.steps:7.3f} ms a step")
    for name, b, c in zip(("x", "weight", "w_gate_up", "w_down"), grads[False], grads[True]):
        off = float((b.double() - c.double()).norm() / b.double().norm())
        print(f"gradient of {name:10s}: {off:.4f} (relative, 8 bits against bf16)")
    if fp8.fp8_sync_status() != 0:
        raise SystemExit("device status")


if __name__ == "__main__":
    main()
