"""A pre-norm SwiGLU block through the fused operators, forward and backward, as a
training step runs it, against the same block in float64."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import fused_ref as ref
import norm_ref as nref

pytestmark = pytest.mark.gpu
DEV, E4M3 = "cuda", fp8.E4M3FN


def matrix(rows, cols, scale, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * scale).bfloat16().to(DEV)


def dequantized(w, fmt, rows=True):
    """What a plain quantize of w (its row layout, or the transposed one) stands for."""
    v = nref.f64(w) if rows else nref.f64(w).T
    q, s = ref.mx_quantize(v, fmt)
    return nref.decode_table(fmt)[q.numpy()] * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)


@pytest.mark.parametrize("tokens,hidden,ffn", [(64, 128, 256), (160, 256, 288)])
def test_block(tokens, hidden, ffn):
    x, res = matrix(tokens, hidden, 1.0, 1), matrix(tokens, hidden, 1.0, 2)
    weight = (1 + 0.2 * torch.randn(hidden, generator=torch.Generator().manual_seed(3))).to(DEV)
    w_gu, w_down = matrix(2 * ffn, hidden, 1 / np.sqrt(hidden), 4), matrix(hidden, ffn, 1 / np.sqrt(ffn), 5)
    dy, dres = matrix(tokens, hidden, 0.1, 6), matrix(tokens, hidden, 0.1, 7)

    halves = torch.tensor([0, ffn, 2 * ffn], dtype=torch.int32)
    gu = fp8.mx_quantize(w_gu, E4M3, group_offsets=halves.to(DEV), host_offsets=halves)
    down = fp8.mx_quantize(w_down, E4M3)
    n = fp8.mx_norm_quantize(x, res, weight, kind=fp8.RMS_NORM)
    f = fp8.mx_swiglu_gemm(n.q.q_row, E4M3, n.q.s_row, gu.q_row, E4M3, gu.s_row, fmt=E4M3, checkpoint_fmt=E4M3)
    y = fp8.mx_gemm(f.q.q_row, E4M3, f.q.s_row, down.q_row, E4M3, down.s_row)
    qd = fp8.mx_quantize(dy, E4M3)
    dw_down = fp8.mx_gemm(qd.q_colT, E4M3, qd.s_col, f.q.q_colT, E4M3, f.q.s_col)
    b = fp8.mx_swiglu_gemm_backward(qd.q_row, E4M3, qd.s_row, down.q_colT, E4M3, down.s_col, f.checkpoint, fmt=E4M3)
    dn = fp8.mx_gemm(b.q.q_row, E4M3, b.q.s_row, gu.q_colT, E4M3, gu.s_col, K=b.q.q_row.shape[1])
    dw_gu = fp8.mx_gemm(b.q.q_colT, E4M3, b.q.s_col, n.q.q_colT, E4M3, n.q.s_col)
    d = fp8.norm_backward(dn, n.sum, None, n.rstd, weight, kind=fp8.RMS_NORM, dsum=dres)
    assert fp8.fp8_sync_status() == 0

    # in float64: the same quantized weights, nothing else rounded
    s = nref.f64(n.sum)
    yn, _, rstd, xh = nref.norm_forward(s, nref.f64(weight), 0.0, True, 1e-5)
    wq = dequantized(w_gu, E4M3)
    g, u = yn @ wq[:ffn].T, yn @ wq[ffn:].T
    h = nref.swiglu(g, u)
    want_y = h @ dequantized(w_down, E4M3).T
    dh = nref.f64(dy) @ dequantized(w_down, E4M3, False).T
    dg, du = nref.swiglu_backward(g, u, dh)
    dgu = np.concatenate([dg, du], 1)
    dn64 = dgu @ nref.f64(w_gu)
    dx, dweight, _ = nref.norm_backward(dn64, xh, rstd, nref.f64(weight), True)

    def far(got, want):
        return np.linalg.norm(nref.f64(got) - want) / np.linalg.norm(want)

    # Each 8-bit rounding is off by at most 2^-4 of its value, a clipped top of a block
    # (448 for up to 512) by 2^-3; with that in each of the k factors that a result
    # has, its 2-norm is off by less than k 2^-3 of sums of magnitudes, whose terms'
    # signs are independent: k 2^-3 of the result.
    for name, got, want, k in (("y", y, want_y, 3), ("dW_down", dw_down, nref.f64(dy).T @ h, 3),
                               ("dW", dw_gu, dgu.T @ yn, 4), ("dx", d.dx, dx + nref.f64(dres), 4),
                               ("dweight", d.dweight, dweight, 4)):
        assert far(got, want) < k * 2 ** -3, (name, far(got, want))


def test_the_graph_of_a_step_beside_an_eager_one():
    """A captured step and an eager one on the same tensors, in turn."""
    x, res, dy = matrix(64, 256, 1.0, 1), matrix(64, 256, 1.0, 2), matrix(64, 256, 0.1, 3)
    w = fp8.mx_quantize(matrix(512, 256, 0.06, 4), E4M3)
    wd = fp8.mx_quantize(matrix(256, 256, 0.06, 5), E4M3)

    def step():
        n = fp8.mx_norm_quantize(x, res, kind=fp8.RMS_NORM)
        f = fp8.mx_swiglu_gemm(n.q.q_row, E4M3, n.q.s_row, w.q_row, E4M3, w.s_row, fmt=E4M3, checkpoint_fmt=E4M3)
        q = fp8.mx_quantize(dy, E4M3)
        b = fp8.mx_swiglu_gemm_backward(q.q_row, E4M3, q.s_row, wd.q_colT, E4M3, wd.s_col, f.checkpoint, fmt=E4M3)
        dn = fp8.mx_gemm(b.q.q_row, E4M3, b.q.s_row, w.q_colT, E4M3, w.s_col)
        return fp8.norm_backward(dn, n.sum, None, n.rstd, kind=fp8.RMS_NORM, dsum=dy), f.q.q_row

    eager = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for _ in range(3):
        g.replay()
        again = step()
    torch.cuda.synchronize()
    for r in (captured, again):
        assert torch.equal(r[0].dx, eager[0].dx) and torch.equal(r[0].dweight, eager[0].dweight)
        assert torch.equal(r[1], eager[1])
