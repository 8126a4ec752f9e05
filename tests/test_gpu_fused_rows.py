"""GPU tests of the SwiGLU products' few-row kernel over long contractions, of E5M2
operands and results, of the wrappers of the stored scale, and of a whole block
stage by stage, against the float64 references (bounds derived in fused_ref and
norm_ref)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import fused_ref as ref
import norm_ref as nref
import test_gpu_norm_quantize as nq
from test_gpu_norm import params, values
from test_gpu_swiglu_gemm import Operand, Out, backward, forward

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, E5M2 = fp8.E4M3FN, fp8.E5M2
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


def varied(R, K, seed, scale):
    """Sizes that differ by up to 2^6 from one block of 32 columns to the next."""
    e = np.random.RandomState(seed + 100).randint(-3, 4, (R, (K + 31) // 32))
    return scale * np.exp2(np.repeat(e, 32, 1)[:, :K].astype(np.float64))


def check_forward(x, w, o, what):
    F = o.F
    (g, tg), (u, tu) = (ref.product(x.v, h) for h in (w.v[:F], w.v[F:]))
    tg, tu = tg + 2 ** -23 * np.abs(g), tu + 2 ** -23 * np.abs(u)
    h, th = ref.swiglu(g, tg, u, tu)
    o.check([h], [th], what)
    if o.gu is not None:
        for i, (v, t) in enumerate(((g, tg), (u, tu))):
            nref.assert_within(nref.f64(o.gu[:, i * F:(i + 1) * F]), v, ref.bf16_tol(v, t), what + " gate|up")
        assert (o.gu[:, 2 * F:] == 7).all()
    if o.ck is not None:
        W = ref.up(F, 32)
        assert (o.ck.q[:, 2 * W:] == 0xA5).all() and (o.ck.s[:, 2 * W // 32:] == 0xA5).all()
        c = fp8.Checkpoint(o.ck.q[:, :2 * W].contiguous(), o.ck.s[:, :2 * W // 32].contiguous(), o.ck.fmt, F, 2)
        ref.check_kept(c, (g, u), (tg, tu), what + " checkpoint")


# one MX row, one or two scaled ones: several steps of 512 along K with a tail, several
# blocks of 32 columns with a tail; beyond K = 24576 (12288 for two rows) tiles again
FEW = [(True, 1, 288, 544), (True, 1, 1504, 2080), (True, 1, 96, 24544), (True, 1, 96, 24608), (True, 1, 4128, 96),
       (False, 1, 720, 2064), (False, 1, 48, 24560), (False, 1, 48, 24592), (False, 2, 272, 12272),
       (False, 2, 272, 12304)]


@pytest.mark.parametrize("mx,M,F,K", FEW)
@pytest.mark.parametrize("kept", ["8bit", "bf16"])
def test_few_rows(mx, M, F, K, kept):
    x = Operand(M, K, E4M3, mx, 1, varied(M, K, 1, 1.0), ld=ref.up(K, 16) + 16)
    w = Operand(2 * F, K, E4M3, mx, 2, varied(2 * F, K, 2, 0.3 / np.sqrt(K)), ld=ref.up(K, 16) + 32, groups=True)
    o = Out(M, F, mx, 1, kept=kept, layouts=1 if mx else 3)
    forward(x, w, o)
    torch.cuda.synchronize()
    check_forward(x, w, o, f"{M}x{F}x{K}")


def test_one_row_nan_stays_in_its_columns():
    F, K = 160, 1056
    x, w = Operand(1, K, E4M3, True, 1, 1.0), Operand(2 * F, K, E4M3, True, 2, 0.03, groups=True)
    w.q[33, 900] = 0x7F  # a gate's column, past the first step of 512
    o = Out(1, F, True, 1, kept="8bit", layouts=1)
    forward(x, w, o)
    torch.cuda.synchronize()
    h, s = nref.f64(o.h[:, :F]), ref.scales_of(o.s, 1, F // 32)
    assert np.isnan(h[0, 33]) and np.isfinite(np.delete(h, 33, 1)).all()
    assert s[0, 1] == 255 and (np.delete(s, 1, 1) != 255).all()
    k = o.ck.s[0, :2 * F // 32].tolist()
    assert [i for i, b in enumerate(k) if b == 255] == [1]
    x.q[0, 1040] = 0x7F
    o = Out(1, F, True, 1, layouts=1)
    forward(x, w, o)
    torch.cuda.synchronize()
    assert torch.isnan(o.h[:, :F]).all() and (ref.scales_of(o.s, 1, F // 32) == 255).all()


# the few-row kernel, one CTA a tile and narrow tiles, pairs
@pytest.mark.parametrize("mx,M,F,K", [(True, 1, 160, 1056), (True, 96, 160, 288), (True, 288, 288, 544),
                                      (False, 1, 208, 1040), (False, 2, 208, 1040), (False, 100, 208, 272),
                                      (False, 1301, 944, 80)])
@pytest.mark.parametrize("fx,fw,fh,fk", [(E5M2, E4M3, E4M3, None), (E4M3, E5M2, E5M2, E5M2), (E5M2, E5M2, E5M2, E5M2),
                                         (E4M3, E4M3, E5M2, E4M3), (E4M3, E4M3, E4M3, E5M2)])
def test_formats(mx, M, F, K, fx, fw, fh, fk):
    x = Operand(M, K, fx, mx, 1, varied(M, K, 1, 1.0))
    w = Operand(2 * F, K, fw, mx, 2, varied(2 * F, K, 2, 0.3 / np.sqrt(K)), groups=True)
    o = Out(M, F, mx, 1, kept=None if fk is None else "8bit", fmt=fh, layouts=3 if not mx or M % 32 == 0 else 1)
    if fk is not None:
        o.ck.fmt = fk
    forward(x, w, o)
    torch.cuda.synchronize()
    check_forward(x, w, o, f"{M}x{F}x{K}")


def test_accumulators_are_the_plain_products():
    """Bit for bit: the same K steps in the same order, whatever the tile."""
    for M in (64, 320):
        x, w = Operand(M, 544, E4M3, True, 1, 1.0), Operand(512, 544, E4M3, True, 2, 0.1)
        r = fp8.mx_swiglu_gemm(x.q, E4M3, x.s, w.q, E4M3, w.s, gate_up=True)
        c = fp8.mx_gemm(x.q, E4M3, x.s, w.q, E4M3, w.s)
        assert torch.equal(r.gate_up, c)


@pytest.mark.parametrize("layouts", [1, 2, 3])
def test_norm_wrapper_with_a_stored_scale(layouts):
    x, res = values(70, 208, BF16, 8), values(70, 208, F32, 9)
    w, b = params(208, F32, 10)
    scale, amax, amax2 = (torch.tensor([v], device=DEV) for v in (60.0, 0.5, 0.5))
    n = fp8.norm_quantize(x, res, w, b, kind=fp8.LAYER_NORM, fmt=E5M2, recipe=fp8.Recipe(kind=fp8.DELAYED),
                          layouts=layouts, scale_in=scale, amax_out=amax)
    o = nq.Out(70, 208, F32, False, 0)
    nq.call(x, res, w, b, fp8.LAYER_NORM, 1e-5, nq.TENSOR, layouts, E5M2, o, scale=scale, amax=amax2)
    torch.cuda.synchronize()
    nq.check(x, res, w, b, fp8.LAYER_NORM, 1e-5, nq.TENSOR, layouts, E5M2, o, scale=scale, amax=amax2, amax0=0.5)
    assert torch.equal(amax, amax2) and torch.equal(n.sum, o.sum)
    if layouts & 1:
        assert torch.equal(n.q.q_row, o.q) and torch.equal(n.q.scale_inv_row, o.st)
    if layouts & 2:
        assert torch.equal(n.q.q_colT[:, :70], o.qt[:, :70]) and torch.equal(n.q.scale_inv_col, o.st)


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("kept", ["8bit", "bf16"])
def test_backward_wrapper_with_a_stored_scale(kept, per_row):
    M, F, K = 100, 208, 272
    dy, wd = Operand(M, K, E5M2, False, 3, 0.05, per_row), Operand(F, K, E4M3, False, 4, 0.1, per_row)
    gu = (torch.from_numpy(np.random.RandomState(5).randn(M, 2 * F)) * 1.5).bfloat16().to(DEV)
    src = fp8.checkpoint(gu, E4M3, parts=2) if kept == "8bit" else gu
    o = Out(M, F, False, 2)
    r = fp8.swiglu_gemm_backward(dy.q, E5M2, wd.q, E4M3, dy.s, wd.s, src, fmt=E4M3, scale_in=o.scale,
                                 amax_out=o.amax, d_gate_up=True)
    o.h[:, :2 * F], o.q, o.qt[:, :M], o.inv = r.d_gate_up, r.q.q_row, r.q.q_colT[:, :M], r.q.scale_inv_row
    torch.cuda.synchronize()
    g, u = np.split(nref.restore(src.q, src.s, F, 2, E4M3) if kept == "8bit" else nref.f64(gu), 2, 1)
    dh, t = ref.product(dy.v, wd.v)
    dg, tg, du, tu = ref.swiglu_backward(g, u, dh, t + 2 ** -23 * np.abs(dh))
    o.check([dg, du], [tg, tu], "wrapper")
    assert torch.equal(r.q.scale_inv_col, r.q.scale_inv_row)


def mx_value(codes, scales, scale_rows=None):
    """What MX codes [R, K] stand for; scale_rows: the scale row of each of theirs, of how many."""
    rows, total = (np.arange(codes.shape[0]), codes.shape[0]) if scale_rows is None else scale_rows
    s = ref.scales_of(scales, total, codes.shape[1] // 32)[rows]
    return ref.decode(codes, E4M3) * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)


@pytest.mark.parametrize("tokens,hidden,ffn", [(64, 128, 256), (160, 256, 288)])
def test_block_stage_by_stage(tokens, hidden, ffn):
    """Every stage of a block's forward and backward against its own inputs as they are."""
    def matrix(rows, cols, scale, seed):
        return (torch.randn((rows, cols), generator=torch.Generator().manual_seed(seed)) * scale).bfloat16().to(DEV)

    x, res, dres = matrix(tokens, hidden, 1.0, 1), matrix(tokens, hidden, 1.0, 2), matrix(tokens, hidden, 0.1, 7)
    weight, _ = params(hidden, F32, 3)
    w_gu, w_down = matrix(2 * ffn, hidden, 1 / np.sqrt(hidden), 4), matrix(hidden, ffn, 1 / np.sqrt(ffn), 5)
    halves = torch.tensor([0, ffn, 2 * ffn], dtype=torch.int32)
    gu = fp8.mx_quantize(w_gu, E4M3, group_offsets=halves.to(DEV), host_offsets=halves)
    down, qd = fp8.mx_quantize(w_down, E4M3), fp8.mx_quantize(matrix(tokens, hidden, 0.1, 6), E4M3)
    n = fp8.mx_norm_quantize(x, res, weight, kind=fp8.RMS_NORM)
    f = fp8.mx_swiglu_gemm(n.q.q_row, E4M3, n.q.s_row, gu.q_row, E4M3, gu.s_row, fmt=E4M3, checkpoint_fmt=E4M3)
    y = fp8.mx_gemm(f.q.q_row, E4M3, f.q.s_row, down.q_row, E4M3, down.s_row)
    dw_down = fp8.mx_gemm(qd.q_colT, E4M3, qd.s_col, f.q.q_colT, E4M3, f.q.s_col)
    b = fp8.mx_swiglu_gemm_backward(qd.q_row, E4M3, qd.s_row, down.q_colT, E4M3, down.s_col, f.checkpoint, fmt=E4M3)
    dn = fp8.mx_gemm(b.q.q_row, E4M3, b.q.s_row, gu.q_colT, E4M3, gu.s_col)
    dw_gu = fp8.mx_gemm(b.q.q_colT, E4M3, b.q.s_col, n.q.q_colT, E4M3, n.q.s_col)
    d = fp8.norm_backward(dn, n.sum, None, n.rstd, weight, kind=fp8.RMS_NORM, dsum=dres)
    assert fp8.fp8_sync_status() == 0

    def mx(q, scales, v, t, what):
        ref.check_mx(q, ref.scales_of(scales, *(v.shape[0], v.shape[1] // 32)), v, t, E4M3, what)

    def product(got, a, c, what):
        v, t = ref.product(a, c)
        nref.assert_within(nref.f64(got), v, ref.bf16_tol(v, t + 2 ** -23 * np.abs(v)), what)

    # the norm, of the stored sum
    assert torch.equal(n.sum, (x.float() + res.float()).bfloat16())
    s, ww = nref.f64(n.sum), nref.f64(weight)
    v, _, rstd, xh = nref.norm_forward(s, ww, 0.0, True, 1e-5)
    t = np.abs(ww) * nref.tol_xhat(s, rstd, xh) + 2 * nref.U * np.abs(xh * ww)
    mx(n.q.q_row, n.q.s_row, v, t, "norm row")
    mx(n.q.q_colT[:, :tokens], n.q.s_col, v.T, t.T, "norm col")
    # gate|up and h, from the norm's codes
    pad = ref.up(ffn, 128)
    at = np.concatenate([np.arange(ffn), pad + np.arange(ffn)])
    wv = mx_value(gu.q_row, gu.s_row, (at, 2 * pad))
    xv = mx_value(n.q.q_row, n.q.s_row)
    (g, tg), (u, tu) = (ref.product(xv, w) for w in (wv[:ffn], wv[ffn:]))
    h, th = ref.swiglu(g, tg, u, tu)
    mx(f.q.q_row, f.q.s_row, h, th, "h row")
    mx(f.q.q_colT[:, :tokens], f.q.s_col, h.T, th.T, "h col")
    ref.check_kept(f.checkpoint, (g, u), (tg, tu), "gate|up")
    # the down projection and its gradients
    product(y, mx_value(f.q.q_row, f.q.s_row), mx_value(down.q_row, down.s_row), "y")
    product(dw_down, mx_value(qd.q_colT[:, :tokens], qd.s_col), mx_value(f.q.q_colT[:, :tokens], f.q.s_col), "dW_down")
    kg, ku = np.split(nref.restore(f.checkpoint.q, f.checkpoint.s, ffn, 2, E4M3), 2, 1)
    dh, tdh = ref.product(mx_value(qd.q_row, qd.s_row), mx_value(down.q_colT[:, :hidden], down.s_col))
    dg, tdg, du, tdu = ref.swiglu_backward(kg, ku, dh, tdh)
    row, trow = np.zeros((tokens, 2 * pad)), np.zeros((tokens, 2 * pad))
    row[:, at], trow[:, at] = np.concatenate([dg, du], 1), np.concatenate([tdg, tdu], 1)
    mx(b.q.q_row, b.q.s_row, row, trow, "d_gate|up row")
    mx(b.q.q_colT[:, :tokens], b.q.s_col, row[:, at].T, trow[:, at].T, "d_gate|up col")
    # the gradients of the norm's result and of gate|up's weight
    product(dn, mx_value(b.q.q_row, b.q.s_row), mx_value(gu.q_colT[:, :2 * pad], gu.s_col), "dn")
    product(dw_gu, mx_value(b.q.q_colT[:, :tokens], b.q.s_col), mx_value(n.q.q_colT[:, :tokens], n.q.s_col), "dW")
    # the norm's backward, with the gradient past it
    rs, dy64 = nref.f64(n.rstd), nref.f64(dn)
    xh = s * rs[:, None]
    tx = 3 * nref.U * (np.abs(xh) + rs[:, None] * np.abs(s))
    dx, dw, _ = nref.norm_backward(dy64, xh, rs, ww, True)
    want, t = dx + nref.f64(dres), nref.tol_dx(dx, dy64, xh, rs, ww, tx, True, F32)
    nref.assert_within(nref.f64(d.dx), want, t + nref.U * np.abs(want) + 2.0 ** -8 * (np.abs(want) + t)
                       + nref.TINY[BF16], "dx")
    nref.assert_within(nref.f64(d.dweight), dw, nref.tol_dw(dw, dy64, xh, tx, F32), "dweight")


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("layouts,h,kept", [(0, True, None), (1, False, None), (2, False, "8bit"), (0, False, "bf16"),
                                            (0, False, "8bit")])
def test_few_rows_each_output_alone(mx, layouts, h, kept):
    M, F, K = 1 if mx else 2, 160, 1056
    if mx and layouts & 2:
        layouts = 1  # the transposed layout has 32 rows at least
    x, w = Operand(M, K, E4M3, mx, 1, 1.0), Operand(2 * F, K, E4M3, mx, 2, 0.03, groups=True)
    both = Out(M, F, mx, 1, kept=kept, layouts=1 if mx else 3)
    o = Out(M, F, mx, 1, h=h, kept=kept, layouts=layouts)
    forward(x, w, both)
    forward(x, w, o)
    torch.cuda.synchronize()
    for a, b, on in ((o.q, both.q, layouts & 1), (o.qt, both.qt, layouts & 2), (o.h, both.h, h)):
        if a is not None:
            assert torch.equal(a, b) if on else (a == 0xA5).all()
    if mx:
        assert torch.equal(o.s, both.s) if layouts & 1 else (o.s == 0xA5).all()
    elif layouts:
        assert torch.equal(o.amax, both.amax) and torch.equal(o.inv, both.inv)
    else:
        assert o.amax.item() == both.amax.new_tensor(1e-3).item() and o.inv.item() == -1
    if kept == "8bit":
        assert torch.equal(o.ck.q, both.ck.q) and torch.equal(o.ck.s, both.ck.s)
    if kept == "bf16":
        assert torch.equal(o.gu, both.gu)


@pytest.mark.parametrize("rows,cols,pad", [(37, 1111, 3), (64, 512, 0), (9, 9000, 0)])
def test_norm_backward_with_dsum_and_no_parameter_gradients(rows, cols, pad):
    """dx is that of the call with all gradients, bit for bit, in rows of another stride too."""
    x, dy, dsum = (values(rows, cols, BF16, s, 1.0, 0.0, pad) for s in (20, 21, 22))
    w, _ = params(cols, F32, 23)
    f = fp8.norm_forward(x, w)
    full = fp8.norm_backward(dy, x, f.mean, f.rstd, w, dsum=dsum)
    out = torch.full((rows, cols + 8), 7.0, dtype=BF16, device=DEV)
    r = fp8.norm_backward(dy, x, f.mean, f.rstd, w, weight_grad=False, bias_grad=False, out=out[:, :cols], dsum=dsum)
    torch.cuda.synchronize()
    assert r.dweight is None and r.dbias is None and full.dbias is not None
    assert torch.equal(out[:, :cols], full.dx) and (out[:, cols:] == 7).all()


@pytest.mark.parametrize("M", [1, 3])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_scales_far_apart(fmt, M):
    """A's and W's scale bytes over their whole range, each block's product of scales 1: a
    few-row kernel that scales A first must not leave fp32 on the way."""
    F, K = 160, 1056
    rng = np.random.RandomState(6)
    byte = rng.randint(0, 255, K // 32)
    byte[:3] = 254, 0, 250
    ops = []
    for rows, b in ((M, byte), (2 * F, 254 - byte)):
        q, _ = ref.mx_quantize(rng.randn(rows, K), fmt)
        q[:, 64:96] = 0  # zeros of W under A's byte 250
        s = np.broadcast_to(b, (rows, K // 32)).astype(np.uint8)
        v = nref.decode_table(fmt)[q.numpy()] * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)
        if rows == 2 * F:
            h = np.zeros((2, ref.up(F, 128), K // 32), np.uint8)
            h[:, :F] = s.reshape(2, F, -1)
            s = h.reshape(-1, K // 32)
        ops.append(SimpleNamespace(q=q.to(DEV), s=ref.layout_of(s).to(DEV), v=v, fmt=fmt, ld=K))
    x, w = ops
    o = Out(M, F, True, 1, kept="bf16", layouts=1)
    forward(x, w, o)
    torch.cuda.synchronize()
    check_forward(x, w, o, f"{M} rows")
