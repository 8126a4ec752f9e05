"""GPU tests of the residual norms into 8 bits and of their backward against the
float64 references (bounds derived in fused_ref and norm_ref)."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import fused_ref as ref
import norm_ref as nref
from test_gpu_norm import params, values

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LAYER, RMS = fp8.LAYER_NORM, fp8.RMS_NORM
MX, ROW, TENSOR = "mx", "row", "tensor"
E4M3, E5M2 = fp8.E4M3FN, fp8.E5M2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


class Out:
    """Output buffers filled with 0xA5 (the sum: 7), sized as the header says, the
    transposed layout with 32 columns more."""

    def __init__(self, rows, cols, rdtype, mx, pad):
        full = lambda n: torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.ld_t = ref.up(max(rows, 1), 16) + 32
        self.q = full(rows * cols)[:rows * cols].view(rows, cols)
        self.qt = full(cols * self.ld_t).view(cols, self.ld_t)
        self.s = full(ref.up(cols // 32, 4) * ref.up(rows, 128)) if mx else torch.full((max(rows, 1),), -1.0, device=DEV)
        self.st = full(ref.up(rows // 32, 4) * ref.up(cols, 128)) if mx else torch.full((1,), -1.0, device=DEV)
        self.mean, self.rstd = torch.full((max(rows, 1),), -1.0, device=DEV), torch.full((max(rows, 1),), -1.0, device=DEV)
        self.sum = None if rdtype is None else torch.full((rows, cols + pad), 7.0, dtype=rdtype, device=DEV)


def call(x, res, w, b, kind, eps, recipe, layouts, fmt, o, scale=None, amax=None, margin=0, stream=None):
    rows, cols = x.shape
    wt = w if w is not None else b
    a = (x, fp8.DTYPES[x.dtype], x.stride(0), res, 0 if res is None else fp8.DTYPES[res.dtype],
         0 if res is None else res.stride(0), rows, cols, kind, eps, w, b, 0 if wt is None else fp8.DTYPES[wt.dtype],
         o.sum, 0 if o.sum is None else o.sum.stride(0), o.mean if kind == LAYER else None, o.rstd, fmt)
    if recipe == MX:
        fp8.fp8_mx_norm_quantize(*a, layouts, o.q, o.s, o.qt, o.ld_t, o.st, stream=stream)
    else:
        rec = fp8.Recipe(kind=fp8.ROWWISE if recipe == ROW else fp8.DELAYED, margin=margin)
        fp8.fp8_norm_quantize(*a, rec, layouts, scale, amax, o.q, o.s if recipe == ROW else o.st, o.qt, o.ld_t, o.st,
                              stream=stream)


def check(x, res, w, b, kind, eps, recipe, layouts, fmt, o, scale=None, amax=None, amax0=0.0, margin=0, what=""):
    """Everything the call wrote, and what it must have left alone."""
    rows, cols = x.shape
    rms = kind == RMS
    t = x
    if res is not None:
        t = (x.float() + res.float()).to(res.dtype)
        assert torch.equal(o.sum[:, :cols].view(torch.uint8), t.view(torch.uint8)), what + " sum"
        assert (o.sum[:, cols:] == 7).all(), what + " behind the sum's rows"
    v = nref.f64(t)
    ww = 1.0 if w is None else nref.f64(w)
    bb = 0.0 if b is None else nref.f64(b)
    y, mean, rstd, xh = nref.norm_forward(v, ww, bb, rms, eps)
    tol = np.abs(ww) * nref.tol_xhat(v, rstd, xh) + 2 * nref.U * (np.abs(xh * ww) + np.abs(bb))
    nref.assert_within(nref.f64(o.rstd[:rows]), rstd, rstd * nref.D * nref.U + rstd ** 2 * nref.D * nref.U
                       * np.abs(v).mean(1), what + " rstd")
    if not rms:
        nref.assert_within(nref.f64(o.mean[:rows]), mean, nref.D * nref.U * np.abs(v).mean(1), what + " mean")
    if recipe == MX:
        if layouts & 1:
            ref.check_mx(o.q, ref.scales_of(o.s, rows, cols // 32), y, tol, fmt, what + " row")
        if layouts & 2:
            ref.check_mx(o.qt[:, :rows], ref.scales_of(o.st, cols, rows // 32), y.T, tol.T, fmt, what + " col")
    elif recipe == ROW:
        top = np.abs(y).max(1)
        inv = nref.f64(o.s[:rows])
        want = np.where(top > 0, top / ref.FMAX[fmt], 1.0) * np.where(top > 0, 2.0 ** margin, 1.0)
        nref.assert_within(inv, want, 4 * nref.U * want + tol.max(1) / ref.FMAX[fmt] * 2.0 ** margin, what + " scales")
        ref.check_scaled(o.q, 1 / inv[:, None], y, tol + 4 * nref.U * np.abs(y), fmt, what + " row")
    else:
        sc = float(scale)
        if layouts & 1:
            ref.check_scaled(o.q, sc, y, tol, fmt, what + " row")
        if layouts & 2:
            ref.check_scaled(o.qt[:, :rows], sc, y.T, tol.T, fmt, what + " col")
        assert abs(float(o.st) - 1 / sc) <= 2 ** -23 / sc
        top = max(np.abs(y).max(), amax0)
        assert abs(float(amax) - top) <= tol.max() + nref.U * top, what + " amax"
    if layouts & 2:
        assert (o.qt[:, rows:] == 0xA5).all(), what + ": bytes behind the transposed rows"
    if not layouts & 1:
        assert (o.q == 0xA5).all()


CASES = [
    # rows, cols, kind, x, residual, weight, recipe, layouts, fmt, pad
    (1, 32, RMS, BF16, BF16, BF16, MX, 1, E4M3, 0),
    (1, 16, LAYER, F16, None, F32, ROW, 1, E4M3, 0),
    (1, 4096, RMS, BF16, BF16, BF16, ROW, 1, E4M3, 0),
    (2, 48, LAYER, BF16, F32, BF16, TENSOR, 3, E4M3, 0),
    (7, 1104, LAYER, F16, F16, F32, TENSOR, 3, E5M2, 2),
    (32, 32, RMS, BF16, BF16, F32, MX, 3, E4M3, 0),
    (32, 160, LAYER, F32, F32, F32, MX, 2, E5M2, 1),
    (33, 112, RMS, BF16, BF16, BF16, ROW, 1, E5M2, 3),
    (96, 4128, LAYER, BF16, BF16, BF16, MX, 3, E4M3, 8),
    (130, 224, RMS, F16, F32, F16, MX, 1, E4M3, 5),
    (129, 8192, RMS, BF16, BF16, BF16, TENSOR, 3, E4M3, 0),
    (160, 1056, LAYER, BF16, F32, F32, MX, 3, E4M3, 7),
    (200, 7168, RMS, BF16, F32, F32, TENSOR, 2, E4M3, 0),
    (65, 96, LAYER, F32, None, None, TENSOR, 3, E4M3, 0),
    (64, 544, RMS, BF16, None, None, MX, 3, E4M3, 0),
    (3, 16400, LAYER, BF16, BF16, BF16, ROW, 1, E4M3, 0),
    (5, 20480, RMS, F16, F16, F16, MX, 1, E4M3, 0),
    (32, 65536, RMS, BF16, BF16, BF16, MX, 3, E4M3, 0),
    (2, 65536, LAYER, F32, F32, F32, ROW, 1, E4M3, 0),
    (1000, 64, RMS, BF16, BF16, F32, ROW, 1, E4M3, 0),
]


@pytest.mark.parametrize("rows,cols,kind,xt,rt,wt,recipe,layouts,fmt,pad", CASES)
def test_forward(rows, cols, kind, xt, rt, wt, recipe, layouts, fmt, pad):
    x = values(rows, cols, xt, 1, 1.0, 0.3, pad)
    res = None if rt is None else values(rows, cols, rt, 2, 2.0, -0.5, pad)
    w, b = (None, None) if wt is None else params(cols, wt, 3)
    if kind == RMS:
        b = None
    o = Out(rows, cols, rt, recipe == MX, pad)
    scale, amax = torch.tensor([60.0], device=DEV), torch.tensor([0.5], device=DEV)
    extra = dict(scale=scale, amax=amax) if recipe == TENSOR else {}
    call(x, res, w, b, kind, 1e-5, recipe, layouts, fmt, o, **extra)
    torch.cuda.synchronize()
    check(x, res, w, b, kind, 1e-5, recipe, layouts, fmt, o, **extra, amax0=0.5,
          what=f"{rows}x{cols}")


@pytest.mark.parametrize("margin", [0, 3, 64])
def test_rowwise_margin_and_zero_rows(margin):
    x = values(5, 64, BF16, 4)
    x[2] = 0
    o = Out(5, 64, None, False, 0)
    call(x, None, None, None, RMS, 1e-5, ROW, 1, E4M3, o, margin=margin)
    torch.cuda.synchronize()
    assert o.s[2] == 1.0 and not (o.q[2] & 0x7F).any()
    check(x, None, None, None, RMS, 1e-5, ROW, 1, E4M3, o, margin=margin)


@pytest.mark.parametrize("what", ["nan", "inf"])
def test_nan_and_inf_stay_in_their_rows(what):
    x, res = values(64, 256, BF16, 5), values(64, 256, BF16, 6)
    x[40, 17] = float(what)
    o = Out(64, 256, BF16, True, 0)
    call(x, res, None, None, RMS, 1e-5, MX, 3, E4M3, o)
    clean = Out(64, 256, BF16, True, 0)
    x[40, 17] = 0
    call(x, res, None, None, RMS, 1e-5, MX, 3, E4M3, clean)
    torch.cuda.synchronize()
    rows = [r for r in range(64) if r != 40]
    assert torch.equal(o.q[rows], clean.q[rows])
    s, c = ref.scales_of(o.s, 64, 8), ref.scales_of(clean.s, 64, 8)
    assert np.array_equal(s[rows], c[rows])
    # a NaN makes the row's statistics NaN, an Inf its reciprocal 0: NaN where it stands
    assert (s[40] == 255).all() if what == "nan" else s[40, 0] == 255 and (s[40, 1:] == 0).all()
    t, tc = ref.scales_of(o.st, 256, 2), ref.scales_of(clean.st, 256, 2)
    assert np.array_equal(t[:, 0], tc[:, 0]) and torch.equal(o.qt[:, :32], clean.qt[:, :32])
    assert (t[:, 1] == 255).all() if what == "nan" else t[17, 1] == 255
    # rowwise: a non-finite largest magnitude gives scale 1
    o = Out(64, 256, None, False, 0)
    x[40, 17] = float(what)
    call(x, None, None, None, RMS, 1e-5, ROW, 1, E4M3, o)
    torch.cuda.synchronize()
    assert o.s[40] == 1.0 and np.isnan(ref.decode(o.q, E4M3)[40, 17])
    assert torch.isfinite(o.s).all()


def test_delayed_amax_takes_a_nan():
    x = values(4, 64, F32, 7)
    x[1, 3] = float("nan")
    o = Out(4, 64, None, False, 0)
    amax = torch.zeros(1, device=DEV)
    call(x, None, None, None, LAYER, 1e-5, TENSOR, 3, E4M3, o, scale=torch.ones(1, device=DEV), amax=amax)
    torch.cuda.synchronize()
    assert torch.isnan(amax).all()


def test_constant_rows_and_eps_zero():
    x = torch.full((32, 96), 3.0, dtype=BF16, device=DEV)
    o = Out(32, 96, None, True, 0)
    call(x, None, None, None, LAYER, 1e-5, MX, 3, E4M3, o)
    torch.cuda.synchronize()
    assert not (o.q & 0x7F).any() and not ref.scales_of(o.s, 32, 3).any()
    assert not ref.scales_of(o.st, 96, 1).any()


def test_no_rows():
    o = Out(0, 64, BF16, True, 0)
    x = torch.empty((0, 64), dtype=BF16, device=DEV)
    n = fp8.mx_norm_quantize(x, x, kind=RMS)
    assert n.q.q_row.shape == (0, 64) and n.sum.shape == (0, 64)
    n = fp8.norm_quantize(x, x, kind=LAYER)
    assert n.q.q_row.shape == (0, 64) and n.mean.numel() == 0
    torch.cuda.synchronize()
    assert (o.q == 0xA5).all()


@pytest.mark.parametrize("layouts", [1, 2, 3])
def test_wrappers(layouts):
    x, res = values(64, 384, BF16, 8), values(64, 384, F32, 9)
    w, b = params(384, F32, 10)
    n = fp8.mx_norm_quantize(x, res, w, b, kind=LAYER, layouts=layouts)
    o = Out(64, 384, F32, True, 0)
    call(x, res, w, b, LAYER, 1e-5, MX, layouts, E4M3, o)
    torch.cuda.synchronize()
    assert torch.equal(n.sum, o.sum) and torch.equal(n.rstd, o.rstd) and torch.equal(n.mean, o.mean)
    if layouts & 1:
        assert torch.equal(n.q.q_row, o.q) and torch.equal(n.q.s_row, o.s)
    if layouts & 2:
        assert torch.equal(n.q.q_colT, o.qt[:, :64]) and torch.equal(n.q.s_col, o.st)
    out = torch.empty_like(res)
    m = fp8.norm_quantize(x, res, w, b, kind=LAYER, out=out)
    assert m.sum is out and torch.equal(out, o.sum)
    assert fp8.norm_quantize(x, kind=RMS).sum is x


def test_replayed_from_a_graph_and_on_another_stream():
    x, res = values(96, 512, BF16, 11), values(96, 512, BF16, 12)
    w, _ = params(512, BF16, 13)
    want = fp8.mx_norm_quantize(x, res, w, kind=RMS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fp8.mx_norm_quantize(x, res, w, kind=RMS, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n = fp8.mx_norm_quantize(x, res, w, kind=RMS)
    for seed in (14, 11):  # other inputs, then the first again
        x.copy_(values(96, 512, BF16, seed))
        g.replay()
    torch.cuda.synchronize()
    for a in (other, n):
        assert torch.equal(a.sum, want.sum) and torch.equal(a.rstd, want.rstd)
        assert torch.equal(a.q.q_row, want.q.q_row) and torch.equal(a.q.s_row, want.q.s_row)
        assert torch.equal(a.q.q_colT, want.q.q_colT) and torch.equal(a.q.s_col, want.q.s_col)


BACK = [
    # rows, cols, kind, sum, dy, weight, checkpoint, pad
    (1, 64, RMS, BF16, BF16, BF16, False, 0),
    (1, 4096, LAYER, F32, BF16, F32, False, 0),
    (37, 1111, LAYER, F16, F16, F32, False, 3),
    (128, 512, RMS, BF16, BF16, BF16, False, 0),
    (70, 7168, LAYER, F32, F32, F32, False, 0),
    (33, 4096, RMS, BF16, BF16, F32, True, 0),
    (21, 200, LAYER, BF16, BF16, BF16, True, 1),
    (9, 9000, RMS, BF16, BF16, BF16, False, 0),
    (9, 9000, LAYER, F32, F16, F32, True, 0),
    (2049, 96, RMS, BF16, BF16, F32, False, 8),
]


@pytest.mark.parametrize("rows,cols,kind,xt,yt,wt,ckpt,pad", BACK)
def test_backward(rows, cols, kind, xt, yt, wt, ckpt, pad):
    x = values(rows, cols, xt, 20, 1.5, 0.25, pad)
    dy, dsum = values(rows, cols, yt, 21, 0.1, 0.0, pad), values(rows, cols, xt, 22, 0.1, 0.0, pad)
    w, _ = params(cols, wt, 23)
    rms = kind == RMS
    f = fp8.norm_forward(x, w, kind=kind, out_dtype=yt, checkpoint_fmt=E4M3 if ckpt else None)
    src = f.checkpoint if ckpt else x
    got = fp8.norm_backward(dy, src, f.mean, f.rstd, w, kind=kind, dx_dtype=xt, dsum=dsum)
    plain = fp8.norm_backward(dy, src, f.mean, f.rstd, w, kind=kind, dx_dtype=xt)
    torch.cuda.synchronize()
    v, rstd = nref.f64(x), nref.f64(f.rstd)
    if ckpt:
        xh, tx = nref.restore(src.q, src.s, cols, 1, E4M3), 0.0
    else:
        xh = (v - (0.0 if rms else nref.f64(f.mean)[:, None])) * rstd[:, None]
        tx = 3 * nref.U * (np.abs(xh) + rstd[:, None] * np.abs(v))
    d64, ww, ds = nref.f64(dy), nref.f64(w), nref.f64(dsum)
    dx, dw, _ = nref.norm_backward(d64, xh, rstd, ww, rms)
    # the bound of dx without its rounding, one fp32 addition, one rounding
    t = nref.tol_dx(dx, d64, xh, rstd, ww, tx + 0 * xh, rms, F32)
    want = dx + ds
    nref.assert_within(nref.f64(got.dx), want, t + nref.U * np.abs(want) + nref.HALF_ULP[xt] * (np.abs(want) + t)
                       + nref.TINY[xt], "dx")
    # the other gradients are the plain backward's, bit for bit
    assert torch.equal(got.dweight, plain.dweight)
    assert (got.dbias is None) == rms and (rms or torch.equal(got.dbias, plain.dbias))
    nref.assert_within(nref.f64(got.dweight), dw, nref.tol_dw(dw, d64, xh, tx + 0 * xh, wt) + 4 * nref.C * nref.U
                       * np.abs(d64 * xh).sum(0), "dweight")


def test_backward_against_differences():
    """d sum of loss(norm(sum) . c) + (sum . e) by central differences in 64 bits."""
    x = values(4, 96, F32, 30, 1.0, 0.5)
    c, e = values(4, 96, F32, 31), values(4, 96, F32, 32)
    w, _ = params(96, F32, 33)
    f = fp8.norm_forward(x, w, kind=LAYER)
    got = nref.f64(fp8.norm_backward(c, x, f.mean, f.rstd, w, kind=LAYER, dsum=e).dx)
    v, ww, cc, ee = (nref.f64(t) for t in (x, w, c, e))

    def loss(v):
        return (nref.norm_forward(v, ww, 0.0, False, 1e-5)[0] * cc + v * ee).sum(1)

    for j in (0, 17, 95):
        d = np.zeros_like(v)
        d[:, j] = 1e-6
        # the differences err by about 1e-9, the kernel by far less than 1e-5 of sums of about 10
        assert np.allclose((loss(v + d) - loss(v - d)) / 2e-6, got[:, j], rtol=0, atol=1e-4)


def test_backward_no_rows_and_refusals():
    e = torch.empty((0, 64), dtype=BF16, device=DEV)
    r = torch.empty(0, dtype=F32, device=DEV)
    b = fp8.norm_backward(e, e, None, r, kind=RMS, dsum=e)
    assert not b.dweight.any()
    x, rs = values(4, 64, BF16, 1), torch.ones(4, device=DEV)
    for bad in (x[:3], x.float(), x[:, :32]):
        with pytest.raises(fp8.Fp8Error):
            fp8.norm_backward(x, x, None, rs, kind=RMS, dsum=bad)


def test_refusals():
    x = values(32, 64, BF16, 1)
    for bad in (dict(residual=x[:4]), dict(residual=x.half()), dict(weight=x[0, :32]), dict(out=x),
                dict(residual=x, out=x.float()), dict(scale_in=x[0, :1])):
        with pytest.raises(fp8.Fp8Error):
            fp8.norm_quantize(x, **bad)
    with pytest.raises(fp8.Fp8Error):
        fp8.norm_quantize(x, layouts=3)
    with pytest.raises(fp8.Fp8Error):
        fp8.norm_quantize(x, recipe=fp8.Recipe(kind=fp8.TENSORWISE))
    with pytest.raises(fp8.Fp8Error):
        fp8.mx_norm_quantize(x[:8], layouts=3)
    with pytest.raises(fp8.Fp8Error):
        fp8.mx_norm_quantize(x[:, :48])
    with pytest.raises(fp8.Fp8Error):
        fp8.mx_norm_quantize(x.cpu())
