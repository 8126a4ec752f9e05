"""GPU tests of the norm's forward and backward against the float64 reference
(tolerances derived in norm_ref), with and without the 8-bit checkpoint."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import norm_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = [fp8.LAYER_NORM, fp8.RMS_NORM]
PAIRS = [(BF16, BF16), (F16, F16), (F32, F32), (F32, BF16), (F32, F16)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


def values(rows, cols, dtype, seed, scale=1.0, shift=0.0, pad=0, offset=0):
    """A [rows, cols] device tensor in rows of cols + pad, `offset` elements
    into its buffer; the rest of the buffer holds NaN."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=dtype, device=DEV)
    x = buf[offset:].view(rows, cols + pad)[:, :cols]
    x.copy_((torch.randn((rows, cols), generator=g) * scale + shift).to(dtype))
    return x


def empty_like_padded(rows, cols, dtype, pad):
    """An output view whose padding must stay as it is (7)."""
    buf = torch.full((rows, cols + pad), 7.0, dtype=dtype, device=DEV)
    return buf, buf[:, :cols]


def params(cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(dtype).to(DEV)
    b = (0.2 * torch.randn(cols, generator=g)).to(dtype).to(DEV)
    return w, b


def check_forward(x, w, b, kind, eps, out_dtype, fmt=None, out=None, what=""):
    f = fp8.norm_forward(x, w, b, kind=kind, eps=eps, out_dtype=out_dtype, checkpoint_fmt=fmt, out=out)
    torch.cuda.synchronize()
    rms = kind == fp8.RMS_NORM
    xx = ref.f64(x)
    ww = ref.f64(w) if w is not None else 1.0
    bb = ref.f64(b) if b is not None else 0.0
    y, mean, rstd, xh = ref.norm_forward(xx, ww, bb, rms, eps)
    ref.assert_within(ref.f64(f.y), y, ref.tol_y(y, xx, rstd, xh, ww, bb, f.y.dtype), what + " y")
    ref.assert_within(ref.f64(f.rstd), rstd, rstd * ref.D * ref.U + np.abs(rstd) ** 2 * ref.D * ref.U
                      * np.abs(xx).mean(1), what + " rstd")
    if rms:
        assert f.mean is None
    else:
        ref.assert_within(ref.f64(f.mean), mean, ref.D * ref.U * np.abs(xx).mean(1), what + " mean")
    if fmt is not None:
        c = f.checkpoint
        got = ref.restore(c.q, c.s, x.shape[1], 1, fmt)
        tx = ref.tol_xhat(xx, rstd, xh)
        # half a step of a normal element, or of the subnormal grid of its block
        unit = np.repeat(np.exp2(c.s.cpu().numpy().astype(np.float64) - 127), 32, 1)[:, :x.shape[1]]
        rel, sub = (2.0 ** -4, 2.0 ** -10) if fmt == 0 else (2.0 ** -3, 2.0 ** -17)
        ref.assert_within(got, xh, np.maximum(rel * (np.abs(xh) + tx), sub * unit) + tx, what + " checkpoint")
        pad = c.q.cpu().numpy()[:, x.shape[1]:]
        assert not pad.any(), what + " codes past the columns"
    return f


def check_backward(dy, src, f, w, kind, x=None, dx_dtype=None, out=None, what="", xh=None):
    rms = kind == fp8.RMS_NORM
    r = fp8.norm_backward(dy, src, f.mean, f.rstd, w, kind=kind, dx_dtype=dx_dtype, out=out)
    torch.cuda.synchronize()
    d = ref.f64(dy)
    rstd = ref.f64(f.rstd)
    ww = ref.f64(w) if w is not None else 1.0
    if xh is None:
        if x is None:
            xh = ref.restore(src.q, src.s, dy.shape[1], 1, src.fmt)
            tx = np.zeros_like(xh)
        else:
            xx = ref.f64(x)
            xh = (xx - (0.0 if rms else ref.f64(f.mean)[:, None])) * rstd[:, None]
            tx = 3 * ref.U * np.abs(xh) + ref.U * np.abs(xx) * rstd[:, None]
    dx, dw, db = ref.norm_backward(d, xh, rstd, ww, rms)
    ref.assert_within(ref.f64(r.dx), dx, ref.tol_dx(dx, d, xh, rstd, ww, tx, rms, r.dx.dtype), what + " dx")
    ref.assert_within(ref.f64(r.dweight), dw, ref.tol_dw(dw, d, xh, tx, r.dweight.dtype), what + " dw")
    if rms:
        assert r.dbias is None
    else:
        ref.assert_within(ref.f64(r.dbias), db, ref.tol_db(db, d, r.dbias.dtype), what + " db")
    return r


COLS = [1, 2, 8, 31, 32, 33, 100, 255, 256, 257, 520, 1000, 1024, 1111, 2048, 2056, 4095, 4096, 5000, 7168, 8192,
        12288, 16384, 20480]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", COLS)
def test_widths(cols, kind):
    """Every width class, contiguous rows, bf16, forward and backward from x
    and from the checkpoint."""
    rows = 37
    x, dy = values(rows, cols, BF16, cols, 1.3, 0.2), values(rows, cols, BF16, cols + 1, 0.05)
    w, b = params(cols, BF16, cols + 2)
    b = b if kind == fp8.LAYER_NORM else None
    for fmt in (None, 0):
        f = check_forward(x, w, b, kind, 1e-5, None, fmt, what=f"{cols}")
        check_backward(dy, x if fmt is None else f.checkpoint, f, w, kind, x if fmt is None else None, what=f"{cols}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [8200, 16385, 16392, 24000, 32768, 32769, 40001, 65536])
def test_rows_shared_by_a_cluster(cols, kind):
    """Widths that two, four and eight blocks share, aligned or not, in bf16
    and with an fp32 x, with few and with several rows a cluster."""
    for rows, tx, pad in ((3, BF16, 0), (170, F32, 0), (41, BF16, 24)):
        x, dy = values(rows, cols, tx, cols, 1.3, 0.2, pad), values(rows, cols, BF16, cols + 1, 0.05, 0.0, pad)
        w, b = params(cols, BF16, cols + 2)
        b = b if kind == fp8.LAYER_NORM else None
        f = check_forward(x, w, b, kind, 1e-5, BF16, 0, what=f"{rows} x {cols}")
        check_backward(dy, x, f, w, kind, x, what=f"{rows} x {cols} from x")
        check_backward(dy, f.checkpoint, f, w, kind, dx_dtype=tx, what=f"{rows} x {cols} from the checkpoint")


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("wt", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(5, 96, 0, 0), (33, 1000, 8, 0), (9, 4096, 3, 1), (12, 7171, 5, 0)])
def test_types_and_strides(pair, wt, shape):
    """Types of x, y and the parameters; padded rows and bases that no vector
    access fits.  Padding is read by nothing (it is NaN) and not written."""
    rows, cols, pad, offset = shape
    tx, ty = pair
    x = values(rows, cols, tx, 3, 2.0, -0.5, pad, offset)
    dy = values(rows, cols, ty, 4, 0.3, 0.0, pad, offset)
    w, b = params(cols, wt, 5)
    for kind in KINDS:
        buf, y = empty_like_padded(rows, cols, ty, pad)
        f = check_forward(x, w, b, kind, 1e-6, ty, 1, out=y, what=f"{shape}")
        assert bool((buf[:, cols:] == 7).all())
        buf, dx = empty_like_padded(rows, cols, tx, pad)
        check_backward(dy, x, f, w, kind, x, out=dx, what=f"{shape} from x")
        assert bool((buf[:, cols:] == 7).all())
        buf, dx = empty_like_padded(rows, cols, tx, pad)
        check_backward(dy, f.checkpoint, f, w, kind, out=dx, what=f"{shape} from the checkpoint")
        assert bool((buf[:, cols:] == 7).all())


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 151, 153, 609, 1300, 4500])
@pytest.mark.parametrize("cols", [64, 1024, 4096])
def test_row_counts(rows, cols):
    """From one row to several per resident block."""
    x, dy = values(rows, cols, BF16, rows, 1.0, 0.1), values(rows, cols, BF16, rows + 1, 0.05)
    w, b = params(cols, F32, 2)
    f = check_forward(x, w, b, fp8.LAYER_NORM, 1e-5, None, what=f"{rows}")
    check_backward(dy, x, f, w, fp8.LAYER_NORM, x, what=f"{rows}")


@pytest.mark.parametrize("cols", [8, 40, 272, 1000, 2056, 4616, 7168])
def test_two_rows_a_step_with_short_last_blocks(cols):
    """Enough rows for every step of the backward to hold two, at widths whose
    last block of 32 columns has only its first lane's half."""
    rows = 700
    x, dy = values(rows, cols, BF16, cols, 1.3, 0.2), values(rows, cols, BF16, cols + 1, 0.05)
    w, b = params(cols, F32, cols + 2)
    f = check_forward(x, w, b, fp8.LAYER_NORM, 1e-5, None, 0, what=f"{cols}")
    check_backward(dy, x, f, w, fp8.LAYER_NORM, x, what=f"{cols} from x")
    check_backward(dy, f.checkpoint, f, w, fp8.LAYER_NORM, what=f"{cols} from the checkpoint")


@pytest.mark.parametrize("cols", [100, 4096])
def test_no_parameters(cols):
    """Without weight and bias y is xh, and the gradients are fp32."""
    x, dy = values(20, cols, BF16, 1), values(20, cols, BF16, 2)
    for kind in KINDS:
        f = check_forward(x, None, None, kind, 1e-5, None, 0)
        r = check_backward(dy, x, f, None, kind, x)
        assert r.dweight.dtype == F32
        r = fp8.norm_backward(dy, x, f.mean, f.rstd, None, kind=kind, weight_grad=False, bias_grad=False)
        assert r.dweight is None and r.dbias is None


def test_bias_only_and_gradient_selection():
    x, dy = values(20, 96, BF16, 1), values(20, 96, BF16, 2)
    w, b = params(96, F32, 3)
    check_forward(x, None, b, fp8.LAYER_NORM, 1e-5, None)
    f = check_forward(x, w, b, fp8.LAYER_NORM, 1e-5, None)
    full = fp8.norm_backward(dy, x, f.mean, f.rstd, w)
    only_w = fp8.norm_backward(dy, x, f.mean, f.rstd, w, bias_grad=False)
    only_b = fp8.norm_backward(dy, x, f.mean, f.rstd, w, weight_grad=False)
    assert only_w.dbias is None and only_b.dweight is None
    assert torch.equal(only_w.dweight, full.dweight) and torch.equal(only_b.dbias, full.dbias)
    assert torch.equal(only_w.dx, full.dx) and torch.equal(only_b.dx, full.dx)


@pytest.mark.parametrize("cols", [96, 4096, 4099])
def test_empty(cols):
    """No rows: empty outputs, gradients of zero."""
    x = torch.empty((0, cols), dtype=BF16, device=DEV)
    w, b = params(cols, F32, 3)
    f = fp8.norm_forward(x, w, b, checkpoint_fmt=0)
    assert f.y.shape == (0, cols) and f.rstd.shape == (0,)
    for src in (x, f.checkpoint):
        torch.full((1 << 20,), float("nan"), device=DEV)   # what the workspace may have held
        r = fp8.norm_backward(x, src, f.mean, f.rstd, w)
        assert r.dx.shape == (0, cols) and not r.dweight.any() and not r.dbias.any()


@pytest.mark.parametrize("cols", [33, 4096])
def test_degenerate_rows(cols):
    """Constant and zero rows give xh = 0 (RMS: x itself over its size), a row
    with NaN or Inf is NaN alone, and its checkpoint restores as NaN."""
    x = values(8, cols, F32, 5)
    x[0] = 0
    x[1] = 3.0
    x[2] = -1e-20
    x[3, 7] = float("nan")
    x[4, 2] = float("inf")
    w, b = params(cols, F32, 6)
    for kind in KINDS:
        f = check_forward(x[[0, 1, 2, 5, 6, 7]], w, b, kind, 1e-5, None)
        f = fp8.norm_forward(x, w, b, kind=kind, checkpoint_fmt=0)
        assert torch.isfinite(f.y[[0, 1, 2, 5, 6, 7]]).all()
        assert torch.isnan(f.y[3]).all()
        if kind == fp8.LAYER_NORM:
            assert torch.isnan(f.y[4]).all() and torch.equal(f.y[0], b)
        back = ref.restore(f.checkpoint.q, f.checkpoint.s, cols, 1, 0)
        assert np.isnan(back[3]).all() and np.isfinite(back[[0, 1, 2, 5, 6, 7]]).all()
        dy = values(8, cols, F32, 7)
        for src in (x, f.checkpoint):
            r = fp8.norm_backward(dy, src, f.mean, f.rstd, w, kind=kind)
            assert torch.isfinite(r.dx[[0, 1, 2, 5, 6, 7]]).all() and torch.isnan(r.dx[3]).all()


def test_large_mean():
    """Rows far from zero: the spread of 0.1 around 1000 is resolved to what
    fp32 holds of x (E[x^2] - mean^2 would have nothing left)."""
    x = values(16, 4096, F32, 5, 0.1, 1000.0)
    w, b = params(4096, F32, 6)
    f = check_forward(x, w, b, fp8.LAYER_NORM, 1e-5, None)
    _, _, rstd, _ = ref.norm_forward(ref.f64(x), 1.0, 0.0, False, 1e-5)
    assert np.abs(ref.f64(f.rstd) / rstd - 1).max() < 1e-5


def test_gradient_is_the_forwards_difference():
    """dx and dweight against central differences of the float64 forward (a
    formula apart from the backward's)."""
    rows, cols = 3, 24
    for kind in KINDS:
        x, dy = values(rows, cols, F32, 8), values(rows, cols, F32, 9)
        w, b = params(cols, F32, 10)
        f = fp8.norm_forward(x, w, b, kind=kind, eps=1e-3)
        r = fp8.norm_backward(dy, x, f.mean, f.rstd, w, kind=kind)
        xx, dd, ww = ref.f64(x), ref.f64(dy), ref.f64(w)
        loss = lambda a, v: (ref.norm_forward(a, v, 0.0, kind == fp8.RMS_NORM, 1e-3)[0] * dd).sum()  # noqa: E731
        for i in np.ndindex(rows, cols):
            e = np.zeros_like(xx)
            e[i] = 1e-5
            num = (loss(xx + e, ww) - loss(xx - e, ww)) / 2e-5
            # differences: 1e-8; the fp32 kernel: tens of u times magnitudes of order one to ten
            assert abs(num - float(r.dx[i])) < 2e-5
        for j in range(cols):
            e = np.zeros_like(ww)
            e[j] = 1e-5
            num = (loss(xx, ww + e) - loss(xx, ww - e)) / 2e-5
            assert abs(num - float(r.dweight[j])) < 2e-5


@pytest.mark.parametrize("shape", [(300, 4096), (300, 1111), (40, 16384)])
def test_same_bits_every_time(shape):
    x, dy = values(*shape, BF16, 1), values(*shape, BF16, 2)
    w, b = params(shape[1], F32, 3)
    f = fp8.norm_forward(x, w, b, checkpoint_fmt=0)
    first = fp8.norm_backward(dy, f.checkpoint, f.mean, f.rstd, w)
    for _ in range(3):
        r = fp8.norm_backward(dy, f.checkpoint, f.mean, f.rstd, w)
        assert torch.equal(r.dx, first.dx) and torch.equal(r.dweight, first.dweight)
        assert torch.equal(r.dbias, first.dbias)


def test_other_stream():
    """A call on a stream of its own while the current one churns through
    allocations: outputs and workspace belong to the call's stream."""
    x, dy = values(2000, 4096, BF16, 1), values(2000, 4096, BF16, 2)
    w, b = params(4096, F32, 3)
    want = fp8.norm_forward(x, w, b, checkpoint_fmt=0)
    back = fp8.norm_backward(dy, want.checkpoint, want.mean, want.rstd, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        for _ in range(5):
            f = fp8.norm_forward(x, w, b, checkpoint_fmt=0, stream=handle)
            r = fp8.norm_backward(dy, f.checkpoint, f.mean, f.rstd, w, stream=handle)
            for _ in range(20):
                torch.full((1 << 22,), float("nan"), device=DEV)
            side.synchronize()
            assert torch.equal(f.y, want.y) and torch.equal(f.checkpoint.q, want.checkpoint.q)
            assert torch.equal(r.dx, back.dx) and torch.equal(r.dweight, back.dweight)
    torch.cuda.synchronize()


def test_graph_capture():
    x, dy = values(300, 4096, BF16, 1), values(300, 4096, BF16, 2)
    w, b = params(4096, F32, 3)
    f = fp8.norm_forward(x, w, b)
    r = fp8.norm_backward(dy, x, f.mean, f.rstd, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2 = fp8.norm_forward(x, w, b)
        r2 = fp8.norm_backward(dy, x, f2.mean, f2.rstd, w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f.y, f2.y) and torch.equal(r.dx, r2.dx) and torch.equal(r.dweight, r2.dweight)


@pytest.mark.parametrize("cols", [4096, 4099])
def test_offsets_past_32_bits(cols):
    """Rows whose element offsets pass 2^32: a stride of 2^27 + 32 elements."""
    rows, ld = 40, (1 << 27) + 32
    x = torch.empty(rows * ld, dtype=BF16, device=DEV).view(rows, ld)[:, :cols]
    dy = torch.empty(rows * ld, dtype=BF16, device=DEV).view(rows, ld)[:, :cols]
    xs, dys = values(rows, cols, BF16, 1), values(rows, cols, BF16, 2)
    x.copy_(xs)
    dy.copy_(dys)
    w, b = params(cols, F32, 3)
    f, want = fp8.norm_forward(x, w, b), fp8.norm_forward(xs, w, b)
    assert torch.equal(f.rstd, want.rstd) or (f.rstd - want.rstd).abs().max() <= 1e-5 * want.rstd.abs().max()
    big = torch.empty(rows * ld, dtype=BF16, device=DEV).view(rows, ld)[:, :cols]
    r = fp8.norm_backward(dy, x, f.mean, f.rstd, w, out=big)
    s = fp8.norm_backward(dys, xs, f.mean, f.rstd, w)
    torch.cuda.synchronize()
    # the two row strides may take kernels that add in another order: one bf16 rounding apart at most
    assert (f.y.float() - want.y.float()).abs().max() <= 2.0 ** -7 * want.y.float().abs().max()
    assert (r.dx.float() - s.dx.float()).abs().max() <= 2.0 ** -7 * s.dx.float().abs().max()
    del x, dy, big, r, f
    torch.cuda.empty_cache()


def test_refusals():
    x = values(8, 64, BF16, 1)
    w, b = params(64, BF16, 2)
    f = fp8.norm_forward(x, w, b, checkpoint_fmt=0)

    def refused(fn, *a, **k):
        with pytest.raises(fp8.Fp8Error):
            fn(*a, **k)

    refused(fp8.norm_forward, x.cpu(), w, b)
    refused(fp8.norm_forward, x.double(), w, b)
    refused(fp8.norm_forward, x, w[:32], b)
    refused(fp8.norm_forward, x, w, b.float())
    refused(fp8.norm_forward, x.t(), None, None)
    refused(fp8.norm_forward, x, w, b, kind=2)
    refused(fp8.norm_forward, x, w, b, eps=-1.0)
    refused(fp8.norm_forward, x, w, b, eps=float("nan"))
    refused(fp8.norm_forward, x, w, b, out_dtype=F32)
    refused(fp8.norm_forward, x, w, b, checkpoint_fmt=fp8.E4M3FNUZ)
    refused(fp8.norm_forward, x, w, b, out=torch.empty((8, 32), dtype=BF16, device=DEV))
    refused(fp8.norm_forward, x[:1].expand(8, 64), w, b)
    wide = torch.zeros((1, 65537), dtype=BF16, device=DEV)
    refused(fp8.norm_forward, wide)
    refused(fp8.norm_backward, wide, wide, f.mean[:1], f.rstd[:1])
    dy = values(8, 64, BF16, 3)
    refused(fp8.norm_backward, dy, x, None, f.rstd, w)
    refused(fp8.norm_backward, dy, x[:4], f.mean, f.rstd, w)
    refused(fp8.norm_backward, dy, x, f.mean, f.rstd[:4], w)
    refused(fp8.norm_backward, dy, x, f.mean, f.rstd.half(), w)
    refused(fp8.norm_backward, dy, x, f.mean, f.rstd, w, dx_dtype=F32)
    refused(fp8.norm_backward, dy[:, :32], f.checkpoint, f.mean, f.rstd, w[:32])
    refused(fp8.norm_backward, dy.float(), x, f.mean, f.rstd, w)
    two = fp8.Checkpoint(f.checkpoint.q, f.checkpoint.s, 0, 32, 2)
    refused(fp8.norm_backward, dy, two, f.mean, f.rstd, w)
    # the workspace is checked against what the shape needs
    need = fp8.fp8_norm_workspace_bytes(8, 64)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(64, dtype=BF16, device=DEV)
    rc = fp8.fp8_norm_backward(dy, 0, 64, x, 64, None, 0, None, 0, 0, 8, 64, 0, f.mean, f.rstd, w, 0, dx, 0, 64, dw,
                               None, ws, need - 1, check=False)
    assert fp8.STATUS[rc] == "FP8_ERR_INVALID_ARG"
    torch.cuda.synchronize()
