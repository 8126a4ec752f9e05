"""GPU tests of the norms into 8 bits and of the SwiGLU products at their edges: rows
without a finite norm beside the padding, no rows."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import fused_ref as ref
import norm_ref as nref
import test_gpu_norm_quantize as nq
from test_gpu_norm import values

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = fp8.E4M3FN
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


@pytest.mark.parametrize("cols,dtype,pad", [(160, BF16, 0), (160, F32, 0), (96, BF16, 3), (224, F16, 0), (32, F32, 1),
                                            (20512, BF16, 0)])
@pytest.mark.parametrize("kind", [fp8.LAYER_NORM, fp8.RMS_NORM])
@pytest.mark.parametrize("what", ["nan", "inf", "eps 0"])
def test_padding_beside_rows_without_a_finite_norm(what, kind, cols, dtype, pad):
    """Widths that are no multiple of 128: the scale bytes behind the data are 0 (scales_of
    asserts it) whatever the rows hold.  With eps = 0 a row of zeros is 0 times Inf."""
    x = values(64, cols, dtype, 41, 1.0, 0.25, pad)
    if what == "eps 0":
        x[40] = 0
    else:
        x[40, 7] = float(what)
    eps = 0.0 if what == "eps 0" else 1e-5
    o = nq.Out(64, cols, None, True, pad)
    nq.call(x, None, None, None, kind, eps, nq.MX, 3, E4M3, o)
    torch.cuda.synchronize()
    v, rms = nref.f64(x), kind == fp8.RMS_NORM
    with np.errstate(all="ignore"):
        y, _, rstd, xh = nref.norm_forward(v, 1.0, 0.0, rms, eps)
        tol = nref.tol_xhat(v, rstd, xh) + 2 * nref.U * np.abs(xh)
    tol = np.where(np.isfinite(tol), tol, 0.0)  # of row 40 only: what is finite there is 0 exactly
    assert np.isfinite(np.delete(y, 40, 0)).all() and not np.isfinite(y[40]).all()
    ref.check_mx(o.q, ref.scales_of(o.s, 64, cols // 32), y, tol, E4M3, "row")
    ref.check_mx(o.qt[:, :64], ref.scales_of(o.st, cols, 2), y.T, tol.T, E4M3, "col")


def delayed():
    return dict(scale_in=torch.tensor([2.5], device=DEV), amax_out=torch.tensor([0.125], device=DEV))


def used_memory():
    """Small blocks of NaN left to the allocator, so that what is not written shows."""
    for t in [torch.full((128,), float("nan"), device=DEV) for _ in range(64)]:
        del t


@pytest.mark.parametrize("layouts", [1, 2, 3])
def test_no_rows_have_the_stored_scale(layouts):
    """The inverse scale follows from the stored one alone."""
    x, e = torch.empty((0, 64), dtype=BF16, device=DEV), torch.empty((0, 64), dtype=torch.uint8, device=DEV)
    w, one = torch.zeros((64, 64), dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV)
    src = torch.empty((0, 128), dtype=BF16, device=DEV)
    calls = [lambda **k: fp8.norm_quantize(x, recipe=fp8.Recipe(kind=fp8.DELAYED), layouts=layouts, **k),
             lambda **k: fp8.swiglu_gemm(e, E4M3, w, E4M3, one, one, fmt=E4M3, layouts=layouts, **k),
             lambda **k: fp8.swiglu_gemm_backward(e, E4M3, w, E4M3, one, one, src, fmt=E4M3, layouts=layouts, **k)]
    for call in calls:
        used_memory()
        d = delayed()
        q = call(**d).q
        for s, on in ((q.scale_inv_row, layouts & 1), (q.scale_inv_col, layouts & 2)):
            assert s.item() == np.float32(1) / np.float32(2.5) if on else s is None
        assert d["amax_out"].item() == 0.125
        with pytest.raises(fp8.Fp8Error):
            call(amax_out=d["amax_out"])


@pytest.mark.parametrize("h,gate_up", [(True, False), (False, True)])
def test_no_rows_of_rowwise_operands(h, gate_up):
    """What a rowwise quantize of no rows leaves goes into the products."""
    n = fp8.norm_quantize(torch.empty((0, 64), dtype=BF16, device=DEV), kind=fp8.RMS_NORM)
    assert n.q.scale_inv_row.numel() == 0
    w, sw = torch.zeros((64, 64), dtype=torch.uint8, device=DEV), torch.ones(64, device=DEV)
    f = fp8.swiglu_gemm(n.q.q_row, E4M3, w, E4M3, n.q.scale_inv_row, sw, h=h, gate_up=gate_up)
    assert (f.h if h else f.gate_up).shape == (0, 32 if h else 64)
    b = fp8.swiglu_gemm_backward(n.q.q_row, E4M3, w, E4M3, n.q.scale_inv_row, sw,
                                 torch.empty((0, 128), dtype=BF16, device=DEV), d_gate_up=True)
    assert b.d_gate_up.shape == (0, 128)
    # no scales are no scales of rows that there are
    with pytest.raises(fp8.Fp8Error):
        fp8.swiglu_gemm(w, E4M3, w, E4M3, n.q.scale_inv_row, sw, h=True)
