"""The float64 references of the norm, SwiGLU and checkpoint tests, checked on
the CPU: gradients against central differences of the forward, the checkpoint
rule against the format's definition and torch's own fp8 conversion."""
import numpy as np
import pytest
import torch

import norm_ref as ref


def central(f, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        out[i] = (f(a) - f(b)) / (2 * step)
    return out


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("cols", [2, 7])
def test_norm_gradients_are_differences(rms, cols):
    rng = np.random.default_rng(cols)
    x, dy = rng.normal(size=(3, cols)), rng.normal(size=(3, cols))
    w, b = rng.normal(size=cols), rng.normal(size=cols)
    eps = 0.1   # keeps a two-column row's statistics smooth
    loss = lambda x_, w_, b_: float((ref.norm_forward(x_, w_, b_, rms, eps)[0] * dy).sum())  # noqa: E731
    _, _, rstd, xh = ref.norm_forward(x, w, b, rms, eps)
    dx, dw, db = ref.norm_backward(dy, xh, rstd, w, rms)
    # central differences of step 1e-6 in float64: truncation 1e-12, cancellation 1e-10
    np.testing.assert_allclose(dx, central(lambda v: loss(v, w, b), x), atol=1e-7)
    np.testing.assert_allclose(dw, central(lambda v: loss(x, v, b), w), atol=1e-7)
    np.testing.assert_allclose(db, central(lambda v: loss(x, w, v), b), atol=1e-7)


def test_swiglu_gradients_are_differences():
    rng = np.random.default_rng(1)
    g, u, dh = (rng.normal(size=40) * 4 for _ in range(3))
    dg, du = ref.swiglu_backward(g, u, dh)
    np.testing.assert_allclose(dg, central(lambda v: float((ref.swiglu(v, u) * dh).sum()), g), atol=1e-6)
    np.testing.assert_allclose(du, central(lambda v: float((ref.swiglu(g, v) * dh).sum()), u), atol=1e-6)


@pytest.mark.parametrize("fmt", [0, 1])
def test_checkpoint_rule(fmt):
    """Scales are the smallest powers of two that hold the block, elements are
    torch's round-to-nearest-even conversion, blocks beside NaN are untouched."""
    rng = np.random.default_rng(fmt)
    x = rng.normal(size=(64, 3 * 32)) * np.exp2(rng.integers(-30, 30, size=(64, 1)))
    x[0, :32] = 0
    x[1, 5] = np.nan
    x[2, 40] = np.inf
    x[3, :32] = ref.FMAX[fmt]              # exactly representable at e = 0
    x[4, 0] = ref.FMAX[fmt] * 1.0625       # one more
    x[4, 1:32] = 0
    t, s = ref.checkpoint(x, 1, fmt)
    assert s[0, 0] == 0 and s[1, 0] == 255 and s[2, 1] == 255 and s[1, 1] != 255 and s[2, 0] != 255
    assert s[3, 0] == 127 and s[4, 0] == 128
    ok = s < 255
    amax = np.abs(np.nan_to_num(x, posinf=0)).reshape(64, 3, 32).max(-1)
    e = s - 127.0
    nz = ok & (amax > 0)
    assert (amax[nz] <= ref.FMAX[fmt] * np.exp2(e[nz])).all() and (amax[nz] > ref.FMAX[fmt] * np.exp2(e[nz] - 1)).all()
    blocks = np.nan_to_num(x, posinf=0).reshape(64, 3, 32)
    want = torch.from_numpy((blocks * np.exp2(-e)[..., None])[ok]).to(ref.TORCH_FP8[fmt]).double().numpy()
    assert np.array_equal(t.reshape(64, 3, 32)[ok], want)
