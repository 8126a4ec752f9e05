"""CPU pins of the references in fused_ref."""
import numpy as np
import pytest
import torch

import fused_ref as ref
import norm_ref as nref
import synth


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (130, 160), (256, 256)])
def test_mx_quantize_is_the_oracles(orc, rows, cols, fmt):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g))).bfloat16()
    x[0, :32] = 0
    want = orc.mx_quantize(synth.bf16_bits(x), fmt, orc.LAYOUT_ROW)
    q, s = ref.mx_quantize(nref.f64(x), fmt)
    assert np.array_equal(q.numpy(), want["q_row"])
    assert np.array_equal(s, want["s_row"])
    assert np.array_equal(ref.scales_of(ref.layout_of(s), rows, cols // 32), s)
    # and is within its own bounds with no error allowed but the rounding's
    ref.check_mx(q, s, nref.f64(x), 0.0, fmt, "self")


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_wrong_code_or_scale_is_found(fmt):
    v = np.random.RandomState(1).randn(4, 64)
    q, s = ref.mx_quantize(v, fmt)
    i = np.abs(v[2]).argmax()  # not a subnormal: one code further is a step off
    bad = q.clone()
    bad[2, i] -= 2
    with pytest.raises(AssertionError):
        ref.check_mx(bad, s, v, 1e-6, fmt, "code")
    off = s.copy()
    off[1, 1] += 1
    with pytest.raises(AssertionError):
        ref.check_mx(q, off, v, 1e-6, fmt, "scale")


def test_swiglu_bounds_hold_for_fp32_arithmetic():
    r = np.random.RandomState(2)
    g, u, dh = (r.randn(20000).astype(np.float32) * s for s in (4, 2, 0.1))
    h, t = ref.swiglu(g.astype(np.float64), 0.0, u.astype(np.float64), 0.0)
    s32 = 1 / (1 + np.exp(-g))
    assert (np.abs(g * s32 * u - h) <= t).all()
    dg, tg, du, tu = ref.swiglu_backward(g.astype(np.float64), u.astype(np.float64), dh.astype(np.float64), 0.0)
    assert (np.abs(dh * u * s32 * (1 + g * (1 - s32)) - dg) <= tg).all()
    assert (np.abs(dh * g * s32 - du) <= tu).all()


def test_swiglu_gradients_are_the_differences_of_h():
    r = np.random.RandomState(3)
    g, u, dh = r.randn(500) * 3, r.randn(500), r.randn(500)
    dg, _, du, _ = ref.swiglu_backward(g, u, dh, 0.0)
    e = 1e-6
    f = lambda g, u: ref.swiglu(g, 0.0, u, 0.0)[0]  # noqa: E731
    assert np.allclose(dh * (f(g + e, u) - f(g - e, u)) / (2 * e), dg, rtol=1e-6, atol=1e-8)
    assert np.allclose(dh * (f(g, u + e) - f(g, u - e)) / (2 * e), du, rtol=1e-6, atol=1e-8)
