"""Host-only checks that a sum, dx or d_gate_up_bf16 that starts where any input of
its call does is refused before anything touches a device."""
import ctypes

import pytest

import fp8_mixed_precision_scale_gb300 as fp8
from fp8_mixed_precision_scale_gb300 import build as fp8build
from test_abi_fused import BACK, BACKWARD, NORM, NORM_ORDER, P

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    fp8build.build()
    return fp8.load_library()


def caller(lib, name, order, base):
    """The entry point with every pointer of `base` (1 for one, None for none) at an address of its own."""
    order, fn = order.split(), getattr(lib, name)
    assert len(order) == len(fn.argtypes)
    at = {k: 0x100000 * (i + 1) for i, (k, t) in enumerate(zip(order, fn.argtypes)) if t is P and k != "stream"}

    def call(same=None, **kw):
        a = dict(base, **kw)
        rec = fp8.fp8_recipe_t(a.get("rkind", 2), 0, 1, 0)
        v = {k: at[k] if k in at and a[k] is not None else a[k] for k in order if k != "recipe"}
        if same is not None:
            v[same[0]] = v[same[1]]
            assert v[same[0]] is not None
        v["recipe"] = ctypes.byref(rec)
        return fn(*[P(v[k]) if t is P else v[k] for k, t in zip(order, fn.argtypes)])
    return call


@pytest.mark.parametrize("name", ["x", "res", "w", "b", "scale"])
@pytest.mark.parametrize("mx", [False, True])
def test_sum(lib, mx, name):
    base = dict(NORM, b=1, mean=1)
    if mx:
        if name == "scale":
            pytest.skip("no stored scale")
        c = caller(lib, "fp8_mx_norm_quantize", NORM_ORDER + "layouts q sr qt ld_t sc stream", base)
    else:
        c = caller(lib, "fp8_norm_quantize", NORM_ORDER + "recipe layouts scale amax q sr qt ld_t sc stream",
                   dict(base, rkind=0, scale=1, amax=1))
    assert c(("sum", name)) == INVALID


RESIDUAL = "dy yt ld_dy x ld_x q ld_q s ld_s fmt dsum ld_d rows cols kind mean rstd w wt dx xt ld_dx dw db ws wsb stream"


@pytest.mark.parametrize("source,name", [("x", n) for n in ("dy", "x", "dsum", "mean", "rstd", "w")] +
                         [("q", n) for n in ("dy", "q", "s", "dsum", "rstd", "w")])
def test_dx(lib, source, name):
    base = dict(dy=1, yt=0, ld_dy=64, x=None, ld_x=64, q=None, ld_q=64, s=None, ld_s=2, fmt=0, dsum=1, ld_d=64,
                rows=4, cols=64, kind=0, mean=1, rstd=1, w=1, wt=2, dx=1, xt=0, ld_dx=64, dw=None, db=None, ws=None,
                wsb=0, stream=None)
    base.update(dict(x=1) if source == "x" else dict(q=1, s=1))
    assert caller(lib, "fp8_residual_norm_backward", RESIDUAL, base)(("dx", name)) == INVALID


@pytest.mark.parametrize("kept,name", [("gu", n) for n in ("A", "W", "sA", "sW", "gu", "scale")] +
                         [("cq", n) for n in ("A", "W", "sA", "sW", "cq", "cs", "scale")])
@pytest.mark.parametrize("mx", [False, True])
def test_d_gate_up(lib, mx, kept, name):
    if mx and name == "scale":
        pytest.skip("no stored scale")
    base = dict(BACK, gu=None, d=1, ld_d=128)
    base.update(dict(gu=1, ld_gu=128) if kept == "gu" else dict(cq=1, cs=1, ld_cq=128, ld_cs=4))
    assert caller(lib, *BACKWARD[mx], base)(("d", name)) == INVALID
