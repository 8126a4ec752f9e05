"""Host-only argument checks of the norms into 8 bits and of the SwiGLU products:
each bad call returns its documented status before anything touches a device."""
import ctypes

import pytest

import fp8_mixed_precision_scale_gb300 as fp8
from fp8_mixed_precision_scale_gb300 import build as fp8build

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
FAKE = 0x10000  # aligned and non-null: validation never dereferences it
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    fp8build.build()
    return fp8.load_library()


def caller(lib, name, order, base):
    order = order.split()
    fn = getattr(lib, name)
    assert len(order) == len(fn.argtypes)
    assert set(order) <= set(base) | {"recipe"}

    def call(**kw):
        a = dict(base, **kw)
        rec = fp8.fp8_recipe_t(a.pop("rkind", 2), a.pop("margin", 0), 1, 0)
        a["recipe"] = a.get("recipe", ctypes.byref(rec))
        unknown = set(kw) - set(order) - {"rkind", "margin"}
        assert not unknown, unknown
        return fn(*[P(a[k]) if t is P else a[k] for k, t in zip(order, fn.argtypes)])
    return call


NORM = dict(x=FAKE, xt=0, ld_x=64, res=FAKE, rt=0, ld_r=64, rows=32, cols=64, kind=1, eps=1e-5, w=FAKE, b=None, wt=2,
            sum=FAKE, ld_s=64, mean=None, rstd=FAKE, fmt=0, layouts=1, scale=None, amax=None, q=FAKE, sr=FAKE, qt=FAKE,
            ld_t=32, sc=FAKE, stream=None)
NORM_ORDER = "x xt ld_x res rt ld_r rows cols kind eps w b wt sum ld_s mean rstd fmt "


@pytest.mark.parametrize("mx", [False, True])
def test_norm_quantize_validation(lib, mx):
    if mx:
        c = caller(lib, "fp8_mx_norm_quantize", NORM_ORDER + "layouts q sr qt ld_t sc stream", NORM)
    else:
        c = caller(lib, "fp8_norm_quantize", NORM_ORDER + "recipe layouts scale amax q sr qt ld_t sc stream", NORM)
    for bad in (dict(x=None), dict(rows=-1), dict(rows=2 ** 31), dict(cols=0), dict(kind=2), dict(xt=3), dict(wt=3),
                dict(rt=5), dict(layouts=0), dict(layouts=4), dict(eps=-1.0), dict(eps=float("nan")), dict(ld_x=63),
                dict(ld_r=63), dict(ld_s=63), dict(sum=None), dict(res=None), dict(q=None), dict(sr=None),
                dict(fmt=4)):
        assert c(**bad) == INVALID, bad
    for bad in (dict(cols=65568), dict(fmt=2), dict(fmt=3), dict(rt=1), dict(xt=2, rt=0), dict(xt=1, rt=0)):
        assert c(**bad) == UNSUPPORTED, bad
    for bad in (dict(cols=40), dict(x=FAKE + 1), dict(res=FAKE + 1), dict(rt=2, res=FAKE + 2), dict(sum=FAKE + 1),
                dict(q=FAKE + 8), dict(w=FAKE + 2), dict(rstd=FAKE + 2), dict(sr=FAKE + 2)):
        assert c(**bad) == ALIGN, bad
    empty = dict(x=None, res=None, sum=None, q=None, sr=None, qt=None, sc=None)
    assert c(rows=0, **empty) == OK
    both = dict(layouts=3) if mx else dict(layouts=3, rkind=0, scale=FAKE, amax=FAKE)
    for bad in (dict(rstd=None), dict(kind=0), dict(qt=None), dict(sc=None), dict(ld_t=16)):
        assert c(**dict(both, **bad)) == INVALID, bad
    for bad in (dict(ld_t=40), dict(qt=FAKE + 8)):
        assert c(**dict(both, **bad)) == ALIGN, bad
    if mx:
        assert c(layouts=3, rows=40, ld_t=48) == ALIGN  # whole blocks of 32 rows
        assert c(cols=48, ld_x=48) == ALIGN
    else:
        assert c(recipe=None) == INVALID
        assert c(rkind=1) == UNSUPPORTED
        assert c(rkind=3) == INVALID
        assert c(margin=-1) == INVALID
        assert c(margin=65) == INVALID
        assert c(layouts=3) == UNSUPPORTED  # column scales need all rows first
        assert c(layouts=2) == UNSUPPORTED
        assert c(scale=FAKE) == INVALID
        assert c(amax=FAKE) == INVALID
        assert c(**dict(both, scale=None)) == INVALID
        assert c(**dict(both, amax=None)) == INVALID
        assert c(**dict(both, amax=FAKE + 2)) == ALIGN


def test_residual_norm_backward_validation(lib):
    base = dict(dy=FAKE, yt=0, ld_dy=64, x=FAKE, ld_x=64, q=None, ld_q=0, s=None, ld_s=0, fmt=0, dsum=FAKE, ld_d=64,
                rows=4, cols=64, kind=1, mean=None, rstd=FAKE, w=FAKE, wt=0, dx=FAKE, xt=0, ld_dx=64, dw=None, db=None,
                ws=None, wsb=0, stream=None)
    c = caller(lib, "fp8_residual_norm_backward", "dy yt ld_dy x ld_x q ld_q s ld_s fmt dsum ld_d rows cols kind mean "
               "rstd w wt dx xt ld_dx dw db ws wsb stream", base)
    for bad in (dict(dsum=None), dict(ld_d=63), dict(dy=None), dict(dx=None), dict(rstd=None), dict(dw=FAKE),
                dict(x=None), dict(q=FAKE, s=FAKE, ld_q=64, ld_s=2), dict(kind=0)):
        assert c(**bad) == INVALID, bad
    assert c(dsum=FAKE + 1) == ALIGN
    assert c(xt=2, yt=0, dsum=FAKE + 2) == ALIGN
    assert c(rows=0, dsum=None) == OK


OUT = dict(fmt=0, layouts=3, scale=FAKE, amax=FAKE, q_row=FAKE, s_row=FAKE, q_colT=FAKE, ld_t=64, s_col=FAKE, inv=FAKE,
           gu=None, ld_gu=0, cfmt=0, cq=None, ld_cq=0, cs=None, ld_cs=0, stream=None)
GEMM = dict(OUT, A=FAKE, fa=0, lda=96, sA=FAKE, W=FAKE, fw=0, ldw=96, sW=FAKE, M=64, F=64, K=96, sam=1, swm=1, h=None,
            ld_h=0)
BACK = dict(GEMM, gu=FAKE, ld_gu=128, d=None, ld_d=0)
FORWARD = {False: ("fp8_swiglu_gemm", "A fa lda W fw ldw M F K sA sam sW swm fmt layouts scale amax q_row q_colT ld_t "
                   "inv h ld_h gu ld_gu cfmt cq ld_cq cs ld_cs stream"),
           True: ("fp8_mx_swiglu_gemm", "A fa lda sA W fw ldw sW M F K fmt layouts q_row s_row q_colT ld_t s_col h "
                  "ld_h gu ld_gu cfmt cq ld_cq cs ld_cs stream")}
BACKWARD = {False: ("fp8_swiglu_gemm_backward", "A fa lda W fw ldw M F K sA sam sW swm gu ld_gu cq ld_cq cs ld_cs cfmt "
                    "fmt layouts scale amax q_row q_colT ld_t inv d ld_d stream"),
            True: ("fp8_mx_swiglu_gemm_backward", "A fa lda sA W fw ldw sW M F K gu ld_gu cq ld_cq cs ld_cs cfmt fmt "
                   "layouts q_row s_row q_colT ld_t s_col d ld_d stream")}


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("mx", [False, True])
def test_swiglu_gemm_validation(lib, mx, back):
    name, order = (BACKWARD if back else FORWARD)[mx]
    c = caller(lib, name, order, BACK if back else GEMM)
    for bad in (dict(A=None), dict(W=None), dict(sA=None), dict(sW=None), dict(M=-1), dict(M=2 ** 31), dict(F=0),
                dict(K=0), dict(K=2 ** 31), dict(F=2 ** 30), dict(lda=64), dict(ldw=64), dict(fa=4), dict(fw=5),
                dict(fmt=4), dict(layouts=4), dict(layouts=-1), dict(q_row=None), dict(q_colT=None), dict(ld_t=48)):
        assert c(**bad) == INVALID, bad
    for bad in (dict(fa=2), dict(fw=3), dict(fmt=2)):
        assert c(**bad) == UNSUPPORTED, bad
    for bad in (dict(F=72), dict(K=72), dict(lda=100), dict(ldw=104), dict(A=FAKE + 8), dict(W=FAKE + 8),
                dict(q_row=FAKE + 8), dict(q_colT=FAKE + 8), dict(ld_t=72)):
        assert c(**bad) == ALIGN, bad
    if mx:
        for bad in (dict(F=48), dict(K=80), dict(M=40), dict(sA=FAKE + 8), dict(sW=FAKE + 4), dict(s_row=FAKE + 2),
                    dict(s_col=FAKE + 1)):
            assert c(**bad) == ALIGN, bad
        assert c(s_row=None) == INVALID
        assert c(s_col=None) == INVALID
    else:
        for bad in (dict(sam=2), dict(swm=-1), dict(scale=None), dict(amax=None), dict(inv=None)):
            assert c(**bad) == INVALID, bad
        for bad in (dict(sA=FAKE + 2), dict(sW=FAKE + 1), dict(scale=FAKE + 2), dict(amax=FAKE + 1)):
            assert c(**bad) == ALIGN, bad
    none = dict(A=None, W=None, sA=None, sW=None)
    assert c(M=0, **none) == OK
    # kept gate|up: bf16, or a checkpoint
    ck = dict(cq=FAKE, cs=FAKE, ld_cq=128, ld_cs=4)
    for bad in (dict(ck, ld_cq=96), dict(ck, ld_cs=3), dict(ck, cs=None), dict(ck, cq=None), dict(ck, cfmt=4)):
        assert c(**dict(dict(gu=None), **bad)) == INVALID, bad
    assert c(**dict(ck, gu=None, cfmt=2)) == UNSUPPORTED
    assert c(**dict(ck, gu=None, cq=FAKE + 16)) == ALIGN
    assert c(**dict(ck, gu=None, ld_cq=136)) == ALIGN
    assert c(gu=FAKE, ld_gu=120) == INVALID
    assert c(gu=FAKE, ld_gu=132) == ALIGN
    assert c(gu=FAKE + 8, ld_gu=128) == ALIGN
    out, ld, least = ("d", "ld_d", 128) if back else ("h", "ld_h", 64)
    assert c(**{out: FAKE, ld: least - 8}) == INVALID
    assert c(**{out: FAKE, ld: least + 4}) == ALIGN
    assert c(**{out: FAKE + 2, ld: least}) == ALIGN
    if back:
        assert c(gu=None) == INVALID              # nothing to read gate|up from
        assert c(**dict(ck, gu=FAKE)) == INVALID  # two
        assert c(layouts=0) == INVALID            # nothing to write
    else:
        assert c(layouts=0) == INVALID


IN = 0x40000  # apart from FAKE


@pytest.mark.parametrize("mx", [False, True])
def test_outputs_that_start_where_an_input_does(lib, mx):
    if mx:
        c = caller(lib, "fp8_mx_norm_quantize", NORM_ORDER + "layouts q sr qt ld_t sc stream", NORM)
    else:
        c = caller(lib, "fp8_norm_quantize", NORM_ORDER + "recipe layouts scale amax q sr qt ld_t sc stream", NORM)
    assert c(x=IN, res=FAKE, sum=FAKE) == INVALID
    assert c(x=FAKE, res=IN, sum=FAKE) == INVALID
    name, order = BACKWARD[mx]
    c = caller(lib, name, order, dict(BACK, gu=IN, d=IN, ld_d=128, layouts=0))
    assert c() == INVALID


@pytest.mark.parametrize("same", ["dy", "x", "dsum"])
def test_residual_norm_backward_in_place(lib, same):
    base = dict(dy=IN, yt=0, ld_dy=64, x=2 * IN, ld_x=64, q=None, ld_q=0, s=None, ld_s=0, fmt=0, dsum=3 * IN, ld_d=64,
                rows=4, cols=64, kind=1, mean=None, rstd=FAKE, w=FAKE, wt=0, dx=FAKE, xt=0, ld_dx=64, dw=None, db=None,
                ws=None, wsb=0, stream=None)
    c = caller(lib, "fp8_residual_norm_backward", "dy yt ld_dy x ld_x q ld_q s ld_s fmt dsum ld_d rows cols kind mean "
               "rstd w wt dx xt ld_dx dw db ws wsb stream", base)
    assert c(**{same: FAKE}) == INVALID
