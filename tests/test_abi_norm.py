"""Host-only argument checks of the norm, SwiGLU and checkpoint entry points:
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


def call(lib, name, order, base, kw):
    a = dict(base, **kw)
    fn = getattr(lib, name)
    return fn(*[P(a[k]) if t is P else a[k] for k, t in zip(order, fn.argtypes)], )


CK = ["x", "dtype", "rows", "cols", "ld_x", "parts", "fmt", "q", "ld_q", "s", "ld_s", "stream"]
CK_BASE = dict(x=FAKE, dtype=0, rows=4, cols=64, ld_x=128, parts=2, fmt=0, q=FAKE, ld_q=128, s=FAKE, ld_s=4,
               stream=None)


def test_checkpoint_validation(lib):
    c = lambda **kw: call(lib, "fp8_checkpoint", CK, CK_BASE, kw)  # noqa: E731
    assert c(x=None) == INVALID
    assert c(rows=-1) == INVALID
    assert c(cols=0) == INVALID
    assert c(parts=0) == INVALID
    assert c(cols=2 ** 31 - 1) == INVALID
    assert c(rows=2 ** 31) == INVALID
    assert c(dtype=3) == INVALID
    assert c(fmt=2) == UNSUPPORTED
    assert c(fmt=4) == INVALID
    assert c(ld_x=127) == INVALID
    assert c(ld_q=96) == INVALID
    assert c(ld_s=3) == INVALID
    assert c(q=None) == INVALID
    assert c(s=None) == INVALID
    assert c(ld_q=136) == ALIGN
    assert c(q=FAKE + 16) == ALIGN
    assert c(x=FAKE + 1) == ALIGN
    assert c(dtype=2, x=FAKE + 2) == ALIGN
    assert c(rows=0, x=None, q=None, s=None) == OK
    r = ["q", "ld_q", "s", "ld_s", "fmt", "rows", "cols", "parts", "x", "dtype", "ld_x", "stream"]
    c = lambda **kw: call(lib, "fp8_checkpoint_restore", r, CK_BASE, kw)  # noqa: E731
    assert c(x=None) == INVALID
    assert c(q=None) == INVALID
    assert c(fmt=3) == UNSUPPORTED
    assert c(ld_x=100) == INVALID
    assert c(rows=0, x=None, q=None, s=None) == OK


def test_swiglu_validation(lib):
    order = ["gu", "rows", "F", "ld", "fmt", "h", "ld_h", "q", "ld_q", "s", "ld_s", "stream"]
    base = dict(gu=FAKE, rows=4, F=40, ld=80, fmt=0, h=FAKE, ld_h=40, q=FAKE, ld_q=128, s=FAKE, ld_s=4, stream=None)
    c = lambda **kw: call(lib, "fp8_swiglu_checkpoint", order, base, kw)  # noqa: E731
    assert c(gu=None) == INVALID
    assert c(h=None) == INVALID
    assert c(F=0) == INVALID
    assert c(ld=79) == INVALID
    assert c(ld_h=39) == INVALID
    assert c(ld_q=96) == INVALID
    assert c(fmt=2) == UNSUPPORTED
    assert c(gu=FAKE + 1) == ALIGN
    assert c(q=FAKE + 8) == ALIGN
    assert c(rows=0, gu=None, h=None, q=None, s=None) == OK
    order = ["dh", "ld_dh", "gu", "ld", "q", "ld_q", "s", "ld_s", "fmt", "rows", "F", "d", "ld_d", "h", "ld_h",
             "stream"]
    base = dict(dh=FAKE, ld_dh=40, gu=None, ld=0, q=FAKE, ld_q=128, s=FAKE, ld_s=4, fmt=0, rows=4, F=40, d=FAKE,
                ld_d=80, h=None, ld_h=0, stream=None)
    c = lambda **kw: call(lib, "fp8_swiglu_backward", order, base, kw)  # noqa: E731
    assert c(dh=None) == INVALID
    assert c(d=None) == INVALID
    assert c(q=None) == INVALID
    assert c(s=None) == INVALID
    assert c(gu=FAKE, ld=80) == INVALID                       # two sources
    assert c(gu=FAKE, ld=79, q=None, s=None) == INVALID
    assert c(fmt=3) == UNSUPPORTED
    assert c(fmt=-1) == INVALID
    assert c(ld_d=79) == INVALID
    assert c(h=FAKE, ld_h=39) == INVALID
    assert c(rows=0, dh=None, q=None, s=None, d=None) == OK


def test_norm_validation(lib):
    order = ["x", "xt", "ld_x", "rows", "cols", "kind", "eps", "w", "b", "wt", "y", "yt", "ld_y", "mean", "rstd",
             "fmt", "q", "ld_q", "s", "ld_s", "stream"]
    base = dict(x=FAKE, xt=0, ld_x=100, rows=4, cols=100, kind=0, eps=1e-5, w=FAKE, b=FAKE, wt=0, y=FAKE, yt=0,
                ld_y=100, mean=FAKE, rstd=FAKE, fmt=0, q=FAKE, ld_q=128, s=FAKE, ld_s=4, stream=None)
    c = lambda **kw: call(lib, "fp8_norm_forward", order, base, kw)  # noqa: E731
    assert c(x=None) == INVALID
    assert c(y=None) == INVALID
    assert c(rows=-1) == INVALID
    assert c(cols=0) == INVALID
    assert c(kind=2) == INVALID
    assert c(eps=-1.0) == INVALID
    assert c(eps=float("nan")) == INVALID
    assert c(xt=3) == INVALID
    assert c(wt=-1) == INVALID
    assert c(yt=2) == UNSUPPORTED                              # bf16 x, fp32 y
    assert c(xt=1) == UNSUPPORTED                              # fp16 x, bf16 y
    assert c(ld_x=99) == INVALID
    assert c(ld_y=99) == INVALID
    assert c(q=None) == INVALID                                # scales without codes
    assert c(s=None) == INVALID
    assert c(fmt=2) == UNSUPPORTED
    assert c(ld_q=100) == INVALID
    assert c(ld_q=136) == ALIGN
    assert c(x=FAKE + 1) == ALIGN
    assert c(w=FAKE + 1) == ALIGN
    assert c(wt=2, b=FAKE + 2) == ALIGN
    assert c(rstd=FAKE + 2) == ALIGN
    assert c(rows=0, x=None, y=None, mean=None, rstd=None, q=None, s=None) == OK
    assert lib.fp8_norm_workspace_bytes(-1, 5) == -1 and lib.fp8_norm_workspace_bytes(5, 0) == -1
    need = lib.fp8_norm_workspace_bytes(4, 100)
    assert need >= 2 * 100 * 4
    order = ["dy", "yt", "ld_dy", "x", "ld_x", "q", "ld_q", "s", "ld_s", "fmt", "rows", "cols", "kind", "mean", "rstd",
             "w", "wt", "dx", "xt", "ld_dx", "dw", "db", "ws", "n", "stream"]
    base = dict(base, dy=FAKE, ld_dy=100, q=None, ld_q=0, s=None, ld_s=0, dx=FAKE, ld_dx=100, dw=FAKE, db=FAKE,
                ws=FAKE, n=need)
    c = lambda **kw: call(lib, "fp8_norm_backward", order, base, kw)  # noqa: E731
    assert c(dy=None) == INVALID
    assert c(dx=None) == INVALID
    assert c(x=None) == INVALID                                # neither x nor a checkpoint
    assert c(q=FAKE, ld_q=128, s=FAKE, ld_s=4) == INVALID      # both
    assert c(x=None, q=FAKE, ld_q=128, s=FAKE, ld_s=3) == INVALID
    assert c(x=None, q=FAKE, ld_q=128, s=FAKE, ld_s=4, fmt=2) == UNSUPPORTED
    assert c(rstd=None) == INVALID
    assert c(mean=None) == INVALID
    assert c(ws=None) == INVALID
    assert c(n=need - 1) == INVALID
    assert c(ws=FAKE + 4) == ALIGN
    assert c(yt=1) == UNSUPPORTED
    assert c(dw=FAKE + 1) == ALIGN


def test_wrappers_refuse_host_tensors():
    """The Python wrappers check where a tensor lies before anything else."""
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c = fp8.Checkpoint(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8), 0, 64)
    for call in (lambda: fp8.norm_forward(x), lambda: fp8.norm_backward(x, x, None, x[:, 0].float()),
                 lambda: fp8.checkpoint(x), lambda: fp8.checkpoint_restore(c), lambda: fp8.swiglu_checkpoint(x),
                 lambda: fp8.swiglu_backward(x, x)):
        with pytest.raises(fp8.Fp8Error) as e:
            call()
        assert e.value.status == INVALID
