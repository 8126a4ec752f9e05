"""GPU tests of the 8-bit checkpoints and the SwiGLU around them: codes and
scales equal the float64 reference's bit for bit, h and the gradients lie
within the tolerances derived in norm_ref."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import norm_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


def values(rows, cols, dtype, seed, scale=1.0, pad=0, offset=0, spread=0):
    """[rows, cols] in rows of cols + pad, `offset` elements into a buffer of
    NaN; with spread, rows of very different size."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=dtype, device=DEV)
    x = buf[offset:].view(rows, cols + pad)[:, :cols]
    v = torch.randn((rows, cols), generator=g) * scale
    if spread:
        v = v * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g).float())
    x.copy_(v.to(dtype))
    return x


def assert_checkpoint(c, x, parts, fmt, what=""):
    t, s = ref.checkpoint(ref.f64(x), parts, fmt)
    assert np.array_equal(c.s.cpu().numpy(), s), f"{what} scales"
    got = ref.decode_table(fmt)[c.q.cpu().numpy()]
    assert np.array_equal(np.isnan(got), np.isnan(t)), f"{what} NaN"
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(t)), f"{what} codes"


def assert_restored(back, c, cols, parts, fmt, what=""):
    want = torch.from_numpy(ref.restore(c.q, c.s, cols, parts, fmt)).to(back.dtype)
    got = back.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(want.double())), what


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 0, 0), (3, 31, 0, 0), (5, 32, 0, 0), (4, 33, 1, 1), (17, 1000, 0, 0),
                                   (9, 1024, 8, 0), (6, 4096, 0, 8), (7, 2999, 5, 3), (2, 16400, 0, 0)])
def test_store_and_restore(shape, dtype, fmt):
    rows, cols, pad, offset = shape
    x = values(rows, cols, dtype, cols, 1.0, pad, offset, spread=6 if dtype == F16 else 40)
    c = fp8.checkpoint(x, fmt)
    assert_checkpoint(c, x, 1, fmt, f"{shape}")
    buf = torch.full((rows, cols + pad), 7.0, dtype=dtype, device=DEV)
    back = fp8.checkpoint_restore(c, out=buf[:, :cols])
    assert_restored(back, c, cols, 1, fmt, f"{shape}")
    assert bool((buf[:, cols:] == 7).all())
    for other in (BF16, F32):
        assert_restored(fp8.checkpoint_restore(c, other), c, cols, 1, fmt, f"{shape} to {other}")


@pytest.mark.parametrize("parts,cols", [(2, 32), (2, 40), (3, 100), (5, 1), (4, 1024)])
def test_parts(parts, cols):
    x = values(11, parts * cols, BF16, cols, spread=10)
    c = fp8.checkpoint(x, 0, parts)
    assert c.q.shape[1] == parts * ref.width(cols)
    assert_checkpoint(c, x, parts, 0)
    assert_restored(fp8.checkpoint_restore(c), c, cols, parts, 0)


@pytest.mark.parametrize("cols", [32, 96, 100])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", [0, 1])
def test_extreme_values(cols, dtype, fmt):
    """Zero blocks, NaN and Inf blocks and their neighbours, the type's
    smallest and largest magnitudes, amax at the scale's boundaries."""
    x = values(16, cols, dtype, 3)
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -133 if dtype == BF16 else 2.0 ** -149
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 20] = float("inf")
    x[3, 1] = -float("inf")
    x[4] = big
    x[5] = -big
    x[6] = tiny
    x[7] = 2.0 ** -126
    x[8] = 0
    x[8, 0] = ref.FMAX[fmt]
    x[9] = 0
    x[9, 0] = ref.FMAX[fmt] * (1 + 2.0 ** -7)
    x[10] = 0
    x[10, 31] = 1.75
    x[11] = x[11] * 1e-38
    x[12, 0] = big
    x[13, :] = 0
    x[13, 5] = -0.0
    c = fp8.checkpoint(x, fmt)
    assert_checkpoint(c, x, 1, fmt)
    assert_restored(fp8.checkpoint_restore(c, dtype), c, cols, 1, fmt)


@pytest.mark.parametrize("fmt", [0, 1])
def test_every_code_restores(fmt):
    """All 256 codes under all 256 scale bytes, as any producer may have
    written them."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).to(DEV)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8).to(DEV)
    c = fp8.Checkpoint(codes, scales, fmt, 256)
    with np.errstate(over="ignore"):
        assert_restored(fp8.checkpoint_restore(c, F32), c, 256, 1, fmt)


def check_swiglu(rows, F, fmt, pad=0, offset=0, scale=2.0, seed=1):
    gu = values(rows, 2 * F, BF16, seed, scale, pad, offset)
    dh = values(rows, F, BF16, seed + 1, 0.1, pad, offset)
    what = f"{rows} x {F}"
    hbuf = torch.full((rows, F + pad), 7.0, dtype=BF16, device=DEV)
    h, c = fp8.swiglu_checkpoint(gu, fmt, h_out=hbuf[:, :F])
    x = ref.f64(gu)
    hr = ref.swiglu(x[:, :F], x[:, F:])
    ref.assert_within(ref.f64(h), hr, 2.0 ** -7 * np.abs(hr) + 2.0 ** -133, what + " h")
    assert_checkpoint(c, gu, 2, fmt, what)
    assert bool((hbuf[:, F:] == 7).all())
    d = ref.f64(dh)
    for src, v in ((gu, x), (c, ref.restore(c.q, c.s, F, 2, fmt))):
        buf = torch.full((rows, 2 * F + pad), 7.0, dtype=BF16, device=DEV)
        dgu, again = fp8.swiglu_backward(dh, src, out=buf[:, :2 * F], return_h=True)
        g, u = v[:, :F], v[:, F:]
        dg, du = ref.swiglu_backward(g, u, d)
        tg, tu = ref.tol_swiglu_backward(dg, du, g, u, d)
        ref.assert_within(ref.f64(dgu)[:, :F], dg, tg, what + " d gate")
        ref.assert_within(ref.f64(dgu)[:, F:], du, tu, what + " d up")
        hr = ref.swiglu(g, u)
        ref.assert_within(ref.f64(again), hr, 2.0 ** -7 * np.abs(hr) + 2.0 ** -133, what + " h again")
        assert bool((buf[:, 2 * F:] == 7).all())
        assert torch.equal(fp8.swiglu_backward(dh, src), dgu)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("F", [1, 7, 8, 31, 32, 33, 40, 128, 1000, 1500, 2048, 2056, 14336])
def test_swiglu_widths(F, fmt):
    check_swiglu(19, F, fmt)


@pytest.mark.parametrize("shape", [(1, 2048, 0, 0), (5, 256, 3, 0), (5, 256, 8, 1), (4, 100, 4, 2), (700, 64, 0, 0),
                                   (3000, 33, 1, 0)])
def test_swiglu_strides_and_rows(shape):
    rows, F, pad, offset = shape
    check_swiglu(rows, F, 0, pad, offset)


def test_swiglu_range():
    """Gates far out on both sides: sigma saturates, nothing overflows."""
    g = torch.linspace(-120, 120, 2048).to(BF16)
    gu = torch.stack([torch.cat([g, torch.full_like(g, v)]) for v in (1.0, -3.0, 1e4)]).to(DEV)
    dh = torch.full((3, 2048), 0.5, dtype=BF16, device=DEV)
    x = ref.f64(gu)
    dg, du = ref.swiglu_backward(x[:, :2048], x[:, 2048:], ref.f64(dh))
    tg, tu = ref.tol_swiglu_backward(dg, du, x[:, :2048], x[:, 2048:], ref.f64(dh))
    got = ref.f64(fp8.swiglu_backward(dh, gu))
    ref.assert_within(got[:, :2048], dg, tg, "d gate")
    ref.assert_within(got[:, 2048:], du, tu, "d up")


def test_swiglu_non_finite():
    """NaN stays in its element from bf16 and in its block from a checkpoint;
    a gate of -Inf gives gradients of 0."""
    gu = values(4, 2 * 96, BF16, 1)
    gu[0, 5] = float("nan")
    gu[1, 96 + 40] = float("nan")
    gu[2, 7] = -float("inf")
    dh = values(4, 96, BF16, 2)
    h, c = fp8.swiglu_checkpoint(gu, 0)
    d = fp8.swiglu_backward(dh, gu)
    assert torch.isnan(d[0, [5, 96 + 5]]).all() and int(torch.isnan(d[0]).sum()) == 2
    assert torch.isnan(d[1, 40]) and not torch.isnan(d[1, 96 + 40])     # d up does not read up
    assert float(d[2, 7]) == 0 and float(d[2, 96 + 7]) == 0 and torch.isfinite(d[2]).all()
    d = fp8.swiglu_backward(dh, c)
    nan = torch.isnan(d)
    assert nan[0, :32].all() and nan[0, 96:128].all() and int(nan[0].sum()) == 64
    assert nan[1, 32:64].all() and int(nan[1].sum()) == 32
    assert not nan[3].any()


def test_swiglu_gradient_is_the_forwards_difference():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn((1, 2 * 64), generator=g) * 2).to(BF16).to(DEV)
    dh = torch.ones((1, 64), dtype=BF16, device=DEV)
    d = ref.f64(fp8.swiglu_backward(dh, x))[0]
    v = ref.f64(x)[0]
    for i in range(128):
        e = np.zeros(128)
        e[i] = 1e-5
        a, b = v + e, v - e
        num = (ref.swiglu(a[:64], a[64:]).sum() - ref.swiglu(b[:64], b[64:]).sum()) / 2e-5
        assert abs(num - d[i]) <= 2.0 ** -8 * abs(num) + 1e-4   # the output's rounding; the fast exponential


def test_empty():
    x = torch.empty((0, 200), dtype=BF16, device=DEV)
    c = fp8.checkpoint(x, 0, 2)
    assert fp8.checkpoint_restore(c).shape == (0, 200)
    h, c = fp8.swiglu_checkpoint(x)
    assert h.shape == (0, 100)
    for src in (x, c):
        assert fp8.swiglu_backward(h, src).shape == (0, 200)


@pytest.mark.parametrize("cols", [4096, 4099])
def test_offsets_past_32_bits(cols):
    rows, ld = 40, (1 << 27) + 32
    buf = torch.empty(rows * ld, dtype=BF16, device=DEV).view(rows, ld)
    x = values(rows, 2 * cols, BF16, 1)
    buf[:, :2 * cols].copy_(x)
    c, want = fp8.checkpoint(buf[:, :2 * cols], 0, 2), fp8.checkpoint(x, 0, 2)
    assert torch.equal(c.q, want.q) and torch.equal(c.s, want.s)
    far = torch.empty(rows * ld, dtype=torch.uint8, device=DEV).view(rows, ld)[:, :want.q.shape[1]]
    far.copy_(want.q)
    c = fp8.Checkpoint(far, want.s, 0, cols, 2)
    buf.fill_(0)
    back = fp8.checkpoint_restore(c, out=buf[:, :2 * cols])
    assert torch.equal(back, fp8.checkpoint_restore(want))
    dh = values(rows, cols, BF16, 2)
    d = fp8.swiglu_backward(dh, c, out=buf[:, :2 * cols])
    assert torch.equal(d, fp8.swiglu_backward(dh, want))
    del buf, far, back, d
    torch.cuda.empty_cache()


def test_many_rows():
    """More rows than a 16-bit grid dimension holds."""
    x = values(200000, 32, BF16, 1)
    c = fp8.checkpoint(x, 0)
    assert_checkpoint(c, x, 1, 0)
    assert_restored(fp8.checkpoint_restore(c), c, 32, 1, 0)


def test_other_stream():
    gu, dh = values(4000, 2 * 2048, BF16, 1), values(4000, 2048, BF16, 2)
    h, c = fp8.swiglu_checkpoint(gu)
    d = fp8.swiglu_backward(dh, c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        h2, c2 = fp8.swiglu_checkpoint(gu, stream=side)
        d2 = fp8.swiglu_backward(dh, c2, stream=side)
        back = fp8.checkpoint_restore(c2, stream=side)
        for _ in range(20):
            torch.full((1 << 22,), float("nan"), device=DEV)
        side.synchronize()
        assert torch.equal(h, h2) and torch.equal(c.q, c2.q) and torch.equal(d, d2)
        assert torch.equal(back, fp8.checkpoint_restore(c))


def test_refusals():
    x = values(8, 64, BF16, 1)
    c = fp8.checkpoint(x)

    def refused(fn, *a, **k):
        with pytest.raises(fp8.Fp8Error):
            fn(*a, **k)

    refused(fp8.checkpoint, x.cpu())
    refused(fp8.checkpoint, x.double())
    refused(fp8.checkpoint, x[0])
    refused(fp8.checkpoint, x.t())
    refused(fp8.checkpoint, x, 0, 3)
    refused(fp8.checkpoint, x, fp8.E5M2FNUZ)
    refused(fp8.checkpoint, x, 9)
    refused(fp8.checkpoint_restore, c, torch.float64)
    refused(fp8.checkpoint_restore, fp8.Checkpoint(c.q, c.s, 0, 65))
    refused(fp8.checkpoint_restore, fp8.Checkpoint(c.q, c.s[:, :1], 0, 64))
    refused(fp8.checkpoint_restore, c, out=torch.empty((8, 63), dtype=BF16, device=DEV))
    off = torch.empty((8 * 64 + 16,), dtype=torch.uint8, device=DEV)[16:].view(8, 64)
    refused(fp8.checkpoint_restore, fp8.Checkpoint(off, c.s, 0, 64))       # codes not 32-byte aligned
    refused(fp8.swiglu_checkpoint, x.float())
    refused(fp8.swiglu_checkpoint, x[:, :63])
    h, k = fp8.swiglu_checkpoint(x)
    refused(fp8.swiglu_backward, h, c)                                      # one part of 64, not two of 32
    refused(fp8.swiglu_backward, h[:4], k)
    refused(fp8.swiglu_backward, h, h)
    refused(fp8.swiglu_backward, h.float(), k)
    refused(fp8.swiglu_backward, h, k, out=torch.empty((8, 32), dtype=BF16, device=DEV))
    torch.cuda.synchronize()
