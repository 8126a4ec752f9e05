"""GPU tests of the norm, SwiGLU and checkpoint operators where callers and
values leave the usual: the default stream by its handle, rows past the last one,
the largest values of a type, gates far below zero, host threads side by side."""
import threading

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


def test_default_stream_by_its_handle():
    """stream=0 is torch's default stream: a call on it comes after what was
    put there before, and before what is put there next."""
    with fp8._on(torch.cuda.default_stream().cuda_stream):
        assert torch.cuda.current_stream().cuda_stream == 0
    x, w = torch.randn((3000, 4096), device=DEV).to(BF16), torch.ones(4096, dtype=BF16, device=DEV)
    want = fp8.norm_forward(x, w, checkpoint_fmt=0)
    dy = want.y * 0.1
    back = fp8.norm_backward(dy, want.checkpoint, want.mean, want.rstd, w)
    gate_up, kept = fp8.checkpoint(x), fp8.checkpoint(x, parts=2)
    h, _ = fp8.swiglu_checkpoint(x)
    grad = fp8.swiglu_backward(h, kept)
    for _ in range(5):
        late = torch.zeros_like(x)
        for _ in range(20):
            late.add_(0.0)
        late.copy_(x)   # after 20 passes over it
        f = fp8.norm_forward(late, w, checkpoint_fmt=0, stream=0)
        b = fp8.norm_backward(dy, f.checkpoint, f.mean, f.rstd, w, stream=0)
        c = fp8.checkpoint(late, stream=0)
        h2, _ = fp8.swiglu_checkpoint(late, stream=0)
        d = fp8.swiglu_backward(h2, kept, stream=0)
        r = fp8.checkpoint_restore(c, stream=0)
        assert torch.equal(f.y, want.y) and torch.equal(b.dx, back.dx) and torch.equal(b.dweight, back.dweight)
        assert torch.equal(c.q, gate_up.q) and torch.equal(h2, h) and torch.equal(d, grad)
        assert torch.equal(r, fp8.checkpoint_restore(gate_up))


@pytest.mark.parametrize("types", [(BF16, BF16), (F16, F16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("cols", [64, 100, 1024, 1111, 8200])
@pytest.mark.parametrize("rows", [37, 700, 4500])
def test_rows_past_the_end_add_nothing(rows, cols, types):
    """Constant rows with mean * rstd above fp32's range: xhat is 0 in every row,
    so dweight is exactly 0, also where a group's last step reaches past the
    rows (the row before's mean * rstd, times a dy of 0, would be NaN)."""
    tx, ty = types
    value = 2.0 ** 15 if tx == F16 else 2.0 ** 120
    x = torch.full((rows, cols), value, dtype=tx, device=DEV)
    dy = torch.ones((rows, cols), dtype=ty, device=DEV)
    mean = torch.full((rows,), value, dtype=F32, device=DEV)
    rstd = torch.full((rows,), 2.0 ** 128 / value * (1 - 2.0 ** -24), dtype=F32, device=DEV) * 2
    b = fp8.norm_backward(dy, x, mean, rstd, torch.ones(cols, dtype=F32, device=DEV))
    assert not b.dx.isnan().any()
    assert int((b.dweight != 0).sum()) == 0
    assert bool((b.dbias == rows).all())   # sums of ones below 2^24 are exact


@pytest.mark.parametrize("fmt", [fp8.E4M3FN, fp8.E5M2])
@pytest.mark.parametrize("cols,pad", [(64, 0), (100, 0), (77, 3)])
def test_finite_fp16_restores_finite(cols, pad, fmt):
    """Every finite fp16 magnitude of the top binade, both signs: back within
    2^-4 (E4M3) or 2^-3 (E5M2) of itself, half a step of a 3 or 2 bit mantissa."""
    top = torch.arange(0x7800, 0x7C00, dtype=torch.int16, device=DEV).view(F16)   # 32768 .. 65504
    x = torch.ones((32, cols + pad), dtype=F16, device=DEV)[:, :cols]
    x[:16, :64] = top.view(16, 64)
    x[16:, :64] = -top.view(16, 64)
    back = fp8.checkpoint_restore(fp8.checkpoint(x, fmt), F16, out=torch.empty_like(x))
    assert torch.isfinite(back).all()
    off = (back.double() - x.double()).abs()[:, :64]
    assert bool((off <= 2.0 ** (-4 if fmt == fp8.E4M3FN else -3) * x.double().abs()[:, :64]).all())
    back = fp8.checkpoint_restore(fp8.checkpoint(x.float() * 4, fmt), F16)        # beyond fp16: Inf, as any conversion
    assert torch.isinf(back[:, :64]).all() and torch.equal(back[:, :64] > 0, x[:, :64] > 0)


def test_host_threads_at_different_widths():
    """Calls of one kernel at different widths from several host threads, on
    streams of their own: none is refused for the shared memory another asked for."""
    calls, rows = 20000, 4
    lib = fp8.load_library()
    refused, wrong = {}, []

    def caller(cols, backward):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            g = torch.Generator(device=DEV).manual_seed(cols)
            x, dy = (torch.randn((rows, cols), generator=g, device=DEV).to(BF16) for _ in range(2))
            w = torch.ones(cols, dtype=F32, device=DEV)
            f = fp8.norm_forward(x, w, w)
            want = fp8.norm_backward(dy, x, f.mean, f.rstd, w)
            y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
            n = fp8.fp8_norm_workspace_bytes(rows, cols)
            ws = torch.empty(n, dtype=torch.uint8, device=DEV)
            P = lambda t: t.data_ptr()  # noqa: E731
            if backward:
                fn, args = lib.fp8_norm_backward, (P(dy), 0, cols, P(x), cols, None, 0, None, 0, 0, rows, cols, 0,
                                                   P(f.mean), P(f.rstd), P(w), 2, P(dx), 0, cols, P(dw), None, P(ws),
                                                   n, side.cuda_stream)
            else:
                fn, args = lib.fp8_norm_forward, (P(x), 0, cols, rows, cols, 0, 1e-5, P(w), P(w), 2, P(y), 0, cols,
                                                  None, None, 0, None, 0, None, 0, side.cuda_stream)
            refused[cols, backward] = sum(fn(*args) != 0 for _ in range(calls))
            side.synchronize()
            if not (torch.equal(dx, want.dx) and torch.equal(dw, want.dweight) if backward else torch.equal(y, f.y)):
                wrong.append((cols, backward))

    threads = [threading.Thread(target=caller, args=a)
               for a in ((8192, True), (4096, True), (6144, True), (16384, False), (8192, False))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(refused) == len(threads) and not any(refused.values()), refused
    assert not wrong


def test_mirrors_of_the_entry_points():
    """The one-to-one mirrors of the C entry points give what the wrappers give."""
    rows, cols = 9, 100
    x, dy = torch.randn((rows, cols), device=DEV).to(BF16), torch.randn((rows, cols), device=DEV).to(BF16)
    w = torch.ones(cols, dtype=BF16, device=DEV)
    codes = lambda parts, n: (torch.empty((rows, parts * n), dtype=torch.uint8, device=DEV),  # noqa: E731
                              torch.empty((rows, parts * n // 32), dtype=torch.uint8, device=DEV))
    f = fp8.norm_forward(x, w, checkpoint_fmt=0)
    (q, s), y, rstd = codes(1, 128), torch.empty_like(x), torch.empty_like(f.rstd)
    fp8.fp8_norm_forward(x, 0, cols, rows, cols, fp8.LAYER_NORM, 1e-5, w, None, 0, y, 0, cols, None, rstd, 0, q, 128,
                         s, 4)
    assert torch.equal(y, f.y) and torch.equal(rstd, f.rstd)
    assert torch.equal(q, f.checkpoint.q) and torch.equal(s, f.checkpoint.s)
    c = fp8.checkpoint(x, parts=2)
    q, s = codes(2, 64)
    fp8.fp8_checkpoint(x, 0, rows, 50, cols, 2, 0, q, 128, s, 4)
    assert torch.equal(q, c.q) and torch.equal(s, c.s)
    back = torch.empty_like(x)
    fp8.fp8_checkpoint_restore(q, 128, s, 4, 0, rows, 50, 2, back, 0, cols)
    assert torch.equal(back, fp8.checkpoint_restore(c))
    h, c = fp8.swiglu_checkpoint(x)
    h2, d = torch.empty_like(h), torch.empty_like(x)
    fp8.fp8_swiglu_checkpoint(x, rows, 50, cols, 0, h2, 50, q, 128, s, 4)
    assert torch.equal(h2, h) and torch.equal(q, c.q) and torch.equal(s, c.s)
    fp8.fp8_swiglu_backward(h, 50, None, 0, q, 128, s, 4, 0, rows, 50, d, cols)
    assert torch.equal(d, fp8.swiglu_backward(h, c))
    assert fp8.fp8_checkpoint(x, 0, rows, 0, cols, 2, 0, q, 128, s, 4, check=False) == 1   # FP8_ERR_INVALID_ARG


def test_swiglu_far_gates():
    """h and the gradients of gates from -150 to 150, relative to themselves.

    Bound: __expf is documented to 2 + 1.173 |x| ulp, 105 of them (2^-16.3) where
    the gate is held at -88; with the reciprocal and the products' roundings sigma
    and silu are within 2^-16, and the slope sigma (1 + gate (1 - sigma)), whose two
    terms keep more than 86 / 88 of their sum's size there, within 2^-15.  bf16
    outputs add half an ulp (2^-8).  The slope crosses zero at -1.28, where both
    terms are about 0.22 and off by under 2^-20 of that each: gates within 8 of zero
    are allowed 2^-20 |dh up| besides.  What gates under -87 leave out is under
    2^-119 of |up|, |dh| or |dh up| (and fp32's own subnormals)."""
    g = torch.cat([torch.linspace(-150, 150, 2047), torch.tensor([-float("inf")])]).to(BF16)
    n = g.numel()
    gu = torch.stack([torch.cat([g, torch.full_like(g, v)]) for v in (1.0, -3.0, 1e4)]).to(DEV)
    dh = torch.full((3, n), 0.5, dtype=BF16, device=DEV)
    h, _ = fp8.swiglu_checkpoint(gu)
    d, again = fp8.swiglu_backward(dh, gu, return_h=True)
    assert torch.equal(h, again)
    x, dd = ref.f64(gu), ref.f64(dh)
    gate, up = x[:, :n].clip(-1e4), x[:, n:]   # e^-1e4 is 0 in float64 too: what the formulas tend to at -Inf
    dg, du = ref.swiglu_backward(gate, up, dd)
    want = ref.swiglu(gate, up)
    lost = lambda scale: 2.0 ** -119 * abs(scale) + 2.0 ** -133  # noqa: E731
    rel = 2.0 ** -8 + 2.0 ** -15
    ref.assert_within(ref.f64(h), want, rel * abs(want) + lost(up), "h")
    ref.assert_within(ref.f64(d)[:, n:], du, rel * abs(du) + lost(dd), "d up")
    ref.assert_within(ref.f64(d)[:, :n], dg,
                      rel * abs(dg) + lost(dd * up) + (abs(gate) < 8) * 2.0 ** -20 * abs(dd * up),
                      "d gate")
    for out in (h, d[:, :n], d[:, n:]):
        assert int(out[:, g < -88].count_nonzero()) == 0
