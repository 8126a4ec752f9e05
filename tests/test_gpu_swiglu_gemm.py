"""GPU tests of the SwiGLU products against the float64 references (bounds derived
in fused_ref), with the padding of every output."""
import numpy as np
import pytest
import torch

import fp8_mixed_precision_scale_gb300 as fp8
import fused_ref as ref
import norm_ref as nref

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3, E5M2 = fp8.E4M3FN, fp8.E5M2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fp8.load_library()


class Operand:
    """An 8-bit operand [R, K] with row stride ld: codes and scales on the device,
    what they stand for in float64.  groups: scale rows in two padded halves."""

    def __init__(self, R, K, fmt, mx, seed, scale, per_row=True, ld=None, groups=False):
        v = np.random.RandomState(seed).randn(R, K) * scale
        if mx:
            q, s = ref.mx_quantize(v, fmt)
            self.v = nref.decode_table(fmt)[q.numpy()] * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)
            if groups:
                h = np.zeros((2, ref.up(R // 2, 128), K // 32), np.uint8)
                h[:, :R // 2] = s.reshape(2, R // 2, -1)
                s = h.reshape(-1, K // 32)
            self.s = ref.layout_of(s).to(DEV)
        else:
            top = np.abs(v).max(1, keepdims=True) if per_row else np.abs(v).max(keepdims=True)
            inv = (top / ref.FMAX[fmt]).astype(np.float32).astype(np.float64)
            q = torch.from_numpy(np.clip(v / inv, -ref.FMAX[fmt], ref.FMAX[fmt])).float().to(nref.TORCH_FP8[fmt])
            self.v = q.double().numpy() * inv
            q = q.view(torch.uint8)
            self.s = torch.from_numpy(inv.ravel().astype(np.float32)).to(DEV)
        ld = ld or K
        buf = torch.full((R, ld), 0x7F, dtype=torch.uint8)  # NaN behind the columns
        buf[:, :K] = q
        self.q, self.fmt, self.ld = buf.to(DEV), fmt, ld


def full(shape, dtype=torch.uint8):
    n = int(np.prod(shape))
    buf = torch.full((max(n, 16),), 0xA5 if dtype == torch.uint8 else 7.0, dtype=dtype, device=DEV)
    return buf[:n].view(shape)


class Out:
    """Outputs of a product with `halves` halves of F columns, filled with 0xA5 or 7."""

    def __init__(self, M, F, mx, halves, h=True, kept=None, fmt=E4M3, layouts=3):
        self.M, self.F, self.mx, self.halves, self.fmt, self.layouts = M, F, mx, halves, fmt, layouts
        self.Fr = ref.up(F, 128) if mx and halves == 2 else F
        self.ld_t = ref.up(M, 16) + 16
        self.q, self.qt = full((M, halves * self.Fr)), full((halves * F, self.ld_t))
        self.s = full((ref.up(halves * self.Fr // 32, 4) * ref.up(M, 128),)) if mx else None
        self.st = full((ref.up(M // 32, 4) * ref.up(halves * F, 128),)) if mx else None
        self.scale, self.amax = torch.tensor([3.0], device=DEV), torch.tensor([1e-3], device=DEV)
        self.inv = torch.full((1,), -1.0, device=DEV)
        self.h = full((M, halves * F + 8), torch.bfloat16) if h else None
        W = ref.up(F, 32)
        self.gu = full((M, 2 * F + 8), torch.bfloat16) if kept == "bf16" else None
        self.ck = fp8.Checkpoint(full((M, 2 * W + 32)), full((M, 2 * W // 32 + 3)), E4M3, F, 2) if kept == "8bit" else None

    def quant(self):
        if not self.layouts:
            return {}
        a = dict(fmt=self.fmt, layouts=self.layouts, q_row=self.q, q_colT=self.qt, ld_colT=self.ld_t)
        return dict(a, s_row=self.s, s_col=self.st) if self.mx else \
            dict(a, scale_in=self.scale, amax_out=self.amax, scale_inv=self.inv)

    def kept(self):
        if self.gu is not None:
            return dict(gate_up=self.gu, ld_gu=self.gu.stride(0))
        if self.ck is not None:
            return dict(q=self.ck.q, ld_q=self.ck.q.stride(0), s=self.ck.s, ld_s=self.ck.s.stride(0), ckpt_fmt=self.ck.fmt)
        return {}

    def check(self, parts, tols, what):
        """parts, tols: the float64 halves [M, F] and their bounds."""
        M, F, Fr = self.M, self.F, self.Fr
        if self.h is not None:
            for i, (v, t) in enumerate(zip(parts, tols)):
                nref.assert_within(nref.f64(self.h[:, i * F:(i + 1) * F]), v, ref.bf16_tol(v, t), what + " bf16")
            assert (self.h[:, self.halves * F:] == 7).all(), what + ": behind the bf16 rows"
        if self.layouts & 1:
            v, t = np.zeros((M, self.halves * Fr)), np.zeros((M, self.halves * Fr))
            for i in range(self.halves):
                v[:, i * Fr:i * Fr + F], t[:, i * Fr:i * Fr + F] = parts[i], tols[i]
            if self.mx:
                ref.check_mx(self.q, ref.scales_of(self.s, M, v.shape[1] // 32), v, t, self.fmt, what + " row")
                for i in range(self.halves):
                    assert not self.q[:, i * Fr + F:(i + 1) * Fr].any(), what + ": between the halves"
            else:
                ref.check_scaled(self.q, 3.0, v, t, self.fmt, what + " row")
        else:
            assert (self.q == 0xA5).all()
        if self.layouts & 2:
            v, t = np.concatenate(parts, 1).T, np.concatenate(tols, 1).T
            if self.mx:
                s = ref.scales_of(self.st, self.halves * F, M // 32)
                ref.check_mx(self.qt[:, :M], s, v, t, self.fmt, what + " col")
            else:
                ref.check_scaled(self.qt[:, :M], 3.0, v, t, self.fmt, what + " col")
            assert (self.qt[:, M:] == 0xA5).all(), what + ": bytes behind the transposed rows"
        if not self.mx and self.layouts:
            top, err = max(np.abs(p).max() for p in parts), max(t.max() for t in tols)
            assert abs(float(self.amax) - max(top, float(np.float32(1e-3)))) <= err + 2 ** -23 * top, what + " amax"
            assert float(self.inv) == float(np.float32(1) / np.float32(3))


def forward(x, w, o, stream=None):
    M, F, K = o.M, o.F, x.v.shape[1]
    more = dict(o.quant(), **o.kept(), h=o.h, ld_h=0 if o.h is None else o.h.stride(0), stream=stream)
    if o.mx:
        fp8.fp8_mx_swiglu_gemm(x.q, x.fmt, x.ld, x.s, w.q, w.fmt, w.ld, w.s, M, F, K, **more)
    else:
        fp8.fp8_swiglu_gemm(x.q, x.fmt, x.ld, w.q, w.fmt, w.ld, M, F, K, x.s, int(x.s.numel() > 1), w.s,
                            int(w.s.numel() > 1), **more)


def backward(dy, wd, kept, o):
    M, F, K = o.M, o.F, dy.v.shape[1]
    more = dict(o.quant(), **kept, d_gate_up=o.h, ld_d=0 if o.h is None else o.h.stride(0))
    if o.mx:
        fp8.fp8_mx_swiglu_gemm_backward(dy.q, dy.fmt, dy.ld, dy.s, wd.q, wd.fmt, wd.ld, wd.s, M, F, K, **more)
    else:
        fp8.fp8_swiglu_gemm_backward(dy.q, dy.fmt, dy.ld, wd.q, wd.fmt, wd.ld, M, F, K, dy.s, int(dy.s.numel() > 1),
                                     wd.s, int(wd.s.numel() > 1), **more)


MX_SIZES = [(1, 32, 32), (5, 96, 64), (32, 64, 160), (64, 128, 128), (96, 160, 96), (127, 192, 288), (128, 256, 512),
            (129, 32, 128), (160, 288, 544), (288, 416, 1056), (257, 512, 96), (3, 1504, 2048),
            # enough tiles for CTA pairs (forward, backward too), and for wide tiles of few rows
            (1312, 928, 96), (2592, 928, 160), (1301, 928, 64), (96, 9760, 64), (64, 19488, 96),
            (96, 288, 2080), (41, 128, 2048)]  # a pair's second rows empty
SIZES = [(1, 16, 16), (4, 48, 80), (33, 112, 128), (128, 128, 256), (130, 144, 272), (300, 400, 1040), (513, 272, 48),
         (2, 720, 2064), (1301, 944, 80), (2600, 944, 48), (100, 9744, 64), (77, 19472, 48)]


def sizes(mx):
    return [(mx, *s) for mx in (True, False) for s in (MX_SIZES if mx else SIZES)]


@pytest.mark.parametrize("mx,M,F,K", sizes(True))
@pytest.mark.parametrize("kept", ["8bit", "bf16"])
def test_forward(mx, M, F, K, kept):
    per_row = M % 2 == 1
    x = Operand(M, K, E4M3, mx, 1, 1.0, per_row, ld=ref.up(K, 16) + 16 * (M % 3))
    w = Operand(2 * F, K, E4M3, mx, 2, 1.3 / np.sqrt(K), per_row, groups=True)
    o = Out(M, F, mx, 1, kept=kept, layouts=3 if not mx or M % 32 == 0 else 1)
    forward(x, w, o)
    torch.cuda.synchronize()
    (g, tg), (u, tu) = (ref.product(x.v, h) for h in (w.v[:F], w.v[F:]))
    tg, tu = tg + 2 ** -23 * np.abs(g), tu + 2 ** -23 * np.abs(u)
    h, th = ref.swiglu(g, tg, u, tu)
    what = f"{M}x{F}x{K}"
    o.check([h], [th], what)
    if kept == "bf16":
        for i, (v, t) in enumerate(((g, tg), (u, tu))):
            nref.assert_within(nref.f64(o.gu[:, i * F:(i + 1) * F]), v, ref.bf16_tol(v, t), what + " gate|up")
        assert (o.gu[:, 2 * F:] == 7).all()
    else:
        W = ref.up(F, 32)
        assert (o.ck.q[:, 2 * W:] == 0xA5).all() and (o.ck.s[:, 2 * W // 32:] == 0xA5).all()
        c = fp8.Checkpoint(o.ck.q[:, :2 * W].contiguous(), o.ck.s[:, :2 * W // 32].contiguous(), E4M3, F, 2)
        ref.check_kept(c, (g, u), (tg, tu), what + " checkpoint")


@pytest.mark.parametrize("mx,M,F,K", sizes(True))
@pytest.mark.parametrize("kept", ["8bit", "bf16"])
def test_backward(mx, M, F, K, kept):
    per_row = M % 2 == 0
    dy = Operand(M, K, E5M2, mx, 3, 0.05, per_row)
    wd = Operand(F, K, E4M3, mx, 4, 1.3 / np.sqrt(F), per_row, ld=ref.up(K, 16) + 16 * (F % 3))
    gu = (torch.from_numpy(np.random.RandomState(5).randn(M, 2 * F)) * 1.5).bfloat16().to(DEV)
    W = ref.up(F, 32)
    if kept == "8bit":
        c = fp8.checkpoint(gu, E5M2, parts=2)
        buf = full((M, 2 * W + 32))
        buf[:, :2 * W] = c.q
        for i in range(2):
            buf[:, i * W + F:(i + 1) * W] = 0x7F  # NaN behind a part's columns: not read into the result
        src = dict(q=buf, ld_q=2 * W + 32, s=c.s, ld_s=c.s.stride(0), ckpt_fmt=E5M2)
        g, u = np.split(nref.restore(c.q, c.s, F, 2, E5M2), 2, 1)
    else:
        buf = full((M, 2 * F + 16), torch.bfloat16)
        buf[:, :2 * F] = gu
        src = dict(gate_up=buf, ld_gu=2 * F + 16)
        g, u = np.split(nref.f64(gu), 2, 1)
    o = Out(M, F, mx, 2, fmt=E4M3 if M % 2 else E5M2, layouts=3 if not mx or M % 32 == 0 else 1)
    backward(dy, wd, src, o)
    torch.cuda.synchronize()
    dh, t = ref.product(dy.v, wd.v)
    t = t + 2 ** -23 * np.abs(dh)
    dg, tg, du, tu = ref.swiglu_backward(g, u, dh, t)
    o.check([dg, du], [tg, tu], f"{M}x{F}x{K}")


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("layouts,h,kept", [(0, True, None), (1, False, None), (2, False, "8bit"), (0, False, "bf16"),
                                            (3, False, None)])
def test_each_output_alone(mx, layouts, h, kept):
    x, w = Operand(64, 128, E4M3, mx, 1, 1.0), Operand(320, 128, E4M3, mx, 2, 0.1, groups=True)
    both = Out(64, 160, mx, 1, kept=kept)
    o = Out(64, 160, mx, 1, h=h, kept=kept, layouts=layouts)
    forward(x, w, both)
    forward(x, w, o)
    torch.cuda.synchronize()
    for a, b, on in ((o.q, both.q, layouts & 1), (o.qt, both.qt, layouts & 2), (o.h, both.h, h)):
        if on:
            assert torch.equal(a, b)
        elif a is not None:
            assert (a == 0xA5).all()
    if kept == "8bit":
        assert torch.equal(o.ck.q, both.ck.q) and torch.equal(o.ck.s, both.ck.s)
    if kept == "bf16":
        assert torch.equal(o.gu, both.gu)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("M", [96, 160])
def test_far_gates_nan_and_inf(mx, M):
    """Gates far below zero give zeros; what is not finite stays in its row."""
    F = K = 128
    x, w = Operand(M, K, E4M3, mx, 1, 1.0), Operand(2 * F, K, E4M3, mx, 2, 0.2, groups=True)
    dy, wd = Operand(M, K, E4M3, mx, 3, 1.0), Operand(F, K, E4M3, mx, 4, 0.1)
    gu = torch.randn((M, 2 * F)).bfloat16()
    gu[3, 0], gu[3, 1], gu[3, 2], gu[3, 3] = -float("inf"), -200.0, -3e38, 100.0
    gu[7, 5], gu[9, F + 5], gu[11, 6] = float("nan"), float("inf"), float("inf")
    gu = gu.to(DEV)
    o = Out(M, F, mx, 2, layouts=1)
    backward(dy, wd, dict(gate_up=gu, ld_gu=2 * F), o)
    torch.cuda.synchronize()
    d = nref.f64(o.h)
    assert not d[3, :3].any() and not d[3, F:F + 3].any()
    dh = ref.product(dy.v, wd.v)[0]
    assert abs(d[3, 3] - dh[3, 3] * float(gu[3, F + 3])) <= 2 ** -7 * abs(d[3, 3]) + 1e-3
    assert np.isnan(d[7, 5]) and np.isnan(d[7, F + 5]) and np.isinf(d[9, 5]) and np.isinf(d[11, F + 6])
    ok = np.ones(M, bool)
    ok[[7, 9, 11]] = False
    assert np.isfinite(d[ok]).all() and np.isfinite(ref.decode(o.q, E4M3)[ok]).all()
    # an operand's NaN stays in its row of the product
    x.q[5, 7] = 0x7F
    o = Out(M, F, mx, 1, layouts=1, kept="8bit")
    forward(x, w, o)
    torch.cuda.synchronize()
    ok = np.arange(M) != 5
    h = nref.f64(o.h[:, :F])
    assert np.isnan(h[5]).all() and np.isfinite(h[ok]).all()
    assert (o.ck.s[5, :2 * F // 32] == 255).all() and (o.ck.s[torch.from_numpy(ok).to(DEV)][:, :2 * F // 32] != 255).all()


def test_gate_up_has_the_products_bits():
    """The accumulators are those of the plain product."""
    for M in (64, 320):
        x, w = Operand(M, 544, E4M3, True, 1, 1.0), Operand(512, 544, E4M3, True, 2, 0.1)
        r = fp8.mx_swiglu_gemm(x.q, E4M3, x.s, w.q, E4M3, w.s, gate_up=True)
        c = fp8.mx_gemm(x.q, E4M3, x.s, w.q, E4M3, w.s)
        # the same products in another order of tiles: at most the bound of the sum apart
        v, t = ref.product(x.v, w.v)
        nref.assert_within(nref.f64(r.gate_up), nref.f64(c), 2 * ref.bf16_tol(v, t), "gate|up")


def test_no_rows():
    e = torch.empty((0, 128), dtype=torch.uint8, device=DEV)
    w = Operand(256, 128, E4M3, True, 2, 0.1)
    s = torch.empty(0, dtype=torch.uint8, device=DEV)
    r = fp8.mx_swiglu_gemm(e, E4M3, s, w.q, E4M3, w.s, fmt=E4M3, h=True, gate_up=True)
    assert r.h.shape == (0, 128) and r.q.q_row.shape == (0, 128) and r.gate_up.shape == (0, 256)
    b = fp8.mx_swiglu_gemm_backward(e, E4M3, s, w.q[:128], E4M3, w.s, r.gate_up, fmt=E4M3, d_gate_up=True)
    assert b.d_gate_up.shape == (0, 256)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mx", [True, False])
def test_on_a_side_stream_and_replayed(mx):
    x, w = Operand(288, 256, E4M3, mx, 1, 1.0), Operand(512, 256, E4M3, mx, 2, 0.1)

    def run(**kw):
        if mx:
            return fp8.mx_swiglu_gemm(x.q, E4M3, x.s, w.q, E4M3, w.s, fmt=E4M3, checkpoint_fmt=E4M3, **kw)
        amax = torch.zeros(1, device=DEV)
        return fp8.swiglu_gemm(x.q, E4M3, w.q, E4M3, x.s, w.s, fmt=E4M3, checkpoint_fmt=E4M3,
                               scale_in=torch.ones(1, device=DEV), amax_out=amax, **kw)

    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = run(stream=side)
    torch.cuda.synchronize()
    first = x.q.clone()
    graphs = []
    for _ in range(2):  # two graphs of the same call
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = run()
        graphs.append((g, r))
    x.q.zero_()
    for g, _ in graphs:
        g.replay()
    x.q.copy_(first)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for r in (other, *(r for _, r in graphs)):
        assert torch.equal(r.q.q_row, want.q.q_row) and torch.equal(r.q.q_colT, want.q.q_colT)
        assert torch.equal(r.checkpoint.q, want.checkpoint.q) and torch.equal(r.checkpoint.s, want.checkpoint.s)
    assert fp8.fp8_sync_status() == 0


def test_refusals():
    x, w = Operand(64, 128, E4M3, True, 1, 1.0), Operand(256, 128, E4M3, True, 2, 0.1)
    gu = torch.zeros((64, 256), dtype=torch.bfloat16, device=DEV)
    go = lambda **k: fp8.mx_swiglu_gemm(*{**dict(A=x.q, fa=0, sA=x.s, W=w.q, fw=0, sW=w.s), **k}.values(), h=True)  # noqa: E731
    go()
    for bad in (dict(A=x.q.float()), dict(sA=x.s[:16]), dict(sW=w.s[:-16]), dict(W=w.q[:255]), dict(W=w.q[:, :96]),
                dict(A=x.q.cpu()), dict(fa=2)):
        with pytest.raises(fp8.Fp8Error):
            go(**bad)
    with pytest.raises(fp8.Fp8Error):
        fp8.mx_swiglu_gemm(x.q, 0, x.s, w.q, 0, w.s)  # nothing asked for
    for src in (gu[:32], gu[:, :128], gu.float(), fp8.checkpoint(gu, parts=1)):
        with pytest.raises(fp8.Fp8Error):
            fp8.mx_swiglu_gemm_backward(x.q, 0, x.s, w.q[:128], 0, w.s, src, d_gate_up=True)
    one = torch.ones(1, device=DEV)
    for bad in (dict(fmt=0), dict(fmt=0, scale_in=one), dict(fmt=0, scale_in=one, amax_out=one.cpu())):
        with pytest.raises(fp8.Fp8Error):
            fp8.swiglu_gemm(x.q, 0, w.q, 0, one, one, **bad)
    with pytest.raises(fp8.Fp8Error):
        fp8.swiglu_gemm(x.q, 0, w.q, 0, torch.ones(3, device=DEV), one, h=True)
    torch.cuda.synchronize()
