"""Float64 references of the norm, SwiGLU and checkpoint operators, and the
tolerances their tests use.

Tolerances (u = 2^-24, the fp32 rounding unit; h = half an ulp of the output
type relative to the value, 2^-8 for bf16, 2^-11 for fp16, u for fp32):

  * D = 128 bounds the longest chain of fp32 additions in a row sum (each
    thread adds at most 80 elements of a row of 20480, then a tree), so a row
    sum is off by at most D u times the sum of magnitudes.
  * xh = (x - mu) r is then off by  tx = r (D u mean|x| + u |x|) + D u |xh|
    (the mean's error, the subtraction's, and half the relative error of the
    variance with the reciprocal square root's few ulps).
  * y: |w| tx + 2 u (|xh w| + |b|) + h |y|.
  * dx: with g = dy w known to u, the two row means to D u of their
    magnitudes, and xh to tx:
    r (4 u |g| + D u mean|g| + D u |xh| mean|g xh| + tx |c2| + |xh| mean(|g| tx))
    + 4 u r |dx/r| + h |dx|.
  * dw, db: column chains of at most C = 512 additions at the sizes used:
    C u sum|dy xh| + sum |dy| tx + h |dw|, and C u sum|dy| + h |db|.
  * SwiGLU: the fast exponential and divide err by less than 2^-20 relative
    in sigma and in its complement; each gradient is within 2^-18 |dh u|
    max(1, |g|) resp. 2^-18 |dh g| of the formula plus the output's rounding
    2^-8; h within one bf16 ulp, 2^-7 relative.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
D, C = 128, 512
FMAX = {0: 448.0, 1: 57344.0}
TORCH_FP8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
BLOCK = 32


def f64(t):
    return t.detach().cpu().double().numpy()


def width(cols):
    return (cols + BLOCK - 1) // BLOCK * BLOCK


# --- checkpoints ----------------------------------------------------------------

def decode_table(fmt):
    return torch.arange(256, dtype=torch.uint8).view(TORCH_FP8[fmt]).double().numpy()


def block_exponents(v, fmt):
    """v [..., 32] -> (e, bad): e the smallest integer with amax <= fmax 2^e,
    clamped to [-127, 127] (-127 for zero blocks), bad: NaN or Inf inside."""
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    m, e = np.frexp(amax / (FMAX[fmt] / 448.0) / 448.0)   # exact: fmax = 7 * 2^k, but 1/7 is not, so test both sides
    e = e.astype(np.int64)
    for _ in range(2):
        e = np.where((amax > 0) & (amax > FMAX[fmt] * np.exp2(e.astype(np.float64))), e + 1, e)
        e = np.where((amax > 0) & (amax <= FMAX[fmt] * np.exp2(e.astype(np.float64) - 1)), e - 1, e)
    return np.where(amax > 0, np.clip(e, -127, 127), -127), bad


def round_to_grid(t, fmt):
    """t / X (|t| <= fmax) rounded to nearest even on the format's grid."""
    bits, low = (3, -6) if fmt == 0 else (2, -14)
    binade = np.floor(np.log2(np.where(t == 0, 1.0, np.abs(t))))
    # log2 can round up across a power of two
    binade = np.where(np.exp2(binade) > np.abs(t), binade - 1, binade)
    step = np.exp2(np.maximum(np.where(t == 0, low, binade), low) - bits)
    return np.round(t / step) * step


def checkpoint(x, parts, fmt):
    """float64 [rows, parts * cols] -> (value on the fp8 grid before scaling
    [rows, parts * W], scale bytes [rows, parts * W / 32])."""
    n, c = x.shape[0], x.shape[1] // parts
    v = np.zeros((n, parts, width(c)))
    v[:, :, :c] = x.reshape(n, parts, c)
    v = v.reshape(n, -1, BLOCK)
    e, bad = block_exponents(v, fmt)
    t = np.where(bad[..., None], np.nan, round_to_grid(np.where(bad[..., None], 0.0, v) * np.exp2(-e[..., None].astype(np.float64)), fmt))
    return t.reshape(n, -1), np.where(bad, 255, e + 127).reshape(n, -1)


def restore(codes, scales, cols, parts, fmt):
    """Codes and scale bytes (any tensors) -> float64 [rows, parts * cols]."""
    n = codes.shape[0]
    t = decode_table(fmt)[codes.cpu().numpy()].reshape(n, -1, BLOCK)
    s = scales.cpu().numpy().astype(np.float64)
    x = np.where(s == 255, np.nan, np.exp2(s - 127))
    v = (t * x[..., None]).reshape(n, parts, -1)[:, :, :cols]
    return v.reshape(n, parts * cols)


# --- norms ----------------------------------------------------------------------

def norm_forward(x, w, b, rms, eps):
    """float64 in and out: (y, mean, rstd, xhat)."""
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    xh = d * rstd[:, None]
    return xh * w + b, mean, rstd, xh


def norm_backward(dy, xh, rstd, w, rms):
    """(dx, dw, db)."""
    g = dy * w
    c1 = 0.0 if rms else g.mean(1, keepdims=True)
    c2 = (g * xh).mean(1, keepdims=True)
    return rstd[:, None] * (g - c1 - xh * c2), (dy * xh).sum(0), dy.sum(0)


def tol_xhat(x, rstd, xh):
    r = rstd[:, None]
    return r * (D * U * np.abs(x).mean(1, keepdims=True) + U * np.abs(x)) + D * U * np.abs(xh)


def tol_y(y, x, rstd, xh, w, b, dtype):
    return np.abs(w) * tol_xhat(x, rstd, xh) + 2 * U * (np.abs(xh * w) + np.abs(b)) + HALF_ULP[dtype] * np.abs(y) \
        + TINY[dtype]


def tol_dx(dx, dy, xh, rstd, w, tx, rms, dtype):
    g = np.abs(dy * w)
    c2 = np.abs((dy * w * xh).mean(1, keepdims=True))
    inner = 4 * U * g + D * U * g.mean(1, keepdims=True) + D * U * np.abs(xh) * (g * np.abs(xh)).mean(1, keepdims=True)
    inner = inner + tx * c2 + np.abs(xh) * (g * tx).mean(1, keepdims=True)
    return rstd[:, None] * inner + (4 * U + HALF_ULP[dtype]) * np.abs(dx) + TINY[dtype]


def tol_dw(dw, dy, xh, tx, dtype):
    return C * U * np.abs(dy * xh).sum(0) + (np.abs(dy) * tx).sum(0) + HALF_ULP[dtype] * np.abs(dw) + TINY[dtype]


def tol_db(db, dy, dtype):
    return C * U * np.abs(dy).sum(0) + HALF_ULP[dtype] * np.abs(db) + TINY[dtype]


# --- SwiGLU ---------------------------------------------------------------------

def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + t), t / (1 + t))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_backward(g, u, dh):
    s = sigmoid(g)
    return dh * u * s * (1 + g * sigmoid(-g)), dh * g * s


def tol_swiglu_backward(dg, du, g, u, dh):
    lim = 2.0 ** -18
    a = lim * np.abs(dh * u) * np.maximum(1, np.abs(g)) + 2.0 ** -8 * np.abs(dg) + 2.0 ** -133
    b = lim * np.abs(dh * g) + 2.0 ** -8 * np.abs(du) + 2.0 ** -133
    return a, b


def assert_within(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol) & ~(np.isnan(got) & np.isnan(ref))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside, first at {i}: {got[i]} for {ref[i]} "
                             f"(off {abs(got[i] - ref[i])}, allowed {np.broadcast_to(tol, ref.shape)[i]})")
