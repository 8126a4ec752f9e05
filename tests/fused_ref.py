"""Float64 references of the norms into 8 bits and of the SwiGLU products, and how
far the kernels may be from them.

A kernel computes a value v in fp32 with an error of at most t (derived below), then
rounds it once: to bf16, off by at most 2^-8 of it, or to 8 bits.

8 bits.  With a scale X the code is rne(v / X), off by at most half a step: 2^-4 of
the value for E4M3 (2^-3 for E5M2), or half the smallest subnormal, 2^-10 (2^-17),
whichever is larger; so |code - v/X| <= h (|v|/X + t/X) + sub + t/X.  A block's scale
byte belongs to some largest magnitude within t of the block's.

Errors t (u = 2^-24):
  * norms: norm_ref.tol_xhat and tol_y without the last rounding.
  * sums of products: every code's product is exact in fp32.  An MMA adds 32 products
    to the accumulator; with each of its K / 32 + 1 results truncated at 2^-21 of
    the sum of magnitudes S (three bits worse than an fp32 truncation):
    t = (K / 32 + 1) 2^-21 S.  Scales applied after: two roundings, 2 u |v|.
  * SwiGLU: e^-g to 2^-16 (|g| log2(e) rounded to fp32, |g| <= 88, times 2 ulp of the
    hardware's exponential), so sigma and 1 - sigma to 2^-15 relative.  h: |dh/dg| <=
    1.1 |u| and |dh/du| = |silu(g)|, so 1.1 |u| tg + |silu| tu + tg tu + 2^-14 |h|.
    d_gate: the slope is at most 1.1 and off by 2^-14 (1 + |g|) s absolutely, at most
    2^-14 * 1.3: 1.1 |u| tdh + |dh u| 2^-13.  d_up: |silu| tdh + 2^-14 |d_up|.
    A gate below -87 gives 0, off by less than 2^-118 of |u| resp. |dh u|, |dh|.
"""
import numpy as np
import torch

import norm_ref as nref

U = 2.0 ** -24
HALF = {0: 2.0 ** -4, 1: 2.0 ** -3}
SUB = {0: 2.0 ** -10, 1: 2.0 ** -17}
EMAX = {0: 8, 1: 15}
FMAX = nref.FMAX


def up(v, unit):
    return (v + unit - 1) // unit * unit


def decode(codes, fmt):
    return nref.decode_table(fmt)[codes.cpu().numpy()]


# --- scale layout -----------------------------------------------------------------


def scale_index(rows, blocks):
    """Byte of block b of row r in the layout of `rows` scale rows."""
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return 4 * ((b // 4) * up(rows, 128) + 128 * (r // 128) + 4 * (r % 32) + (r // 32) % 4) + b % 4


def scales_of(buf, rows, blocks):
    """Scale codes [rows, blocks]; asserts that the rest of the layout is 0."""
    b = buf.cpu().numpy()
    n = up(blocks, 4) * up(rows, 128)
    at = scale_index(rows, blocks)
    rest = np.ones(n, bool)
    rest[at.ravel()] = False
    assert not b[:n][rest].any(), "scale bytes behind the data are not 0"
    return b[at]


def layout_of(codes):
    """Scale codes [rows, blocks] -> the layout's bytes."""
    rows, blocks = codes.shape
    out = np.zeros(max(16, up(blocks, 4) * up(rows, 128)), np.uint8)
    out[scale_index(rows, blocks).ravel()] = codes.ravel()
    return torch.from_numpy(out)


# --- quantize ---------------------------------------------------------------------


def mx_code(amax, fmt):
    """floor(log2 amax) - emax + 127 in [0, 254]; 0 for 0."""
    m, e = np.frexp(amax)
    return np.where(amax > 0, np.clip(e - 1 - EMAX[fmt] + 127, 0, 254), 0).astype(np.int64)


def mx_quantize(v, fmt):
    """float64 [R, C] -> (u8 codes, scale codes [R, C / 32])."""
    b = v.reshape(v.shape[0], -1, 32)
    s = mx_code(np.abs(b).max(2), fmt)
    t = np.clip(b * np.exp2(127.0 - s)[..., None], -FMAX[fmt], FMAX[fmt])
    q = torch.from_numpy(nref.round_to_grid(t, fmt)).to(torch.float32).to(nref.TORCH_FP8[fmt]).view(torch.uint8)
    return q.reshape(v.shape), s.astype(np.uint8)


def close_codes(got, want, tol, fmt, what):
    """got: decoded codes; want, tol: in the codes' units, want not yet held to the range."""
    want = np.clip(want, -FMAX[fmt], FMAX[fmt])
    nref.assert_within(got, want, HALF[fmt] * (np.abs(want) + tol) + SUB[fmt] + tol, what)


def check_mx(codes, scales, v, tol, fmt, what):
    """codes u8 [R, C] and scale codes [R, C / 32] against v, tol [R, C]."""
    R, C = v.shape
    t = decode(codes, fmt).reshape(R, -1, 32)
    b, e = v.reshape(R, -1, 32), np.broadcast_to(tol, v.shape).reshape(R, -1, 32)
    bad = ~np.isfinite(b).all(2)
    assert (scales[bad] == 255).all() and np.isnan(t[bad]).all(), what + ": blocks with a NaN or Inf"
    b, e = np.where(bad[..., None], 0.0, b), np.where(bad[..., None], 0.0, e)
    lo, hi = np.maximum(np.abs(b) - e, 0).max(2), (np.abs(b) + e).max(2)
    ok = (scales >= mx_code(lo, fmt)) & (scales <= mx_code(hi, fmt)) | bad
    assert ok.all(), (what, "scales", np.argwhere(~ok)[:3], scales[~ok][:3], mx_code(hi, fmt)[~ok][:3])
    inv = np.exp2(127.0 - scales.astype(np.float64))[..., None]
    got = np.where(bad[..., None], 0.0, t)
    close_codes(got, b * inv, e * inv, fmt, what)


def check_scaled(codes, scale, v, tol, fmt, what):
    """codes against v scale (a stored or a row's scale)."""
    want = v * scale
    close_codes(decode(codes, fmt), want, tol * scale + U * np.abs(want), fmt, what)


def check_kept(c, parts, tol, what):
    """A checkpoint of the float64 parts [M, F] (tol alike) side by side."""
    M, F = parts[0].shape
    W = up(F, 32)
    t, s = decode(c.q, c.fmt), c.s.cpu().numpy()
    for i, (v, e) in enumerate(zip(parts, tol)):
        b = np.zeros((M, W)), np.zeros((M, W))
        b[0][:, :F], b[1][:, :F] = v, e
        got = t[:, i * W:(i + 1) * W]
        assert not got[:, F:].any(), what + ": codes behind the columns"
        lo, hi = (np.maximum(np.abs(b[0]) + k * b[1], 0).reshape(M, -1, 32) for k in (-1, 1))
        code = s[:, i * W // 32:(i + 1) * W // 32]
        e_lo, e_hi = (nref.block_exponents(x, c.fmt)[0] + 127 for x in (lo, hi))
        assert ((code >= e_lo) & (code <= e_hi)).all(), what + ": scales"
        inv = np.repeat(np.exp2(127.0 - code.astype(np.float64)), 32, 1)
        close_codes(got, b[0] * inv, b[1] * inv, c.fmt, what)


# --- products ---------------------------------------------------------------------


def product(a, b):
    """a [M, K], b [N, K] in float64: (a b^T, its error bound)."""
    s = np.abs(a) @ np.abs(b).T
    return a @ b.T, (a.shape[1] / 32 + 1) * 2.0 ** -21 * s


def swiglu(g, tg, u, tu):
    silu = g * nref.sigmoid(g)
    h = silu * u
    return h, 1.1 * np.abs(u) * tg + np.abs(silu) * tu + tg * tu + 2.0 ** -14 * np.abs(h) + 2.0 ** -118 * np.abs(u)


def swiglu_backward(g, u, dh, tdh):
    """(d_gate, its bound, d_up, its bound) from exact gate and up."""
    dg, du = nref.swiglu_backward(g, u, dh)
    silu = g * nref.sigmoid(g)
    tg = 1.1 * np.abs(u) * tdh + 2.0 ** -13 * np.abs(dh * u)
    tu = np.abs(silu) * tdh + 2.0 ** -14 * np.abs(du) + 2.0 ** -118 * np.abs(dh)
    return dg, tg, du, tu


def bf16_tol(v, t):
    return t + 2.0 ** -8 * (np.abs(v) + t) + nref.TINY[torch.bfloat16]
