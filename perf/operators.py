"""Workloads of the normalization, 8-bit checkpoint and SwiGLU operators: their
plain forms in elementary torch operations, and the calls of this package.

The block they come from is a pre-norm SwiGLU MLP trained in FP8: a layer or RMS
norm in front of the quantize of the gate|up projection's input, the SwiGLU
between the projections, and the backward pass through both.  What the backward
needs of them (the normalized rows, gate|up) is kept in 8 bits.

A checkpoint: each row in blocks of 32; a block's scale is 2^e, the smallest
power of two with amax <= fp8_max * 2^e, e in [-127, 127], stored as the byte
e + 127; each element is rne_fp8(v * 2^-e).  `parts` tensors of the same width
side by side (gate | up) each start a block of their own.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 32
EPS = 1e-5
LARGEST = 32768 * 7168


def norm(op, rows, cols, kind, x="bf16", y="bf16", w="bf16", pad=0, **more):
    return dict(op=op, rows=rows, cols=cols, kind=kind, x=x, y=y, w=w, pad=pad, **more)


def listed():
    return [
        # one token of a Llama-3-8B sized block: latency
        dict(norm("norm_forward", 1, 4096, "layer"), name="norm fwd 1x4096"),
        # the norm in front of the MLP benchmark's 8192 tokens
        dict(norm("norm_forward", 8192, 4096, "layer"), name="norm fwd 8192x4096"),
        # top-8 routed width of the MoE layer, residual stream kept in fp32
        dict(norm("norm_forward", 32768, 7168, "rms", x="f32"), name="rms fwd f32 32768x7168"),
        # the same norm's backward, from the bf16 input
        dict(norm("norm_backward", 8192, 4096, "layer", w="f32"), name="norm bwd 8192x4096"),
        # a width and a row stride that no vector load fits
        dict(norm("norm_backward", 3001, 1111, "layer", x="f16", y="f16", w="f32", pad=2), name="norm bwd 3001x1111"),
        # forward and backward through the 8-bit checkpoint: a short sequence's
        # tail, and a long batch of the MoE model's hidden size
        dict(norm("norm_step", 16, 7168, "rms", fmt="e4m3"), name="rms step ckpt 16x7168"),
        dict(norm("norm_step", 32768, 7168, "layer", fmt="e4m3"), name="norm step ckpt 32768x7168"),
        # SwiGLU of the Llama MLP benchmark, forward and backward through the checkpoint
        dict(op="swiglu_step", rows=8192, cols=14336, fmt="e4m3", name="swiglu step 8192x14336"),
        # the same of a handful of tokens and an expert width that is no multiple of 32
        dict(op="swiglu_step", rows=7, cols=1500, fmt="e4m3", name="swiglu step 7x1500"),
        # backward of the MoE experts' SwiGLU from a checkpoint in hand; h once more for the down projection's wgrad
        dict(op="swiglu_backward", rows=32768, cols=2048, fmt="e4m3", again=True, name="swiglu bwd 32768x2048"),
        # any activation to 8 bits and back: the MLP's hidden tensor, and a ragged one of the wider-range format
        dict(op="checkpoint", rows=8192, cols=14336, x="bf16", fmt="e4m3", pad=0, name="ckpt 8192x14336"),
        dict(op="checkpoint", rows=513, cols=2999, x="f32", fmt="e5m2", pad=5, name="ckpt f32 513x2999"),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_forward", "norm_backward", "norm_step", "swiglu_step", "swiglu_backward", "checkpoint"])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    cols = size(48, 16384)
    if rng.random() < 0.6:  # most models' widths are multiples of 64
        cols = max(64, cols // 64 * 64)
    most = LARGEST // 4 if op.startswith("swiglu") else LARGEST // 2
    rows = min(size(1, 40000), max(1, most // cols))
    pad = rng.choice([0, 0, 0, 8, rng.randrange(1, 40)])
    kind = rng.choice(["layer", "rms"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm_forward" or op == "norm_backward":
        y = rng.choice(["bf16", "f32"]) if x == "f32" else x
        return norm(op, rows, cols, kind, x, y, rng.choice(["f32", y]), pad)
    if op == "norm_step":  # the benchmark configurations' type: everything bf16
        return norm(op, rows, cols, kind, pad=pad, fmt=fmt)
    if op == "swiglu_step":
        return dict(op=op, rows=rows, cols=cols, fmt=fmt)
    if op == "swiglu_backward":
        return dict(op=op, rows=rows, cols=cols, fmt=fmt, again=rng.random() < 0.5)
    return dict(op=op, rows=rows, cols=cols, x=x, fmt=fmt, pad=pad)


def width(cols):
    return (cols + BLOCK - 1) // BLOCK * BLOCK


def work(case):
    n, c, op = case["rows"], case["cols"], case["op"]
    ck = n * width(c) * (1 + 1 / BLOCK)  # bytes of one part's codes and scales
    if op.startswith("norm"):
        ex, ey, ew = SIZE[case["x"]], SIZE[case["y"]], SIZE[case["w"]]
        layer = case["kind"] == "layer"
        stats = n * (8 if layer else 4)
        params = c * ew * (2 if layer else 1)
        if op == "norm_forward":
            return {"bytes": n * c * (ex + ey) + stats + params, "flops": 8 * n * c}
        grads = c * ew * (2 if layer else 1)
        if op == "norm_backward":
            return {"bytes": n * c * (2 * ex + ey) + stats + c * ew + grads, "flops": 14 * n * c}
        # the checkpoint is written by the forward and read by the backward
        return {"bytes": n * c * (2 * ex + 2 * ey) + 2 * ck + 2 * stats + params + c * ew + grads, "flops": 26 * n * c}
    if op == "swiglu_step":  # gate|up -> h, checkpoint; dh, checkpoint -> d gate|up
        return {"bytes": n * c * (4 + 2 + 2 + 4) + 4 * ck, "flops": 30 * n * c}
    if op == "swiglu_backward":
        return {"bytes": n * c * (2 + 4 + (2 if case["again"] else 0)) + 2 * ck, "flops": 18 * n * c}
    return {"bytes": 2 * n * c * SIZE[case["x"]] + 2 * ck, "flops": 4 * n * c}


# --- inputs -------------------------------------------------------------------


def rows_of(gen, n, c, dtype, pad, scale=1.0, outliers=False):
    """[n, c] values in rows of c + pad.  With outliers, as a residual stream has
    them: channels of unequal size, one in 256 twenty times the others."""
    buf = torch.empty((n, c + pad), dtype=dtype, device="cuda")
    per = torch.full((c,), scale, device="cuda")
    if outliers:
        per = per * torch.exp(0.4 * torch.randn(c, generator=gen, device="cuda"))
        per = torch.where(torch.rand(c, generator=gen, device="cuda") < 1 / 256, 20 * per, per)
    buf.zero_()
    buf[:, :c] = (torch.randn((n, c), generator=gen, device="cuda") + (0.05 if outliers else 0.0)) * per
    return buf[:, :c]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, c, op = case["rows"], case["cols"], case["op"]
    s = dict(case)
    if op.startswith("norm"):
        tx, ty, tw = (DTYPES[case[k]] for k in ("x", "y", "w"))
        s["xs"] = rows_of(gen, n, c, tx, case["pad"], outliers=True)
        s["weight"] = (1 + 0.2 * torch.randn(c, generator=gen, device="cuda")).to(tw)
        s["bias"] = (0.1 * torch.randn(c, generator=gen, device="cuda")).to(tw) if case["kind"] == "layer" else None
        if op != "norm_forward":
            s["dy"] = rows_of(gen, n, c, ty, case["pad"], scale=0.02)
        if op == "norm_backward":  # the forward's statistics, kept from it
            s["mean"], s["rstd"] = statistics(s["xs"], case["kind"])
        return s
    if op == "checkpoint":
        s["xs"] = rows_of(gen, n, c, DTYPES[case["x"]], case["pad"], scale=1.5)
        return s
    gate_up = rows_of(gen, n, 2 * c, torch.bfloat16, 0, scale=1.5)
    s["dh"] = rows_of(gen, n, c, torch.bfloat16, 0, scale=0.02)
    if op == "swiglu_step":
        s["gate_up"] = gate_up
    else:
        s["codes"], s["scales"] = store(gate_up, 2, case["fmt"])
    return s


# --- the operators in plain form ------------------------------------------------


def statistics(x, kind):
    x = x.float()
    mean = x.mean(1) if kind == "layer" else None
    d = x - mean[:, None] if kind == "layer" else x
    return mean, torch.rsqrt((d * d).mean(1) + EPS)


def normalized(x, mean, rstd):
    x = x.float()
    return (x if mean is None else x - mean[:, None]) * rstd[:, None]


def store(x, parts, fmt):
    """Codes [rows, parts * width] and scale bytes of `parts` equal parts of x."""
    n, c = x.shape[0], x.shape[1] // parts
    v = torch.zeros((n, parts, width(c)), dtype=torch.float32, device=x.device)
    v[:, :, :c] = x.reshape(n, parts, c)
    v = v.view(n, -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))  # amax = m 2^e, m in [1/2, 1); fp8_max = 7/8 2^k
    k = 9 if fmt == "e4m3" else 16
    e = torch.clamp(e - k + (m > 0.875), -127, 127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    codes = torch.ldexp(v, -e[:, :, None]).to(CODES[fmt]).view(torch.uint8)
    return codes.view(n, -1), (e + 127).to(torch.uint8)


def load(codes, scales, parts, c, fmt):
    """[rows, parts * c] in fp32."""
    n = codes.shape[0]
    v = codes.view(CODES[fmt]).view(n, -1, BLOCK).float()
    v = torch.ldexp(v, (scales.to(torch.int32) - 127)[:, :, None])
    return v.view(n, parts, -1)[:, :, :c].reshape(n, parts * c)


def plain_norm_backward(s, xhat, rstd):
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    c2 = (g * xhat).mean(1, keepdim=True)
    d = g - xhat * c2
    if s["kind"] == "layer":
        d = d - g.mean(1, keepdim=True)
    out = {"dx": (d * rstd[:, None]).to(DTYPES[s["x"]]), "dw": (dy * xhat).sum(0).to(DTYPES[s["w"]])}
    if s["kind"] == "layer":
        out["db"] = dy.sum(0).to(DTYPES[s["w"]])
    return out


def plain_norm_forward(s, xhat):
    y = xhat * s["weight"].float()
    return (y if s["bias"] is None else y + s["bias"].float()).to(DTYPES[s["y"]])


def plain_swiglu_backward(gate_up, dh):
    g, u = gate_up.chunk(2, 1)
    dh = dh.float()
    sg = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1).to(torch.bfloat16)


def plain_swiglu(gate_up):
    g, u = gate_up.chunk(2, 1)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


def plain(s):
    op = s["op"]
    if op == "norm_backward":
        return plain_norm_backward(s, normalized(s["xs"], s["mean"], s["rstd"]), s["rstd"])
    if op.startswith("norm"):
        mean, rstd = statistics(s["xs"], s["kind"])
        xhat = normalized(s["xs"], mean, rstd)
        out = {"y": plain_norm_forward(s, xhat), "rstd": rstd}
        if mean is not None:
            out["mean"] = mean
        if op == "norm_step":
            xhat = load(*store(xhat, 1, s["fmt"]), 1, s["cols"], s["fmt"])
            out.update(plain_norm_backward(s, xhat, rstd))
        return out
    if op == "checkpoint":
        return load(*store(s["xs"], 1, s["fmt"]), 1, s["cols"], s["fmt"]).to(DTYPES[s["x"]])
    if op == "swiglu_step":
        kept = store(s["gate_up"], 2, s["fmt"])
        return {"h": plain_swiglu(s["gate_up"].float()),
                "d_gate_up": plain_swiglu_backward(load(*kept, 2, s["cols"], s["fmt"]), s["dh"])}
    gate_up = load(s["codes"], s["scales"], 2, s["cols"], s["fmt"])
    out = {"d_gate_up": plain_swiglu_backward(gate_up, s["dh"])}
    if s["again"]:
        out["h"] = plain_swiglu(gate_up)
    return out


# --- the package's operators -----------------------------------------------------


def kernels(s):
    import fp8_mixed_precision_scale_gb300 as fp8

    op = s["op"]
    fmt = {"e4m3": fp8.E4M3FN, "e5m2": fp8.E5M2}[s["fmt"]] if "fmt" in s else None
    if op.startswith("norm"):
        kind = fp8.LAYER_NORM if s["kind"] == "layer" else fp8.RMS_NORM
        out = {}
        if op == "norm_backward":
            src, mean, rstd = s["xs"], s["mean"], s["rstd"]
        else:
            f = fp8.norm_forward(s["xs"], s["weight"], s["bias"], kind=kind, eps=EPS, out_dtype=DTYPES[s["y"]],
                                 checkpoint_fmt=fmt)
            out = {"y": f.y, "rstd": f.rstd}
            if f.mean is not None:
                out["mean"] = f.mean
            src, mean, rstd = f.checkpoint, f.mean, f.rstd
        if op != "norm_forward":
            b = fp8.norm_backward(s["dy"], src, mean, rstd, s["weight"], kind=kind, dx_dtype=DTYPES[s["x"]])
            out["dx"], out["dw"] = b.dx, b.dweight
            if s["kind"] == "layer":
                out["db"] = b.dbias
        return out
    if op == "checkpoint":
        return fp8.checkpoint_restore(fp8.checkpoint(s["xs"], fmt), DTYPES[s["x"]])
    if op == "swiglu_step":
        h, kept = fp8.swiglu_checkpoint(s["gate_up"], fmt)
        return {"h": h, "d_gate_up": fp8.swiglu_backward(s["dh"], kept)}
    kept = fp8.Checkpoint(s["codes"], s["scales"], fmt, s["cols"], parts=2)
    if s["again"]:
        d, h = fp8.swiglu_backward(s["dh"], kept, return_h=True)
        return {"d_gate_up": d, "h": h}
    return {"d_gate_up": fp8.swiglu_backward(s["dh"], kept)}


def run(state):
    return kernels(state) if own else plain(state)


# --- in 64 bits --------------------------------------------------------------------


def exact_kept(v, fmt):
    """What a checkpoint of v (float64, blocks along the last axis from its start)
    gives back: each value on the grid of its block's scale and its own binade."""
    n, c = v.shape
    p = torch.nn.functional.pad(v, (0, width(c) - c)).view(n, -1, BLOCK)
    amax = p.abs().amax(2, keepdim=True)
    unit = torch.exp2(torch.clamp(torch.ceil(torch.log2(amax / FMAX[fmt])), -127, 127))
    unit = torch.where(amax > 0, unit, torch.ones_like(unit))
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    t = p / unit
    binade = torch.clamp(torch.floor(torch.log2(t.abs())), min=low)
    grid = torch.exp2(binade - bits)
    return (torch.round(t / grid) * grid * unit).view(n, -1)[:, :c]


def exact_rows(case, s, i, j):
    """The outputs of rows i..j-1 in float64; dw and db are these rows' share."""
    op = case["op"]
    out = {}
    if op.startswith("norm"):
        x = s["xs"][i:j].double()
        layer = case["kind"] == "layer"
        w = s["weight"].double()
        if op == "norm_backward":  # the statistics are inputs
            mean, rstd = s["mean"][i:j].double() if layer else 0.0, s["rstd"][i:j].double()
        else:
            mean = x.sum(1) / case["cols"] if layer else 0.0
            var = ((x - (mean[:, None] if layer else 0.0)) ** 2).sum(1) / case["cols"]
            rstd = 1 / torch.sqrt(var + EPS)
        xh = (x - (mean[:, None] if layer else 0.0)) * rstd[:, None]
        if op != "norm_backward":
            out["y"] = xh * w + (s["bias"].double() if layer else 0.0)
            out["rstd"] = rstd
            if layer:
                out["mean"] = mean
        if op == "norm_step":
            xh = exact_kept(xh, case["fmt"])
        if op != "norm_forward":
            dy = s["dy"][i:j].double()
            c2 = (dy * w * xh).sum(1) / case["cols"]
            c1 = (dy * w).sum(1) / case["cols"] if layer else torch.zeros_like(c2)
            out["dx"] = rstd[:, None] * (dy * w - c1[:, None] - xh * c2[:, None])
            out["dw"] = (dy * xh).sum(0)
            if layer:
                out["db"] = dy.sum(0)
        return out
    if op == "checkpoint":
        return {"x": exact_kept(s["xs"][i:j].double(), case["fmt"])}
    c = case["cols"]
    if op == "swiglu_step":
        g, u = s["gate_up"][i:j, :c].double(), s["gate_up"][i:j, c:].double()
        out["h"] = g * torch.sigmoid(g) * u
        g, u = exact_kept(g, case["fmt"]), exact_kept(u, case["fmt"])
    else:
        codes = s["codes"][i:j].view(CODES[case["fmt"]]).double()
        v = codes * torch.exp2(s["scales"][i:j].double() - 127).repeat_interleave(BLOCK, 1)
        g, u = v[:, :c], v[:, width(c):width(c) + c]
        if case["again"]:
            out["h"] = g * torch.sigmoid(g) * u
    dh = s["dh"][i:j].double()
    sg = torch.sigmoid(g)
    out["d_gate_up"] = torch.cat([dh * u * (sg + g * sg * torch.sigmoid(-g)), dh * g * sg], 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n = case["rows"]
    step = max(1, (1 << 25) // case["cols"])
    got = [exact_rows(case, s, i, min(n, i + step)) for i in range(0, n, step)]
    out = {k: sum(p[k] for p in got) if k in ("dw", "db") else torch.cat([p[k] for p in got]) for k in got[0]}
    return out["x"] if case["op"] == "checkpoint" else out
