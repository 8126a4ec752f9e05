"""Workloads of the operators that run straight into and out of the FP8 matrix
products of a SwiGLU block: their plain forms in elementary torch operations, and
the calls of this package.

    sum = x + residual,  y = norm(sum) w + b, quantized        (norm_quantize)
    gate | up = y W^T,  h = silu(gate) up, quantized           (swiglu_gemm)
    dh = dY W_down,  d_gate | d_up from it and the kept gate | up, quantized
                                                               (swiglu_gemm_backward)
    d_sum = the norm's backward of dy, plus the gradient that reaches the sum past
            the norm                                           (norm_backward with dsum)

Three recipes.  `mx`: blocks of 32 along the contraction share a scale 2^e, e =
floor(log2 amax) - 8, stored as the byte e + 127; elements sat_rne_e4m3(v 2^-e).
`row`: one fp32 scale per row, 448 / amax.  `tensor`: a stored scale per tensor, the
current amax beside it.  Everything in 8 bits is E4M3 here, and comes back as the
float8 values of the codes and, for `mx`, of the scale bytes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
FMAX = 448.0
EPS = 1e-5
MOST_NORM = 32768 * 7168
MOST_FFN = 8192 * 4096 * 14336


def norm(op, rows, cols, kind, recipe, both, x="bf16", r="bf16", w="bf16", pad=0):
    return dict(op=op, rows=rows, cols=cols, kind=kind, recipe=recipe, both=both, x=x, r=r, w=w, pad=pad)


def ffn(op, tokens, hidden, ffn, recipe, both=True, keep="8bit"):
    return dict(op=op, tokens=tokens, hidden=hidden, ffn=ffn, recipe=recipe, both=both, keep=keep)


def listed():
    return [
        # one token of a Llama-3-8B sized block, for serving: latency
        dict(norm("norm_quantize", 1, 4096, "rms", "row", False), name="norm row 1x4096"),
        # in front of the MLP benchmark's gate|up projection, both operands of training
        dict(norm("norm_quantize", 8192, 4096, "rms", "mx", True), name="norm mx 8192x4096"),
        # top-8 routed width of the MoE model's hidden size, residual stream in fp32
        dict(norm("norm_quantize", 32768, 7168, "rms", "mx", True, r="f32", w="f32"), name="norm mx f32 32768x7168"),
        # the delayed recipe, a layer norm, odd rows and a width that is no multiple of 128
        dict(norm("norm_quantize", 3001, 1104, "layer", "tensor", True, x="f16", r="f16", w="f32", pad=2),
             name="norm tensor 3001x1104"),
        # a training step through the norm: forward, and backward with the gradient past it
        dict(norm("norm_step", 8192, 4096, "rms", "mx", True), name="norm step 8192x4096"),
        dict(norm("norm_step", 77, 7168, "layer", "row", False, r="f32"), name="norm step 77x7168"),
        # one token through the gate|up projection: the weights are read, little else
        dict(ffn("ffn_forward", 1, 4096, 14336, "mx", False, ""), name="ffn fwd 1x4096x14336"),
        # the MLP benchmark's 8192 tokens in training: h in both layouts, gate|up kept in 8 bits
        dict(ffn("ffn_forward", 8192, 4096, 14336, "mx"), name="ffn fwd 8192x4096x14336"),
        # a ragged batch of the rowwise recipe: h and gate|up in bf16
        dict(ffn("ffn_forward", 1000, 2064, 1504, "row", False, "bf16"), name="ffn fwd row 1000x2064x1504"),
        # backward of the MLP benchmark's block
        dict(ffn("ffn_backward", 8192, 4096, 14336, "mx"), name="ffn bwd 8192x4096x14336"),
        # forward and backward with the gradients of the input and the weights, an expert's width
        dict(ffn("ffn_step", 4096, 7168, 2048, "mx"), name="ffn step 4096x7168x2048"),
        # the delayed recipe's backward of a short odd batch
        dict(ffn("ffn_backward", 333, 1040, 720, "tensor", True, "bf16"), name="ffn bwd tensor 333x1040x720"),
    ]


def draw(rng):
    def size(lo, hi, unit=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // unit * unit)

    op = rng.choice(["norm_quantize", "norm_quantize", "norm_step", "ffn_forward", "ffn_forward", "ffn_backward",
                     "ffn_step"])
    recipe = rng.choice(["mx", "mx", "row", "tensor"])
    both = recipe != "row" and rng.random() < 0.6
    unit = 32 if recipe == "mx" else 16  # of the contraction that the 8-bit operand goes into
    if op.startswith("norm"):
        cols = size(64, 16384, rng.choice([unit, 64]))
        rows = size(1, 32768)
        rows = min(rows, max(1, MOST_NORM // 2 // cols))
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        r = rng.choice(["", x, x, "f32"])
        if both and recipe == "mx":
            rows = max(32, rows // 32 * 32)
        return norm(op, rows, cols, rng.choice(["layer", "rms"]), recipe, both, x, r,
                    rng.choice(["f32", "f32" if x == "f32" else x]), rng.choice([0, 0, 8, rng.randrange(1, 40)]))
    if op == "ffn_step":
        recipe, both = "mx", True
        unit = 32
    hidden = size(128, 8192, rng.choice([unit, 128]))
    width = size(128, 16384, rng.choice([unit, 128]))
    tokens = min(size(1, 8192), max(1, MOST_FFN // 3 // (hidden * width)))
    if both and recipe == "mx":
        tokens = max(32, tokens // 32 * 32)
    keep = rng.choice(["8bit", "bf16"]) if op != "ffn_forward" else rng.choice(["8bit", "bf16", ""])
    return ffn(op, tokens, hidden, width, recipe, both, keep)


def up(v, unit):
    return (v + unit - 1) // unit * unit


def work(case):
    mx = case["recipe"] == "mx"
    e8 = 1 + 1 / 32 if mx else 1  # bytes of an 8-bit operand's element with its share of the scales
    layouts = 2 if case["both"] else 1
    if case["op"].startswith("norm"):
        n, c = case["rows"], case["cols"]
        ex, ew = SIZE[case["x"]], SIZE[case["w"]]
        er = SIZE[case["r"]] if case["r"] else 0
        layer = case["kind"] == "layer"
        stats = n * (8 if layer else 4) + (4 * n if case["recipe"] == "row" else 0)
        params = c * ew * (2 if layer else 1)
        b = n * c * (ex + 2 * er + layouts * e8) + stats + params
        if case["op"] == "norm_quantize":
            return {"bytes": b, "flops": 10 * n * c}
        es, ey = er or ex, min(2, ex)  # of the sum and of dy; the backward reads sum, dy, dsum and writes d_sum
        return {"bytes": b + n * c * (3 * es + ey) + stats + params + c * ew, "flops": 26 * n * c}
    m, k, f = case["tokens"], case["hidden"], case["ffn"]
    kept = {"8bit": 2 * m * up(f, 32) * (1 + 1 / 32), "bf16": 4 * m * f, "": 0}[case["keep"]]
    out = m * f * (2 if case["recipe"] == "row" else layouts * e8)
    forward = (m * k + 2 * f * k) * e8 + out + kept
    backward = (m * k + f * k) * e8 + kept + 2 * out
    if case["op"] == "ffn_forward":
        return {"bytes": forward, "flops": 4 * m * k * f}
    if case["op"] == "ffn_backward":
        return {"bytes": backward, "flops": 2 * m * k * f}
    # the gradients of the input and of the weights: two more products of 2 f
    grads = (2 * m * f * 2 + 2 * f * k + m * k) * e8 + 2 * m * k + 4 * f * k
    return {"bytes": forward + backward + grads, "flops": 14 * m * k * f}


# --- inputs -------------------------------------------------------------------


def rows_of(gen, n, c, dtype, pad, scale=1.0, outliers=False):
    """[n, c] values in rows of c + pad.  With outliers, as a residual stream has
    them: channels of unequal size, one in 256 twenty times the others."""
    per = torch.full((c,), scale, device="cuda")
    if outliers:
        per = per * torch.exp(0.4 * torch.randn(c, generator=gen, device="cuda"))
        per = torch.where(torch.rand(c, generator=gen, device="cuda") < 1 / 256, 20 * per, per)
    buf = torch.zeros((n, c + pad), dtype=dtype, device="cuda")
    buf[:, :c] = torch.randn((n, c), generator=gen, device="cuda") * per
    return buf[:, :c]


def operand(v, recipe, scale_rows=None):
    """An 8-bit matrix operand of v [R, C], blocks and rows along C: its codes and
    its scales as the package's products take them."""
    if recipe == "mx":
        codes, e = mx_codes(v)
        return codes.view(torch.uint8), mx_layout(e if scale_rows is None else scale_rows(e))
    amax = v.abs().amax(1) if recipe == "row" else v.abs().max().view(1)
    return (v * (FMAX / amax)[:, None]).to(FP8).view(torch.uint8), amax / FMAX


def halves(e):
    """Gate and up rows, each padded to whole groups of 128 rows."""
    f = e.shape[0] // 2
    out = e.new_zeros((2, up(f, 128), e.shape[1]))
    out[:, :f] = e.view(2, f, -1)
    return out.view(-1, e.shape[1])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    recipe = case["recipe"]
    if case["op"].startswith("norm"):
        n, c = case["rows"], case["cols"]
        t = DTYPES[case["r"] or case["x"]]
        s["xs"] = rows_of(gen, n, c, DTYPES[case["x"]], case["pad"], outliers=not case["r"])
        s["res"] = rows_of(gen, n, c, DTYPES[case["r"]], case["pad"], outliers=True) if case["r"] else None
        s["weight"] = (1 + 0.2 * torch.randn(c, generator=gen, device="cuda")).to(DTYPES[case["w"]])
        s["bias"] = (0.1 * torch.randn(c, generator=gen, device="cuda")).to(DTYPES[case["w"]]) \
            if case["kind"] == "layer" else None
        if case["op"] == "norm_step":
            s["dy"] = rows_of(gen, n, c, torch.bfloat16 if t == torch.float32 else t, case["pad"], scale=0.02)
            s["dsum"] = rows_of(gen, n, c, t, case["pad"], scale=0.02)
        # the stored scale of an amax history
        s["scale"] = torch.full((1,), FMAX / 40, device="cuda")
        return s
    m, k, f = case["tokens"], case["hidden"], case["ffn"]
    s["scale"] = torch.full((1,), FMAX / (0.3 if case["op"] == "ffn_backward" else 12.0), device="cuda")
    if case["op"] != "ffn_backward":
        x = rows_of(gen, m, k, torch.float32, 0)
        s["x"], s["sx"] = operand(x, recipe)
        w = rows_of(gen, 2 * f, k, torch.float32, 0, scale=1.28 / math.sqrt(k))
        s["w"], s["sw"] = operand(w, recipe, halves)
    if case["op"] != "ffn_forward":
        s["dy"], s["sdy"] = operand(rows_of(gen, m, k, torch.float32, 0, scale=0.02), recipe)
        # the down projection's transposed layout
        s["wd"], s["swd"] = operand(rows_of(gen, f, k, torch.float32, 0, scale=1.28 / math.sqrt(f)), recipe)
    if case["op"] == "ffn_backward":  # what the forward kept
        gate_up = rows_of(gen, m, 2 * f, torch.bfloat16, 0, scale=1.28)
        if case["keep"] == "8bit":
            s["codes"], s["scales"] = store(gate_up.float())
        else:
            s["gate_up"] = gate_up
    if case["op"] == "ffn_step":
        s["xt"], s["sxt"] = operand(x.t().contiguous(), recipe)
        # the transposed layout of gate|up: gate's and up's rows as groups padded to 128
        w = halves(w).t().contiguous()
        s["wt"], s["swt"] = operand(w, recipe)
    return s


# --- the operators in plain form ------------------------------------------------


def mx_codes(v):
    """Codes [R, C] and scale bytes [R, C / 32] of v."""
    b = v.reshape(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(2))
    e = torch.where(m == 0, torch.full_like(e, -127), torch.clamp(e - 1 - 8, -127, 127))
    q = torch.clamp(torch.ldexp(b, -e[:, :, None]), -FMAX, FMAX).to(FP8)
    return q.view(v.shape), (e + 127).to(torch.uint8)


def mx_layout(e):
    """Scale bytes [R, KB] in the order of the products: [KB / 4][R / 128][32][4][4]."""
    r, kb = e.shape
    p = e.new_zeros((up(r, 128), up(kb, 4)))
    p[:r, :kb] = e
    return p.view(-1, 4, 32, up(kb, 4) // 4, 4).permute(3, 0, 2, 1, 4).reshape(-1)


def mx_values(codes, scales, r, rows=None):
    """The fp32 matrix of codes [R, C] and the scale bytes of r rows; `rows`: those of the codes among them."""
    c = codes.shape[1]
    e = scales.view(up(c // 32, 4) // 4, -1, 32, 4, 4).permute(1, 3, 2, 0, 4).reshape(up(r, 128), -1)[:, :c // 32]
    e = e[:r] if rows is None else e[rows]
    v = codes.view(FP8).float().view(codes.shape[0], -1, 32)
    return torch.ldexp(v, (e.to(torch.int32) - 127)[:, :, None]).view(codes.shape)


def values(codes, scales, recipe, halved=False):
    """The fp32 matrix of an 8-bit operand; `halved`: of gate and up rows in groups."""
    if recipe != "mx":
        return codes.view(FP8).float() * scales[:, None]
    r = codes.shape[0]
    if not halved:
        return mx_values(codes, scales, r)
    f = r // 2
    rows = torch.arange(r, device=codes.device)
    return mx_values(codes, scales, 2 * up(f, 128), torch.where(rows < f, rows, rows - f + up(f, 128)))


def quantized(v, s, out):
    """v in 8 bits by the case's recipe, into `out`."""
    recipe = s["recipe"]
    if recipe == "mx":
        q, e = mx_codes(v)
        out["row"], out["row_scales"] = q, mx_layout(e).view(E8M0)
        if s["both"]:
            q, e = mx_codes(v.t().contiguous())
            out["col"], out["col_scales"] = q, mx_layout(e).view(E8M0)
    elif recipe == "row":
        amax = v.abs().amax(1)
        scale = torch.where(amax > 0, FMAX / amax, torch.ones_like(amax))
        out["row"], out["row_scales"] = (v * scale[:, None]).to(FP8), 1 / scale
    else:
        out["row"] = torch.clamp(v * s["scale"], -FMAX, FMAX).to(FP8)
        if s["both"]:
            out["col"] = out["row"].t().contiguous()
        out["amax"] = v.abs().max().view(1)


def store(gate_up):
    """Codes [M, 2 W] and scale bytes of gate | up, W the width in whole blocks of 32;
    a block's scale is the smallest power of two that leaves nothing above 448."""
    m, f = gate_up.shape[0], gate_up.shape[1] // 2
    v = gate_up.new_zeros((m, 2, up(f, 32)))
    v[:, :, :f] = gate_up.view(m, 2, f)
    v = v.view(m, -1, 32)
    fr, e = torch.frexp(v.abs().amax(2))
    e = torch.where(fr == 0, torch.full_like(e, -127), torch.clamp(e - 9 + (fr > 0.875), -127, 127))
    codes = torch.ldexp(v, -e[:, :, None]).to(FP8).view(torch.uint8)
    return codes.view(m, -1), (e + 127).to(torch.uint8)


def load(codes, scales, f):
    v = codes.view(FP8).view(codes.shape[0], -1, 32).float()
    v = torch.ldexp(v, (scales.to(torch.int32) - 127)[:, :, None])
    return v.view(codes.shape[0], 2, -1)[:, :, :f].reshape(codes.shape[0], -1)


def plain_norm(s):
    x = s["xs"]
    t = x if s["res"] is None else (x.float() + s["res"].float()).to(s["res"].dtype)
    v = t.float()
    mean = v.mean(1) if s["kind"] == "layer" else None
    d = v if mean is None else v - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    xhat = d * rstd[:, None]
    y = xhat * s["weight"].float()
    y = y if s["bias"] is None else y + s["bias"].float()
    out = {"rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    if s["res"] is not None:
        out["sum"] = t
    quantized(y, s, out)
    if s["op"] == "norm_step":
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        ds = g - xhat * (g * xhat).mean(1, keepdim=True)
        if s["kind"] == "layer":
            ds = ds - g.mean(1, keepdim=True)
            out["db"] = dy.sum(0).to(s["weight"].dtype)
        out["d_sum"] = (ds * rstd[:, None] + s["dsum"].float()).to(t.dtype)
        out["dw"] = (dy * xhat).sum(0).to(s["weight"].dtype)
    return out


def plain_forward(s, out):
    g, u = (values(s["x"], s["sx"], s["recipe"]) @ values(s["w"], s["sw"], s["recipe"], True).t()).chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    if s["recipe"] == "row":
        out["h"] = h.to(torch.bfloat16)
    else:
        quantized(h, s, out)
    gate_up = torch.cat([g, u], 1)
    if s["keep"] == "bf16":
        out["gate_up"] = gate_up.to(torch.bfloat16)
    elif s["keep"]:
        out["codes"], out["scales"] = (v.view(t) for v, t in zip(store(gate_up), (FP8, E8M0)))
    return out


def plain_backward(s, kept, out):
    g, u = kept.chunk(2, 1)
    dh = values(s["dy"], s["sdy"], s["recipe"]) @ values(s["wd"], s["swd"], s["recipe"]).t()
    sg = 1 / (1 + torch.exp(-g))
    d = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1)
    if s["recipe"] == "row":
        out["d_gate_up"] = d.to(torch.bfloat16)
        return out
    quantized(d, s, out)
    if s["recipe"] == "mx" and s["ffn"] % 128:  # the row layout's halves start at whole groups of 128
        q, e = mx_codes(halves(d.t()).t())
        out["row"], out["row_scales"] = q, mx_layout(e).view(E8M0)
    return out


def plain(s):
    if s["op"].startswith("norm"):
        return plain_norm(s)
    if s["op"] == "ffn_forward":
        return plain_forward(s, {})
    f = s["ffn"]
    if s["op"] == "ffn_backward":
        kept = s["gate_up"].float() if s["keep"] == "bf16" else load(s["codes"], s["scales"], f)
        return plain_backward(s, kept, {})
    out = plain_forward(s, {})
    kept = out["gate_up"].float() if s["keep"] == "bf16" else \
        load(out["codes"].view(torch.uint8), out["scales"].view(torch.uint8), f)
    d = plain_backward(s, kept, {})
    row, col = (mx_values(d[n].view(torch.uint8), d[n + "_scales"].view(torch.uint8), d[n].shape[0])
                for n in ("row", "col"))
    out["dx"] = (row @ values(s["wt"], s["swt"], "mx").t()).to(torch.bfloat16)
    out["dw"] = (col @ values(s["xt"], s["sxt"], "mx").t()).to(torch.bfloat16)
    return out


# --- the package's operators -----------------------------------------------------


def handed(q, s, out, rows):
    """The 8-bit results of a call as float8 values."""
    out["row"] = q.q_row.view(FP8)
    if s["recipe"] == "mx":
        out["row_scales"] = q.s_row.view(E8M0)
        if s["both"]:
            out["col"], out["col_scales"] = q.q_colT.view(FP8), q.s_col.view(E8M0)
    elif s["recipe"] == "row":
        out["row_scales"] = q.scale_inv_row
    elif s["both"]:
        out["col"] = q.q_colT.view(FP8)[:, :rows]


def own_norm(s, fp8):
    kind = fp8.LAYER_NORM if s["kind"] == "layer" else fp8.RMS_NORM
    layouts = fp8.LAYOUT_ROW | (fp8.LAYOUT_COLT if s["both"] else 0)
    out = {}
    if s["recipe"] == "mx":
        n = fp8.mx_norm_quantize(s["xs"], s["res"], s["weight"], s["bias"], kind=kind, eps=EPS, fmt=fp8.E4M3FN,
                                 layouts=layouts)
    elif s["recipe"] == "row":
        n = fp8.norm_quantize(s["xs"], s["res"], s["weight"], s["bias"], kind=kind, eps=EPS, fmt=fp8.E4M3FN,
                              recipe=fp8.Recipe(kind=fp8.ROWWISE), layouts=layouts)
    else:
        out["amax"] = torch.zeros(1, device=s["xs"].device)
        n = fp8.norm_quantize(s["xs"], s["res"], s["weight"], s["bias"], kind=kind, eps=EPS, fmt=fp8.E4M3FN,
                              recipe=fp8.Recipe(kind=fp8.DELAYED), layouts=layouts, scale_in=s["scale"],
                              amax_out=out["amax"])
    handed(n.q, s, out, s["rows"])
    out["rstd"] = n.rstd
    if n.mean is not None:
        out["mean"] = n.mean
    if s["res"] is not None:
        out["sum"] = n.sum
    if s["op"] == "norm_step":
        b = fp8.norm_backward(s["dy"], n.sum, n.mean, n.rstd, s["weight"], kind=kind, dsum=s["dsum"])
        out["d_sum"], out["dw"] = b.dx, b.dweight
        if b.dbias is not None:
            out["db"] = b.dbias
    return out


def own_forward(s, fp8, out):
    layouts = fp8.LAYOUT_ROW | (fp8.LAYOUT_COLT if s["both"] else 0)
    keep = dict(checkpoint_fmt=fp8.E4M3FN) if s["keep"] == "8bit" else dict(gate_up=bool(s["keep"]))
    x, w, e4m3 = s["x"], s["w"], fp8.E4M3FN
    if s["recipe"] == "mx":
        r = fp8.mx_swiglu_gemm(x, e4m3, s["sx"], w, e4m3, s["sw"], fmt=e4m3, layouts=layouts, **keep)
    elif s["recipe"] == "row":
        r = fp8.swiglu_gemm(x, e4m3, w, e4m3, s["sx"], s["sw"], h=True, **keep)
        out["h"] = r.h
    else:
        out["amax"] = torch.zeros(1, device=x.device)
        r = fp8.swiglu_gemm(x, e4m3, w, e4m3, s["sx"], s["sw"], fmt=e4m3, layouts=layouts, scale_in=s["scale"],
                            amax_out=out["amax"], **keep)
    if r.q is not None:
        handed(r.q, s, out, s["tokens"])
    if r.gate_up is not None:
        out["gate_up"] = r.gate_up
    if r.checkpoint is not None:
        out["codes"], out["scales"] = r.checkpoint.q.view(FP8), r.checkpoint.s.view(E8M0)
    return r


def own_backward(s, fp8, kept, out):
    layouts = fp8.LAYOUT_ROW | (fp8.LAYOUT_COLT if s["both"] else 0)
    dy, wd, e4m3 = s["dy"], s["wd"], fp8.E4M3FN
    if s["recipe"] == "mx":
        return fp8.mx_swiglu_gemm_backward(dy, e4m3, s["sdy"], wd, e4m3, s["swd"], kept, fmt=e4m3, layouts=layouts).q
    if s["recipe"] == "row":
        out["d_gate_up"] = fp8.swiglu_gemm_backward(dy, e4m3, wd, e4m3, s["sdy"], s["swd"], kept,
                                                    d_gate_up=True).d_gate_up
        return None
    out["amax"] = torch.zeros(1, device=dy.device)
    return fp8.swiglu_gemm_backward(dy, e4m3, wd, e4m3, s["sdy"], s["swd"], kept, fmt=e4m3, layouts=layouts,
                                    scale_in=s["scale"], amax_out=out["amax"]).q


def kernels(s):
    import fp8_mixed_precision_scale_gb300 as fp8

    if s["op"].startswith("norm"):
        return own_norm(s, fp8)
    out = {}
    if s["op"] == "ffn_forward":
        own_forward(s, fp8, out)
        return out
    if s["op"] == "ffn_backward":
        kept = s["gate_up"] if s["keep"] == "bf16" else \
            fp8.Checkpoint(s["codes"], s["scales"], fp8.E4M3FN, s["ffn"], parts=2)
        q = own_backward(s, fp8, kept, out)
        if q is not None:
            handed(q, s, out, s["tokens"])
        return out
    r = own_forward(s, fp8, out)
    q = own_backward(s, fp8, r.gate_up if r.checkpoint is None else r.checkpoint, {})
    out["dx"] = fp8.mx_gemm(q.q_row, fp8.E4M3FN, q.s_row, s["wt"], fp8.E4M3FN, s["swt"])
    out["dw"] = fp8.mx_gemm(q.q_colT, fp8.E4M3FN, q.s_col, s["xt"], fp8.E4M3FN, s["sxt"])
    return out


def run(state):
    return kernels(state) if own else plain(state)


# --- in 64 bits --------------------------------------------------------------------
# An 8-bit result is given as what its code would be without the rounding, a value
# over its block's scale held to 448; what an operator reads back of it is rounded.


def exact_blocks(v, whole):
    """v over its blocks' scales, and those: blocks of 32 along the last axis.
    `whole`: a scale that leaves nothing above 448, else one that holds to it."""
    b = v.unflatten(1, (-1, 32))
    amax = b.abs().amax(2)
    e = torch.ceil(torch.log2(amax / FMAX)) if whole else torch.floor(torch.log2(amax)) - 8
    x = torch.exp2(torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127)))
    return (b / x[:, :, None]).clamp(-FMAX, FMAX).flatten(1), x


def exact_rounded(t):
    """t on the grid of E4M3."""
    grid = torch.exp2(torch.clamp(torch.floor(torch.log2(t.abs())), min=-6) - 3)
    return torch.round(t / grid) * grid


def exact_scales(x):
    """Scales [R, KB] where the products want them, 2^-127 in what is left over."""
    r, kb = x.shape
    out = torch.full((up(kb, 4) // 4 * up(r, 128) * 4,), 2.0 ** -127, dtype=torch.float64, device=x.device)
    i, b = torch.arange(r, device=x.device)[:, None], torch.arange(kb, device=x.device)[None]
    at = 4 * ((b // 4) * up(r, 128) + 128 * (i // 128) + 4 * (i % 32) + (i // 32) % 4) + b % 4
    out[at.flatten()] = x.flatten()
    return out


def exact_operand(codes, scales, recipe, row=None):
    """The matrix of an operand; `row`: the scale row of each of its rows."""
    v = codes.view(FP8).double()
    if recipe != "mx":
        return v * scales.double()[:, None]
    i = (torch.arange(v.shape[0], device=v.device) if row is None else row)[:, None]
    b = torch.arange(v.shape[1] // 32, device=v.device)[None]
    r128 = scales.numel() // up(b.shape[1], 4)
    at = 4 * ((b // 4) * r128 + 128 * (i // 128) + 4 * (i % 32) + (i // 32) % 4) + b % 4
    return v * torch.exp2(scales.double()[at] - 127).repeat_interleave(32, 1)


def exact_quantized(v, case, out, padded=None):
    if case["recipe"] == "mx":
        t, x = exact_blocks(v if padded is None else padded, False)
        out["row"], out["row_scales"] = t, exact_scales(x)
        if case["both"]:
            t, x = exact_blocks(v.t().contiguous(), False)
            out["col"], out["col_scales"] = t, exact_scales(x)
    elif case["recipe"] == "row":
        amax = v.abs().amax(1, keepdim=True)
        amax = torch.where(amax > 0, amax, torch.full_like(amax, FMAX))
        out["row"], out["row_scales"] = v * FMAX / amax, amax[:, 0] / FMAX
    else:
        scale = FMAX / (40 if case["op"].startswith("norm") else 0.3 if case["op"] == "ffn_backward" else 12)
        out["row"] = (v * scale).clamp(-FMAX, FMAX)
        if case["both"]:
            out["col"] = out["row"].t().contiguous()
        out["amax"] = v.abs().max().view(1)


def exact_norm(case, s):
    v = s["xs"].double()
    if case["r"]:
        v = v + s["res"].double()
    out = {"sum": v} if case["r"] else {}
    if case["r"]:  # the norm is of the sum as it is stored
        v = v.to(DTYPES[case["r"]]).double()
    layer = case["kind"] == "layer"
    mean = v.sum(1, keepdim=True) / case["cols"] if layer else torch.zeros_like(v[:, :1])
    rstd = 1 / torch.sqrt(((v - mean) ** 2).sum(1, keepdim=True) / case["cols"] + EPS)
    w = s["weight"].double()
    xh = (v - mean) * rstd
    out["rstd"] = rstd[:, 0]
    if layer:
        out["mean"] = mean[:, 0]
    exact_quantized(xh * w + s["bias"].double() if layer else xh * w, case, out)
    if case["op"] == "norm_step":
        dy = s["dy"].double()
        c2 = (dy * w * xh).sum(1, keepdim=True) / case["cols"]
        c1 = (dy * w).sum(1, keepdim=True) / case["cols"] if layer else 0.0
        out["d_sum"] = rstd * (dy * w - c1 - xh * c2) + s["dsum"].double()
        out["dw"] = (dy * xh).sum(0)
        if layer:
            out["db"] = dy.sum(0)
    return out


def exact_kept(v, f):
    """Gate and up, [M, f] each, as a checkpoint gives them back: (g, u, codes, scales)."""
    w = up(f, 32)
    p = torch.cat([torch.nn.functional.pad(t, (0, w - f)) for t in v], 1)
    t, x = exact_blocks(p, True)
    back = exact_rounded(t) * x.repeat_interleave(32, 1)
    return back[:, :f], back[:, w:w + f], t, x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return exact_norm(case, s)
    f, recipe, out = case["ffn"], case["recipe"], {}
    fp = up(f, 128)
    if case["op"] != "ffn_backward":
        x = exact_operand(s["x"], s["sx"], recipe)
        row = torch.arange(2 * f, device=x.device)
        row = row + (fp - f) * (row >= f)
        w = exact_operand(s["w"], s["sw"], recipe, row)
        g, u = x @ w[:f].t(), x @ w[f:].t()
        del x, w
        h = g * torch.sigmoid(g) * u
        if recipe == "row":
            out["h"] = h
        else:
            exact_quantized(h, case, out)
        if case["keep"] == "8bit":
            g, u, out["codes"], out["scales"] = exact_kept((g, u), f)
        elif case["keep"] == "bf16":
            out["gate_up"] = torch.cat([g, u], 1)
            g, u = g.to(torch.bfloat16).double(), u.to(torch.bfloat16).double()
        if case["op"] == "ffn_forward":
            return out
    elif case["keep"] == "8bit":
        kept = s["codes"].view(FP8).double() * torch.exp2(s["scales"].double() - 127).repeat_interleave(32, 1)
        g, u = kept[:, :f], kept[:, up(f, 32):up(f, 32) + f]
    else:
        g, u = s["gate_up"][:, :f].double(), s["gate_up"][:, f:].double()
    dh = exact_operand(s["dy"], s["sdy"], recipe) @ exact_operand(s["wd"], s["swd"], recipe).t()
    sg = torch.sigmoid(g)
    dg, du = dh * u * (sg + g * sg * torch.sigmoid(-g)), dh * g * sg
    d = torch.cat([dg, du], 1)
    padded = torch.cat([torch.nn.functional.pad(t, (0, fp - f)) for t in (dg, du)], 1) if recipe == "mx" else None
    if case["op"] == "ffn_backward":
        if recipe == "row":
            return {"d_gate_up": d}
        exact_quantized(d, case, out, padded)
        return out
    for name, left, right in (("dx", padded, ("wt", "swt")), ("dw", d.t().contiguous(), ("xt", "sxt"))):
        t, scale = exact_blocks(left, False)
        out[name] = exact_rounded(t) * scale.repeat_interleave(32, 1) @ exact_operand(s[right[0]], s[right[1]], "mx").t()
    return out
