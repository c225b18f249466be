"""Cases, plain forms and 64-bit values of the 8-bit projection operators.

The operators take a representation's rows from the residual stream through a
projection in 8-bit floating point (e4m3, one fp32 scale for each group of 128
values) and back:

    norm       h = x + residual;  n = h / rms(h) * weight;  n in 8 bits, a scale per row and 128 channels
    norm_bwd   the gradients of that norm
    quantize   a tensor in 8 bits with scales per 1 x 128 group or per 128 x 128 block, as it lies or transposed
    linear     y = x @ w^T + bias of two 8-bit tensors with such scales
    train      norm and linear as one differentiable step: outputs and every gradient

e4m3 has its largest value at 448: a group whose largest magnitude is m keeps
q = e4m3(448 * v / m) and scale = m / 448, where m is held at 2^-100 or above.
"""
import torch

own = False

GROUP = 128
TOP = 448.0
LEAST = 2.0 ** -100
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a wide residual stream, as while answering: latency alone
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True},
        # the MSA representation at 512 sequences x 384 residues, 256 channels: the rows ahead of q, k, v and g
        {"name": "norm msa 196608x256", "op": "norm", "rows": 196608, "cols": 256, "dtype": "bf16", "residual": True},
        # an fp32 residual stream with an odd number of rows and channels that end inside a group
        {"name": "norm f32 4099x2500", "op": "norm", "rows": 4099, "cols": 2500, "dtype": "f32", "residual": True},
        # the gradient of the MSA norm at 512 x 384 rows
        {"name": "norm_bwd msa 196608x256", "op": "norm_bwd", "rows": 196608, "cols": 256, "dtype": "bf16", "residual": True},
        # a short ragged batch, wide rows, fp32
        {"name": "norm_bwd f32 777x5001", "op": "norm_bwd", "rows": 777, "cols": 5001, "dtype": "f32", "residual": True},
        # a wide layer's weight, once per optimizer step: 128 x 128 blocks
        {"name": "quantize weight 4096x4096", "op": "quantize", "rows": 4096, "cols": 4096, "dtype": "f32",
         "square": True, "transpose": False},
        # the gradient of the q, k, v, g projection over 512 x 256 rows, laid out for the weight's gradient
        {"name": "quantize grad^T 131072x1024", "op": "quantize", "rows": 131072, "cols": 1024, "dtype": "bf16",
         "square": False, "transpose": True},
        # one token through a wide layer: the weight is read once
        {"name": "linear 1x8192x8192", "op": "linear", "rows": 1, "cols": 8192, "n_out": 8192, "square": True,
         "bias": True, "dtype": "bf16"},
        # q, k, v and g (8 heads x 32) of the MSA at 512 x 256 rows: bound by writing the output
        {"name": "linear msa 131072x256x1024", "op": "linear", "rows": 131072, "cols": 256, "n_out": 1024,
         "square": True, "bias": True, "dtype": "bf16"},
        # a wide layer over a long batch with an odd number of rows: bound by the products
        {"name": "linear 8191x4096x8192", "op": "linear", "rows": 8191, "cols": 4096, "n_out": 8192, "square": True,
         "bias": False, "dtype": "bf16"},
        # that projection's weight gradient: a small result, a sum over every row
        {"name": "linear grad 1024x131072x256", "op": "linear", "rows": 1024, "cols": 131072, "n_out": 256,
         "square": False, "bias": False, "dtype": "f32"},
        # norm and projection of 64 x 256 MSA rows, forward and backward
        {"name": "train 16384x256x1024", "op": "train", "rows": 16384, "cols": 256, "n_out": 1024, "dtype": "bf16"},
    ]


def _size(rng, low, high):
    """A whole number in [low, high], spread over its logarithm; one in three is a multiple of 128 (where there is one)."""
    n = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 1 / 3:
        n = max(GROUP, n // GROUP * GROUP)
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quantize", "linear", "linear", "linear", "train"])
    if op in ("norm", "norm_bwd"):
        cols = _size(rng, 64, 8192)
        return {"op": op, "rows": _size(rng, 1, 196608 * 256 // cols), "cols": cols, "dtype": rng.choice(["bf16", "f32"]),
                "residual": rng.random() < 0.75}
    if op == "quantize":
        cols = _size(rng, 64, 8192)
        return {"op": op, "rows": _size(rng, 1, min(131072, 131072 * 1024 // cols)), "cols": cols,
                "dtype": rng.choice(["bf16", "f32"]), "square": rng.random() < 0.5, "transpose": rng.random() < 0.5}
    if op == "linear" and rng.random() < 0.3:  # a weight's gradient: many rows summed
        rows, n_out = _size(rng, 64, 4096), _size(rng, 64, 4096)
        most = min(131072, 8191 * 4096 * 8192 // (4 * rows * n_out))
        return {"op": op, "rows": rows, "cols": _size(rng, 128, max(256, most)), "n_out": n_out, "square": False,
                "bias": False, "dtype": "f32"}
    cols, n_out = _size(rng, 64, 8192), _size(rng, 64, 8192)
    if op == "linear":
        most = min(131072, 8191 * 4096 * 8192 // (cols * n_out))
        return {"op": op, "rows": _size(rng, 1, most), "cols": cols, "n_out": n_out, "square": True,
                "bias": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    cols, n_out = min(cols, 4096), min(n_out, 4096)
    most = min(65536, 8191 * 4096 * 8192 // (8 * cols * n_out))
    return {"op": op, "rows": _size(rng, 1, most), "cols": cols, "n_out": n_out, "dtype": "bf16"}


def _pitch16(q):
    """The 8-bit rows at a distance that is a multiple of 16 bytes, as the framework's own producers lay them out."""
    rows, cols = q.shape
    wide = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=q.device)
    wide[:, :cols] = q.view(torch.uint8)
    return wide.view(torch.float8_e4m3fn)[:, :cols]


def _rows(gen, rows, cols, dtype):
    """Rows of a residual stream: normal values, a different size from row to row, a few wide channels."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda"))
    x *= 1 + 7 * (torch.rand((1, cols), generator=gen, device="cuda") < 0.01)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, rows, cols, dtype = case["op"], case["rows"], case["cols"], DTYPES[case["dtype"]]
    s = dict(case)
    if op in ("norm", "norm_bwd", "train"):
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
    if op in ("norm", "train"):
        s["x"] = _rows(gen, rows, cols, dtype)
        s["res"] = _rows(gen, rows, cols, dtype) if case.get("residual", True) else None
    if op == "norm_bwd":
        s["h"] = _rows(gen, rows, cols, dtype)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dy"] = torch.randn((rows, cols), generator=gen, device="cuda").to(dtype)
        s["dh"] = torch.randn((rows, cols), generator=gen, device="cuda").to(dtype) if case["residual"] else None
    if op == "quantize":
        s["x"] = _rows(gen, rows, cols, dtype)
    if op == "linear":
        x, xs = _quantized(_rows(gen, rows, cols, torch.float32), False)
        w, ws = _quantized(torch.randn((case["n_out"], cols), generator=gen, device="cuda") / cols ** 0.5, case["square"])
        # scales lie with the groups outermost, as the framework's own producers write them
        s.update(xq=_pitch16(x), xs=xs.t().contiguous().t(), wq=_pitch16(w), ws=ws if case["square"] else ws.t().contiguous().t())
        s["b"] = torch.randn(case["n_out"], generator=gen, device="cuda") if case["bias"] else None
    if op == "train":
        n_out = case["n_out"]
        s["w"] = (torch.randn((n_out, cols), generator=gen, device="cuda") / cols ** 0.5).to(dtype)
        s["dy"] = torch.randn((rows, n_out), generator=gen, device="cuda").to(dtype)
        s["dh"] = torch.randn((rows, cols), generator=gen, device="cuda").to(dtype)
        for name in ("x", "res", "weight", "w"):
            s[name].requires_grad_(True)
    return s


# ---------------------------------------------------------------- plain forms, 32 bits

def _padded(v, square):
    """v [R, C] with zeros up to whole groups, as [R or R/128, 1 or 128, C/128, 128]."""
    r, c = v.shape
    v = torch.nn.functional.pad(v, (0, -c % GROUP, 0, (-r % GROUP) if square else 0))
    return v.reshape(-1, GROUP if square else 1, v.shape[1] // GROUP, GROUP)


def _quantized(v, square):
    """v (fp32) as e4m3 values and fp32 scales [R or R/128, C/128]."""
    p = _padded(v, square)
    m = p.abs().amax((1, 3), keepdim=True).clamp_min(LEAST)
    q = (p * TOP / m).to(torch.float8_e4m3fn)
    return q.reshape(-1, p.shape[2] * GROUP)[: v.shape[0], : v.shape[1]].contiguous(), (m / TOP)[:, 0, :, 0].contiguous()


def _values(q, scale, square):
    """What an 8-bit tensor stands for, fp32."""
    s = scale.repeat_interleave(GROUP, 1)[:, : q.shape[1]]
    if square:
        s = s.repeat_interleave(GROUP, 0)[: q.shape[0]]
    return q.float() * s


def _norm(x, res, weight, dtype):
    h = x if res is None else (x.float() + res.float()).to(dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    return h, rstd, f * rstd[:, None] * weight.float()


def _norm_grads(dy, dh, h, rstd, weight, dtype):
    n = h.float() * rstd[:, None]
    g = dy.float() * weight.float()
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.float()
    return dx.to(dtype), (dy.float() * n).sum(0)


def _plain(s):
    op, dtype = s["op"], DTYPES[s["dtype"]]
    if op == "norm":
        h, rstd, n = _norm(s["x"], s["res"], s["weight"], dtype)
        q, scale = _quantized(n, False)
        return {"q": q, "scale": scale, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight = _norm_grads(s["dy"], s["dh"], s["h"], s["rstd"], s["weight"], dtype)
        return {"dx": dx, "dweight": dweight}
    if op == "quantize":
        v = s["x"].float()
        q, scale = _quantized(v.t() if s["transpose"] else v, s["square"])
        return {"q": q, "scale": scale}
    if op == "linear":
        x, w = _values(s["xq"], s["xs"], False), _values(s["wq"], s["ws"], s["square"])
        if x.shape[1] > 8192:  # a long sum
            x, w = x.double(), w.double()
        y = x @ w.t()
        return {"y": (y if s["b"] is None else y + s["b"]).to(dtype)}
    with torch.no_grad():
        h, rstd, n = _norm(s["x"], s["res"], s["weight"], dtype)
        xv = _values(*_quantized(n, False), False)
        wv = _values(*_quantized(s["w"].float(), True), True)
        y = (xv @ wv.t()).to(dtype)
        dn = (_values(*_quantized(s["dy"].float(), False), False) @ wv).to(dtype)
        dyt = _values(*_quantized(s["dy"].float().t(), False), False)
        nt = _values(*_quantized(n.to(dtype).float().t(), False), False)
        dw = (dyt @ nt.t()).to(dtype)
        dx, dweight = _norm_grads(dn, s["dh"], h, rstd, s["weight"], dtype)
        return {"h": h, "y": y, "dx": dx, "dres": dx, "dweight": dweight.to(dtype), "dw": dw}


# ---------------------------------------------------------------- the framework's calls

def _called(s):
    from evoformer_pair_bias_b200 import fp8

    op = s["op"]
    if op == "norm":
        q, scale, h, rstd = fp8.add_rms_norm_fp8(s["x"], s["res"], s["weight"], EPS)
        return {"q": q, "scale": scale, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight = fp8.add_rms_norm_bwd(s["dy"], s["dh"], s["h"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dweight}
    if op == "quantize":
        q, scale = fp8.quantize_fp8(s["x"], square=s["square"], transpose=s["transpose"])
        return {"q": q, "scale": scale}
    if op == "linear":
        return {"y": fp8.fp8_linear(s["xq"], s["xs"], s["wq"], s["ws"], s["b"], out_dtype=DTYPES[s["dtype"]])}
    h, y = fp8.add_rms_norm_linear(s["x"], s["res"], s["weight"], EPS, s["w"])
    leaves = (s["x"], s["res"], s["weight"], s["w"])
    dx, dres, dweight, dw = torch.autograd.grad((h, y), leaves, (s["dh"], s["dy"]))
    return {"h": h, "y": y, "dx": dx, "dres": dres, "dweight": dweight, "dw": dw}


def run(state):
    return _called(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, r, c = case["op"], case["rows"], case["cols"]
    e = 2 if case["dtype"] == "bf16" else 4
    groups = -(-c // GROUP)
    if op == "norm":
        both = case["residual"]
        return {"bytes": r * c * (e * (3 if both else 1) + 1) + 4 * r * (groups + 1) + e * c, "flops": 8 * r * c}
    if op == "norm_bwd":
        return {"bytes": r * c * e * (4 if case["residual"] else 3) + 4 * r + (e + 4) * c, "flops": 10 * r * c}
    if op == "quantize":
        n = -(-r // GROUP) * groups if case["square"] else (c * -(-r // GROUP) if case["transpose"] else r * groups)
        return {"bytes": r * c * (e + 1) + 4 * n, "flops": 4 * r * c}
    n = case["n_out"]
    if op == "linear":
        ws = -(-n // GROUP) * groups if case["square"] else n * groups
        return {"bytes": r * c + n * c + r * n * e + 4 * (r * groups + ws + (n if case["bias"] else 0)), "flops": 2 * r * n * c}
    # reads x, res, weight, w, dh, dy; writes h, y, dx, dweight, dw
    return {"bytes": e * (5 * r * c + 2 * r * n + 2 * n * c + 2 * c), "flops": 6 * r * n * c}


# ---------------------------------------------------------------- the definitions in 64 bits

def _e4m3_64(v):
    """v rounded to the nearest e4m3 value, ties to even: 4 significant bits, none below 2^-9."""
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 4).clamp_min(-9))
    return torch.round(v / step) * step


def _exact_quantized(v, square):
    r, c = v.shape
    rows = GROUP if square else 1
    q = torch.empty_like(v)
    scale = torch.empty((-(-r // rows), -(-c // GROUP)), dtype=torch.float64, device=v.device)
    full = r // rows * rows  # whole blocks of rows first, then the rest
    for r0, r1 in ((0, full), (full, r)):
        if r0 == r1:
            continue
        for g in range(scale.shape[1]):
            part = v[r0:r1, g * GROUP : (g + 1) * GROUP]
            block = part.reshape(-1, min(rows, r1 - r0) * part.shape[1])
            top = block.abs().max(1).values.clamp(min=LEAST)
            q[r0:r1, g * GROUP : (g + 1) * GROUP] = _e4m3_64(block * TOP / top[:, None]).view(part.shape)
            scale[r0 // rows : r0 // rows + len(top), g] = top / TOP
    return q, scale


def _exact_values(q, scale, square):
    out = q.double().clone()
    for g in range(scale.shape[1]):
        f = scale[:, g].double()
        if square:
            f = f[torch.arange(q.shape[0], device=q.device) // GROUP]
        out[:, g * GROUP : (g + 1) * GROUP] *= f[:, None]
    return out


def _exact_norm(x, res, weight, dtype):
    h = x.double() if res is None else (x.double() + res.double())
    h = h.to(dtype).double()
    rstd = 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
    return h, rstd, h * rstd[:, None] * weight.double()


def _exact_norm_grads(dy, dh, h, rstd, weight):
    dy, h, weight, rstd = dy.double(), h.double(), weight.double(), rstd.double()
    dot = torch.einsum("rc,c,rc->r", dy, weight, h)
    dx = dy * weight * rstd[:, None] - h * (rstd ** 3 * dot / h.shape[1])[:, None]
    return dx if dh is None else dx + dh.double(), torch.einsum("rc,rc,r->c", dy, h, rstd)


def exact(case, seed):
    s = prepare(case, seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    with torch.no_grad():
        if op == "norm":
            h, rstd, n = _exact_norm(s["x"], s["res"], s["weight"], dtype)
            q, scale = _exact_quantized(n, False)
            return {"q": q, "scale": scale, "h": h, "rstd": rstd}
        if op == "norm_bwd":
            dx, dweight = _exact_norm_grads(s["dy"], s["dh"], s["h"], s["rstd"], s["weight"])
            return {"dx": dx, "dweight": dweight}
        if op == "quantize":
            v = s["x"].double()
            q, scale = _exact_quantized(v.t().contiguous() if case["transpose"] else v, case["square"])
            return {"q": q, "scale": scale}
        if op == "linear":
            y = torch.mm(_exact_values(s["xq"], s["xs"], False), _exact_values(s["wq"], s["ws"], case["square"]).t())
            return {"y": y if s["b"] is None else y + s["b"].double()}
        h, rstd, n = _exact_norm(s["x"], s["res"], s["weight"], dtype)
        w = _exact_values(*_exact_quantized(s["w"].double(), True), True)
        dy = s["dy"].double()
        y = torch.mm(_exact_values(*_exact_quantized(n, False), False), w.t())
        dn = torch.mm(_exact_values(*_exact_quantized(dy, False), False), w).to(dtype)
        n_t = n.to(dtype).double().t().contiguous()
        dw = torch.mm(_exact_values(*_exact_quantized(dy.t().contiguous(), False), False),
                      _exact_values(*_exact_quantized(n_t, False), False).t())
        dx, dweight = _exact_norm_grads(dn, s["dh"], h, rstd, s["weight"])
        return {"h": h, "y": y, "dx": dx, "dres": dx, "dweight": dweight, "dw": dw}
