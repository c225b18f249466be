"""Projections in 8-bit floating point around the attention (include/evo_attn.h).

Argument marshalling only, like ``attention``: torch tensors in, calls of
libevo_attn.so on the current CUDA stream of the tensors' device, no fallback.

    q8, s8, h, rstd = add_rms_norm_fp8(x, residual, weight, eps)   # norm of the stream, in 8 bits
    w8, ws = quantize_fp8(w, square=True)                           # a weight [n_out, c_in], once per update
    y = fp8_linear(q8, s8, w8, ws, bias)                            # [..., n_out]
    q, k, v, g = attention.qkvg_views(y, H)                         # into the attention, no copy

An 8-bit tensor is a ``torch.float8_e4m3fn`` tensor of codes and an fp32 tensor
of scales, one for each 128 values along the last axis (``[..., G]``) or for
each 128 x 128 block (``[ceil(R/128), G]``); a value is code * scale.  Rows of
codes start at multiples of 16 bytes (``empty_codes``), so for widths that are
not a multiple of 16 the codes are a view of wider rows.

Training: ``add_rms_norm_linear`` and ``fp8_linear_train`` are differentiable.
Their products run in 8 bits in both directions; the rounding itself is passed
over by the gradient.
"""
from __future__ import annotations

import torch

from .attention import DTYPES, _check, _opt_f32, _ptr, _stream, load_library

GROUP = 128
CODES = torch.float8_e4m3fn


def _groups(n: int) -> int:
    return -(-n // GROUP)


def _on(*tensors):
    """Every tensor on one CUDA device, which is returned."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device")
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    return dev


def _call(where, dev, *args):
    """One library call with `dev` current, on its current stream."""
    fn = getattr(load_library(), where)
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    _check(where, rc)


def _dtype(t, name):
    if t.dtype not in DTYPES:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return DTYPES[t.dtype]


def _rows(t):
    """t [..., C] as (rows, C, 2-D view); a copy only where the leading axes do not fold into one."""
    if t.dim() < 1:
        raise ValueError("expected at least one axis")
    c = t.shape[-1]
    if t.dim() == 2 and (t.stride(1) == 1 or c <= 1):
        return t.shape[0], c, t
    t2 = t.reshape(t.numel() // c if c else 0, c)
    return t2.shape[0], c, t2 if c <= 1 or t2.stride(1) == 1 else t2.contiguous()


def empty_codes(rows: int, cols: int, device) -> torch.Tensor:
    """Uninitialised codes [rows, cols] whose rows start at multiples of 16 bytes."""
    pitch = (cols + 15) // 16 * 16
    return torch.empty_strided((rows, cols), (pitch, 1), dtype=CODES, device=device)


def empty_scales(rows: int, groups: int, device) -> torch.Tensor:
    """Uninitialised scales [rows, groups], laid out group by group (the rows of a group contiguous)."""
    return torch.empty_strided((rows, groups), (1, max(rows, 1)), dtype=torch.float32, device=device)


def _scale_strides(s):
    return max(s.stride(0), 1), max(s.stride(1), 1)


def _check_dense(t, shape, dtype, name, dev):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != dev or \
            (t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} with a contiguous last axis")


def _weight(weight, cols):
    if weight is None:
        return 0
    if weight.dim() != 1 or weight.shape[0] != cols or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{cols}] tensor")
    return _dtype(weight, "weight")


def add_rms_norm_fp8(x, residual=None, weight=None, eps=1e-6, want_n=False):
    """Residual addition, root-mean-square norm, and its output in 8 bits: ``(q, scale, h, rstd)``.

    h = x + residual (in x's type; x itself where residual is None), n = h / rms(h) * weight.
    x, residual: bf16 or fp32 ``[..., C]``; weight: bf16 or fp32 ``[C]`` or None.  q ``[..., C]``
    codes and scale ``[..., G]`` of n; rstd fp32 ``[...]`` is 1 / rms, which the backward takes.
    ``want_n=True`` returns n, rounded to x's type, as a fifth value.
    """
    dev = _on(x, residual, weight)
    dt = _dtype(x, "x")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")
    rows, c, x2 = _rows(x)
    wd = _weight(weight, c)
    r2 = None if residual is None else _rows(residual)[2]
    lead = x.shape[:-1]
    q, scale = empty_codes(rows, c, dev), empty_scales(rows, _groups(c), dev)
    h = None if residual is None else torch.empty((rows, c), dtype=x.dtype, device=dev)
    n = torch.empty((rows, c), dtype=x.dtype, device=dev) if want_n else None
    rstd = torch.empty(lead, dtype=torch.float32, device=dev)
    sr, sg = _scale_strides(scale)
    _call("evo_add_rms_norm_fp8", dev, rows, c, dt, _ptr(x2), x2.stride(0), _ptr(r2),
          0 if r2 is None else r2.stride(0), _ptr(weight), wd, float(eps), _ptr(q), q.stride(0), _ptr(scale), sr, sg,
          _ptr(h), c, _ptr(n), c, _ptr(rstd))
    if x.dim() != 2:
        q, scale = q.unflatten(0, lead) if lead else q[0], scale.unflatten(0, lead) if lead else scale[0]
    out = (q, scale, x if h is None else h.view(x.shape), rstd)
    return out + (n.view(x.shape),) if want_n else out


def add_rms_norm_bwd(dy, dh, h, rstd, weight=None, want_dweight=True):
    """Gradients of add_rms_norm_fp8 with its rounding to 8 bits passed over: ``(dx, dweight)``.

    dy: gradient with respect to n; dh: the one that reaches h by the residual stream, or None;
    h, rstd: the forward's.  dx (h's type) is the gradient of x and of residual alike; dweight is
    fp32 ``[C]`` (None with ``want_dweight=False``).
    """
    dev = _on(dy, dh, h, rstd, weight)
    dt = _dtype(h, "h")
    for name, t in (("dy", dy), ("dh", dh)):
        if t is not None and (t.shape != h.shape or t.dtype != h.dtype):
            raise ValueError(f"{name} must have h's shape and dtype")
    rows, c, h2 = _rows(h)
    if rstd.dtype != torch.float32 or rstd.shape != h.shape[:-1] or not rstd.is_contiguous():
        raise ValueError(f"rstd must be a contiguous fp32 tensor of shape {tuple(h.shape[:-1])}")
    wd = _weight(weight, c)
    dy2 = _rows(dy)[2]
    dh2 = None if dh is None else _rows(dh)[2]
    dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    dweight = ws = None
    nbytes = 0
    if want_dweight:
        dweight = torch.empty(c, dtype=torch.float32, device=dev)
        nbytes = int(load_library().evo_add_rms_norm_bwd_workspace_bytes(rows, c))
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _call("evo_add_rms_norm_bwd", dev, rows, c, dt, _ptr(dy2), dy2.stride(0), _ptr(dh2),
          0 if dh2 is None else dh2.stride(0), _ptr(h2), h2.stride(0), _ptr(rstd), _ptr(weight), wd, _ptr(dx), c,
          _ptr(dweight), _ptr(ws), nbytes)
    return dx, dweight


def quantize_fp8(x, square=False, transpose=False):
    """x (bf16 or fp32) in 8 bits: ``(q, scale)``.

    Default: 1 x 128 groups along the last axis of ``[..., C]``.  ``square=True``: 128 x 128 blocks
    of a matrix ``[R, C]`` (weights).  ``transpose=True``: of ``x.T`` -- q is ``[C, R]``, its groups
    along R -- for a matrix, or for ``[..., C]`` with the leading axes as R.
    """
    dev = _on(x)
    dt = _dtype(x, "x")
    if square and x.dim() != 2:
        raise ValueError("square blocks are of a matrix [R, C]")
    rows, c, x2 = _rows(x)
    qr, qc = (c, rows) if transpose else (rows, c)
    q = empty_codes(qr, qc, dev)
    if square:
        scale = torch.empty((_groups(qr), _groups(qc)), dtype=torch.float32, device=dev)
    else:
        scale = empty_scales(qr, _groups(qc), dev)
    sr, sg = _scale_strides(scale)
    _call("evo_quantize_fp8", dev, rows, c, dt, _ptr(x2), x2.stride(0), int(square), int(transpose), _ptr(q),
          q.stride(0), _ptr(scale), sr, sg)
    if not transpose and x.dim() != 2:
        lead = x.shape[:-1]
        q, scale = (q.unflatten(0, lead), scale.unflatten(0, lead)) if lead else (q[0], scale[0])
    return q, scale


def _codes(t, name):
    """Codes [..., C] as a matrix, without a copy."""
    if t.dtype != CODES:
        raise ValueError(f"{name} must hold {CODES} codes, got {t.dtype}")
    if t.dim() == 2:
        t2 = t
    else:
        t2 = t.view(-1, t.shape[-1]) if t.is_contiguous() else t.flatten(0, -2) if t.dim() > 1 else t[None]
        if t2.data_ptr() != t.data_ptr():
            raise ValueError(f"{name}: the leading axes must fold into one without a copy")
    if t2.shape[1] > 1 and t2.stride(1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if (t2.shape[0] > 1 and t2.stride(0) % 16) or t2.data_ptr() % 16:
        raise ValueError(f"{name}: rows must start at multiples of 16 bytes (see empty_codes)")
    return t2


def fp8_linear(xq, x_scale, wq, w_scale, bias=None, out_dtype=torch.bfloat16):
    """y = x @ w.T + bias of two 8-bit tensors, bf16 or fp32 ``[..., N]``.

    xq ``[..., K]`` with x_scale ``[..., G]`` (1 x 128 groups); wq ``[N, K]`` with w_scale
    ``[ceil(N/128), G]`` (128 x 128 blocks) or ``[N, G]`` (1 x 128 groups; for N = 1, where the two
    shapes are the same, they also mean the same); bias ``[N]`` or None.  Everything accumulates
    in fp32.
    """
    dev = _on(xq, x_scale, wq, w_scale, bias)
    if out_dtype not in DTYPES:
        raise ValueError(f"out_dtype must be bf16 or fp32, got {out_dtype}")
    x2, w2 = _codes(xq, "xq"), _codes(wq, "wq")
    M, K = x2.shape
    N = w2.shape[0]
    G = _groups(K)
    if wq.dim() != 2 or w2.shape[1] != K:
        raise ValueError(f"wq must be [N, {K}], got {tuple(wq.shape)}")
    if tuple(x_scale.shape) != tuple(xq.shape[:-1]) + (G,) or x_scale.dtype != torch.float32:
        raise ValueError(f"x_scale must be fp32 of shape {tuple(xq.shape[:-1]) + (G,)}")
    if w_scale.dtype != torch.float32 or w_scale.dim() != 2 or w_scale.shape[1] != G or \
            w_scale.shape[0] not in (N, _groups(N)):
        raise ValueError(f"w_scale must be fp32 of shape [{_groups(N)}, {G}] (blocks) or [{N}, {G}] (rows)")
    w_rows = w_scale.shape[0] != _groups(N)
    xs = x_scale if x_scale.dim() == 2 else x_scale.reshape(M, G)
    y = torch.empty(xq.shape[:-1] + (N,), dtype=out_dtype, device=dev)
    b = _opt_f32(bias, N, dev)
    _call("evo_fp8_linear", dev, M, N, K, _ptr(x2), x2.stride(0), _ptr(xs), xs.stride(0), xs.stride(1), _ptr(w2),
          w2.stride(0), _ptr(w_scale), w_scale.stride(0), w_scale.stride(1), int(w_rows), _ptr(b), DTYPES[out_dtype],
          _ptr(y), N)
    return y


def _input_grad(dy, w):
    """dy @ w in 8 bits: dy [..., N] in 1 x 128 groups, the transposed w [N, K] in blocks."""
    return fp8_linear(*quantize_fp8(dy), *quantize_fp8(w, square=True, transpose=True), out_dtype=dy.dtype)


def _weight_grad(dy, x, dtype):
    """dy^T @ x in 8 bits, both in groups of 128 rows."""
    return fp8_linear(*quantize_fp8(dy, transpose=True), *quantize_fp8(x, transpose=True), out_dtype=dtype)


def _training_weight(x, w):
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError(f"w must be [N, {x.shape[-1]}], got {tuple(w.shape)}")
    _dtype(w, "w")


class Fp8Linear(torch.autograd.Function):
    """y = x @ w.T in 8 bits, both directions (x: bf16 or fp32; y in x's type; w [N, K])."""

    @staticmethod
    def forward(ctx, x, w):
        _training_weight(x, w)
        ctx.save_for_backward(x, w)
        return fp8_linear(*quantize_fp8(x), *quantize_fp8(w, square=True), out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dx = _input_grad(dy, w) if ctx.needs_input_grad[0] else None
        dw = _weight_grad(dy, x, w.dtype) if ctx.needs_input_grad[1] else None
        return dx, dw


class AddRmsNormLinear(torch.autograd.Function):
    """(h, y): h = x + residual, y = norm(h) @ w.T with the norm and the product in 8 bits, both directions."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps, w):
        _training_weight(x, w)
        q, scale, h, rstd, n = add_rms_norm_fp8(x, residual, weight, eps, want_n=True)
        y = fp8_linear(q, scale, *quantize_fp8(w, square=True), out_dtype=x.dtype)
        if residual is None:
            h = x.view_as(x)
        ctx.set_materialize_grads(False)         # an unused output costs nothing
        ctx.save_for_backward(h, rstd, n, weight, w)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, rstd, n, weight, w = ctx.saved_tensors
        if dy is None:
            return dh if ctx.needs_input_grad[0] else None, dh if ctx.needs_input_grad[1] else None, None, None, None
        dw = _weight_grad(dy, n, w.dtype) if ctx.needs_input_grad[4] else None
        dx = dweight = None
        if any(ctx.needs_input_grad[:3]):
            want = weight is not None and ctx.needs_input_grad[2]
            dx, dweight = add_rms_norm_bwd(_input_grad(dy, w), dh, h, rstd, weight, want_dweight=want)
            dweight = dweight.to(weight.dtype) if want else None
        return (dx if ctx.needs_input_grad[0] else None, dx if ctx.needs_input_grad[1] else None, dweight, None, dw)


def fp8_linear_train(x, w):
    """Differentiable x @ w.T with 8-bit products forward and backward; x ``[..., K]``, w ``[N, K]``."""
    return Fp8Linear.apply(x, w)


def add_rms_norm_linear(x, residual, weight, eps, w):
    """Differentiable ``(h, y)``: h = x + residual, y = (h / rms(h) * weight) @ w.T, products in 8 bits."""
    return AddRmsNormLinear.apply(x, residual, weight, eps, w)
