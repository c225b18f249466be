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

from math import prod

import torch
from torch.autograd.function import once_differentiable

from .attention import DTYPES, EVO_OK, EvoError, _opt_f32, load_library

GROUP = 128
CODES = torch.float8_e4m3fn
EVO_ERR_WORKSPACE_TOO_SMALL = 3

# A call costs the host some ten microseconds, as much as the smaller kernels take on the
# GPU: the functions below avoid objects where a number will do (addresses and the raw
# stream go to ctypes as integers) and ask each tensor once.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty_strided


def _groups(n: int) -> int:
    return -(-n // GROUP)


def _on(first, *others):
    """Every tensor (or None) on first's CUDA device, which is returned."""
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device")
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    return dev


def _addr(t):
    return None if t is None else t.data_ptr()


def _status(where, dev, *args):
    """The status of one library call with `dev` current, on its current stream."""
    fn = getattr(load_library(), where)
    i = dev.index
    if i == _current_device():
        return fn(*args, _raw_stream(i))
    with torch.cuda.device(i):
        return fn(*args, _raw_stream(i))


def _call(where, dev, *args):
    rc = _status(where, dev, *args)
    if rc != EVO_OK:
        raise EvoError(where, rc)


def _dtype(t, name):
    if t.dtype not in DTYPES:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return DTYPES[t.dtype]


def _rows(t):
    """t [..., C] as (rows, C, matrix, row pitch); a copy only where the leading axes do not fold into one."""
    shape = t.shape
    if not shape:
        raise ValueError("expected at least one axis")
    c = shape[-1]
    t2 = t
    if len(shape) != 2:
        t2 = t.reshape(t.numel() // c if c else prod(shape[:-1]), c)
    pitch, step = t2.stride()
    if step != 1 and c > 1:
        t2 = t2.contiguous()
        pitch = c
    return t2.shape[0], c, t2, pitch


def empty_codes(rows: int, cols: int, device) -> torch.Tensor:
    """Uninitialised codes [rows, cols] whose rows start at multiples of 16 bytes."""
    return _empty((rows, cols), ((cols + 15) // 16 * 16, 1), dtype=CODES, device=device)


def empty_scales(rows: int, groups: int, device) -> torch.Tensor:
    """Uninitialised scales [rows, groups], laid out group by group (the rows of a group contiguous)."""
    return _empty((rows, groups), (1, rows or 1), dtype=torch.float32, device=device)


def _weight(weight, cols):
    if weight is None:
        return 0
    if weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{cols}] tensor")
    return _dtype(weight, "weight")


def _lead(t, lead):
    """A result [rows, ...] with the leading axes of its input."""
    return t.unflatten(0, lead) if lead else t[0]


def add_rms_norm_fp8(x, residual=None, weight=None, eps=1e-6, want_n=False):
    """Residual addition, root-mean-square norm, and its output in 8 bits: ``(q, scale, h, rstd)``.

    h = x + residual (in x's type; x itself where residual is None), n = h / rms(h) * weight.
    x, residual: bf16 or fp32 ``[..., C]``; weight: bf16 or fp32 ``[C]`` or None.  q ``[..., C]``
    codes and scale ``[..., G]`` of n; rstd fp32 ``[...]`` is 1 / rms, which the backward takes.
    Any eps >= 0: below 2^-20 rows of a small rms take a factor more (6 % at 196608 x 256); with
    eps = 0 a row of zeros has no norm, and NaN scales.  C is 1 to 32768.
    ``want_n=True`` returns n, rounded to x's type, as a fifth value.
    """
    dev = _on(x, residual, weight)
    dtype, shape = x.dtype, x.shape
    dt = _dtype(x, "x")
    rows, c, x2, ldx = _rows(x)
    wd = _weight(weight, c)
    q, scale = empty_codes(rows, c, dev), empty_scales(rows, -(-c // GROUP), dev)
    r2 = h = n = None
    ldr = 0
    if residual is not None:
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must have x's shape and dtype")
        r2, ldr = _rows(residual)[2:]
        h = _empty((rows, c), (c, 1), dtype=dtype, device=dev)
    if want_n:
        n = _empty((rows, c), (c, 1), dtype=dtype, device=dev)
    rstd = _empty((rows,), (1,), dtype=torch.float32, device=dev)
    _call("evo_add_rms_norm_fp8", dev, rows, c, dt, x2.data_ptr(), ldx, _addr(r2), ldr, _addr(weight), wd, eps,
          q.data_ptr(), (c + 15) // 16 * 16, scale.data_ptr(), 1, rows or 1, _addr(h), c, _addr(n), c, rstd.data_ptr())
    if h is None:
        h = x
    if len(shape) != 2:
        lead = shape[:-1]
        q, scale, rstd = _lead(q, lead), _lead(scale, lead), _lead(rstd, lead)
        h = h.view(shape) if residual is not None else h
        n = n.view(shape) if want_n else None
    return (q, scale, h, rstd, n) if want_n else (q, scale, h, rstd)


def add_rms_norm_bwd(dy, dh, h, rstd, weight=None, want_dweight=True, dweight_dtype=torch.float32):
    """Gradients of add_rms_norm_fp8 with its rounding to 8 bits passed over: ``(dx, dweight)``.

    dy: gradient with respect to n; dh: the one that reaches h by the residual stream, or None;
    h, rstd: the forward's.  dx (h's type) is the gradient of x and of residual alike; dweight
    ``[C]`` is summed in fp32 and fp32 or, with ``dweight_dtype``, bf16 (None with ``want_dweight=False``).
    """
    dev = _on(h, dy, dh, rstd, weight)
    dtype, shape = h.dtype, h.shape
    dt = _dtype(h, "h")
    rows, c, h2, ldh = _rows(h)
    if dy.shape != shape or dy.dtype != dtype or (dh is not None and (dh.shape != shape or dh.dtype != dtype)):
        raise ValueError("dy and dh must have h's shape and dtype")
    if rstd.dtype != torch.float32 or rstd.shape != shape[:-1] or not rstd.is_contiguous():
        raise ValueError(f"rstd must be a contiguous fp32 tensor of shape {tuple(shape[:-1])}")
    if dweight_dtype not in DTYPES:
        raise ValueError(f"dweight_dtype must be bf16 or fp32, got {dweight_dtype}")
    wd = _weight(weight, c)
    dy2, lddy = _rows(dy)[2:]
    dh2, lddh = (None, 0) if dh is None else _rows(dh)[2:]
    dx = _empty((rows, c), (c, 1), dtype=dtype, device=dev)
    dweight = ws = None
    nbytes = 0
    if want_dweight:
        dweight = _empty((c,), (1,), dtype=dweight_dtype, device=dev)
        nbytes = load_library().evo_add_rms_norm_bwd_workspace_bytes(rows, c)
        ws = _empty((nbytes // 4,), (1,), dtype=torch.float32, device=dev)
    _call("evo_add_rms_norm_bwd", dev, rows, c, dt, dy2.data_ptr(), lddy, _addr(dh2), lddh, h2.data_ptr(), ldh,
          rstd.data_ptr(), _addr(weight), wd, dx.data_ptr(), c, _addr(dweight), DTYPES[dweight_dtype], _addr(ws), nbytes)
    return dx if len(shape) == 2 else dx.view(shape), dweight


def quantize_fp8(x, square=False, transpose=False):
    """x (bf16 or fp32) in 8 bits: ``(q, scale)``.

    Default: 1 x 128 groups along the last axis of ``[..., C]``.  ``square=True``: 128 x 128 blocks
    of a matrix ``[R, C]`` (weights).  ``transpose=True``: of ``x.T`` -- q is ``[C, R]``, its groups
    along R -- for a matrix, or for ``[..., C]`` with the leading axes as R.
    """
    dev = _on(x)
    dt = _dtype(x, "x")
    shape = x.shape
    if square and len(shape) != 2:
        raise ValueError("square blocks are of a matrix [R, C]")
    rows, c, x2, ldx = _rows(x)
    qr, qc = (c, rows) if transpose else (rows, c)
    g = -(-qc // GROUP)
    q = empty_codes(qr, qc, dev)
    if square:
        scale = _empty((-(-qr // GROUP), g), (g or 1, 1), dtype=torch.float32, device=dev)
        sr, sg = g or 1, 1
    else:
        scale = empty_scales(qr, g, dev)
        sr, sg = 1, qr or 1
    _call("evo_quantize_fp8", dev, rows, c, dt, x2.data_ptr(), ldx, bool(square), bool(transpose), q.data_ptr(),
          (qc + 15) // 16 * 16, scale.data_ptr(), sr, sg)
    if not transpose and len(shape) != 2:
        q, scale = _lead(q, shape[:-1]), _lead(scale, shape[:-1])
    return q, scale


def quantize_fp8_both(x, square=False):
    """quantize_fp8 of x and of x.T in one pass over x: ``(q, scale, q_t, scale_t)``.

    For training: a weight's blocks serve its product and, transposed, the input's gradient; an output
    gradient's groups along both axes serve the input's and the weight's gradient.  With
    ``square=True`` the two hold the same values, transposed.
    """
    dev = _on(x)
    dt = _dtype(x, "x")
    shape = x.shape
    if square and len(shape) != 2:
        raise ValueError("square blocks are of a matrix [R, C]")
    rows, c, x2, ldx = _rows(x)
    gr, gc = -(-rows // GROUP), -(-c // GROUP)
    q, qt = empty_codes(rows, c, dev), empty_codes(c, rows, dev)
    if square:
        scale = _empty((gr, gc), (gc or 1, 1), dtype=torch.float32, device=dev)
        scale_t = scale.t()
        strides = gc or 1, 1, 1, gc or 1
    else:
        scale, scale_t = empty_scales(rows, gc, dev), empty_scales(c, gr, dev)
        strides = 1, rows or 1, 1, c or 1
    _call("evo_quantize_fp8_both", dev, rows, c, dt, x2.data_ptr(), ldx, bool(square), q.data_ptr(),
          (c + 15) // 16 * 16, scale.data_ptr(), strides[0], strides[1], qt.data_ptr(), (rows + 15) // 16 * 16,
          scale_t.data_ptr(), strides[2], strides[3])
    if len(shape) != 2:
        q, scale = _lead(q, shape[:-1]), _lead(scale, shape[:-1])
    return q, scale, qt, scale_t


def _codes(t, name):
    """Codes [..., C] as (rows, C, address, pitch), without a copy."""
    if t.dtype != CODES:
        raise ValueError(f"{name} must hold {CODES} codes, got {t.dtype}")
    if t.dim() != 2:
        flat = t[None] if t.dim() == 1 else t.flatten(0, -2)
        if flat.numel() and flat.data_ptr() != t.data_ptr():
            raise ValueError(f"{name}: the leading axes must fold into one without a copy")
        t = flat
    rows, c = t.shape
    pitch, step = t.stride()
    at = t.data_ptr()
    if step != 1 and c > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if at % 16 or (rows > 1 and pitch % 16):
        raise ValueError(f"{name}: rows must start at multiples of 16 bytes (see empty_codes)")
    return rows, c, at, pitch


def fp8_linear(xq, x_scale, wq, w_scale, bias=None, out_dtype=torch.bfloat16):
    """y = x @ w.T + bias of two 8-bit tensors, bf16 or fp32 ``[..., N]``.

    xq ``[..., K]`` with x_scale ``[..., G]`` (1 x 128 groups); wq ``[N, K]`` with w_scale
    ``[ceil(N/128), G]`` (128 x 128 blocks) or ``[N, G]`` (1 x 128 groups; for N = 1, where the two
    shapes are the same, they also mean the same); bias ``[N]`` or None.  Everything accumulates
    in fp32.  K is at least 1; the other axes may be empty.
    """
    dev = _on(xq, x_scale, wq, w_scale, bias)
    if out_dtype not in DTYPES:
        raise ValueError(f"out_dtype must be bf16 or fp32, got {out_dtype}")
    M, K, x_at, ldx = _codes(xq, "xq")
    N, wk, w_at, ldw = _codes(wq, "wq")
    if wq.dim() != 2 or wk != K:
        raise ValueError(f"wq must be [N, {K}], got {tuple(wq.shape)}")
    G = -(-K // GROUP)
    lead = xq.shape[:-1]
    if x_scale.shape != (*lead, G) or x_scale.dtype != torch.float32:
        raise ValueError(f"x_scale must be fp32 of shape {(*lead, G)}")
    sn = w_scale.shape[0] if w_scale.dim() == 2 and w_scale.shape[1] == G else -1
    blocks = -(-N // GROUP)
    if w_scale.dtype != torch.float32 or sn not in (N, blocks):
        raise ValueError(f"w_scale must be fp32 of shape [{blocks}, {G}] (blocks) or [{N}, {G}] (rows)")
    xs = x_scale if len(lead) == 1 else x_scale.reshape(M, G)
    sxr, sxg = xs.stride()
    swr, swg = w_scale.stride()
    y = _empty((M, N), (N, 1), dtype=out_dtype, device=dev)
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (N,) or not bias.is_contiguous()):
        bias = _opt_f32(bias, N, dev)
    args = (M, N, K, x_at, ldx, xs.data_ptr(), sxr, sxg, w_at, ldw, w_scale.data_ptr(), swr, swg, sn != blocks,
            _addr(bias), DTYPES[out_dtype], y.data_ptr(), N)
    # most sizes need no workspace: a call without one is refused before anything is enqueued
    rc = _status("evo_fp8_linear", dev, *args, None, 0)
    if rc == EVO_ERR_WORKSPACE_TOO_SMALL:
        nbytes = load_library().evo_fp8_linear_workspace_bytes(M, N, K)
        ws = _empty((nbytes // 4,), (1,), dtype=torch.float32, device=dev)
        rc = _status("evo_fp8_linear", dev, *args, ws.data_ptr(), nbytes)
    if rc != EVO_OK:
        raise EvoError("evo_fp8_linear", rc)
    return y if len(lead) == 1 else y.view(*lead, N)


def _training_weight(x, w):
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError(f"w must be [N, {x.shape[-1]}], got {tuple(w.shape)}")
    _dtype(w, "w")


def _forward(ctx, q, scale, w, dtype):
    """q @ w.T; keeps on ctx what the input's gradient wants of w, quantised in the same pass."""
    if ctx.needs_input_grad[0] or any(ctx.needs_input_grad[1:-1]):
        wq, ws, wqt, wst = quantize_fp8_both(w, square=True)
    else:
        (wq, ws), wqt, wst = quantize_fp8(w, square=True), None, None
    return fp8_linear(q, scale, wq, ws, out_dtype=dtype), wqt, wst


def fp8_linear_bwd(dy, x, wq_t, w_scale_t, dw_dtype=torch.float32, want_dx=True, want_dw=True):
    """Gradients of ``y = x @ w.T`` in 8 bits: ``(dx, dw)``, each None where it is not wanted.

    dy ``[..., N]`` and x ``[..., K]`` (bf16 or fp32, one type) are quantised here; wq_t ``[K, N]`` and
    w_scale_t are the transposed half of ``quantize_fp8_both(w, square=True)``.  dx ``[..., K]`` is of
    dy's type, dw ``[N, K]`` of dw_dtype.  x may be None without dw, wq_t and w_scale_t without dx.
    K is at least 1; with M or N of 0 the gradients are the empty sums, zeros.
    """
    dev = _on(dy, x, wq_t, w_scale_t)
    dtype, shape = dy.dtype, dy.shape
    dt = _dtype(dy, "dy")
    if dw_dtype not in DTYPES:
        raise ValueError(f"dw_dtype must be bf16 or fp32, got {dw_dtype}")
    M, N, dy2, lddy = _rows(dy)
    dx = dw = x2 = None
    ldx = w_at = ldw = s_at = sr = sg = nbytes = 0
    if want_dw:
        if x is None or x.dtype != dtype or x.shape[:-1] != shape[:-1]:
            raise ValueError("x must have dy's type and leading axes")
        x2, ldx = _rows(x)[2:]
        K = x.shape[-1]
        dw = _empty((N, K), (K, 1), dtype=dw_dtype, device=dev)
    if want_dx:
        wk, wn, w_at, ldw = _codes(wq_t, "wq_t")
        if wn != N or (want_dw and wk != K):
            raise ValueError(f"wq_t must be [K, {N}], got {tuple(wq_t.shape)}")
        K = wk
        if w_scale_t.shape != (-(-K // GROUP), -(-N // GROUP)) or w_scale_t.dtype != torch.float32:
            raise ValueError(f"w_scale_t must be fp32 of shape {(-(-K // GROUP), -(-N // GROUP))}")
        sr, sg = w_scale_t.stride()
        s_at = w_scale_t.data_ptr()
        dx = _empty((M, K), (K, 1), dtype=dtype, device=dev)
    if dx is None and dw is None:
        return None, None
    ws = None
    nbytes = load_library().evo_fp8_linear_bwd_workspace_bytes(M, N, K, want_dx, want_dw)
    if nbytes:
        ws = _empty((nbytes,), (1,), dtype=torch.uint8, device=dev)
    _call("evo_fp8_linear_bwd", dev, M, N, K, dt, dy2.data_ptr(), lddy, _addr(x2), ldx, w_at, ldw, s_at, sr, sg,
          _addr(dx), K, _addr(dw), DTYPES[dw_dtype], K, _addr(ws), nbytes)
    return dx if dx is None or len(shape) == 2 else dx.view(*shape[:-1], K), dw


class Fp8Linear(torch.autograd.Function):
    """y = x @ w.T in 8 bits, both directions (x: bf16 or fp32; y in x's type; w [N, K])."""

    @staticmethod
    def forward(ctx, x, w):
        _training_weight(x, w)
        y, wqt, wst = _forward(ctx, *quantize_fp8(x), w, x.dtype)
        ctx.save_for_backward(x, wqt, wst)
        ctx.w_dtype = w.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, wqt, wst = ctx.saved_tensors
        return fp8_linear_bwd(dy, x, wqt, wst, ctx.w_dtype, *ctx.needs_input_grad)


class AddRmsNormLinear(torch.autograd.Function):
    """(h, y): h = x + residual, y = norm(h) @ w.T with the norm and the product in 8 bits, both directions."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps, w):
        _training_weight(x, w)
        q, scale, h, rstd, *n = add_rms_norm_fp8(x, residual, weight, eps, want_n=ctx.needs_input_grad[4])
        y, wqt, wst = _forward(ctx, q, scale, w, x.dtype)
        if residual is None:
            h = x.view_as(x)
        ctx.set_materialize_grads(False)         # an unused output costs nothing
        ctx.save_for_backward(h, rstd, n[0] if n else None, weight, wqt, wst)
        ctx.w_dtype = w.dtype
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        h, rstd, n, weight, wqt, wst = ctx.saved_tensors
        for_x, for_res, for_weight, _, for_w = ctx.needs_input_grad
        if dy is None:
            return dh if for_x else None, dh if for_res else None, None, None, None
        dn, dw = fp8_linear_bwd(dy, n, wqt, wst, ctx.w_dtype, for_x or for_res or for_weight, for_w)
        dx = dweight = None
        if dn is not None:
            dx, dweight = add_rms_norm_bwd(dn, dh, h, rstd, weight, for_weight,
                                           weight.dtype if for_weight else torch.float32)
        return dx if for_x else None, dx if for_res else None, dweight, None, dw


def fp8_linear_train(x, w):
    """Differentiable x @ w.T with 8-bit products forward and backward; x ``[..., K]``, w ``[N, K]``."""
    return Fp8Linear.apply(x, w)


def add_rms_norm_linear(x, residual, weight, eps, w):
    """Differentiable ``(h, y)``: h = x + residual, y = (h / rms(h) * weight) @ w.T, products in 8 bits."""
    return AddRmsNormLinear.apply(x, residual, weight, eps, w)
