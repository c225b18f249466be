"""The 8-bit operators from their definitions, in 64 bits (torch, any device).

Shares no code with the library.  e4m3: sign, 4 exponent bits (bias 7), 3 bits of
fraction, largest value 448, steps of 2^-9 below 2^-6.
"""
import torch

GROUP = 128
LEAST = 2.0 ** -100


def e4m3(v):
    """Nearest e4m3 value, ties to even (|v| <= 448; NaN stays NaN)."""
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 4).clamp_min(-9))
    return torch.round(v / step) * step


def blocks(v, square):
    """v [R, C] padded with zeros to whole groups: [R', h, G, 128] with h = 128 or 1."""
    r, c = v.shape
    h = GROUP if square else 1
    p = torch.zeros((-(-r // h) * h, -(-c // GROUP) * GROUP), dtype=v.dtype, device=v.device)
    p[:r, :c] = v
    return p.view(p.shape[0] // h, h, p.shape[1] // GROUP, GROUP)


def quotients(v, square):
    """448 * v / m per value, and m [R', G]."""
    p = blocks(v.double(), square)
    m = p.abs().amax((1, 3)).clamp_min(LEAST)
    t = p * 448 / m[:, None, :, None]
    return t.reshape(-1, p.shape[2] * GROUP)[: v.shape[0], : v.shape[1]], m


def quantize(v, square=False):
    t, m = quotients(v, square)
    return e4m3(t), m / 448


def values(q, scale, square=None):
    """What codes stand for; scale [R or R/128, G]."""
    r, c = q.shape
    if square is None:
        square = scale.shape[0] != r
    s = scale.double().repeat_interleave(GROUP, 1)[:, :c]
    if square:
        s = s.repeat_interleave(GROUP, 0)[:r]
    return q.double() * s


def norm(x, residual, weight, eps):
    """h, rstd, n; h rounded to x's type."""
    h = x.double() if residual is None else (x.double() + residual.double()).to(x.dtype).double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    n = h * rstd[:, None]
    return h, rstd, n if weight is None else n * weight.double()


def norm_bwd(dy, dh, h, rstd, weight):
    dy, h, rstd = dy.double(), h.double(), rstd.double()
    g = dy if weight is None else dy * weight.double()
    n = h * rstd[:, None]
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return dx if dh is None else dx + dh.double(), (dy * n).sum(0)


def tie_distance(t):
    """Relative distance of |t| from the nearest border between two e4m3 values."""
    a = t.abs()
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 4).clamp_min(-9))
    f = a / step
    return ((f - torch.floor(f) - 0.5).abs() * step) / a.clamp_min(1e-30)
