"""GPU parity of the 8-bit projection operators with their definitions in 64 bits.

Tolerances, from the arithmetic:

quantise   bf16: every quotient is correctly rounded and 448 v / m of two 8-bit
           significands is either on a border between two codes or further from it
           than 2^-24, so the codes are equal.  fp32: v is rounded once more (0.875 v),
           so a code may be the neighbour where the quotient is within 2^-22 of a border.
           scale: one division, 2^-23.
norm       a row's sum of squares takes at most 32 additions per lane, 5 across the
           lanes and 32 across the warps, each 2^-24: rstd within 70 * 2^-24 / 2 plus
           its own roundings, held to 2^-17; scale the same.  The quotient does not
           depend on rstd, and h * weight is exact for bf16: the codes are equal;
           fp32 rounds h * weight too: neighbours within 2^-21 of a border.
product    within a block the tensor core adds 128 exact products in fp32, allowed 2^-21 of the
           sum of their magnitudes; the blocks are added by fp32 fused multiply-adds (2^-24
           each) and the scales' product rounds twice; then one rounding to y's type.
gradients  dx: fp32 sums as in the norm (2^-17 of the terms' magnitudes) and one rounding;
           dweight: at most rows / blocks + 64 + 32 additions of 2^-24 each.
"""
import pytest
import torch

import _fp8 as R
from evoformer_pair_bias_b200 import attention as A
from evoformer_pair_bias_b200 import fp8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from evoformer_pair_bias_b200 import build
    build.build()
    A.load_library()
    yield
    assert A.device_status(clear=True) == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(shape, g, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def stream_rows(rows, cols, g, dtype):
    x = randn((rows, cols), g) * torch.exp(randn((rows, 1), g))
    return x.to(dtype)


def check_codes(q, t, margin):
    """Codes equal to the rounded quotients t; neighbours allowed within `margin` of a border."""
    want, got = R.e4m3(t), q.double()
    off = got != want
    if off.any():
        assert margin > 0, (int(off.sum()), got[off][:4], want[off][:4])
        assert (R.tie_distance(t[off]) <= margin).all(), (got[off][:4], want[off][:4])
        assert ((got[off] - want[off]).abs() <= 2.0 ** -3 * want[off].abs().clamp_min(2.0 ** -6)).all()


def close(got, ref, rel):
    assert torch.isfinite(got).all()
    assert ((got.double() - ref).abs() <= rel * ref.abs() + 1e-300).all(), \
        float(((got.double() - ref).abs() / ref.abs().clamp_min(1e-300)).max())


# ------------------------------------------------------------------- quantise
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("square,transpose", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 7), (128, 128), (129, 127), (127, 129), (256, 512),
                                       (130, 264), (257, 1001), (5, 8192), (1000, 72), (131, 260)])
def test_quantize(rows, cols, square, transpose, dtype):
    g = gen(rows * 1000 + cols)
    x = stream_rows(rows, cols, g, dtype)
    q, scale = fp8.quantize_fp8(x, square=square, transpose=transpose)
    v = x.t() if transpose else x
    t, m = R.quotients(v, square)
    assert q.shape == v.shape and tuple(scale.shape) == tuple(m.shape)
    check_codes(q, t, 0 if dtype == BF16 else 2.0 ** -22)
    close(scale, m / 448, 2.0 ** -23)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (128, 128), (129, 127), (300, 512), (257, 1001), (5, 2048)])
def test_quantize_both_is_the_two_calls(rows, cols, square, dtype):
    x = stream_rows(rows, cols, gen(rows + cols), dtype)
    q, s, qt, st = fp8.quantize_fp8_both(x, square=square)
    for got, want in (((q, s), fp8.quantize_fp8(x, square=square)), ((qt, st), fp8.quantize_fp8(x, square=square, transpose=True))):
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    if square:
        assert torch.equal(q.view(torch.uint8).t(), qt.view(torch.uint8)) and torch.equal(s.t(), st)


def test_quantize_breaks_ties_to_even():
    # 448 * v / m is a border for many bf16 pairs (448 = 7 * 64): v = 3 m / 2^k, 21 k / m ...
    m = torch.arange(128, 256, device="cuda", dtype=F32)[:, None]
    v = torch.arange(0, 256, device="cuda", dtype=F32)[None, :]
    for scale_bits in (0, -60, 60):
        x = torch.minimum(v.expand(128, 256), m).clone()
        x[:, 0] = m[:, 0]
        x[:, 128] = m[:, 0]
        x = (x * 2.0 ** scale_bits).to(BF16)
        t, _ = R.quotients(x, False)
        assert (R.tie_distance(t) == 0).sum() > 100
        for kw in ({}, {"transpose": True}):
            xx = x.t().contiguous() if kw else x
            q, _s = fp8.quantize_fp8(xx, **kw)
            check_codes(q, t, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_small_and_extreme_groups(dtype):
    x = torch.zeros((6, 256), device="cuda")
    x[1, 3], x[1, 4] = 1e-38, -3e-38                # below the least maximum
    x[2] = 3.0e38
    x[2, 5] = -1e30
    x[3, :128] = 2.0 ** -100
    x[4, 7] = 2.0 ** -126
    x = x.to(dtype)
    for kw in ({}, {"transpose": True}, {"square": True}):
        q, scale = fp8.quantize_fp8(x.t().contiguous() if kw.get("transpose") else x, **kw)
        t, m = R.quotients(x, kw.get("square", False))
        check_codes(q, t, 0)
        close(scale, m / 448, 2.0 ** -23)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_non_finite_groups_have_a_nan_scale(bad, dtype):
    x = torch.ones((300, 300), device="cuda", dtype=dtype)
    x[200, 130] = bad
    for transpose in (False, True):
        _, s = fp8.quantize_fp8(x, transpose=transpose)
        want = torch.zeros_like(s, dtype=torch.bool)
        want[(130, 1) if transpose else (200, 1)] = True
        assert torch.equal(s.isnan(), want) and torch.isfinite(s[~want]).all()
        _, s = fp8.quantize_fp8(x, square=True, transpose=transpose)
        assert s.isnan().sum() == 1 and s[1, 1].isnan()


def test_quantize_writes_only_its_codes_and_scales():
    lib = A.load_library()
    for dtype, dt in ((BF16, 0), (F32, 1)):
        for square in (0, 1):
            for transpose in (0, 1):
                for rows, cols in ((5, 3), (130, 133), (64, 40)):
                    x = randn((rows, cols), gen(3), dtype)
                    qr, qc = (cols, rows) if transpose else (rows, cols)
                    gr, gc = (-(-qr // 128) if square else qr), -(-qc // 128)
                    pitch = (qc + 15) // 16 * 16 + 16
                    buf = torch.full((qr + 2, pitch), 0x55, dtype=torch.uint8, device="cuda")
                    sbuf = torch.full((gr + 1, gc + 1), -7.0, device="cuda")
                    rc = lib.evo_quantize_fp8(rows, cols, dt, A._ptr(x), cols, square, transpose, A._ptr(buf), pitch,
                                              A._ptr(sbuf), gc + 1, 1, A._stream(x.device))
                    assert rc == 0
                    assert (buf[:qr, qc:] == 0x55).all() and (buf[qr:] == 0x55).all()
                    assert (sbuf[:gr, gc:] == -7).all() and (sbuf[gr:] == -7).all()
                    t, m = R.quotients(x.t() if transpose else x, bool(square))
                    check_codes(buf[:qr, :qc].contiguous().view(fp8.CODES), t, 0 if dtype == BF16 else 2.0 ** -22)
                    close(sbuf[:gr, :gc], m / 448, 2.0 ** -23)


def test_quantize_strided_and_offset_rows():
    big = randn((70, 400), gen(5), BF16)
    for view in (big[:, 8:264], big[:, 3:260], big[::2, :128], big[1:2].expand(33, 400), big.t()[5:200]):
        for transpose in (False, True):
            q, s = fp8.quantize_fp8(view, transpose=transpose)
            t, m = R.quotients(view.t() if transpose else view, False)
            check_codes(q, t, 0)
            close(s, m / 448, 2.0 ** -23)


# ------------------------------------------------------------------- norm
def check_norm(x, res, w, eps, out, want_n=False):
    rows, cols = x.shape
    q, scale, h, rstd = out[:4]
    rh, rrstd, rn = R.norm(x, res, w, eps)
    assert torch.equal(h.double(), rh)
    close(rstd, rrstd, 2.0 ** -17)
    t, m = R.quotients(rn, False)
    exact = x.dtype == BF16 and (w is None or w.dtype == BF16)
    check_codes(q, t, 2.0 ** -44 if exact else 2.0 ** -21)   # exact: only where fp64's own n lies beside a border
    close(scale, m / 448, 2.0 ** -17)
    if want_n:
        n = out[4]
        bound = (torch.finfo(x.dtype).eps / 2 + 2.0 ** -17) * rn.abs() + 1e-38
        assert ((n.double() - rn).abs() <= bound).all()


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, None), (BF16, None)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (17, 64), (9, 128), (1000, 256), (129, 257),
                                       (40, 512), (33, 1000), (65, 1024), (20, 2500), (7, 5001), (4, 8192),
                                       (3, 9000), (2, 16384), (2, 32768), (3, 32767), (700, 700), (301, 1500), (50, 2049),
                                       (9, 4100), (4, 10300)])
def test_add_rms_norm(rows, cols, residual, dtype, wdtype):
    g = gen(rows * 7 + cols)
    x = stream_rows(rows, cols, g, dtype)
    res = stream_rows(rows, cols, g, dtype) if residual else None
    w = None if wdtype is None else (1 + 0.3 * randn((cols,), g)).to(wdtype)
    out = fp8.add_rms_norm_fp8(x, res, w, 1e-5, want_n=True)
    check_norm(x, res, w, 1e-5, out, want_n=True)
    if not residual:
        assert out[2] is x


def test_add_rms_norm_many_rows_and_strides():
    g = gen(11)
    x, res = stream_rows(20001, 256, g, BF16), stream_rows(20001, 256, g, BF16)
    w = (1 + 0.3 * randn((256,), g)).to(BF16)
    check_norm(x, res, w, 1e-5, fp8.add_rms_norm_fp8(x, res, w, 1e-5))
    big = stream_rows(300, 700, g, BF16)
    for view in (big[:, 8:264], big[:, 1:258], big[::3, :256]):
        w = (1 + 0.3 * randn((view.shape[1],), g)).to(BF16)
        r = stream_rows(*view.shape, g, BF16)
        check_norm(view, r, w, 1e-5, fp8.add_rms_norm_fp8(view, r, w, 1e-5))
    x3 = stream_rows(24, 256, g, BF16).view(2, 3, 4, 256)
    q, s, h, rstd = fp8.add_rms_norm_fp8(x3, x3, None, 1e-5)
    assert q.shape == x3.shape and s.shape == (2, 3, 4, 2) and rstd.shape == (2, 3, 4) and h.shape == x3.shape
    q2, s2, _, _ = fp8.add_rms_norm_fp8(x3.view(24, 256), x3.view(24, 256), None, 1e-5)
    assert torch.equal(q.view(24, 256).view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s.reshape(24, 2), s2)


def test_add_rms_norm_zero_rows_nan_rows_and_least_maximum():
    x = torch.zeros((6, 300), device="cuda", dtype=BF16)
    x[1] = 1e-30                                     # n = 1e-30 / sqrt(eps): below the least maximum
    x[2, 7] = float("nan")
    x[3, 299] = float("inf")
    x[4] = 3.0
    q, s, h, rstd = fp8.add_rms_norm_fp8(x, None, None, 1e-5)
    ok = [0, 1, 4, 5]
    rh, rrstd, rn = R.norm(x[ok], None, None, 1e-5)
    t, m = R.quotients(rn, False)
    check_codes(q[ok], t, 2.0 ** -21)
    close(s[ok], m / 448, 2.0 ** -17)
    assert s[[2, 3]].isnan().all()


def test_rows_off_16_bytes_and_their_neighbours():
    # bf16 rows at even and odd element offsets inside wider ones: the values beside them are NaN
    # on the way in, and on the way out they stay as they were
    g = gen(20)
    lib = A.load_library()
    for cols in (1, 7, 8, 9, 255, 263, 1001):
        for off in range(4):
            for pitch in (cols + 5, (cols + 15) // 8 * 8):
                wide = torch.full((6, pitch + 8), float("nan"), dtype=BF16, device="cuda")
                x = wide[:, off:off + cols]
                x.copy_(stream_rows(6, cols, g, BF16))
                want = fp8.add_rms_norm_fp8(x.contiguous(), x.contiguous(), None, 1e-5, want_n=True)
                h_buf = torch.full((6, pitch + 8), 5.0, dtype=BF16, device="cuda")
                n_buf = h_buf.clone()
                q, s = fp8.empty_codes(6, cols, x.device), fp8.empty_scales(6, -(-cols // 128), x.device)
                at = lambda b: b.data_ptr() + 2 * off  # noqa: E731
                rc = lib.evo_add_rms_norm_fp8(6, cols, 0, at(wide), pitch + 8, at(wide), pitch + 8, None, 0, 1e-5,
                                              A._ptr(q), q.stride(0), A._ptr(s), 1, 6, at(h_buf), pitch + 8, at(n_buf),
                                              pitch + 8, None, A._stream(x.device))
                assert rc == 0
                for buf, ref in ((h_buf, want[2]), (n_buf, want[4])):
                    assert torch.equal(buf[:, off:off + cols], ref)
                    assert (buf[:, :off] == 5).all() and (buf[:, off + cols:] == 5).all()
                assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
                for kw in ({}, {"transpose": True}, {"square": True}):
                    for a, b in zip(fp8.quantize_fp8(x, **kw), fp8.quantize_fp8(x.contiguous(), **kw)):
                        assert torch.equal(a.view(torch.uint8) if a.dtype == fp8.CODES else a,
                                           b.view(torch.uint8) if b.dtype == fp8.CODES else b)


def test_add_rms_norm_in_place_on_the_residual_stream():
    # h may be x or the residual itself: the C call, with the rows of both pitches
    g = gen(21)
    lib = A.load_library()
    for cols in (256, 250, 5000):
        x, res = stream_rows(37, cols, g, BF16), stream_rows(37, cols, g, BF16)
        want = fp8.add_rms_norm_fp8(x, res, None, 1e-5)
        for target in ("x", "res"):
            xx, rr = x.clone(), res.clone()
            h = xx if target == "x" else rr
            q, s = fp8.empty_codes(37, cols, x.device), fp8.empty_scales(37, -(-cols // 128), x.device)
            rc = lib.evo_add_rms_norm_fp8(37, cols, 0, A._ptr(xx), cols, A._ptr(rr), cols, None, 0, 1e-5, A._ptr(q),
                                          q.stride(0), A._ptr(s), 1, 37, A._ptr(h), cols, None, 0, None,
                                          A._stream(x.device))
            assert rc == 0
            assert torch.equal(h, want[2]) and torch.equal(s, want[1])
            assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8))


# ------------------------------------------------------------------- norm, backward
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, None)])
@pytest.mark.parametrize("stream", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (17, 64), (1000, 256), (129, 257), (40, 512),
                                       (33, 1000), (6001, 1024), (20, 2500), (7, 5001), (3, 9000), (2, 32767), (700, 700), (301, 1500), (50, 2049),
                                       (400, 4100), (4, 10300)])
def test_add_rms_norm_bwd(rows, cols, stream, dtype, wdtype):
    g = gen(rows * 13 + cols)
    h = stream_rows(rows, cols, g, dtype)
    rstd = R.norm(h, None, None, 1e-5)[1].float()
    dy, dh = randn((rows, cols), g, dtype), randn((rows, cols), g, dtype) if stream else None
    w = None if wdtype is None else (1 + 0.3 * randn((cols,), g)).to(wdtype)
    dx, dw = fp8.add_rms_norm_bwd(dy, dh, h, rstd, w)
    rdx, rdw = R.norm_bwd(dy, dh, h, rstd, w)
    gg = dy.double().abs() if w is None else (dy.double() * w.double()).abs()
    n = h.double().abs() * rstd.double()[:, None]
    terms = rstd.double()[:, None] * (gg + n * (gg * n).mean(1, keepdim=True))
    if dh is not None:
        terms = terms + dh.double().abs()
    assert dx.dtype == dtype and ((dx.double() - rdx).abs() <= torch.finfo(dtype).eps / 2 * rdx.abs() + 2.0 ** -17 * terms).all()
    # 148 blocks at least walk many rows; each block adds up to 8 rows' partial sums, then the blocks' rows 32 at a time
    adds = rows / 148 + 64 + 32
    assert ((dw.double() - rdw).abs() <= adds * 2.0 ** -24 * (dy.double().abs() * n).sum(0) + 1e-30).all()
    dx2, none = fp8.add_rms_norm_bwd(dy, dh, h, rstd, w, want_dweight=False)
    assert none is None and torch.equal(dx, dx2)
    assert torch.equal(fp8.add_rms_norm_bwd(dy, dh, h, rstd, w)[1], dw)
    assert torch.equal(fp8.add_rms_norm_bwd(dy, dh, h, rstd, w, dweight_dtype=BF16)[1], dw.to(BF16))


def test_add_rms_norm_bwd_against_differences():
    # directional central differences of the plain norm in 64 bits: error of order step^2
    g = gen(31)
    x, w = randn((5, 300), g), 1 + 0.3 * randn((300,), g)
    dy, dh = randn((5, 300), g), randn((5, 300), g)
    _, rstd, _ = R.norm(x, None, w, 1e-5)
    dx, dw = fp8.add_rms_norm_bwd(dy, dh, x, rstd.float(), w)

    def loss(xx, ww):
        rs = 1 / torch.sqrt((xx * xx).mean(1) + 1e-5)
        return (dy.double() * (xx * rs[:, None] * ww)).sum() + (dh.double() * xx).sum()

    step = 1e-4
    for _ in range(4):
        vx, vw = randn((5, 300), g).double(), randn((300,), g).double()
        d = (loss(x.double() + step * vx, w.double() + step * vw) - loss(x.double() - step * vx, w.double() - step * vw)) / (2 * step)
        got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        scale = (dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum()
        assert abs(float(d - got)) <= 1e-5 * float(scale)     # 2^-17 of the terms, and step^2 = 1e-8


# ------------------------------------------------------------------- product
def operands(M, N, K, square, g):
    """Codes and scales of random matrices, from the reference."""
    out = []
    for r, sq in ((M, False), (N, square)):
        q, s = R.quantize(stream_rows(r, K, g, F32), sq)
        codes = fp8.empty_codes(r, K, "cuda")
        codes.copy_(q.float().to(fp8.CODES))
        out += [codes, s.float()]
    return out


def check_linear(y, xq, xs, wq, ws, bias):
    x, w = R.values(xq, xs, False), R.values(wq, ws)
    ref = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    nb = -(-xq.shape[1] // 128) + 10
    bound = (2.0 ** -21 + nb * 2.0 ** -24) * mag + torch.finfo(y.dtype).eps / 2 * ref.abs()
    assert torch.isfinite(y).all()
    assert ((y.double() - ref).abs() <= bound).all(), float(((y.double() - ref).abs() / bound.clamp_min(1e-300)).max())


SHAPES = [(1, 1, 1), (1, 128, 128), (3, 5, 17), (1, 4096, 4096), (128, 128, 128), (129, 127, 129), (64, 1024, 256),
          (200, 136, 4000), (5, 300, 12345), (257, 1000, 384), (300, 2048, 512), (1, 8, 8192), (17, 777, 1040),
          (2500, 1024, 256), (700, 1001, 130),
          (2, 77, 530), (3, 1000, 4097), (4, 129, 700), (4, 4096, 1024), (5, 4096, 1024), (2, 1, 8191),
          (1, 8192, 8192), (1, 3, 50000), (6, 3, 50000), (100, 77, 40001), (129, 257, 16384)]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_fp8_linear(M, N, K, square, out_dtype):
    g = gen(M + 3 * N + 7 * K)
    xq, xs, wq, ws = operands(M, N, K, square, g)
    bias = randn((N,), g) if (M + N) % 2 else None
    y = fp8.fp8_linear(xq, xs, wq, ws, bias, out_dtype=out_dtype)
    assert y.shape == (M, N) and y.dtype == out_dtype
    check_linear(y, xq, xs, wq, ws, bias)
    assert torch.equal(y, fp8.fp8_linear(xq, xs, wq, ws, bias, out_dtype=out_dtype))


@pytest.mark.parametrize("M,N,K", [(20000, 1024, 256), (4099, 4100, 1000), (3000, 2000, 2100), (1024, 256, 40000)])
@pytest.mark.parametrize("square", [True, False])
def test_fp8_linear_large(M, N, K, square):
    g = gen(M + N + K)
    xq, xs, wq, ws = operands(M, N, K, square, g)
    for out_dtype in (BF16, F32):
        check_linear(fp8.fp8_linear(xq, xs, wq, ws, None, out_dtype=out_dtype), xq, xs, wq, ws, None)


def test_fp8_linear_scale_layouts_pitches_and_untouched_bytes():
    g = gen(41)
    lib = A.load_library()
    work = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for M, N, K in ((130, 200, 300), (70, 129, 128), (520, 264, 1000), (2000, 1024, 256), (4000, 2056, 130),
                    (3, 130, 20000), (200, 77, 30000)):
        xq, xs, wq, ws = operands(M, N, K, True, g)
        want = fp8.fp8_linear(xq, xs, wq, ws)
        assert torch.equal(want, fp8.fp8_linear(xq, xs.t().contiguous().t(), wq, ws.t().contiguous().t()))
        # codes inside wider rows whose other bytes are NaN codes; y inside a wider buffer
        wide = torch.full((M, (K + 15) // 16 * 16 + 48), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, 16:16 + K] = xq.contiguous().view(torch.uint8)
        xw = wide.view(fp8.CODES)[:, 16:16 + K]
        assert torch.equal(want, fp8.fp8_linear(xw, xs, wq, ws))
        for off, ld in ((0, N + 8), (1, N + 3)):         # the second: rows at odd addresses
            buf = torch.full((M + 1, ld), 9.0, dtype=BF16, device="cuda")
            rc = lib.evo_fp8_linear(M, N, K, A._ptr(xq), xq.stride(0), A._ptr(xs), xs.stride(0), xs.stride(1),
                                    A._ptr(wq), wq.stride(0), A._ptr(ws), ws.stride(0), ws.stride(1), 0, None, 0,
                                    buf.data_ptr() + 2 * off, ld, A._ptr(work), work.numel(), A._stream(xq.device))
            assert rc == 0
            flat = buf.view(-1)
            y = flat[off:off + M * ld].view(M, ld) if off == 0 else torch.as_strided(flat, (M, N), (ld, 1), off)
            assert torch.equal(y[:, :N], want)
            mask = torch.ones_like(flat, dtype=torch.bool)
            torch.as_strided(mask, (M, N), (ld, 1), off).fill_(False)
            assert (flat[mask] == 9.0).all()


@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("M,N,K", [(2500, 2056, 1024), (2500, 2056, 1025), (2049, 2571, 1700)])
def test_fp8_linear_long_sums_bias_and_odd_pitches(M, N, K, square):
    # both sides of the sum where whole tiles change their summing warps
    g = gen(M + N + K)
    xq, xs, wq, ws = operands(M, N, K, square, g)
    bias = randn((N,), g)
    lib = A.load_library()
    for dtype in (BF16, F32):
        y = fp8.fp8_linear(xq, xs, wq, ws, bias, out_dtype=dtype)
        check_linear(y, xq, xs, wq, ws, bias)
        ld = N + 3
        buf = torch.full((M * ld + 1,), 9.0, dtype=dtype, device="cuda")
        rc = lib.evo_fp8_linear(M, N, K, A._ptr(xq), xq.stride(0), A._ptr(xs), xs.stride(0), xs.stride(1),
                                A._ptr(wq), wq.stride(0), A._ptr(ws), ws.stride(0), ws.stride(1), int(not square),
                                A._ptr(bias), int(dtype == F32), buf.data_ptr() + buf.element_size(), ld, None, 0,
                                A._stream(xq.device))
        assert rc == 0
        assert torch.equal(torch.as_strided(buf, (M, N), (ld, 1), 1), y)
        torch.as_strided(buf, (M, N), (ld, 1), 1).fill_(9.0)
        assert (buf == 9.0).all()


def test_fp8_linear_nan_scales_reach_their_rows_only():
    g = gen(43)
    x = randn((300, 260), g, BF16)
    x[7, 200] = float("nan")
    x[299, 0] = float("inf")
    w = randn((140, 260), g, BF16)
    y = fp8.fp8_linear(*fp8.quantize_fp8(x), *fp8.quantize_fp8(w, square=True))
    bad = torch.zeros(300, dtype=torch.bool, device="cuda")
    bad[[7, 299]] = True
    assert y[bad].isnan().all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("M", [1, 2, 70, 20000])
def test_fp8_linear_nan_codes(M):
    # a NaN code under a finite scale: its row of y, and in w its column
    g = gen(44)
    xq, xs = fp8.quantize_fp8(randn((M, 300), g, BF16))
    wq, ws = fp8.quantize_fp8(randn((140, 300), g, BF16), square=True)
    xq.view(torch.uint8)[M - 1, 299] = 0x7F
    wq.view(torch.uint8)[5, 7] = 0xFF
    y = fp8.fp8_linear(xq, xs, wq, ws)
    bad = torch.zeros((M, 140), dtype=torch.bool, device="cuda")
    bad[M - 1] = True
    bad[:, 5] = True
    assert torch.equal(y.isnan(), bad)


def test_training_functions_are_once_differentiable():
    g = gen(45)
    x, w = randn((8, 64), g, BF16).requires_grad_(True), randn((16, 64), g, BF16).requires_grad_(True)
    dy = randn((8, 16), g, BF16).requires_grad_(True)
    (gx,) = torch.autograd.grad(fp8.fp8_linear_train(x, w), x, dy, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.sum().backward()


def test_fp8_linear_leading_axes_and_empty_calls():
    g = gen(47)
    x = randn((2, 3, 5, 200), g, BF16)
    w8, ws = fp8.quantize_fp8(randn((64, 200), g, BF16), square=True)
    q, s = fp8.quantize_fp8(x)
    y = fp8.fp8_linear(q, s, w8, ws)
    assert y.shape == (2, 3, 5, 64)
    assert torch.equal(y.view(30, 64), fp8.fp8_linear(*fp8.quantize_fp8(x.view(30, 200)), w8, ws))
    q1, s1 = fp8.quantize_fp8(x[0, 0, 0])
    assert torch.equal(fp8.fp8_linear(q1, s1, w8, ws), y[0, 0, 0])
    e = x[:, :0]
    q, s = fp8.quantize_fp8(e)
    assert q.shape == (2, 0, 5, 200) and fp8.fp8_linear(q, s, w8, ws).shape == (2, 0, 5, 64)
    q, s, h, rstd = fp8.add_rms_norm_fp8(e, e, None, 1e-5)
    assert q.shape == e.shape and rstd.shape == (2, 0, 5)
    dx, dw = fp8.add_rms_norm_bwd(e, None, h, rstd, None)
    assert dx.shape == e.shape and (dw == 0).all()


# ------------------------------------------------------------------- a run of them
def test_norm_projection_attention_projection_norm():
    """The stream's norm, q/k/v/g in 8 bits, the attention on views of that output, the output
    projection in 8 bits, and the next norm, which adds it to the stream."""
    B, S, N, H, C = 1, 6, 40, 2, 32
    D = 96
    g = gen(53)
    stream, x = randn((B, S, N, D), g, BF16), randn((B, S, N, D), g, BF16)
    w_in, w_out = randn((4 * H * C, D), g, BF16) / D ** 0.5, randn((D, H * C), g, BF16) / (H * C) ** 0.5
    gamma = (1 + 0.2 * randn((D,), g)).to(BF16)
    pb = randn((B, 1, H, N, N), g, BF16)
    wi, wis = fp8.quantize_fp8(w_in, square=True)
    wo, wos = fp8.quantize_fp8(w_out, square=True)
    q8, s8, h, _ = fp8.add_rms_norm_fp8(x, stream, gamma, 1e-5)
    y = fp8.fp8_linear(q8, s8, wi, wis)
    rn = R.norm(x.view(-1, D), stream.view(-1, D), gamma, 1e-5)[2]
    check_linear(y.view(-1, 4 * H * C), q8.flatten(0, 2), s8.reshape(-1, 1), wi, wis, None)
    ref = R.values(*R.quantize(rn), False) @ R.values(wi, wis).t()
    assert float((y.view(-1, 4 * H * C).double() - ref).norm() / ref.norm()) <= 2.0 ** -8
    q, k, v, gate = A.qkvg_views(y, H)
    out, _ = A.evo_attn_fwd(q, k, v, gate, None, pb)
    o = out.reshape(B, S, N, H * C)
    z = fp8.fp8_linear(*fp8.quantize_fp8(o), wo, wos)
    ref_z = R.values(*R.quantize(o.view(-1, H * C)), False) @ R.values(wo, wos).t()
    assert float((z.view(-1, D).double() - ref_z).norm() / ref_z.norm()) <= 2.0 ** -8
    n8, ns, h2, _ = fp8.add_rms_norm_fp8(z, h, gamma, 1e-5)
    check_norm(z.view(-1, D), h.view(-1, D), gamma, 1e-5, (n8.flatten(0, 2), ns.reshape(-1, 1), h2.view(-1, D),
                                                           1 / torch.sqrt(h2.double().square().mean(-1) + 1e-5).view(-1).float()))


# ------------------------------------------------------------------- training
def rel(a, b):
    return float((a.detach().double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,K,N", [(300, 256, 384), (77, 100, 33), (1, 130, 8), (1030, 64, 257)])
def test_fp8_linear_train(rows, K, N, dtype):
    g = gen(rows + K + N)
    x, w, dy = randn((rows, K), g, dtype), (randn((N, K), g) / K ** 0.5).to(dtype), randn((rows, N), g, dtype)
    x.requires_grad_(True), w.requires_grad_(True)
    y = fp8.fp8_linear_train(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert (y.dtype, dx.dtype, dw.dtype) == (dtype,) * 3
    x, w = x.detach(), w.detach()
    # the formula, with every operand quantised as documented: what is left are the roundings of
    # the outputs (bf16 2^-8 at most) and, in fp32, codes beside a border
    xv, wv = R.values(*R.quantize(x), False), R.values(*R.quantize(w, True), True)
    ref_dx = R.values(*R.quantize(dy), False) @ wv
    ref_dw = R.values(*R.quantize(dy.t()), False) @ R.values(*R.quantize(x.t()), False).t()
    for got, ref in ((y, xv @ wv.t()), (dx, ref_dx), (dw, ref_dw)):
        assert rel(got, ref) <= (2.0 ** -8 if dtype == BF16 else 1e-3)
    # and the gradients without quantisation: each operand within 2^-4 of itself, or 2^-10 / 448 of its
    # group's maximum where its code is subnormal
    err = lambda v, sq=False: 2.0 ** -4 * v.double().abs() + 2.0 ** -10 * R.values(torch.ones_like(v, dtype=torch.float64), R.quotients(v, sq)[1] / 448, sq)  # noqa: E731
    edy, ew = err(dy), err(w, True)
    bound = edy @ (w.double().abs() + ew) + dy.double().abs() @ ew
    true = dy.double() @ w.double()
    assert ((dx.double() - true).abs() <= 1.01 * bound + torch.finfo(dtype).eps * (true.abs() + bound)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [True, False])
def test_add_rms_norm_linear_gradients(dtype, residual):
    g = gen(61)
    rows, K, N = 200, 260, 140
    x, res, dh = (randn((2, 100, K), g, dtype) for _ in range(3))
    gamma, w = (1 + 0.2 * randn((K,), g)).to(dtype), (randn((N, K), g) / K ** 0.5).to(dtype)
    dy = randn((2, 100, N), g, dtype)
    leaves = [x, gamma, w] + ([res] if residual else [])
    for t in leaves:
        t.requires_grad_(True)
    h, y = fp8.add_rms_norm_linear(x, res if residual else None, gamma, 1e-5, w)
    grads = torch.autograd.grad((h, y), leaves, (dh, dy))
    with torch.no_grad():
        flat = lambda t: t.reshape(rows, -1)  # noqa: E731
        rh, rrstd, rn = R.norm(flat(x), flat(res) if residual else None, gamma, 1e-5)
        wv = R.values(*R.quantize(w, True), True)
        ref_y = R.values(*R.quantize(rn), False) @ wv.t()
        dn = (R.values(*R.quantize(flat(dy)), False) @ wv).to(dtype)
        rdx, rdg = R.norm_bwd(dn, flat(dh), rh, rrstd, gamma)
        nq = R.values(*R.quantize(rn.to(dtype).t()), False)
        rdw = R.values(*R.quantize(flat(dy).t()), False) @ nq.t()
        tol = 2.0 ** -8 if dtype == BF16 else 1e-3
        assert torch.equal(flat(h).double(), rh)
        assert rel(flat(y), ref_y) <= tol
        for got, ref in zip(grads, [rdx, rdg, rdw] + ([rdx] if residual else [])):
            assert got.dtype == dtype and rel(got.reshape(ref.shape), ref) <= tol


def test_training_functions_with_unused_outputs_and_expanded_gradients():
    g = gen(67)
    x, w = randn((40, 128), g, BF16).requires_grad_(True), randn((64, 128), g, BF16).requires_grad_(True)
    fp8.fp8_linear_train(x, w).sum().backward()
    assert torch.isfinite(x.grad).all() and torch.isfinite(w.grad).all()
    x2, r2 = (randn((40, 128), g, BF16).requires_grad_(True) for _ in range(2))
    h, y = fp8.add_rms_norm_linear(x2, r2, None, 1e-5, w)
    (gx,) = torch.autograd.grad(h.sum(), x2, retain_graph=True)
    assert torch.equal(gx, torch.ones_like(gx))
    gx, gr = torch.autograd.grad(y.sum(), (x2, r2))
    assert torch.equal(gx, gr) and torch.isfinite(gx).all()
    e = torch.zeros((0, 128), dtype=BF16, device="cuda", requires_grad=True)
    ge, gw = torch.autograd.grad(fp8.fp8_linear_train(e, w).sum(), (e, w))
    assert ge.shape == (0, 128) and (gw == 0).all()
    h, y = fp8.add_rms_norm_linear(e, e, None, 1e-5, w)
    ge, gw = torch.autograd.grad((h.sum() + y.sum()), (e, w))
    assert ge.shape == (0, 128) and (gw == 0).all()


def test_gradients_use_the_weight_of_the_forward():
    g = gen(68)
    x, w = randn((40, 128), g, BF16).requires_grad_(True), randn((64, 128), g, BF16).requires_grad_(True)
    dy = randn((40, 64), g, BF16)
    (want,) = torch.autograd.grad(fp8.fp8_linear_train(x, w), x, dy)
    y = fp8.fp8_linear_train(x, w)
    with torch.no_grad():
        w.mul_(3)
    (got,) = torch.autograd.grad(y, x, dy)
    assert torch.equal(got, want)


# ------------------------------------------------------------------- streams and graphs
def test_graph_replay_matches_eager():
    g = gen(71)
    x, res = randn((200, 512), g, BF16), randn((200, 512), g, BF16)
    gamma, w = randn((512,), g, BF16), randn((384, 512), g, BF16)
    w8, ws = fp8.quantize_fp8(w, square=True)

    def step():
        q, s, h, rstd = fp8.add_rms_norm_fp8(x, res, gamma, 1e-5)
        y = fp8.fp8_linear(q, s, w8, ws)
        dx, dw = fp8.add_rms_norm_bwd(h, None, h, rstd, gamma)
        return y, h, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        x.copy_(randn((200, 512), gen(seed), BF16))
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_captured_training_step_matches_eager():
    # the capture has leaves of its own: no eager graph of them is alive beside it
    g = gen(72)
    data = [randn(s, g, BF16) for s in ((130, 200), (130, 200), (200,), (96, 200))]
    dh, dy = randn((130, 200), g, BF16), randn((130, 96), g, BF16)

    def step(leaves):
        h, y = fp8.add_rms_norm_linear(leaves[0], leaves[1], leaves[2], 1e-5, leaves[3])
        return (h, y) + torch.autograd.grad((h, y), leaves, (dh, dy))

    want = [t.detach().clone() for t in step([t.clone().requires_grad_(True) for t in data])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step([t.clone().requires_grad_(True) for t in data])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    leaves = [t.clone().requires_grad_(True) for t in data]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(leaves)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_captured_products_keep_their_own_workspaces():
    g = gen(74)
    sets = [operands(8, 512, 16384, True, g) for _ in range(2)]
    want = [fp8.fp8_linear(*s) for s in sets]
    graphs, got = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(fp8.fp8_linear(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_on_two_streams_do_not_disturb_each_other():
    g = gen(73)
    sets = [operands(8, 512, 16384, True, g) for _ in range(2)]   # both with a workspace
    want = [fp8.fp8_linear(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(fp8.fp8_linear(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_offsets_beyond_32_bits():
    """Rows behind 2^31 elements: 2.2 M rows x 1024 in bf16 (4.5 GB), the last rows against the reference."""
    rows, cols = 2_200_000, 1024
    x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    tail = randn((300, cols), gen(79), BF16)
    x[-300:] = tail
    q, s = fp8.quantize_fp8(x)
    t, m = R.quotients(tail, False)
    check_codes(q[-300:], t, 0)
    close(s[-300:], m / 448, 2.0 ** -23)
    w = randn((1024, cols), gen(80), BF16)
    w8, ws = fp8.quantize_fp8(w, square=True)
    y = fp8.fp8_linear(q, s, w8, ws)
    check_linear(y[-300:], q[-300:], s[-300:], w8, ws, None)
    del y
    out = fp8.add_rms_norm_fp8(x, x, None, 1e-5)
    check_norm(tail, tail, None, 1e-5, [o[-300:] for o in out])
