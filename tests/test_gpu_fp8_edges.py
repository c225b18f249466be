"""GPU parity of the 8-bit operators at the edges of their arguments: tiny rows and small eps,
empty axes, ties of fp32 values, layouts of the products of one and two rows, long sums.

The tolerances are those of test_gpu_fp8.py and, for a group held at the least maximum 2^-100,
2^-21 for the codes: there 448 v / m depends on rms, which takes an approximate reciprocal square
root (2^-22) and a mean in fp32.
"""
import pytest
import torch

import _fp8 as R
from evoformer_pair_bias_b200 import attention as A
from evoformer_pair_bias_b200 import fp8
from test_gpu_fp8 import BF16, F32, check_codes, check_linear, close, gen, operands, randn, stream_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from evoformer_pair_bias_b200 import build
    build.build()
    A.load_library()
    yield
    assert A.device_status(clear=True) == 0


# ------------------------------------------------------------------- norm of tiny rows
def tiny_rows(cols, g, dtype):
    x = randn((8, cols), g) * 10.0 ** torch.tensor([0, -6, -9, -15, -4, 0, -30, 3], device="cuda")[:, None]
    x[0] = 0                                         # as padding and masked rows are
    x[1, :128] = 0                                   # a group of zeros beside small values
    x[3, -100:] *= 1e-10                             # far below the row's rms
    x[4, 1:] = 0
    return x.to(dtype)                               # 6: its squares leave fp32's range


@pytest.mark.parametrize("dtype,wdtype", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32)])
@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-16, 1e-12, 1e-10, 1e-8, 9.5e-7, 1e-6])
@pytest.mark.parametrize("cols", [128, 300, 1001, 5000, 9000])
def test_norm_of_tiny_rows(cols, eps, dtype, wdtype):
    g = gen(cols + int(eps * 1e20) % 97)
    x = tiny_rows(cols, g, dtype)
    w = None if wdtype is None else (1 + 0.3 * randn((cols,), g)).to(wdtype)
    q, scale, h, rstd, n = fp8.add_rms_norm_fp8(x, None, w, eps, want_n=True)
    # rows whose mean of squares + eps is 0 in fp32 have no norm: NaN scales
    none = [r for r in range(8) if eps == 0 and not x[r].float().square().any()]
    assert none == ([] if eps else [0, 6] if cols > 128 else [0, 1, 6])
    assert scale[none].isnan().all()
    rows = [r for r in range(8) if r not in none]
    q, scale, rstd, n = q[rows], scale[rows], rstd[rows], n[rows]
    _, rrstd, rn = R.norm(x[rows], None, w, eps)
    close(rstd, rrstd, 2.0 ** -17)
    t, m = R.quotients(rn, False)
    close(scale, m / 448, 2.0 ** -17)
    exact = dtype == BF16 and wdtype != F32
    held = (m <= R.LEAST * (1 + 2.0 ** -16)).repeat_interleave(128, 1)[:, :cols]
    for part, margin in ((held, 2.0 ** -21), (~held, 2.0 ** -44 if exact else 2.0 ** -21)):
        if part.any():
            check_codes(q.contiguous()[part], t[part], margin)
    # n: rounded in its type, subnormal where fp32 is
    bound = (torch.finfo(dtype).eps / 2 + 2.0 ** -17) * rn.abs() + (2.0 ** -133 if dtype == BF16 else 2.0 ** -149)
    assert ((n.double() - rn).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_projection_of_zero_rows_is_zero_for_any_eps(dtype):
    g = gen(7)
    x = randn((5, 260), g, dtype)
    x[[1, 4]] = 0
    w = (randn((40, 260), g) / 16).to(dtype)
    gamma = (1 + 0.3 * randn((260,), g)).to(dtype)
    for eps in (1e-5, 1e-12, 1e-16, 1e-30):
        h, y = fp8.add_rms_norm_linear(x, None, gamma, eps, w)
        assert (y[[1, 4]] == 0).all() and torch.isfinite(y).all() and (y[[0, 2, 3]] != 0).any(1).all()


# ------------------------------------------------------------------- empty axes
def leave_nans(*shapes, dtype=BF16):
    """Memory that the next results of these shapes may get, full of NaN."""
    for s in shapes:
        for t in [torch.full(s, float("nan"), dtype=dtype, device="cuda") for _ in range(4)]:
            del t


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_a_projection_without_outputs(dtype):
    # n_out = 0: the input's gradient is the empty sum
    g = gen(83)
    x, w = randn((37, 200), g, dtype).requires_grad_(True), randn((0, 200), g, dtype).requires_grad_(True)
    y = fp8.fp8_linear_train(x, w)
    assert y.shape == (37, 0)
    leave_nans((37, 200), dtype=dtype)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert dx.shape == x.shape and dx.dtype == dtype and (dx == 0).all() and dw.shape == (0, 200)
    dh = randn((37, 200), g, dtype)
    gamma = (1 + 0.3 * randn((200,), g)).to(dtype).requires_grad_(True)
    h, y = fp8.add_rms_norm_linear(x, None, gamma, 1e-5, w)
    leave_nans((37, 200), dtype=dtype)
    dx, dgamma, dw = torch.autograd.grad((h, y), (x, gamma, w), (dh, torch.zeros_like(y)))
    assert torch.equal(dx, dh) and (dgamma == 0).all() and dw.shape == (0, 200)


def test_linear_bwd_without_outputs_zeroes_the_rows_of_dx_only():
    lib = A.load_library()
    for dt, dtype in ((0, BF16), (1, F32)):
        for ld in (40, 43):
            buf = torch.full((7, ld), 9.0, dtype=dtype, device="cuda")
            rc = lib.evo_fp8_linear_bwd(6, 0, 40, dt, None, 0, None, 0, None, 0, None, 1, 1, A._ptr(buf), ld, None, 1, 0,
                                        None, 0, A._stream(buf.device))
            assert rc == 0
            assert (buf[:6, :40] == 0).all() and (buf[:6, 40:] == 9).all() and (buf[6:] == 9).all()


def test_gradients_without_outputs_in_a_captured_graph():
    dy = torch.empty((5, 0), dtype=BF16, device="cuda")
    wq_t, ws_t = fp8.quantize_fp8(torch.empty((0, 64), dtype=BF16, device="cuda"), square=True, transpose=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = fp8.fp8_linear_bwd(dy, None, wq_t, ws_t, want_dw=False)[0]
    dx.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    assert (dx == 0).all()


def test_leading_axes_of_an_empty_last_axis():
    g = gen(84)
    x, w = randn((2, 3, 200), g, BF16).requires_grad_(True), randn((0, 200), g, BF16).requires_grad_(True)
    y = fp8.fp8_linear_train(x, w)
    assert y.shape == (2, 3, 0)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert dx.shape == x.shape and (dx == 0).all() and dw.shape == (0, 200)
    h, y = fp8.add_rms_norm_linear(x, x, None, 1e-5, w)
    assert h.shape == x.shape and y.shape == (2, 3, 0)
    dx, dw = torch.autograd.grad((h, y), (x, w), (torch.ones_like(h), torch.zeros_like(y)))
    assert (dx == 2).all() and dw.shape == (0, 200)
    e = torch.empty((2, 3, 0), dtype=BF16, device="cuda")
    q, s = fp8.quantize_fp8(e)
    assert q.shape == (2, 3, 0) and s.shape == (2, 3, 0)
    q, s = fp8.quantize_fp8(e, transpose=True)
    assert q.shape == (0, 6) and s.shape == (0, 1)
    q, s, qt, st = fp8.quantize_fp8_both(e)
    assert q.shape == (2, 3, 0) and s.shape == (2, 3, 0) and qt.shape == (0, 6) and st.shape == (0, 1)


# ------------------------------------------------------------------- rounding of fp32 quotients
def test_quantize_fp32_breaks_ties_to_even():
    # m = 7 n and v = (2 j + 1) n 2^e with odd n of 18 bits: 448 v / m = (2 j + 1) 2^(e + 6) lies on a
    # border for j = 8 .. 15, and 0.875 v has up to 26 bits
    g = gen(85)
    n = torch.randint(1 << 17, 1 << 18, (500, 1), generator=g, device="cuda") | 1
    j = torch.randint(8, 16, (500, 128), generator=g, device="cuda")
    sign = torch.randint(0, 2, (500, 128), generator=g, device="cuda") * 2.0 - 1
    e = torch.randint(-7, -2, (500, 128), generator=g, device="cuda")
    x = sign.double() * (2 * j + 1) * n * torch.tensor([2.0 ** k for k in range(-7, -2)], dtype=torch.float64, device="cuda")[e + 7]
    x[:, 0] = 7.0 * n[:, 0]
    assert torch.equal(x, x.float().double()) and (x.abs() <= 7 * n).all()
    x = x.float()
    t, m = R.quotients(x, False)
    assert (R.tie_distance(t)[:, 1:] == 0).float().mean() > 0.9
    for q, s in (fp8.quantize_fp8(x), fp8.quantize_fp8(x[:, :127].contiguous()), fp8.quantize_fp8_both(x)[:2]):
        check_codes(q, t[:, : q.shape[1]], 0)
    q, s = fp8.quantize_fp8(x.t().contiguous(), transpose=True)
    check_codes(q, t, 0)
    q, s = fp8.quantize_fp8_both(x.t().contiguous())[2:]
    check_codes(q, t, 0)
    one = x[:1].expand(128, 128).contiguous()
    for q, s in (fp8.quantize_fp8(one, square=True), fp8.quantize_fp8(one.t().contiguous(), square=True, transpose=True)):
        check_codes(q, t[:1].expand(128, 128), 0)


@pytest.mark.parametrize("rows,cols", [(1000, 1024), (257, 1001), (5, 130)])
def test_quantize_fp32_beside_borders(rows, cols):
    # values a few units in the last place around the borders of their groups.  The quotient is within
    # 0.65 of a unit in the last place, at most 2^-23 of the value: neighbours that far from a border only
    g = gen(rows + cols)
    x = randn((rows, cols), g)
    m = R.quotients(x, False)[1].repeat_interleave(128, 1)[:, :cols]
    code = torch.randint(16, 127, (rows, cols), generator=g, device="cuda", dtype=torch.uint8).view(fp8.CODES).double()
    up = torch.ldexp(torch.ones_like(code), torch.frexp(code)[1] - 5)    # half a step
    near = ((code + up) * m / 448).float()
    near = (near.view(torch.int32) + torch.randint(-3, 4, (rows, cols), generator=g, device="cuda", dtype=torch.int32)).view(F32)
    x = torch.where((near < m) & (torch.rand((rows, cols), generator=g, device="cuda") < 0.9) & (x.abs() < m), near, x)
    t, m = R.quotients(x, False)
    assert (R.tie_distance(t) <= 2.0 ** -21).float().mean() > 0.5
    for v, kw in ((x, {}), (x.t().contiguous(), {"transpose": True})):
        q, s = fp8.quantize_fp8(v, **kw)
        close(s, m / 448, 2.0 ** -23)
        check_codes(q, t, 0.65 * 2.0 ** -23)


# ------------------------------------------------------------------- layouts of the product
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("M,N,K", [(1, 77, 530), (2, 77, 530), (1, 131, 8191), (2, 9, 12345), (1, 1, 17), (2, 257, 128),
                                   (3, 77, 530), (130, 200, 300), (2000, 1024, 256)])
def test_linear_layouts_and_neighbours(M, N, K, square):
    # both operands inside wider rows whose other bytes are NaN codes, scales in either order inside a
    # wider buffer of NaN, y at odd addresses inside a buffer that stays as it was
    g = gen(M + N + K)
    lib = A.load_library()
    xq, xs, wq, ws = operands(M, N, K, square, g)
    bias = randn((N,), g)

    def wide(q):
        buf = torch.full((q.shape[0] + 1, (K + 15) // 16 * 16 + 48), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:-1, 16:16 + K] = q.contiguous().view(torch.uint8)
        return buf.view(fp8.CODES)[:-1, 16:16 + K]

    def spread(s, by_group):
        r, c = s.shape
        buf = torch.full((c + 2, r + 3) if by_group else (r + 3, c + 2), float("nan"), device="cuda")
        view = buf[1:-1, 1:-2].t() if by_group else buf[1:-2, 1:-1]
        view.copy_(s)
        return view

    for dtype, dt in ((BF16, 0), (F32, 1)):
        want = fp8.fp8_linear(xq, xs, wq, ws, bias, out_dtype=dtype)
        check_linear(want, xq, xs, wq, ws, bias)
        for by_group in (False, True):
            xw, ww, sx, sw = wide(xq), wide(wq), spread(xs, by_group), spread(ws, by_group)
            assert torch.equal(want, fp8.fp8_linear(xw, sx, ww, sw, bias, out_dtype=dtype))
            for off, ld in ((0, N + 8), (1, N + 3)):
                buf = torch.full(((M + 1) * ld + 1,), 9.0, dtype=dtype, device="cuda")
                rc = lib.evo_fp8_linear(M, N, K, xw.data_ptr(), xw.stride(0), sx.data_ptr(), sx.stride(0), sx.stride(1),
                                        ww.data_ptr(), ww.stride(0), sw.data_ptr(), sw.stride(0), sw.stride(1),
                                        int(not square), A._ptr(bias), dt, buf.data_ptr() + off * buf.element_size(), ld,
                                        None, 0, A._stream(buf.device))
                assert rc == 0
                y = torch.as_strided(buf, (M, N), (ld, 1), off)
                assert torch.equal(y, want)
                y.fill_(9.0)
                assert (buf == 9.0).all()


# ------------------------------------------------------------------- long axes
def test_weight_gradient_over_131072_rows():
    # quantised along the rows and summed over them: 1024 x 131072 x 256, as for 512 x 256 rows of an MSA
    g = gen(86)
    dy, n = stream_rows(131072, 1024, g, BF16), stream_rows(131072, 256, g, BF16)
    dq, ds = fp8.quantize_fp8(dy, transpose=True)
    nq, ns = fp8.quantize_fp8(n, transpose=True)
    for q, s, v in ((dq, ds, dy), (nq, ns, n)):
        for c0 in range(0, v.shape[1], 256):             # the reference in parts, for its memory
            part = v[:, c0:c0 + 256].t()
            t, m = R.quotients(part, False)
            check_codes(q[c0:c0 + 256], t, 0)
            close(s[c0:c0 + 256], m / 448, 2.0 ** -23)
    dw = fp8.fp8_linear(dq, ds, nq, ns, out_dtype=F32)
    for r0 in range(0, 1024, 256):
        check_linear(dw[r0:r0 + 256], dq[r0:r0 + 256], ds[r0:r0 + 256], nq, ns, None)


def test_projection_of_131072_outputs():
    g = gen(87)
    xq, xs, wq, ws = operands(5, 131072, 140, True, g)
    check_linear(fp8.fp8_linear(xq, xs, wq, ws), xq, xs, wq, ws, None)
    xq, xs = xq[:1], xs[:1]
    check_linear(fp8.fp8_linear(xq, xs, wq, ws), xq, xs, wq, ws, None)


# ------------------------------------------------------------------- gradients through projection and attention
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_through_norm_projection_and_attention(dtype):
    """The stream's norm, q/k/v/g in 8 bits, and the attention on views of that output, as one graph."""
    B, S, N, H, C, D = 1, 3, 24, 2, 32, 96
    g = gen(88)
    x, res = (randn((B, S, N, D), g, dtype).requires_grad_(True) for _ in range(2))
    gamma = (1 + 0.2 * randn((D,), g)).to(dtype).requires_grad_(True)
    w = (randn((4 * H * C, D), g) / D ** 0.5).to(dtype).requires_grad_(True)
    pb = randn((B, 1, H, N, N), g, dtype).requires_grad_(True)
    dout, dh = randn((B, S, N, H, C), g, dtype), randn((B, S, N, D), g, dtype)
    h, y = fp8.add_rms_norm_linear(x, res, gamma, 1e-5, w)
    out = A.evoformer_attention(*A.qkvg_views(y, H), None, pb)
    got = torch.autograd.grad((h, out), (y, x, res, gamma, w, pb), (dh, dout))
    # the attention's part from its formula in 64 bits, from the same y
    y64 = y.detach().double().requires_grad_(True)
    pb64 = pb.detach().double().requires_grad_(True)
    q, k, v, gate = A.qkvg_views(y64, H)
    scores = torch.einsum("bsihc,bsjhc->bshij", q, k) / C ** 0.5 + pb64
    o64 = torch.einsum("bshij,bsjhc->bsihc", scores.softmax(-1), v) * gate.sigmoid()
    dy64, dpb64 = torch.autograd.grad(o64, (y64, pb64), dout.double())
    rel = lambda a, b: float((a.detach().double() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    tol = 5e-3 if dtype == BF16 else 1e-4                # the attention's own tests' bounds
    assert rel(out, o64) <= tol and rel(got[0], dy64) <= tol and rel(got[-1], dpb64) <= tol
    # and from there the projection and the norm, from y's gradient as computed
    dy = got[0].reshape(-1, 4 * H * C)
    flat = lambda t: t.detach().reshape(-1, D)  # noqa: E731
    rh, rrstd, rn = R.norm(flat(x), flat(res), gamma.detach(), 1e-5)
    dn = (R.values(*R.quantize(dy), False) @ R.values(*R.quantize(w.detach(), True), True)).to(dtype)
    rdx, rdg = R.norm_bwd(dn, flat(dh), rh, rrstd, gamma.detach())
    rdw = R.values(*R.quantize(dy.t()), False) @ R.values(*R.quantize(rn.to(dtype).t()), False).t()
    tol = 2.0 ** -8 if dtype == BF16 else 1e-3
    for a, b in zip(got[1:5], (rdx, rdx, rdg, rdw)):
        assert rel(a.reshape(b.shape), b) <= tol
