"""Host-side checks of the 8-bit operators, and their 64-bit reference: no GPU needed."""
import ctypes

import pytest
import torch

import _fp8 as R
from evoformer_pair_bias_b200 import attention as A
from evoformer_pair_bias_b200 import build as B
from evoformer_pair_bias_b200 import fp8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.load_library()


FAKE, ODD, ODD4, NUL = (ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 4), None)


def test_reference_rounding_is_torchs_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = torch.unique(codes[~codes.isnan()])
    assert torch.equal(R.e4m3(codes), codes)
    mid = (codes[1:] + codes[:-1]) / 2
    for v in (mid, mid * (1 + 2.0 ** -12), mid * (1 - 2.0 ** -12)):
        assert torch.equal(R.e4m3(v), v.float().to(torch.float8_e4m3fn).double())


def test_reference_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    x, w, dy = (torch.randn((4, 50), generator=g, dtype=torch.float64) for _ in range(3))
    w = w[0]
    rstd = R.norm(x, None, w, 1e-3)[1]
    dx, dw = R.norm_bwd(dy, None, x, rstd, w)
    loss = lambda a, b: (dy * R.norm(a, None, b, 1e-3)[2]).sum()  # noqa: E731
    for _ in range(3):
        vx, vw = torch.randn((4, 50), generator=g, dtype=torch.float64), torch.randn(50, generator=g, dtype=torch.float64)
        d = (loss(x + 1e-5 * vx, w + 1e-5 * vw) - loss(x - 1e-5 * vx, w - 1e-5 * vw)) / 2e-5
        assert abs(float(d - (dx * vx).sum() - (dw * vw).sum())) < 1e-6


def test_quantize_refusals(lib):
    f = lib.evo_quantize_fp8
    assert f(0, 8, 0, NUL, 8, 0, 0, NUL, 16, NUL, 1, 1, NUL) == 0                 # empty
    assert f(8, 0, 0, NUL, 8, 0, 0, NUL, 16, NUL, 1, 1, NUL) == 0
    assert f(-1, 8, 0, FAKE, 8, 0, 0, FAKE, 16, FAKE, 1, 1, NUL) == 1
    assert f(8, 8, 2, FAKE, 8, 0, 0, FAKE, 16, FAKE, 1, 1, NUL) == 1              # unknown type
    assert f(8, 8, 0, NUL, 8, 0, 0, FAKE, 16, FAKE, 1, 1, NUL) == 1               # null
    assert f(8, 8, 0, FAKE, 8, 0, 0, FAKE, 16, FAKE, 0, 1, NUL) == 1              # scale stride
    assert f(8, 32, 0, FAKE, 32, 0, 0, FAKE, 16, FAKE, 1, 8, NUL) == 1            # ldq < cols
    assert f(8, 8, 0, FAKE, 8, 0, 0, FAKE, 24, FAKE, 1, 8, NUL) == 2              # ldq % 16
    assert f(8, 8, 0, FAKE, 8, 0, 0, ODD4, 16, FAKE, 1, 8, NUL) == 2              # q alignment
    assert f(8, 8, 1, ODD, 8, 0, 0, FAKE, 16, FAKE, 1, 8, NUL) == 1               # fp32 alignment
    assert f(1 << 40, 1 << 20, 0, FAKE, 1 << 20, 1, 0, FAKE, 1 << 20, FAKE, 1, 8, NUL) == 2   # more blocks than a grid


def test_quantize_both_refusals(lib):
    def f(rows=8, cols=8, dtype=0, x=FAKE, ldx=8, q=FAKE, ldq=16, s=FAKE, sr=1, qt=FAKE, ldqt=16, st=FAKE, stg=8):
        return lib.evo_quantize_fp8_both(rows, cols, dtype, x, ldx, 0, q, ldq, s, sr, 8, qt, ldqt, st, 1, stg, NUL)
    assert f(rows=0, x=NUL, q=NUL) == 0 and f(cols=0, x=NUL, qt=NUL) == 0
    assert f(rows=-1) == 1 and f(dtype=4) == 1 and f(x=NUL) == 1 and f(ldx=-8) == 1
    assert f(q=NUL) == 1 and f(qt=NUL) == 1 and f(s=NUL) == 1 and f(st=NUL) == 1 and f(sr=0) == 1 and f(stg=0) == 1
    assert f(cols=32, ldx=32, ldq=16) == 1 and f(rows=32, ldqt=16) == 1
    assert f(ldq=24) == 2 and f(ldqt=24) == 2 and f(q=ODD4) == 2 and f(qt=ODD4) == 2


def test_norm_refusals(lib):
    def f(rows=8, cols=64, dtype=0, x=FAKE, ldx=64, res=NUL, ldr=0, w=NUL, wd=0, eps=1e-5, q=FAKE, ldq=64, s=FAKE, sr=1,
          sg=8, h=NUL, ldh=0, n=NUL, ldn=0, rstd=NUL):
        return lib.evo_add_rms_norm_fp8(rows, cols, dtype, x, ldx, res, ldr, w, wd, eps, q, ldq, s, sr, sg, h, ldh, n,
                                        ldn, rstd, NUL)
    assert f(rows=0, x=NUL, q=NUL, s=NUL) == 0
    assert f(rows=-1) == 1 and f(cols=0) == 1 and f(dtype=5) == 1 and f(wd=5) == 1
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(x=NUL) == 1 and f(q=NUL) == 1 and f(s=NUL) == 1
    assert f(ldq=48) == 1 and f(h=FAKE, ldh=32) == 1 and f(n=FAKE, ldn=32) == 1 and f(ldx=-1) == 1
    assert f(cols=32769, ldq=32784) == 2 and f(ldq=72) == 2 and f(q=ODD4) == 2
    assert f(dtype=1, x=ODD) == 1 and f(w=ODD, wd=1) == 1 and f(s=ODD) == 1 and f(rstd=ODD) == 1


def test_norm_bwd_refusals_and_workspace(lib):
    def f(rows=8, cols=64, dtype=0, dy=FAKE, dh=NUL, h=FAKE, rstd=FAKE, w=NUL, wd=0, dx=FAKE, lddx=64, dw=NUL, ws=NUL,
          nb=0, dwd=1):
        return lib.evo_add_rms_norm_bwd(rows, cols, dtype, dy, 64, dh, 64, h, 64, rstd, w, wd, dx, lddx, dw, dwd, ws, nb,
                                        NUL)
    assert f(rows=0, dy=NUL, h=NUL, rstd=NUL, dx=NUL) == 0
    assert f(rows=-1) == 1 and f(cols=0) == 1 and f(dtype=2) == 1 and f(wd=2) == 1
    assert f(dwd=9) == 1 and f(dw=ODD, ws=FAKE, nb=1 << 30) == 1
    assert f(dy=NUL) == 1 and f(h=NUL) == 1 and f(rstd=NUL) == 1 and f(dx=NUL) == 1 and f(lddx=8) == 1
    assert f(cols=40000, lddx=40000) == 2
    assert f(dw=FAKE) == 3 and f(dw=FAKE, ws=FAKE, nb=255) == 3
    need = lib.evo_add_rms_norm_bwd_workspace_bytes
    assert need(8, 64) >= 256 and need(0, 64) == 0 and need(8, 0) == 0 and need(8, 40000) == 0
    assert need(1 << 30, 256) == need(1 << 20, 256)                               # bounded by the grid
    assert f(dw=FAKE, ws=ODD4, nb=1 << 30) == 1                                   # workspace alignment


def test_linear_refusals(lib):
    def f(M=8, N=8, K=64, x=FAKE, ldx=64, xs=FAKE, w=FAKE, ldw=64, ws=FAKE, bias=NUL, yd=0, y=FAKE, ldy=8, sxr=1,
          work=NUL, nb=0):
        return lib.evo_fp8_linear(M, N, K, x, ldx, xs, sxr, 8, w, ldw, ws, 1, 1, 0, bias, yd, y, ldy, work, nb, NUL)
    assert f(M=0, x=NUL, y=NUL) == 0 and f(N=0, w=NUL) == 0
    assert f(M=-1) == 1 and f(K=0) == 1 and f(yd=3) == 1
    assert f(x=NUL) == 1 and f(xs=NUL) == 1 and f(w=NUL) == 1 and f(ws=NUL) == 1 and f(y=NUL) == 1
    assert f(ldx=48) == 1 and f(ldw=48) == 1 and f(ldy=4) == 1 and f(sxr=-1) == 1
    assert f(ldx=72) == 2 and f(ldw=72) == 2 and f(x=ODD4) == 2 and f(w=ODD4) == 2
    assert f(M=1 << 31) == 2 and f(N=1 << 31, ldy=1 << 31) == 2 and f(K=1 << 31, ldx=1 << 31, ldw=1 << 31) == 2
    assert f(xs=ODD) == 1 and f(bias=ODD) == 1 and f(yd=1, y=ODD) == 1
    need = lib.evo_fp8_linear_workspace_bytes
    assert need(0, 8, 8) == 0 and need(8, 8, 0) == 0 and need(8, 8, 1 << 40) == 0 and need(8, 8, 64) == 0
    assert need(131072, 1024, 256) == 0 and need(8192, 8192, 1 << 20) == 0        # tiles enough
    big = need(1024, 256, 131072)                                                  # few tiles, a long sum: parts
    assert 0 < big <= 64 << 20 and big == need(1024, 256, 131072)
    long = dict(M=1024, N=256, K=131072, ldx=131072, ldw=131072, ldy=256)
    assert f(**long) == 3 and f(work=FAKE, nb=big - 1, **long) == 3
    assert f(work=ctypes.c_void_p((1 << 20) + 16), nb=big, **long) == 1
    for M, N, K in ((1, 8192, 8192), (3, 77, 1 << 20), (129, 257, 70001), (1, 1, 1 << 30)):
        assert need(M, N, K) <= 148 * 128 * 256 * 4 + (1 << 22)                   # bounded by the GPU, not by K


def test_linear_bwd_refusals_and_workspace(lib):
    need = lib.evo_fp8_linear_bwd_workspace_bytes
    assert need(0, 8, 8, 1, 1) == 0 and need(8, 0, 8, 1, 1) == 0 and need(8, 8, 0, 1, 1) == 0
    assert need(300, 64, 128, 1, 0) < need(300, 64, 128, 1, 1) and need(300, 64, 128, 0, 1) < need(300, 64, 128, 1, 1)

    def f(M=8, N=8, K=64, dt=0, dy=FAKE, lddy=8, x=FAKE, ldx=64, w=FAKE, ldw=16, ws=FAKE, wr=1, dx=FAKE, lddx=64, dw=FAKE,
          dwd=1, lddw=64, work=FAKE, nb=1 << 30):
        return lib.evo_fp8_linear_bwd(M, N, K, dt, dy, lddy, x, ldx, w, ldw, ws, wr, 1, dx, lddx, dw, dwd, lddw, work, nb,
                                      NUL)
    assert f(N=0, dy=NUL) == 0 and f(dx=NUL, dw=NUL, dy=NUL) == 0 and f(M=0, dw=NUL, dy=NUL) == 0
    assert f(M=-1) == 1 and f(K=0) == 1 and f(dt=3) == 1 and f(dwd=3) == 1 and f(lddw=8) == 1 and f(lddx=8) == 1
    assert f(dy=NUL) == 1 and f(x=NUL) == 1 and f(w=NUL) == 1 and f(ws=NUL) == 1 and f(wr=-1) == 1 and f(ldx=-1) == 1
    assert f(dt=1, dx=ODD) == 1 and f(dw=ODD) == 1 and f(dt=1, dy=ODD) == 1 and f(dt=1, x=ODD) == 1
    assert f(ldw=24) == 2 and f(w=ODD4) == 2 and f(M=1 << 31) == 2
    assert f(nb=100) == 3 and f(work=NUL) == 3 and f(work=ODD4) == 1


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.quantize_fp8(x)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.add_rms_norm_fp8(x, x)
    c = torch.zeros((4, 64), dtype=torch.uint8).view(fp8.CODES)
    with pytest.raises(ValueError, match="codes"):
        fp8._codes(x, "xq")
    assert fp8._codes(c, "xq") == (4, 64, c.data_ptr(), 64)
    with pytest.raises(ValueError, match="multiples of 16"):
        fp8._codes(torch.zeros((4, 60), dtype=torch.uint8).view(fp8.CODES), "xq")
    with pytest.raises(ValueError, match="contiguous"):
        fp8._codes(c.t(), "xq")
    with pytest.raises(ValueError, match="fold"):
        fp8._codes(torch.zeros((4, 3, 64), dtype=torch.uint8).view(fp8.CODES).transpose(0, 1), "xq")
    with pytest.raises(ValueError, match="weight"):
        fp8._weight(torch.zeros(63), 64)
    with pytest.raises(ValueError, match="weight"):
        fp8._weight(torch.zeros(64, dtype=torch.float16), 64)
    with pytest.raises(ValueError, match=r"w must be"):
        fp8._training_weight(x, torch.zeros((8, 63)))
    assert fp8.empty_codes(5, 33, "cpu").stride() == (48, 1) and fp8.empty_scales(5, 2, "cpu").stride() == (1, 5)


def test_rows_folds_leading_axes_without_a_copy_where_it_can():
    x = torch.zeros((2, 3, 4, 8))
    r, c, v, ld = fp8._rows(x)
    assert (r, c, ld) == (24, 8, 8) and v.data_ptr() == x.data_ptr()
    r, c, v, ld = fp8._rows(x[..., 2:6])
    assert (r, c, ld) == (24, 4, 8) and v.data_ptr() == x.data_ptr() + 8
    r, c, v, ld = fp8._rows(x.transpose(0, 3))               # no contiguous last axis: copied
    assert (r, c, ld) == (8 * 3 * 4, 2, 2) and v.stride(1) == 1
    assert fp8._rows(torch.zeros(0, 8))[0] == 0 and fp8._rows(torch.zeros(8))[0] == 1
