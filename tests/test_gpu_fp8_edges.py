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
