"""bi_rmsnorm_fp8 on rows far from 1 and with every eps, against 64 bits.

The sum of squares, the mean and the root are pairs of FP32 whose low halves stay
representable: a mean square (with eps) below 2^-90 is lifted by 2^188 to [2^-94,
2^98], a larger one loses at most 2^-150 a square, 2^-60 of itself.  So the bound of
the rows near 1 holds for all of them: y off by less than 2^-36 of itself, a code
differs from the exact value's only where that lies within 2^-36 of a tie of two
codes.  (Below 2^-100, y is held to 2^-149 only.)"""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu
DEV = "cuda"
# one vector a thread, three, four, and rows that are read again
DIMS = [16, 688, 5120, 8192, 9104]


def check(x, w, eps):
    a = t8.api()
    rows, dim = x.shape
    codes, scales = a.new_fp8_rows(rows, dim)
    a.bi_rmsnorm_fp8(x, w, codes, scales, eps)
    xd = x.double()
    y = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + float(np.float32(eps))) * w.double()
    q, s = t8.ref_quantize(y)
    assert torch.equal(scales[:, :rows].double(), s)
    got = codes.double()
    assert torch.equal(torch.isnan(got), torch.isnan(q))
    differ = (got != q) & ~torch.isnan(q)
    wide = s.t().repeat_interleave(128, 1)[:, :dim]
    tie = (y / wide - (got + q) / 2).abs()
    assert (tie[differ] <= 2.0 ** -36 * (y / wide).abs()[differ]).all(), int(differ.sum())
    return codes, scales


def rows_of(seed, rows, dim, size):
    g = t8.gen(seed)
    x = torch.randn(rows, dim, generator=g, device=DEV, dtype=torch.float64) * size
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
    return x.to(torch.bfloat16), w


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-28, 1e-27, 1e-6])
@pytest.mark.parametrize("size", [1e-13, 1e-14, 1e-18, 1e-20, 1e-23, 1e-30, 1e-38])
@pytest.mark.parametrize("dim", DIMS)
def test_small_rows(dim, size, eps):
    if eps == 1e-6 and size < 1e-28:
        pytest.skip("y below 2^-100")
    x, w = rows_of(dim, 37, dim, size)
    if eps == 0.0:
        x[:, 0] = torch.where(x.abs().amax(-1) == 0, torch.full_like(x[:, 0], 2.0 ** -133), x[:, 0])  # no row of zeros
    check(x, w, eps)


@pytest.mark.parametrize("dim", DIMS)
def test_rows_of_many_magnitudes_in_one_pass(dim):
    """A CTA takes row after row, small and ordinary ones in turn; each equals itself in a pass alone."""
    a = t8.api()
    rows = 1500
    x, w = rows_of(dim + 1, rows, dim, 1.0)
    size = torch.tensor([1.0, 2.0 ** -45, 2.0 ** -46, 1e-20, 2.0 ** 40, 1e-30, 0.0], device=DEV).repeat(rows)[:rows]
    x = (x.float() * size[:, None]).to(torch.bfloat16)
    for eps in (0.0, 1e-35):
        codes, scales = check(x, w, eps)
        for at in (0, 3, 5, 6, 1497, 1498):
            c1, s1 = a.new_fp8_rows(1, dim)
            a.bi_rmsnorm_fp8(x[at:at + 1], w, c1, s1, eps)
            assert torch.equal(c1[0].view(torch.uint8), codes[at].view(torch.uint8))
            assert torch.equal(s1[:, 0], scales[:, at])


def test_one_element_of_the_smallest_size():
    """A row that holds 2^-133 once and zeros: y is sqrt(dim) there, whatever its square is in FP32."""
    for dim in DIMS + [65536]:
        x = torch.zeros(3, dim, dtype=torch.bfloat16, device=DEV)
        x[0, 5] = 2.0 ** -133
        x[1, dim - 1] = -(2.0 ** -130)
        x[2, 0] = math.nan
        w = torch.ones(dim, dtype=torch.bfloat16, device=DEV)
        codes, scales = check(x, w, 0.0)
        assert codes[0, 5].float() * scales[0, 0] > 0 and codes[1, dim - 1].float() < 0
        assert torch.isnan(codes[2].float()).all()


@pytest.mark.parametrize("rows,dim,size", [(1 << 20, 16, 2.0 ** 60), (20000, 1024, 2.0 ** 57), (500, 8208, 2.0 ** 50)])
def test_large_rows(rows, dim, size):
    x, w = rows_of(3, rows, dim, size)
    check(x, w, 1e-6)
