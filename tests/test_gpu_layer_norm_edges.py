"""Rows of layer norm at the ends of what its types hold, against what the formulas give there."""
import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("rows", [5, 9601])
@pytest.mark.parametrize("cols", [256, 896, 1792, 3584, 1021])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows(rows, cols, dtype):
    """A row of one value whose sums are exact in fp32 has that mean: y is the bias, and dx of one dy is 0.

    1000 * cols and all partial sums are multiples of 1000 below 1000 * 2^24 / 1000, so exact; so are
    multiples of 0.5."""
    x = torch.full((rows, cols), 1000.0, dtype=dtype, device="cuda")
    y, mean, rstd = nsb.muon_layer_norm(x)
    assert (mean == 1000).all() and (y == 0).all()
    assert ((rstd.double() * 1e-5 ** 0.5 - 1).abs() <= 4 * U + 1e-7).all()
    dx, _, _ = nsb.muon_layer_norm_backward(torch.full_like(x, 0.5), x, mean, rstd)
    assert (dx == 0).all()


@pytest.mark.parametrize("cols", [4, 32, 1024])
@pytest.mark.parametrize("power", [-74, -70, -62, 0, 40, 58])
def test_variance_at_the_ends_of_fp32(cols, power):
    """A row of +-2^power in half of its places (a quarter each), no eps: every sum is exact, the variance is
    2^(2 power - 1), down to the smallest number there is."""
    q = cols // 4
    x = torch.zeros(3, cols, device="cuda")
    x[:, :q], x[:, q:2 * q] = 2.0 ** power, -2.0 ** power
    y, mean, rstd = nsb.muon_layer_norm(x, eps=0.0)
    want = 2.0 ** (0.5 - power)
    assert (mean == 0).all()
    assert ((rstd.double() / want - 1).abs() <= 4 * U).all()
    assert ((y.double() - x.double() * want).abs() <= 5 * U * 2 ** 0.5).all()


@pytest.mark.parametrize("rows", [3, 40000])
@pytest.mark.parametrize("cols", [5, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_constant_rows_far_from_zero(rows, cols, dtype):
    """Equal values of 2^120 in a row: mean * rstd has no fp32 number, but no value of the formula needs it.

    The sums are exact (40 * 2^120 is below 2^126), xhat is 0, so dx = rstd (dy - mean(dy))."""
    x = torch.full((rows, cols), 2.0 ** 120, dtype=dtype, device="cuda")
    dy = torch.arange(1, cols + 1, device="cuda").to(dtype).repeat(rows, 1)
    y, mean, rstd = nsb.muon_layer_norm(x)
    assert (mean == 2.0 ** 120).all() and (y == 0).all()
    dx, _, db = nsb.muon_layer_norm_backward(dy, x, mean, rstd, bias=True)
    R = rstd.double()[:, None]
    want = (dy.double() - (cols + 1) / 2) * R
    half = torch.finfo(dtype).eps / 2
    assert ((dx.double() - want).abs() <= (half + 4 * U) * want.abs() + 4 * U * cols * R).all()
    assert (db.double() == dy.double().sum(0)).all()
