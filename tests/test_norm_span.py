"""dsa_norm_q8 where values span more than fp32 does with their squares, their products with gamma, or a block's scale."""
import numpy as np
import pytest
import torch

from _parity import np64
from test_projections import check_norm, gen, randn, run_norm

pytestmark = pytest.mark.gpu

DIMS = [144, 512, 1040, 4096, 16384]   # a warp's rows, a CTA's, the widest


def small_block_beside(dim, big, small):
    """Rows with one value `big`, zeros, and a last block of `small`."""
    x = torch.zeros((3, dim), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = big
    x[:, (dim - 1) // 128 * 128:] = small
    x[2] = 1.0
    return x


@pytest.mark.parametrize("dim", DIMS)
def test_no_scale_below_its_least(dim):
    """One value of 1.0625 2^63 beside a block of 1.5 2^-60: its largest norm / 448 is 2^-127.7 at a width of 144, the scale 2^-126."""
    x = small_block_beside(dim, 1.0625 * 2.0 ** 63, 1.5 * 2.0 ** -60)
    out, scale, total = run_norm(x, None, None)
    check_norm(x, None, None, out, scale, total)
    assert (scale >= 2.0 ** -126).all()
    if dim == 144:
        assert (scale[:2, -1] == 2.0 ** -126).all()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("big,small", [(2.0 ** 66, 1.1875 * 2.0 ** -57), (-3.0e38, 1.7 * 2.0 ** -12), (2.0 ** 126, 2.0 ** 9)])
def test_small_values_beside_ones_whose_squares_overflow(dim, big, small):
    """The small block's values and scale keep their bits."""
    x = small_block_beside(dim, big, small)
    x[1, -7:] *= -0.8125
    r = torch.zeros_like(x)
    for residual in (None, r):
        check_norm(x, residual, None, *run_norm(x, residual, None))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("size,weight,eps", [(2.0 ** 62, 2.0 ** 70, 1e-6), (2.0 ** 50, 2.0 ** 80, 1e-6), (2.0 ** -55, 2.0 ** -75, 2.0 ** -118), (2.0 ** 100, 2.0 ** 90, 1e-6),
                                             (2.0 ** 100, 2.0 ** -90, 1e-6), (2.0 ** 15, 2.0 ** 90, 1e-6), (2.0 ** -15, 2.0 ** -90, 2.0 ** -60)])
def test_gamma_times_a_value_beyond_fp32(dim, size, weight, eps):
    """gamma * h may leave fp32 at either end where gamma times the norm does not."""
    g = gen(dim)
    x = (randn(g, 5, dim) * size).to(torch.bfloat16)
    gamma = (1 + 0.2 * randn(g, dim)) * weight
    out, scale, total = run_norm(x, None, gamma, eps=eps)
    assert np.isfinite(np64(scale)).all()
    check_norm(x, None, gamma, out, scale, total, eps=eps)
