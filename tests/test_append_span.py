"""dsa_cache_append with the norm where values span more than fp32 does with their squares or their products with gamma."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from oracle import projection as OP
from oracle.codecs import e4m3_decode
from _parity import np64
from _rows8 import half_step
from test_projections import BF16, EPS, NORM_OFF, gen, ints, make_pool, physical, randn, schedule, tables

pytestmark = pytest.mark.gpu

FORMS = [("fp8", 512), ("bf16", 512), ("fp8", 128), ("bf16", 64)]


def check(x, gamma, fmt, eps=EPS):
    n, dim = x.shape
    cu, req, pos = schedule([250], [n])
    bt, blocks = tables([250], [n], gen(1))
    pool, data, scale = make_pool(blocks, dim, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_append(ints(cu), ints([250]), x, dsa.rope(64), pool, dsa.block_table(bt), norm=True, rms_gamma=gamma, rms_eps=eps,
                         dev_status=status)
    assert int(status) == 0
    want = OP.append_rows(np64(x), pos, 1.0 if gamma is None else np64(gamma), eps, True, 64)
    off = NORM_OFF * np.abs(want)
    tail = want[:, dim - 64:]
    off[:, dim - 64:] = (1e-6 + NORM_OFF) * np.repeat(np.hypot(tail[:, 0::2], tail[:, 1::2]), 2, axis=1)
    rows = physical(bt, req, pos)
    if fmt == "bf16":   # below 2^-126 the steps no longer shrink with the value: half of bf16's is 2^-134, of fp32's 2^-150, a few times
        tiny = np.where(np.abs(want) < 2.0 ** -125, 2.0 ** -134 + 2.0 ** -146, 0)
        err = np.abs(np64(data[rows]) - want) - (BF16 * np.abs(want) + off * (1 + BF16) + tiny)
        worst = np.unravel_index(np.argmax(err), err.shape)
        assert err[worst] <= 0, (worst, err[worst], want[worst])
        return
    s = np64(scale[rows])[:, None]
    ideal = np.max(np.abs(want), axis=1, keepdims=True) / 448
    assert (np.abs(s - ideal) <= np.max(off, axis=1, keepdims=True) / 448 + 2.0 ** -23 * ideal).all(), (s, ideal)
    q = np.clip(want / s, -448, 448)
    err = np.abs(e4m3_decode(data[rows].cpu().numpy()) - q) - (half_step(q) + off / s + 2.0 ** -22 * np.abs(q))
    worst = np.unravel_index(np.argmax(err), err.shape)
    assert err[worst] <= 0, (worst, err[worst], want[worst])


@pytest.mark.parametrize("fmt,dim", FORMS)
@pytest.mark.parametrize("size,weight,eps", [(2.0 ** 50, 2.0 ** 80, EPS), (2.0 ** -50, 2.0 ** -85, 2.0 ** -118), (2.0 ** 100, 2.0 ** 90, EPS),
                                             (2.0 ** 100, 2.0 ** -90, EPS), (2.0 ** 15, 2.0 ** 90, EPS), (2.0 ** -15, 2.0 ** -105, 2.0 ** -60)])
def test_gamma_times_a_value_beyond_fp32(fmt, dim, size, weight, eps):
    g = gen(dim)
    check((randn(g, 5, dim) * size).to(torch.bfloat16), (1 + 0.2 * randn(g, dim)) * weight, fmt, eps)


@pytest.mark.parametrize("fmt,dim", FORMS)
@pytest.mark.parametrize("big,small", [(2.0 ** 66, 1.6171875 * 2.0 ** -64), (2.0 ** 66, 1.6171875 * 2.0 ** -40), (-3.0e38, 1.7 * 2.0 ** -12)])
def test_small_values_beside_ones_whose_squares_overflow(fmt, dim, big, small):
    """Values of a row whose largest ones' squares leave fp32 keep their bits."""
    x = torch.full((4, dim), small, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = big
    x[1, 1::2] *= -0.75
    x[2, ::3] = 0
    x[3] = 1.0
    check(x, None, fmt)
