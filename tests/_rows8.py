"""Checks of 8-bit rows (e4m3 codes with a scale per block) against float64 values.

A code is a rounding of value / scale: off by at most half a step of e4m3's grid there (2^-4 of the value in the normal range,
2^-10 below 2^-6), and by what the kernel's fp32 value was off before the rounding."""
import numpy as np

from oracle.codecs import e4m3_decode
from oracle.projection import blocks_of, per_value


def half_step(q):
    """Half the distance between neighbouring e4m3 values around |q|."""
    e = np.maximum(np.frexp(np.abs(q))[1] - 1, -6)
    return np.ldexp(1.0, e - 4)


def block_max(v):
    n = v.shape[-1]
    return np.stack([np.max(v[..., b * 128:(b + 1) * 128], axis=-1) for b in range(blocks_of(n))], axis=-1)


def assert_rows8(codes, scale, want, off):
    """codes [..., n], scale [..., blocks] are the 8-bit rows of values that differ from `want` by at most `off`."""
    n = want.shape[-1]
    scale = scale.astype(np.float64)
    amax = block_max(np.abs(want))
    near = block_max(off * np.ones_like(want)) / 448 + 2.0 ** -23 * amax / 448
    ideal = np.where(amax > 0, np.maximum(amax / 448, 2.0 ** -126), 1.0)
    bad = np.abs(scale - ideal) > near
    bad &= ~((amax <= block_max(off * np.ones_like(want))) & (scale == 1.0))
    assert not bad.any(), ("scale", np.argwhere(bad)[:4], scale[bad][:4], ideal[bad][:4])
    s = per_value(scale, n)
    q = np.clip(want / s, -448, 448)
    err = np.abs(e4m3_decode(codes) - q)
    room = half_step(q) + off / s + 2.0 ** -22 * np.abs(q)
    worst = np.unravel_index(np.argmax(err - room), err.shape)
    assert (err <= room).all(), ("code", worst, err[worst], room[worst], want[worst])
