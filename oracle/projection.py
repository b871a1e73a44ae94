"""Norm, projections and appended rows around the attention (oracle; test infrastructure only).

[P2] "DeepSeek V4 稀疏注意力完全解剖", 融合点 1 (RMSNorm), 融合点 2 (rows in fp8 for the products around the attention),
融合点 3 (keys rotated, then inserted).  8-bit rows: e4m3 codes with one scale per 128 consecutive values, scale =
max |v| / 448 (1 for zeros, at least 2^-126); the last block of a row may be shorter.

Everything in float64; the rounding to codes is left to the caller (codes decide an integer from a float, so a test
compares the kernel's code with the unrounded quotient).
"""
import numpy as np

from .codecs import e4m3_decode
from .rope import rope

BLOCK = 128


def blocks_of(n):
    return -(-n // BLOCK)


def block_scales(v):
    """Scales [..., blocks] of rows v [..., n]."""
    n = v.shape[-1]
    out = np.ones((*v.shape[:-1], blocks_of(n)))
    for b in range(blocks_of(n)):
        amax = np.max(np.abs(v[..., b * BLOCK:(b + 1) * BLOCK]), axis=-1)
        out[..., b] = np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 1.0)
    return out


def per_value(scales, n):
    """Block scales as one for each of n values."""
    return np.repeat(scales, BLOCK, axis=-1)[..., :n]


def rms_norm(h, gamma, eps):
    """gamma * h / sqrt(mean(h^2) + eps) over the last axis."""
    return (1.0 if gamma is None else gamma) * h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)


def gemm(a, a_scale, w, w_scale):
    """(out, size) of codes a [m][g][k], w [g][n][k] with their block scales: the products' sums, and the sums of the
    products' magnitudes (what an error bound of a sum goes by)."""
    m, groups, k = a.shape
    n = w.shape[1]
    out, size = np.empty((m, groups, n)), np.empty((m, groups, n))
    for g in range(groups):
        av = e4m3_decode(a[:, g]) * per_value(a_scale[:, g].astype(np.float64), k)
        ws = np.repeat(per_value(w_scale[g].astype(np.float64), k), BLOCK, axis=0)[:n]
        wv = e4m3_decode(w[g]) * ws
        out[:, g] = av @ wv.T
        size[:, g] = np.abs(av) @ np.abs(wv).T
    return out, size


def append_rows(x, pos, gamma, eps, norm, rope_dim, theta=10000.0):
    """The values of appended rows: normed where asked, then rotated by their positions."""
    v = rms_norm(x, gamma, eps) if norm else x
    return rope(v, pos, rope_dim, theta) if rope_dim else v
