"""4-bit cache rows (e2m1 codes, an e4m3 scale per 16 elements, a power-of-two scale per row): the format's definition,
storing rows (dsa_cache_write, dsa_compress), reading them back (dsa_cache_read) and attention over them.

Exactness.  The row scale s is a power of two, so x / s is exact; the block scale has 4 significant bits.  For a bf16
input x (8 significant bits) and a border b between two codes (3 significant bits) the quotient x / (s bs) is either b
itself or differs from it by a relative 2^-16 or more, far above fp32 rounding: the stored bytes equal the oracle's.
A stored value has at most 6 significant bits: reading back as bf16 is exact.

Attention tolerance (element, u = 2^-8 half a bf16 step): with w_j = softmax weights and the fp32 logit error
eps = 2^-14 * sm * sum_d |q_d k_jd| + 2^-20 (512 products summed in fp32, worst case 512 * 2^-24 < 2^-14; the exponential
a few 2^-23), the kernel's weights are w_j (1 + 2 eps), each rounded to bf16 once (the row scale is a power of two and
rounds nothing), a CTA's partial sum is rounded to bf16 once more when a cluster merges, and the output once:
    |err_d| <= (2 u + 4 eps + 2^-16) * sum_j w_j |k_jd| * sqrt2 (rotated pairs, the larger of the two) + u |o_d|
"""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa, synth
from oracle import codecs, layer as OL
from oracle.compress import RollingState
from oracle.rope import ROPE_THETA
from _parity import np64

gpu = pytest.mark.gpu
U = 2.0 ** -8
D = 512
SM = 1.0 / math.sqrt(512.0)


# ---- the format on the CPU ----------------------------------------------------------------------------------------
def test_format_is_the_nearest_value_on_its_grids():
    """Against a search over every code: the row scale is the least that holds the row, each block scale and code the
    nearest (ties to the even code)."""
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal((6, D)) * 2.0 ** rng.integers(-30, 30, (6, 1)),
                        np.zeros((1, D)), rng.integers(-12, 13, (4, D)) / 2.0, np.full((1, D), 2688.0)])
    x = codecs.bf16_round(x)
    data, s = codecs.fp4_block_quantize_rows(x)
    assert data.shape == (len(x), 288)
    amax = np.max(np.abs(x), axis=1)
    assert np.all((amax <= 2688 * s) & ((amax > 2688 * s / 2) | (amax == 0))) and np.all(s[amax == 0] == 1)
    el, bs = codecs.e2m1_decode(codecs.fp4_unpack(data[:, :256])), codecs.e4m3_decode(data[:, 256:])
    grid8 = codecs.e4m3_decode(np.arange(127))
    grid4 = codecs.e2m1_decode(np.arange(8))

    def nearest(v, grid):
        d = np.abs(v[..., None] - grid)
        tie = d == d.min(-1, keepdims=True)
        best = np.argmax(tie, -1)
        return np.where((tie.sum(-1) > 1) & (best % 2 == 1), best + 1, best)

    b = x.reshape(len(x), 32, 16) / s[:, None, None]
    assert np.array_equal(bs, grid8[nearest(np.minimum(np.max(np.abs(b), -1) / 6, 448.0), grid8)])
    q = np.divide(b, bs[..., None], out=np.zeros_like(b), where=bs[..., None] > 0)
    assert np.array_equal(np.abs(el).reshape(b.shape), grid4[nearest(np.minimum(np.abs(q), 6.0), grid4)])
    v = codecs.fp4_block_dequantize_rows(data, s)
    assert np.array_equal(codecs.bf16_round(v), v)                 # exact in bf16
    again, s2 = codecs.fp4_block_quantize_rows(codecs.fp4_block_dequantize_rows(data, s))
    assert np.all(s2 <= s)
    # half a step of the grid, and of the block scale where the block's largest value saturates
    err = np.abs(v.reshape(b.shape) / s[:, None, None] - b)
    assert np.all(err <= bs[..., None] + np.max(np.abs(b), -1, keepdims=True) * 2.0 ** -4 + 2.0 ** -9 * 6)


def _pool(dim=D, dtype=dsa.DSA_FP4_BLOCK, epb=64, data=256, scale=512):
    return dsa.DsaPool(data, scale, 4, epb, dim, dtype)


def test_refusals_host_only():
    """Every argument that the calls refuse, decided before anything is launched."""
    P = ctypes.c_void_p
    bt = dsa.DsaBlockTable(64, 2, 4)
    ok = _pool()

    def write(batch=2, n=8, cu=P(16), start=P(16), x=P(16), pool=ok, table=bt):
        return dsa._lib.dsa_cache_write(batch, cu, start, n, x, None if pool is None else ctypes.byref(pool),
                                        None if table is None else ctypes.byref(table), None, None)

    INV, UNS, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK
    assert write(batch=0) == OK and write(n=0) == OK
    assert write(batch=-1) == INV and write(n=-1) == INV
    assert write(cu=None) == INV and write(start=None) == INV and write(x=None) == INV
    assert write(x=P(24)) == INV and write(pool=None) == INV and write(table=None) == INV
    assert write(batch=3) == INV                                     # more requests than the table has rows
    assert write(pool=_pool(dim=128)) == UNS and write(pool=_pool(dim=96, dtype=dsa.DSA_BF16)) == UNS
    assert write(pool=_pool(scale=None)) == INV and write(pool=_pool(data=264)) == INV
    assert write(pool=_pool(dtype=9)) == INV

    def read(n=8, req=P(16), ids=P(16), out=P(16), pool=ok, table=bt):
        return dsa._lib.dsa_cache_read(ctypes.byref(pool), ctypes.byref(table), n, req, ids, out, None, None)

    assert read(n=0) == OK and read(n=-1) == INV
    assert read(req=None) == INV and read(ids=None) == INV and read(out=None) == INV and read(out=P(40)) == INV
    assert read(pool=_pool(dim=64)) == UNS and read(table=dsa.DsaBlockTable(64, 2, 0)) == INV

    rope = dsa.DsaRope(64, 10000.0)
    f = dsa._lib.dsa_sparse_attn_decode

    def attend(main, swa, q=P(16)):
        return f(1, 64, q, P(16), 0, P(16), 8, ctypes.byref(main), ctypes.byref(bt), ctypes.byref(swa),
                 ctypes.byref(bt), 128, SM, ctypes.byref(rope), P(16), None, None, 0, None, None)

    swa = _pool(epb=256)
    assert attend(ok, _pool(dtype=dsa.DSA_BF16, epb=256)) == UNS     # both pools in one format
    assert attend(_pool(dtype=dsa.DSA_FP4_E2M1), swa) == UNS
    assert attend(ok, swa, q=P(8)) == INV
    assert attend(_pool(dim=128), swa) == UNS
    assert dsa.dsa_attn_plan(32, 64, 640, "fp4_block")[0] == 64
    # indexer keys are e4m3 or e2m1 with a scale per row; the compressor stores block rows at dim 512 only
    keys = _pool(dim=128)
    assert dsa._lib.dsa_index_scores(1, 8, 128, P(16), P(16), P(16), P(16), P(16), 1, ctypes.byref(keys),
                                     ctypes.byref(bt), P(16), 64, None, None, None, None, None) == UNS
    comp = [0, 1, P(16), P(16), 1, P(16), P(16), P(16), P(16), P(16), 4, None, ctypes.c_float(1e-6),
            ctypes.byref(rope), ctypes.byref(keys), ctypes.byref(bt), None, None, None, None]
    assert dsa._lib.dsa_compress(*comp) == UNS


def test_binding_pool_dim_from_its_rows():
    assert dsa.pool(torch.zeros((64, 288), dtype=torch.uint8), 64, torch.zeros(64), fmt="fp4_block").dim == 512
    with pytest.raises(AssertionError):
        dsa.pool(torch.zeros((64, 256), dtype=torch.uint8), 64, torch.zeros(64), fmt="fp4_block")


# ---- storing and reading back ---------------------------------------------------------------------------------------
def _bf16(x):
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def _awkward_rows(n, seed):
    """bf16 rows that meet the borders: exact ties, zero rows and blocks, one large element, tiny and huge rows."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, D)) * 2.0 ** g.integers(-8, 8, (n, 1))
    for i in range(n):
        m = i % 8
        if m == 1:
            x[i] = g.integers(-24, 25, D) / 4.0          # quarters: many quotients sit on a border
        elif m == 2:
            x[i] = 0.0
        elif m == 3:
            x[i, 16:] = 0.0
        elif m == 4:
            x[i] *= 2.0 ** -20
            x[i, 77] = 300.0                             # the other blocks' scales fall among e4m3's subnormals
        elif m == 5:
            x[i] *= 2.0 ** g.integers(-110, -60)
        elif m == 6:
            x[i] *= 2.0 ** 100
        elif m == 7:
            x[i] = np.sign(x[i]) * 1344.0 * 2.0 ** g.integers(-3, 3)
    return _bf16(x)


def _paged(counts, first, epb, seed, spare=3):
    """A shuffled block table that maps every block up to each request's last row."""
    g = torch.Generator().manual_seed(seed)
    need = [max(1, (a + n + epb - 1) // epb) for a, n in zip(first, counts)]
    perm = torch.randperm(sum(need) + spare, generator=g).to(torch.int32)
    bt = torch.full((len(counts), max(need)), -1, dtype=torch.int32)
    at = 0
    for r, b in enumerate(need):
        bt[r, :b] = perm[at:at + b]
        at += b
    return bt, sum(need) + spare


def _physical(bt, r, i, epb):
    return int(bt[r, i // epb]) * epb + i % epb


def _schedule(counts, first):
    cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    return cu, torch.tensor(first, dtype=torch.int32)


RAGGED = [([1], [0]), ([1] * 32, [0] * 32), ([5, 0, 131, 1, 0, 64, 0], [0, 9, 63, 64, 5, 250, 0]),
          ([0, 3], [2, 61]), ([1] * 70 + [0] * 5 + [9], [i % 3 for i in range(76)]), ([2] * 1100, [1] * 1100)]


@gpu
@pytest.mark.parametrize("case", range(len(RAGGED)))
@pytest.mark.parametrize("epb", [64, 256])
def test_write_then_read_is_the_oracle_bit_for_bit(case, epb):
    """Stored bytes and scales equal the oracle's; other rows of the pool, and the rows of x behind the last request,
    change nothing; every row reads back as the value it stands for, in any order and more than once."""
    counts, first = RAGGED[case]
    total = sum(counts)
    bt, blocks = _paged(counts, first, epb, case)
    x = torch.cat([_awkward_rows(total, case), _bf16(np.full((5, D), 7.0))])     # five rows of padding
    cu, start = _schedule(counts, first)
    data = torch.randint(0, 256, (blocks * epb, 288), dtype=torch.uint8, generator=torch.Generator().manual_seed(case))
    scale = torch.arange(blocks * epb, dtype=torch.float32)
    gd, gs, status = data.cuda(), scale.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, table = dsa.pool(gd, epb, gs, fmt="fp4_block"), bt.cuda()
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, dsa.block_table(table), dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    req = np.repeat(np.arange(len(counts)), counts)
    ids = np.concatenate([np.arange(n) + f for n, f in zip(counts, first)]).astype(int)
    rows = np.array([_physical(bt, r, i, epb) for r, i in zip(req, ids)])
    want, ws = codecs.fp4_block_quantize_rows(np64(x[:total]))
    got = gd.cpu().numpy()
    # the sign of a zero code is not part of the value: compare codes with -0 taken as 0
    def plain(b):
        lo, hi = b[:, :256] & 15, b[:, :256] >> 4
        lo, hi = np.where(lo == 8, 0, lo), np.where(hi == 8, 0, hi)
        return np.concatenate([lo | (hi << 4), b[:, 256:]], axis=1)
    assert np.array_equal(np64(gs)[rows], ws)
    assert np.array_equal(plain(got[rows]), plain(want))
    rest = np.setdiff1d(np.arange(blocks * epb), rows)
    assert np.array_equal(got[rest], data.numpy()[rest]) and np.array_equal(np64(gs)[rest], np64(scale)[rest])
    # read back: every row, twice over and shuffled, with pads
    order = np.random.default_rng(case).permutation(np.concatenate([np.arange(total), np.arange(total)]))
    r2, i2 = np.append(req[order], 0), np.append(ids[order], -1)
    out = torch.full((len(r2), D), 3.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read(pool, dsa.block_table(table), torch.tensor(r2, dtype=torch.int32, device="cuda"),
                       torch.tensor(i2, dtype=torch.int32, device="cuda"), out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    vals = codecs.fp4_block_dequantize_rows(want, ws)
    assert np.array_equal(np64(out)[:-1], vals[order]) and not np64(out)[-1].any()


@gpu
def test_rows_with_infinities_or_nan_read_back_as_nan():
    x = _awkward_rows(6, 3)
    x[1, 5], x[3, 500], x[4, 0] = float("nan"), float("inf"), float("-inf")
    data = torch.zeros((64, 288), dtype=torch.uint8, device="cuda")
    scale = torch.zeros(64, device="cuda")
    pool = dsa.pool(data, 64, scale, fmt="fp4_block")
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu, start = _schedule([6], [0])
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, dsa.block_table(bt))
    out = torch.empty((6, D), dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(6, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_read(pool, dsa.block_table(bt), torch.zeros_like(ids), ids, out)
    got = np64(out)
    assert np.isnan(got[[1, 3, 4]]).all() and np.isfinite(got[[0, 2, 5]]).all()
    want = codecs.fp4_block_dequantize_rows(*codecs.fp4_block_quantize_rows(np64(x[[0, 2, 5]])))
    assert np.array_equal(got[[0, 2, 5]], want)


@gpu
@pytest.mark.parametrize("fmt,dim", [("bf16", 64), ("bf16", 512), ("fp8", 64), ("fp8", 128), ("fp8", 512), ("fp4", 64),
                                     ("fp4", 128), ("fp4", 512)])
def test_write_and_read_in_the_other_formats(fmt, dim):
    """bf16 rows come back as they were; e4m3 / e2m1 rows carry scale amax/448, amax/6 (fp32, one rounding) and the
    codes nearest to x / scale; reading returns scale * code rounded to bf16."""
    counts, first, epb = [3, 0, 66], [62, 4, 1], 64
    bt, blocks = _paged(counts, first, epb, 5)
    g = torch.Generator().manual_seed(dim)
    x = (torch.randn((69, dim), generator=g) * 4).to(torch.bfloat16)
    x[7] = 0
    cu, start = _schedule(counts, first)
    cols = {"bf16": dim, "fp8": dim, "fp4": dim // 2}[fmt]
    gd = torch.zeros((blocks * epb, cols), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")
    gs = None if fmt == "bf16" else torch.zeros(blocks * epb, device="cuda")
    pool, table = dsa.pool(gd, epb, gs, fmt=fmt), dsa.block_table(bt.cuda())
    tb = bt.cuda()
    table = dsa.block_table(tb)
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, table)
    req = np.repeat(np.arange(3), counts)
    ids = np.concatenate([np.arange(n) + f for n, f in zip(counts, first)]).astype(int)
    out = torch.empty((69, dim), dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read(pool, table, torch.tensor(req, dtype=torch.int32, device="cuda"),
                       torch.tensor(ids, dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    if fmt == "bf16":
        assert torch.equal(out.cpu(), x)
        return
    rows = [_physical(bt, r, i, epb) for r, i in zip(req, ids)]
    xs = np64(x)
    amax = np.abs(xs).max(1)
    top, half = (448.0, 2.0 ** -4) if fmt == "fp8" else (6.0, 0.5)
    s = np64(gs)[rows]
    assert np.all(np.abs(s - np.where(amax > 0, amax / top, 1.0)) <= 2.0 ** -24 * np.maximum(s, 1e-30))
    codes = gd.cpu().numpy()[rows]
    dec = codecs.e4m3_decode(codes) if fmt == "fp8" else codecs.e2m1_decode(codecs.fp4_unpack(codes))
    q = xs / s[:, None]
    # half a step of the grid at |q| (e4m3: relative 2^-4, at least half its subnormal step; e2m1: 1/4, 1/2 or 1)
    step = np.maximum(np.abs(q) * half, 2.0 ** -10) if fmt == "fp8" else np.where(np.abs(q) < 2, 0.25, np.where(np.abs(q) < 4, 0.5, 1.0))
    assert np.all(np.abs(dec - q) <= step * (1 + 2.0 ** -20))
    want = dec * s[:, None]
    assert np.all(np.abs(np64(out) - want) <= U * np.abs(want))


@gpu
def test_bad_rows_fault_and_the_others_are_written():
    """Unmapped and out-of-pool blocks, rows beyond the table, a negative start, a request outside the table."""
    counts, first = [4, 4, 4, 4, 4], [62, 62, 126, -2, 0]
    bt = torch.tensor([[0, -1], [1, 99], [2, 3], [4, 5], [6, 7]], dtype=torch.int32)   # 8 blocks
    x = _awkward_rows(20, 8)
    cu, start = _schedule(counts, first)
    gd = torch.full((512, 288), 17, dtype=torch.uint8, device="cuda")
    gs = torch.full((512,), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, tb = dsa.pool(gd, 64, gs, fmt="fp4_block"), bt.cuda()
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, dsa.block_table(tb), dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    good = {0: 62, 1: 63, 4: 64 + 62, 5: 64 + 63, 8: 192 + 62, 9: 192 + 63, 14: 256, 15: 257,
            16: 384, 17: 385, 18: 386, 19: 387}
    want, ws = codecs.fp4_block_quantize_rows(np64(x))
    vals = codecs.fp4_block_dequantize_rows(want, ws)
    got = codecs.fp4_block_dequantize_rows(gd.cpu().numpy(), np64(gs))
    for j, row in good.items():
        assert np.array_equal(got[row], vals[j]), j
    rest = np.setdiff1d(np.arange(512), list(good.values()))
    assert (gd.cpu().numpy()[rest] == 17).all() and (np64(gs)[rest] == 5.0).all()
    # reads
    req = torch.tensor([0, 0, 1, 2, -1, 5, 4, 4], dtype=torch.int32, device="cuda")
    ids = torch.tensor([62, 64, 64, 128, 0, 0, -2, 1], dtype=torch.int32, device="cuda")
    out = torch.full((8, D), 9.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    dsa.dsa_cache_read(pool, dsa.block_table(tb), req, ids, out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    o = np64(out)
    assert np.array_equal(o[0], vals[0]) and np.array_equal(o[7], vals[17]) and not o[1:7].any()


@gpu
@pytest.mark.parametrize("kind,cached,new", [("c4a", [1000, 6, 0], [1, 1, 40]), ("c128a", [127, 300], [1, 200])])
def test_compressor_stores_block_rows(kind, cached, new):
    """dsa_compress into block pools (entries and window rows): each row is a correct quantisation of the oracle's
    float64 row: the same row scale (or its neighbour when amax / 2688 lies within 1e-5 of a power of two), block scales
    within half an e4m3 step of amax_b / (6 s), codes within half an e2m1 step, with a slack of 1e-4 of the value for the
    kernel's fp32 row."""
    spec = synth.CaseSpec("block", kind=kind, cached=cached, new=new, queries="all", idx_heads=0, topk=0,
                          main_dtype="fp4_block", swa_dtype="fp4_block", seed=41)
    case = synth.make_case(spec, "cpu")
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in case.items()}
    from compressed_sparse_attention_c4a_gb300.step import LayerStep
    step = LayerStep(dev)
    step.compress_main()
    torch.cuda.synchronize()
    assert int(step.status) == 0
    epb = case["epb"]
    main = OL.Pool(epb, OL.FP4_BLOCK, case["main_data"].numpy().copy(), np64(case["main_scale"]))
    swa = OL.Pool(256, OL.FP4_BLOCK, case["swa_data"].numpy().copy(), np64(case["swa_scale"]))
    bt, sbt = np64(case["bt_main"]), np64(case["bt_swa"])
    cu = np64(case["cu_new"])
    xs, zs = np64(case["x_new"]), np64(case["z_new"])
    states = [RollingState(kind, D, np64(case["state_x"])[r], np64(case["state_z"])[r]) for r in range(len(cached))]
    rec = {}
    OL.compress(kind, np64(case["start_pos"]), [xs[cu[r]:cu[r + 1]] for r in range(len(new))],
                [zs[cu[r]:cu[r + 1]] for r in range(len(new))], states, 64, main, bt, swa, sbt, record=rec)
    assert any(k[0] == "entry" for k in rec)
    for (what, r, i), v in rec.items():
        table, per, data, scale = (bt, epb, dev["main_data"], dev["main_scale"]) if what == "entry" else \
            (sbt, 256, dev["swa_data"], dev["swa_scale"])
        row = int(table[r][i // per]) * per + i % per
        b, s = data[row].cpu().numpy(), float(scale[row])
        ratio = np.max(np.abs(v)) / 2688 / s
        assert 0.5 * (1 - 1e-5) <= ratio <= 1 + 1e-5, (what, r, i, ratio)
        blocks = v.reshape(32, 16) / s
        want = np.max(np.abs(blocks), -1) / 6
        bs = codecs.e4m3_decode(b[256:])
        assert np.all(np.abs(bs - np.minimum(want, 448)) <= np.maximum(want * 2.0 ** -4, 2.0 ** -10) + 1e-4 * want)
        q = np.divide(blocks, bs[:, None], out=np.zeros_like(blocks), where=bs[:, None] > 0)
        el = codecs.e2m1_decode(codecs.fp4_unpack(b[:256])).reshape(32, 16)
        a = np.minimum(np.abs(q), 6.0)
        half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
        assert np.all(np.abs(np.abs(el) - a) <= half + 1e-4 * a + 1e-12), (what, r, i)


# ---- attention ------------------------------------------------------------------------------------------------------
def _attn_case(spec, topk="random", seed=0):
    case = synth.make_case(spec, "cpu")
    nq = case["nq"]
    g = np.random.default_rng(seed)
    w, s = synth.WINDOW[spec.kind]
    pos = np64(case["q_pos"])
    nvis = np.where(pos + 1 < w, 0, (pos + 1 - w) // s + 1)
    tk = None
    if topk == "random":
        tk = np.full((nq, spec.topk), -1, dtype=np.int32)
        for j in range(nq):
            n = min(int(nvis[j]), spec.topk - (j % 3) * (spec.topk // 5))
            pick = np.sort(g.choice(int(nvis[j]), n, replace=False)) if n > 0 else np.zeros(0, int)
            at = np.sort(g.choice(spec.topk, n, replace=False)) if j % 2 else np.arange(n)   # -1 between entries, too
            tk[j, at] = pick
        case["topk"] = torch.tensor(tk)
    case["nvis"] = nvis
    return case


def _pools(case, dev):
    f = case["spec"].main_dtype
    return (dsa.pool(dev["main_data"], case["epb"], dev["main_scale"], fmt=f), dsa.block_table(dev["bt_main"]),
            dsa.pool(dev["swa_data"], 256, dev["swa_scale"], fmt=f), dsa.block_table(dev["bt_swa"]))


def _expected(case, rows=None):
    """{row: (o, lse, sum_j w_j |k_jd| after the pair's larger, eps)} in 64 bits."""
    spec, epb = case["spec"], case["epb"]
    bt, sbt = np64(case["bt_main"]), np64(case["bt_swa"])
    pos, req, q = np64(case["q_pos"]), np64(case["q_req"]), np64(case["q"])
    tk = case.get("topk")
    md, ms = case["main_data"].numpy(), np64(case["main_scale"])
    sd, ss = case["swa_data"].numpy(), np64(case["swa_scale"])
    out = {}
    for j in range(len(pos)) if rows is None else rows:
        m, r = int(pos[j]), int(req[j])
        ids = np.arange(case["nvis"][j]) if tk is None else np64(tk)[j]
        ids = ids[ids >= 0].astype(int)
        win = np.arange(max(0, m - spec.window + 1), m + 1)
        mr = bt[r][ids // epb].astype(int) * epb + ids % epb
        sr = sbt[r][win // 256].astype(int) * 256 + win % 256
        keys = np.concatenate([codecs.fp4_block_dequantize_rows(md[mr], ms[mr]),
                               codecs.fp4_block_dequantize_rows(sd[sr], ss[sr])])
        logits = q[j] @ keys.T * SM
        top = logits.max(-1, keepdims=True)
        e = np.exp(logits - top)
        wgt = e / e.sum(-1, keepdims=True)
        o, reach = wgt @ keys, wgt @ np.abs(keys)
        eps = 2.0 ** -14 * SM * np.max(np.abs(q[j]) @ np.abs(keys).T, axis=-1) + 2.0 ** -20
        ang = m * ROPE_THETA ** (-np.arange(0, 64, 2) / 64.0)
        c, s = np.cos(ang), np.sin(ang)
        a, b = o[:, 448::2].copy(), o[:, 449::2].copy()
        o[:, 448::2], o[:, 449::2] = a * c + b * s, b * c - a * s
        pair = np.maximum(reach[:, 448::2], reach[:, 449::2]) * math.sqrt(2.0)
        reach[:, 448::2] = reach[:, 449::2] = pair
        out[j] = (o, (top[:, 0] + np.log(e.sum(-1))), reach, eps)
    return out


def _check(got, lse, want, vm=None):
    for j, (o, l, reach, eps) in want.items():
        tol = (2 * U + 4 * eps[:, None] + 2.0 ** -16) * reach + U * np.abs(o) + 1e-30
        err = np.abs(np64(got[j]) - o)
        assert np.all(err <= tol), (j, float((err / tol).max()), np.unravel_index(np.argmax(err / tol), err.shape))
        if lse is not None:
            assert np.all(np.abs(np64(lse[j]) - l) <= 2 * eps + 2.0 ** -20 * np.maximum(1, np.abs(l))), j


S = synth.CaseSpec
F = dict(main_dtype="fp4_block", swa_dtype="fp4_block")
ATTN = {
    # decode rows of lengths 1, 8 (the first entry), a block's border, below and above k, in one call
    "ragged": S("ragged", cached=[0, 7, 8, 126, 127, 255, 256, 1000, 2999], new=[1] * 9, topk=200, seed=51, **F),
    "heads16": S("heads16", cached=[4095], new=[1], heads=16, seed=52, **F),
    "heads32": S("heads32", cached=[4095, 77], new=[1, 1], heads=32, topk=500, seed=53, **F),
    "heads128": S("heads128", cached=[3000, 10], new=[1, 1], heads=128, topk=33, seed=54, **F),
    "one_entry": S("one_entry", cached=[700] * 3, new=[1] * 3, topk=1, window=1, seed=55, **F),
    "wide_window": S("wide_window", cached=[5000, 600], new=[1, 1], topk=64, window=1024, seed=56, **F),
    "many_rows": S("many_rows", cached=[300 + 7 * i for i in range(90)], new=[1] * 90, topk=63, heads=64, seed=57, **F),
    "pairs": S("pairs", cached=[200 + 31 * i for i in range(40)], new=[1] * 40, topk=250, heads=64, seed=63, **F),
    "many_splits": S("many_splits", cached=[4999, 4200], new=[1, 1], topk=1024, seed=64, **F),
    "dense": S("dense", kind="c128a", cached=[60000, 1279, 126, 127, 0], new=[1] * 5, idx_heads=0, topk=0, seed=58, **F),
    "dense_c4a": S("dense_c4a", kind="c4a", cached=[3001, 5], new=[1] * 2, topk=0, heads=16, seed=59, **F),
    "prefill": S("prefill", cached=[1037, 0], new=[130, 70], queries="all", topk=100, seed=60, **F),
    "prefill_few": S("prefill_few", cached=[500], new=[3], queries="all", heads=16, topk=100, window=77, seed=61, **F),
    "prefill_many": S("prefill_many", cached=[0], new=[400], queries="all", heads=32, topk=90, window=128, seed=62, **F),
}


def _run(case, dev, mode="plain", stream=None):
    spec, nq = case["spec"], case["nq"]
    main, bt, swa, sbt = _pools(case, dev)
    rope = dsa.rope(64)
    out = torch.full((nq, spec.heads, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq, spec.heads), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tk, k = (dev["topk"], spec.topk) if "topk" in case else (None, 0)
    keys = (k if k else bt.max_blocks * case["epb"]) + spec.window
    ws = torch.empty(max(16, dsa.dsa_attn_workspace_size(nq, spec.heads, keys)), dtype=torch.uint8, device="cuda")
    if spec.queries == "last":
        dsa.dsa_sparse_attn_decode(dev["q"], dev["q_pos"], spec.kind, tk, k, main, bt, swa, sbt, spec.window, SM, rope,
                                   out, lse, ws, dev_status=status, stream=stream)
    else:
        dsa.dsa_sparse_attn_prefill(dev["q"], dev["q_pos"], dev["q_req"], spec.kind, tk, k, main, bt, swa, sbt,
                                    spec.window, SM, rope, out, lse, ws, dev_status=status, stream=stream)
    return out, lse, status, ws


def _on_gpu(case):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in case.items()}


@gpu
@pytest.mark.parametrize("name", list(ATTN))
def test_attention_over_block_rows(name):
    spec = ATTN[name]
    case = _attn_case(spec, "random" if spec.topk else None, seed=spec.seed)
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    rows = None if case["nq"] <= 60 else list(range(0, case["nq"], 7)) + [case["nq"] - 1]
    _check(out, lse, _expected(case, rows))


@gpu
@pytest.mark.parametrize("name", ["ragged", "dense", "prefill_few", "heads128"])
def test_attention_when_the_running_maximum_moves(name):
    """Queries 12 times as long: the maxima of later tiles exceed the earlier ones by more than the lazy margin, for some
    heads and not for others (every fourth head keeps its length), so accumulated outputs are rescaled."""
    spec = ATTN[name]
    case = _attn_case(spec, "random" if spec.topk else None, seed=spec.seed)
    long = torch.full((spec.heads, 1), 12.0)
    long[::4] = 1.0
    case["q"] = (case["q"].float() * long).to(torch.bfloat16)
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check(out, lse, _expected(case))


@gpu
@pytest.mark.parametrize("heads,nq", [(64, 500), (128, 170), (16, 700)])
def test_attention_many_rows_in_turn(heads, nq):
    """More rows than the GPU holds at once, of lengths from one key to many, in an order that mixes them."""
    spec = S("many", cached=[0] * 2, new=[nq // 2, nq - nq // 2], queries="all", heads=heads, topk=150, window=128,
             seed=70 + heads, **F)
    case = _attn_case(spec, "random", seed=heads)
    order = torch.randperm(nq, generator=torch.Generator().manual_seed(1))
    for k in ("q", "q_pos", "q_req", "topk"):
        case[k] = case[k][order].contiguous()
    case["nvis"] = case["nvis"][order.numpy()]
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check(out, lse, _expected(case, range(0, nq, 3)))


@gpu
@pytest.mark.parametrize("rows,heads", [(3, 64), (200, 64), (200, 16)])
def test_attention_faults_zero_their_rows_only(rows, heads):
    """A position below zero, a request outside the tables, an unmapped or out-of-pool block of each pool, an entry that is
    not visible: zeros, lse -inf and the device status; every other row is right."""
    spec = S("faults", cached=[900 + i for i in range(rows)], new=[1] * rows, heads=heads, topk=40, seed=81, **F)
    case = _attn_case(spec, "random", seed=5)
    g = np.random.default_rng(0)
    bad = {}
    for i, j in enumerate(range(0, rows, 1 if rows < 10 else 7)):
        kind = i % 6 if rows >= 10 else [1, 3, 5][i]
        bad[j] = kind
        if kind == 0:
            case["q_pos"][j] = -1
        elif kind == 1:
            first = int(case["topk"][j][case["topk"][j] >= 0][0])
            case["bt_main"][j, first // case["epb"]] = -1
        elif kind == 2:
            first = int(case["topk"][j][case["topk"][j] >= 0][0])
            case["bt_main"][j, first // case["epb"]] = 10 ** 6
        elif kind == 3:
            case["bt_swa"][j, int(case["q_pos"][j]) // 256] = -1
        elif kind == 4:
            case["bt_swa"][j, int(case["q_pos"][j]) // 256] = 2 ** 30
        else:
            case["topk"][j, int((case["topk"][j] >= 0).nonzero()[0])] = int(case["nvis"][j])
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    for j in bad:
        assert not np64(out[j]).any() and np.isneginf(np64(lse[j])).all(), (j, bad[j])
    _check(out, lse, _expected(case, [j for j in range(rows) if j not in bad][:40]) if rows > 3 else {})


@gpu
@pytest.mark.parametrize("rows", [4, 200])
def test_a_row_of_nan_reaches_only_the_queries_that_read_it(rows):
    spec = S("nan", cached=[600] * rows, new=[1] * rows, heads=64, topk=30, window=16, seed=91, **F)
    case = _attn_case(spec, "random", seed=6)
    hit = list(range(0, rows, 3))
    for j in hit:      # the row of one of j's selected entries, or (every other) of its own window
        if j % 2:
            p = int(case["q_pos"][j]) - 3
            case["swa_scale"][_physical(case["bt_swa"], j, p, 256)] = float("nan")
        else:
            i = int(case["topk"][j][case["topk"][j] >= 0][2])
            case["main_scale"][_physical(case["bt_main"], j, i, case["epb"])] = float("nan")
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    for j in hit:
        assert np.isnan(np64(out[j])).all() and np.isnan(np64(lse[j])).all(), j
    _check(out, lse, _expected(case, [j for j in range(rows) if j not in hit][:40]))


@gpu
@pytest.mark.parametrize("epb", [64, 256])
def test_many_rows_at_16_byte_addresses(epb):
    """Enough rows that a warp takes four, requests that begin and end inside such a group, empty ones between them; x and
    out start 16 bytes past a 32-byte boundary."""
    counts, first = [9001, 0, 0, 1, 37, 0, 700, 2, 0, 1259], [3, 0, 5, 64, 250, 1, 0, 63, 9, 77]
    total = sum(counts)
    bt, blocks = _paged(counts, first, epb, 5)
    x = torch.empty(total * D + 8, dtype=torch.bfloat16, device="cuda")[8:].view(total, D)
    x.copy_(_awkward_rows(total, 12))
    assert x.data_ptr() % 32 == 16
    cu, start = _schedule(counts, first)
    gd = torch.full((blocks * epb, 288), 17, dtype=torch.uint8, device="cuda")
    gs, status = torch.full((blocks * epb,), 5.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, table = dsa.pool(gd, epb, gs, fmt="fp4_block"), bt.cuda()
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x, pool, dsa.block_table(table), dev_status=status)
    req = np.repeat(np.arange(len(counts)), counts)
    ids = np.concatenate([np.arange(n) + f for n, f in zip(counts, first)]).astype(int)
    out = torch.empty((total + 1) * D + 8, dtype=torch.bfloat16, device="cuda")[8:].view(total + 1, D)
    out.fill_(3.0)
    order = np.random.default_rng(3).permutation(total)
    dsa.dsa_cache_read(pool, dsa.block_table(table), torch.tensor(req[order], dtype=torch.int32, device="cuda"),
                       torch.tensor(ids[order], dtype=torch.int32, device="cuda"), out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    want, ws = codecs.fp4_block_quantize_rows(np64(x))
    assert np.array_equal(np64(out)[:-1], codecs.fp4_block_dequantize_rows(want, ws)[order])
    assert (np64(out)[-1] == 3.0).all()                                          # behind the n rows
    rows = np.array([_physical(bt, r, i, epb) for r, i in zip(req, ids)])
    rest = np.setdiff1d(np.arange(blocks * epb), rows)
    assert (gd.cpu().numpy()[rest] == 17).all() and (np64(gs)[rest] == 5.0).all()


@gpu
@pytest.mark.parametrize("name", ["ragged", "many_rows", "heads16"])
def test_attention_through_the_other_entry_points(name):
    """The call with the library's own scratch, and top-k and attention in one call: the same bits.  e4m3 output with an
    amax / 448 scale per 128 dims: half an e4m3 step (2^-4 of the value, 2^-10 of the scale below its normal range) on top
    of the attention's own error, which here has no bf16 rounding of the output."""
    spec = ATTN[name]
    case = _attn_case(spec, "random", seed=spec.seed)
    nq, nvis = case["nq"], case["nvis"]
    g = torch.Generator().manual_seed(2)
    ld = (int(nvis.max()) + 3) // 4 * 4 + 4
    scores = torch.randn((nq, ld), generator=g).cuda()
    n_visible = torch.tensor(nvis, dtype=torch.int32, device="cuda")
    topk = torch.full((nq, spec.topk), -7, dtype=torch.int32, device="cuda")
    dsa.dsa_topk(scores, n_visible, spec.topk, topk)
    case["topk"] = topk.cpu()
    dev = _on_gpu(case)
    out, lse, status, ws = _run(case, dev)
    main, bt, swa, sbt = _pools(case, dev)
    rope = dsa.rope(64)
    o2, l2 = torch.full_like(out, 4.0), torch.full_like(lse, 4.0)
    dsa.dsa_sparse_attn_decode_static(dev["q"], dev["q_pos"], spec.kind, topk, spec.topk, main, bt, swa, sbt, spec.window,
                                      SM, rope, o2, l2, dev_status=status)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3, t3 = torch.full_like(out, 4.0), torch.full_like(lse, 4.0), torch.full_like(topk, -7)
    dsa.dsa_topk_sparse_attn_decode(dev["q"], dev["q_pos"], spec.kind, scores, n_visible, spec.topk, t3, main, bt, swa, sbt,
                                    spec.window, SM, rope, o3, l3, workspace=ws, dev_status=status)
    assert torch.equal(topk, t3) and torch.equal(out, o3) and torch.equal(lse, l3)
    o8 = torch.zeros((nq, spec.heads, D), dtype=torch.uint8, device="cuda")
    s8, l8 = torch.zeros((nq, spec.heads, 4), device="cuda"), torch.full_like(lse, 4.0)
    dsa.dsa_sparse_attn_q8(dev["q"], dev["q_pos"], dev["q_req"], spec.kind, topk, spec.topk, main, bt, swa, sbt, spec.window,
                           SM, rope, o8, s8, l8, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(lse, l8)
    sc = np.repeat(np64(s8), 128, axis=-1)
    got = codecs.e4m3_decode(o8.cpu().numpy()) * sc
    for j, (o, l, reach, eps) in _expected(case).items():
        tol = (2 * U + 4 * eps[:, None] + 2.0 ** -16) * reach
        tol = tol + np.maximum(2.0 ** -4 * (np.abs(o) + tol), 2.0 ** -10 * sc[j]) + 1e-30
        assert np.all(np.abs(got[j] - o) <= tol), j


@gpu
@pytest.mark.parametrize("name", ["ragged", "prefill_many"])
def test_rows_that_no_query_selects_are_never_used(name):
    """Every row that is neither selected nor in a window, NaN scales and all: the same bits."""
    spec = ATTN[name]
    case = _attn_case(spec, "random", seed=spec.seed)
    out, lse, status, _ = _run(case, _on_gpu(case))
    pos, req, tk, epb = np64(case["q_pos"]), np64(case["q_req"]), np64(case["topk"]).astype(int), case["epb"]
    keep, keep_w = set(), set()
    for j in range(case["nq"]):
        r, m = int(req[j]), int(pos[j])
        keep |= {_physical(case["bt_main"], r, i, epb) for i in tk[j] if i >= 0}
        keep_w |= {_physical(case["bt_swa"], r, i, 256) for i in range(max(0, m - spec.window + 1), m + 1)}
    for data, scale, kept in ((case["main_data"], case["main_scale"], keep), (case["swa_data"], case["swa_scale"], keep_w)):
        drop = torch.tensor(np.setdiff1d(np.arange(data.shape[0]), sorted(kept)))
        data[drop], scale[drop] = 0x7F, float("nan")
    o2, l2, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(out, o2) and torch.equal(lse, l2)


@gpu
def test_the_same_entry_twice_counts_twice():
    spec = ATTN["ragged"]
    case = _attn_case(spec, "random", seed=spec.seed)
    tk = case["topk"]
    for j in range(case["nq"]):
        got = tk[j][tk[j] >= 0]
        if len(got):
            tk[j] = got[torch.arange(spec.topk) % max(1, len(got) // 3)]
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check(out, lse, _expected(case))


@gpu
def test_offsets_beyond_32_bits():
    """Blocks at the end of a pool of 4.8 GB: stored, read back and attended to; the bytes at the offsets' low 32 bits keep
    their values."""
    blocks, epb, n = 262144, 64, 200
    data = torch.empty((blocks * epb, 288), dtype=torch.uint8, device="cuda")
    scale = torch.empty((blocks * epb,), device="cuda")
    far = [blocks - 1, blocks - 4, blocks - 2, blocks - 3]
    assert far[1] * epb * 288 > 2 ** 32
    low = [(b * epb * 288 % 2 ** 32) // 288 for b in far]
    for row in low:
        data[row:row + epb + 1], scale[row:row + epb + 1] = 23, 0.5
    x = _awkward_rows(n, 9)
    x[5::8] = x[4::8]                   # no row so tiny or large that it alone decides the softmax
    x[6::8] = x[0::8]
    x = (x.float() * 2.0 ** -6).to(torch.bfloat16)
    bt = torch.tensor([far], dtype=torch.int32)
    cu, start = _schedule([n], [0])
    gbt = bt.cuda()
    pool, table = dsa.pool(data, epb, scale, fmt="fp4_block"), dsa.block_table(gbt)
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, table)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.empty((n, D), dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read(pool, table, torch.zeros_like(ids), ids, out)
    vals = codecs.fp4_block_dequantize_rows(*codecs.fp4_block_quantize_rows(np64(x)))
    assert np.array_equal(np64(out), vals)
    for row in low:
        assert bool((data[row:row + epb + 1] == 23).all()) and bool((scale[row:row + epb + 1] == 0.5).all())
    # the same rows in a small pool give the same attention
    pos = torch.tensor([4 * n + 7], dtype=torch.int32, device="cuda")            # all n entries visible
    q = _bf16(np.random.default_rng(1).standard_normal((1, 64, D))).cuda()
    swa = torch.zeros((256 * 4, 288), dtype=torch.uint8, device="cuda")
    ss = torch.ones(1024, device="cuda")
    sbt = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    topk = torch.randperm(n, generator=torch.Generator().manual_seed(4))[:96].to(torch.int32).cuda().view(1, 96)
    small = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    sd, sc = torch.empty((256, 288), dtype=torch.uint8, device="cuda"), torch.empty(256, device="cuda")
    for i, b in enumerate(far):
        sd[i * 64:i * 64 + 64], sc[i * 64:i * 64 + 64] = data[b * 64:b * 64 + 64], scale[b * 64:b * 64 + 64]
    res = []
    for p, t in ((pool, table), (dsa.pool(sd, epb, sc, fmt="fp4_block"), dsa.block_table(small))):
        o, l = torch.zeros((1, 64, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 64), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(16, dsa.dsa_attn_workspace_size(1, 64, 96 + 128)), dtype=torch.uint8, device="cuda")
        dsa.dsa_sparse_attn_decode(q, pos, "c4a", topk, 96, p, t, dsa.pool(swa, 256, ss, fmt="fp4_block"),
                                   dsa.block_table(sbt), 128, SM, dsa.rope(64), o, l, ws, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        res.append((o, l))
    assert np.isfinite(np64(res[0][0])).all() and np64(res[0][0]).any()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def _append_and_attend(case, dev, x, cu, start, out, lse, ws, status, stream=None):
    """A decode step as served: the new window rows stored, then attention over both caches."""
    spec = case["spec"]
    main, bt, swa, sbt = _pools(case, dev)
    dsa.dsa_cache_write(cu, start, x, swa, sbt, dev_status=status, stream=stream)
    dsa.dsa_sparse_attn_decode(dev["q"], dev["q_pos"], spec.kind, dev["topk"], spec.topk, main, bt, swa, sbt, spec.window, SM,
                               dsa.rope(64), out, lse, ws, dev_status=status, stream=stream)


@gpu
@pytest.mark.parametrize("name", ["heads16", "many_rows"])
def test_append_and_attend_eager_on_a_stream_and_in_two_graphs(name):
    """Rows stored and attended to in one go: against the 64-bit form over the stored rows; on another stream; and captured
    twice with one workspace, the graphs replayed in turn over changed inputs: the same bits as eager calls."""
    spec = ATTN[name]
    case = _attn_case(spec, "random", seed=spec.seed)
    nq = case["nq"]
    dev = _on_gpu(case)
    cu = torch.arange(nq + 1, dtype=torch.int32, device="cuda")
    xs = [_bf16(np.random.default_rng(20 + i).standard_normal((nq, D))).cuda() for i in range(3)]
    x = xs[0].clone()
    ws = torch.empty(max(16, dsa.dsa_attn_workspace_size(nq, spec.heads, spec.topk + spec.window)), dtype=torch.uint8,
                     device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers():
        return (torch.full((nq, spec.heads, D), 9.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((nq, spec.heads), 9.0, device="cuda"))

    eager = []
    for xi in xs:
        x.copy_(xi)
        o, l = buffers()
        _append_and_attend(case, dev, x, cu, dev["q_pos"], o, l, ws, status)
        torch.cuda.synchronize()
        eager.append((o, l))
    assert not torch.equal(eager[0][0], eager[1][0])
    stored = dict(case, swa_data=dev["swa_data"].cpu(), swa_scale=dev["swa_scale"].cpu())
    _check(*eager[2], _expected(stored, range(0, nq, max(1, nq // 12))))
    # another stream
    side = torch.cuda.Stream()
    x.copy_(xs[0])
    o, l = buffers()
    side.wait_stream(torch.cuda.current_stream())
    _append_and_attend(case, dev, x, cu, dev["q_pos"], o, l, ws, status, stream=side)
    side.synchronize()
    assert torch.equal(o, eager[0][0]) and torch.equal(l, eager[0][1])
    # two graphs
    graphs = []
    for _ in range(2):
        o, l = buffers()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _append_and_attend(case, dev, x, cu, dev["q_pos"], o, l, ws, status)
        graphs.append((g, o, l))
    for which, i in ((0, 1), (1, 2), (0, 0), (1, 1), (0, 2)):
        x.copy_(xs[i])
        g, o, l = graphs[which]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[i][0]) and torch.equal(l, eager[i][1]), (which, i)
    assert int(status) == 0


@gpu
def test_two_calls_at_once():
    """Calls on two streams with a workspace each, over one cache: each as if alone."""
    cases = [_attn_case(ATTN[n], "random", seed=ATTN[n].seed) for n in ("heads16", "many_rows")]
    devs = [_on_gpu(c) for c in cases]
    alone = [_run(c, d)[:2] for c, d in zip(cases, devs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, d, s in zip(cases, devs, streams):
            with torch.cuda.stream(s):
                got.append(_run(c, d, stream=s))
        torch.cuda.synchronize()
        for (o, l, status, _), (ao, al) in zip(got, alone):
            assert int(status) == 0 and torch.equal(o, ao) and torch.equal(l, al)


@gpu
@pytest.mark.parametrize("kind,cached,new,queries", [("c4a", [2100, 39, 7], [1, 1, 1], "last"),
                                                     ("c4a", [1000, 0], [37, 81], "all"),
                                                     ("c128a", [5000, 126], [1, 1], "last")])
def test_layer_step_over_block_caches(kind, cached, new, queries):
    """Compress, index, select and attend as one layer step with both caches in 4 bits: the attention against the 64-bit form
    over the rows that the step stored and the entries that it selected; fused calls and a second stream give the same bits."""
    from compressed_sparse_attention_c4a_gb300.step import LayerStep
    spec = synth.CaseSpec("step", kind=kind, cached=cached, new=new, queries=queries, idx_heads=16 if kind == "c4a" else 0,
                          topk=64 if kind == "c4a" else 0, main_dtype="fp4_block", swa_dtype="fp4_block", seed=71)
    runs = []
    for opts in ({}, {"fused_select": True}, {"two_streams": True}):
        case = synth.make_case(spec, "cpu")
        dev = _on_gpu(case)
        step = LayerStep(dev, **opts)
        step.run()
        torch.cuda.synchronize()
        assert int(step.status) == 0
        runs.append((step, dev, case))
    step, dev, case = runs[0]
    w, s = synth.WINDOW[kind]
    pos = np64(case["q_pos"])
    case["nvis"] = np.where(pos + 1 < w, 0, (pos + 1 - w) // s + 1)
    for k in ("main_data", "main_scale", "swa_data", "swa_scale"):
        case[k] = dev[k].cpu()
    if kind == "c4a":
        case["topk"] = step.topk.cpu()
        for j in range(case["nq"]):
            picked = case["topk"][j][case["topk"][j] >= 0]
            assert len(set(picked.tolist())) == len(picked) == min(int(case["nvis"][j]), 64)
    _check(step.out, step.lse, _expected(case))
    for other, d, _ in runs[1:]:
        assert torch.equal(other.out, step.out) and torch.equal(other.lse, step.lse)
        assert torch.equal(d["main_data"], dev["main_data"]) and torch.equal(d["swa_data"], dev["swa_data"])


@gpu
@pytest.mark.parametrize("heads,topk,window", [(64, 1, 1), (64, 3, 2), (128, 40, 30), (16, 2, 60)])
def test_many_rows_of_one_or_two_tiles(heads, topk, window):
    """Rows so short that a CTA's next rows are resolved, multiplied and normalised while the first is still being stored: every
    row, its log-sum-exp and its own position's rotation."""
    spec = S("tiny", cached=[0] * 3, new=[700, 500, 311], queries="all", heads=heads, topk=topk, window=window,
             seed=90 + heads + topk, **F)
    case = _attn_case(spec, "random", seed=heads + topk)
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check(out, lse, _expected(case))


@gpu
@pytest.mark.parametrize("nq,heads", [(3, 64), (40, 64), (500, 16)])
def test_tiles_without_a_key_are_left_out(nq, heads):
    """Top-k rows with runs of -1 as long as several tiles, at the front, in the middle, at the end and all along: the same
    values as rows without the padding, whatever tiles are left."""
    spec = S("gaps", cached=[3000 - i for i in range(nq)], new=[1] * nq, heads=heads, topk=600, window=40, seed=97, **F)
    case = _attn_case(spec, "random", seed=7)
    tk = case["topk"]
    for j in range(nq):
        cut = [(0, 200), (150, 430), (10, 600), (0, 600), (0, 0), (48, 96), (1, 599), (300, 600)][j % 8]
        tk[j, cut[0]:cut[1]] = -1
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == 0
    _check(out, lse, _expected(case, range(0, nq, max(1, nq // 60))))
    for j in (3 % nq, 2 % nq):      # an unmapped block whose only entry is alone in its tile
        pick = int((tk[j] >= 0).nonzero()[0]) if (tk[j] >= 0).any() else 300
        tk[j, pick] = 17
        case["bt_main"][j, 17 // case["epb"]] = -1
    out, lse, status, _ = _run(case, _on_gpu(case))
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    for j in (3 % nq, 2 % nq):
        assert not np64(out[j]).any() and np.isneginf(np64(lse[j])).all()
