"""The operators around the attention: dsa_norm_q8, dsa_gemm_q8, dsa_cache_append, against float64 and, where an operation
exists twice, bit for bit.

Tolerances, from the arithmetic (u = 2^-24 in fp32; a rounding is off by at most half a step: bf16 2^-8, e4m3 2^-4 of a value):
  * norm: h is rounded once (u); the sum of squares adds at most 32 terms a thread, then 5 and 16 more, all of one sign, each
    square off by 3 u: 56 u, halved by the root; the root, the division and two products 6 u: below 2^-18 of a value;
  * gemm: products of e4m3 values are exact in fp32; a sum of k of them by blocks takes at most 128 + ceil(k / 128) additions
    of fp32, whichever way they go, each off by at most 2 u (the tensor cores may cut off instead of rounding) of the sum of the
    magnitudes, the scales' product and its use 3 u of it;
  * append: as the norm, and the rotation: cosine and sine within 1e-6 of the exact ones, times the pair's length."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa, synth
from compressed_sparse_attention_c4a_gb300.step import LayerStep
from oracle import projection as OP
from oracle.codecs import fp4_dequantize_rows, fp8_dequantize_rows
from _parity import np64
from _rows8 import assert_rows8

pytestmark = pytest.mark.gpu

EPS = 1e-6
NORM_OFF = 2.0 ** -18
BF16 = 2.0 ** -8
FORMATS = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ---- norm -------------------------------------------------------------------------------------------------------------
def run_norm(x, residual, gamma, sum_out="new", eps=EPS):
    n, d = x.shape
    out = torch.full((n, d), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((n, -(-d // 128)), float("nan"), device="cuda")
    total = torch.empty((n, d), dtype=torch.bfloat16, device="cuda") if sum_out == "new" else sum_out
    dsa.dsa_norm_q8(x, gamma, eps, out, scale, residual=residual, sum_out=total)
    return out, scale, total


def check_norm(x, residual, gamma, out, scale, total, eps=EPS):
    h = np64(x) + (0 if residual is None else np64(residual))
    v = OP.rms_norm(h, None if gamma is None else np64(gamma), eps)
    assert_rows8(out.cpu().numpy(), np64(scale), v, NORM_OFF * np.abs(v))
    if total is not None:
        assert (np.abs(np64(total) - h) <= BF16 * np.abs(h) + 2.0 ** -24 * np.abs(h)).all()


@pytest.mark.parametrize("n,dim", [(1, 16), (1, 128), (3, 144), (37, 256), (9, 272), (64, 512), (5, 1008), (17, 1024),
                                   (7, 1040), (33, 2048), (2, 2064), (700, 4096), (1, 4112), (11, 8192), (3, 8208),
                                   (2, 16384), (1300, 1024), (1, 8176)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(n, dim, residual):
    g = gen(n * 31 + dim)
    x = (randn(g, n, dim) * torch.exp2(2 * randn(g, n, 1)) * torch.exp2(randn(g, 1, dim))).to(torch.bfloat16)
    r = (randn(g, n, dim) * 3).to(torch.bfloat16) if residual else None
    gamma = 1 + 0.3 * randn(g, dim) if (n + dim) % 3 else None
    check_norm(x, r, gamma, *run_norm(x, r, gamma))


def test_norm_extreme_rows():
    """Zeros, single values, tiny and huge rows (whose squares leave fp32), and rows that cancel against the residual."""
    d = 400
    x = torch.zeros((8, d), dtype=torch.bfloat16, device="cuda")
    x[1, 5] = 1.0
    x[2] = 1e-30
    x[3] = 1e30
    x[4, ::2], x[4, 1::2] = 3e38, -1e-3
    x[5, 130] = -2.0 ** -120
    x[6] = randn(gen(1), d).to(torch.bfloat16)
    x[7, :128], x[7, 128:256] = 1e-20, 1e10
    r = torch.zeros_like(x)
    r[6] = -x[6]
    for residual in (None, r):
        out, scale, total = run_norm(x, residual, None)
        check_norm(x, residual, None, out, scale, total)
        assert (np64(scale[0]) == 1).all() and not out[0].any()


def test_norm_infinities_and_nan():
    g = gen(3)
    x = randn(g, 4, 304).to(torch.bfloat16)
    x[1, 140] = float("inf")
    x[2, 7] = float("nan")
    out, scale, _ = run_norm(x, None, None)
    codes = out.cpu().numpy() & 0x7f
    for row in (0, 3):
        check_norm(x[row:row + 1], None, None, out[row:row + 1], scale[row:row + 1], None)
    assert codes[1, 140] == 0x7f and (np.delete(codes[1], 140) == 0).all()
    assert (codes[2] == 0x7f).all()


@pytest.mark.parametrize("dim", [256, 4096])
def test_norm_strides_and_in_place(dim):
    """Rows cut out of a wider buffer, and the sum written over x or over the residual."""
    g = gen(4)
    wide = randn(g, 6, 3, dim).to(torch.bfloat16)
    x, r = wide[:, 0], wide[:, 2]
    gamma = 1 + 0.1 * randn(g, dim)
    out, scale, total = run_norm(x, r, gamma)
    check_norm(x, r, gamma, out, scale, total)
    for where in (0, 2):
        again = wide.clone()
        o2, s2, _ = run_norm(again[:, 0], again[:, 2], gamma, sum_out=again[:, where])
        assert torch.equal(o2, out) and torch.equal(s2, scale) and torch.equal(again[:, where], total)
        assert torch.equal(again[:, 2 - where], wide[:, 2 - where]) and torch.equal(again[:, 1], wide[:, 1])


# ---- gemm -------------------------------------------------------------------------------------------------------------
def rows8(g, *shape):
    """Random 8-bit rows: codes over the whole range but NaN, scales over a few powers of two."""
    codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    codes = torch.where((codes & 0x7f) == 0x7f, codes & 0x80, codes)
    n = shape[-1]
    scale = torch.exp2(2 * randn(g, *shape[:-1], -(-n // 128))) / 448
    return codes, scale


def weights8(g, groups, n, k):
    codes, _ = rows8(g, groups, n, k)
    return codes, torch.exp2(2 * randn(g, groups, -(-n // 128), -(-k // 128))) / 448


def gemm_off(k, size):
    return (2 * (128 + -(-k // 128)) + 3) * 2.0 ** -24 * size


def check_gemm(a, a_scale, w, w_scale, out, out_scale):
    want, size = OP.gemm(a.cpu().numpy(), np64(a_scale), w.cpu().numpy(), np64(w_scale))
    off = gemm_off(a.shape[-1], size)
    if out_scale is not None:
        assert_rows8(out.cpu().numpy(), np64(out_scale), want, off)
        return
    room = off + (BF16 * np.abs(want) if out.dtype == torch.bfloat16 else 0)
    err = np.abs(np64(out) - want)
    worst = np.unravel_index(np.argmax(err - room), err.shape)
    assert (err <= room).all(), (worst, err[worst], room[worst], want[worst])


def new_out(m, groups, n, fmt):
    out = torch.full((m, groups, n), 0x55 if fmt == "fp8" else float("nan"), dtype=FORMATS[fmt], device="cuda")
    return out, torch.full((m, groups, -(-n // 128)), float("nan"), device="cuda") if fmt == "fp8" else None


SHAPES = [(1, 1, 16, 1), (1, 520, 4096, 1), (3, 130, 144, 2), (16, 128, 128, 1), (17, 257, 272, 3), (32, 1024, 4096, 8),
          (33, 96, 1040, 1), (64, 384, 512, 1), (65, 1000, 1040, 1), (130, 300, 2064, 2), (300, 640, 384, 1),
          (2, 4096, 8192, 1), (48, 512, 16400, 1), (127, 2, 48, 5), (5, 129, 1024, 1),
          # every number of CTAs that share a tile, of 16 and of 32 rows
          (3, 2000, 2048, 8), (1, 64, 1040, 1), (1, 64, 2048, 1), (17, 4096, 128, 8), (20, 2000, 4096, 8), (17, 520, 1040, 8),
          (31, 256, 2048, 8),
          # tiles of 256 x 256 by pairs: one round of tiles and several, ends inside a tile, a half and a block
          (2560, 2048, 144, 1), (5000, 1000, 400, 1), (700, 300, 272, 16), (19500, 130, 1168, 1), (513, 520, 16, 13),
          (4100, 2900, 2064, 1)]


def test_gemm_shapes_reach_every_form():
    plans = {dsa.dsa_gemm_q8_plan(*s) for s in SHAPES}
    assert plans >= {(128, rows, share) for rows in (16, 32) for share in (1, 2, 4, 8)} | {(256, 256, 2)}


@pytest.mark.parametrize("m,n,k,groups", SHAPES)
@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8"])
def test_gemm(m, n, k, groups, fmt):
    g = gen(m + 3 * n + 7 * k)
    a, a_scale = rows8(g, m, groups, k)
    w, w_scale = weights8(g, groups, n, k)
    out, out_scale = new_out(m, groups, n, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale=out_scale, dev_status=status)
    check_gemm(a, a_scale, w, w_scale, out, out_scale)
    assert int(status) == 0


def test_gemm_strides_and_untouched_bytes():
    """Rows of a wider activation buffer into columns of a wider output: what lies between is left as it was."""
    g = gen(9)
    m, groups, k, n = 21, 2, 272, 37
    buf, sbuf = rows8(g, m, 3 * groups * k + 16)[0], torch.rand((m, 11), generator=g, device="cuda")
    a = buf[:, 16:16 + groups * k].unflatten(1, (groups, k))
    a_scale = sbuf[:, 4:4 + groups * 3].unflatten(1, (groups, 3))
    w, w_scale = weights8(g, groups, n, k)
    wide = torch.full((m, 100), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 13:13 + groups * n].unflatten(1, (groups, n))
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out)
    check_gemm(a, a_scale, w, w_scale, out, None)
    assert (wide[:, :13] == 7).all() and (wide[:, 13 + groups * n:] == 7).all()


def test_gemm_zero_rows_infinite_scales_and_nan():
    """A row of zeros gives zeros (8-bit rows: scale 1); a NaN code or scale reaches only the outputs that it enters, a
    scale of infinity makes infinities."""
    g = gen(10)
    m, n, k = 40, 260, 400
    a, a_scale = rows8(g, m, 1, k)
    w, w_scale = weights8(g, 1, n, k)
    a[3] = 0
    for fmt in FORMATS:
        out, scale = new_out(m, 1, n, fmt)
        dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale=scale)
        assert not out[3].any() and (scale is None or (scale[3] == 1).all())
    a2, s2, w2 = a.clone(), a_scale.clone(), w.clone()
    a2[5, 0, 399], s2[7, 0, 1], w2[0, 131, 128] = 0x7f, float("inf"), 0xff
    base, _ = new_out(m, 1, n, "f32")
    out, _ = new_out(m, 1, n, "f32")
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, base)
    dsa.dsa_gemm_q8(a2, s2, w2, w_scale, out)
    nan = torch.isnan(out[:, 0])
    assert nan[5].all() and nan[:, 131].all()
    rest = torch.ones(m, n, dtype=torch.bool, device="cuda")
    rest[5], rest[7], rest[:, 131] = False, False, False
    assert torch.equal(out[:, 0][rest], base[:, 0][rest])
    assert not torch.isfinite(out[7, 0]).any()


def test_gemm_two_calls_give_the_same_bits_and_streams():
    """Two products at once on two streams, and the same ones again from a captured graph, replayed on new inputs."""
    g = gen(11)
    shapes = [(32, 1024, 4096, 2), (200, 640, 1040, 1)]
    data = [(*rows8(g, m, gr, k), *weights8(g, gr, n, k)) for m, n, k, gr in shapes]
    fresh = [rows8(g, m, gr, k) for m, n, k, gr in shapes]
    outs = [new_out(m, gr, n, "bf16")[0] for m, n, k, gr in shapes]
    first = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for d, o, s in zip(data, outs, streams):
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            dsa.dsa_gemm_q8(*d, o, stream=s)
    torch.cuda.synchronize()
    for d, o in zip(data, outs):
        check_gemm(*d, o, None)
        first.append(o.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for d, o in zip(data, outs):
            dsa.dsa_gemm_q8(*d, o)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, f) for o, f in zip(outs, first))
    for d, (a, s) in zip(data, fresh):
        d[0].copy_(a), d[1].copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    for d, o in zip(data, outs):
        check_gemm(*d, o, None)


@pytest.mark.parametrize("m,n,k", [(4, 256, 4096), (100, 200, 512), (2100, 2048, 1040)])
def test_gemm_bounded_waits_expire_then_the_next_call_is_correct(m, n, k):
    g = gen(12)
    a, a_scale = rows8(g, m, 1, k)
    w, w_scale = weights8(g, 1, n, k)
    out, _ = new_out(m, 1, n, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_debug_gemm_q8_stalled(a, a_scale, w, w_scale, out, 20_000_000, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_TIMEOUT and not out.any()
    status.zero_()
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, dev_status=status)
    check_gemm(a, a_scale, w, w_scale, out, None)
    assert int(status) == 0


# ---- append -----------------------------------------------------------------------------------------------------------
def make_pool(blocks, dim, fmt, fill=0x33):
    """A pool of 256-row blocks whose bytes are all `fill`, and its tensors."""
    rows = blocks * 256
    width = {"bf16": 2 * dim, "fp8": dim, "fp4": dim // 2, "fp4_block": dim // 16 * 9}[fmt]
    data = torch.full((rows, width), fill, dtype=torch.uint8, device="cuda")
    scale = None if fmt == "bf16" else torch.full((rows,), 5.0, device="cuda")
    view = data.view(torch.bfloat16) if fmt == "bf16" else data
    return dsa.pool(view, 256, scale, fmt=fmt if fmt.startswith("fp4") else None), view, scale


def tables(starts, counts, g, extra=2):
    most = max((s + c + 255) // 256 for s, c in zip(starts, counts)) + 1
    need = [((s + c + 255) // 256 - s // 256) if c else 0 for s, c in zip(starts, counts)]
    perm = torch.randperm(sum(need) + extra, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(starts), most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, (s, c, b) in enumerate(zip(starts, counts, need)):
        bt[r, s // 256:s // 256 + b] = perm[at:at + b]
        at += b
    return bt, len(perm)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def schedule(starts, counts):
    cu = np.concatenate([[0], np.cumsum(counts)])
    req = np.repeat(np.arange(len(counts)), counts)
    pos = np.array(starts)[req] + np.arange(cu[-1]) - cu[req]
    return cu, req, pos


def physical(bt, req, pos):
    return bt.cpu().numpy()[req, pos // 256].astype(np.int64) * 256 + pos % 256


CASES = [([0], [1]), ([65535], [1]), ([255, 0, 1000], [3, 0, 700]), ([511, 131071, 2 ** 24 + 5, 0], [1, 300, 2, 513]),
         ([100 * i for i in range(40)], [1] * 40), ([0, 5], [6000, 4300])]


@pytest.mark.parametrize("starts,counts", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("fmt,dim,rope_dim", [("bf16", 512, 64), ("fp8", 512, 64), ("fp4_block", 512, 64), ("fp4", 512, 64),
                                              ("bf16", 128, 64), ("fp8", 128, 10), ("fp4", 64, 64), ("bf16", 64, 0),
                                              ("fp8", 64, 64)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(starts, counts, fmt, dim, rope_dim, norm):
    g = gen(len(starts) + sum(counts) + dim)
    cu, req, pos = schedule(starts, counts)
    n = int(cu[-1])
    bt, blocks = tables(starts, counts, g)
    pool, data, scale = make_pool(blocks, dim, fmt)
    before = data.clone()
    x = (randn(g, n + 3, dim) * torch.exp2(randn(g, n + 3, 1))).to(torch.bfloat16)   # three rows behind the last
    gamma = 1 + 0.2 * randn(g, dim)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_append(ints(cu), ints(starts), x, dsa.rope(rope_dim, 10000.0), pool, dsa.block_table(bt), norm=norm,
                         rms_gamma=gamma, rms_eps=EPS, dev_status=status)
    assert int(status) == 0
    rows = physical(bt, req, pos)
    left = np.setdiff1d(np.arange(blocks * 256), rows)
    assert torch.equal(data[left].view(torch.uint8), before[left].view(torch.uint8))
    assert scale is None or (scale[left] == 5).all()
    want = OP.append_rows(np64(x[:n]), pos, np64(gamma), EPS, norm, rope_dim)
    off = (NORM_OFF if norm else 0) * np.abs(want)
    if rope_dim:
        tail = want[:, dim - rope_dim:]
        pair = np.repeat(np.hypot(tail[:, 0::2], tail[:, 1::2]), 2, axis=1)
        off[:, dim - rope_dim:] = (1e-6 + NORM_OFF) * pair
    if fmt == "bf16":
        assert (np.abs(np64(data[rows]) - want) <= BF16 * np.abs(want) + off * (1 + BF16)).all()
    elif fmt == "fp8":
        s = np64(scale[rows])[:, None]
        amax = np.max(np.abs(want), axis=1, keepdims=True)
        assert (np.abs(s - amax / 448) <= np.max(off, axis=1, keepdims=True) / 448 + 2.0 ** -23 * s).all()
        from _rows8 import half_step
        from oracle.codecs import e4m3_decode
        q = np.clip(want / s, -448, 448)
        assert (np.abs(e4m3_decode(data[rows].cpu().numpy()) - q) <= half_step(q) + off / s + 2.0 ** -22 * np.abs(q)).all()
    elif fmt == "fp4":   # a code is within half of its grid's widest step there: 1 of 6 of the row's largest value
        s = np64(scale[rows])
        amax = np.max(np.abs(want), axis=1)
        assert (np.abs(s - amax / 6) <= np.max(off, axis=1) / 6 + 2.0 ** -23 * s).all()
        got = fp4_dequantize_rows(data[rows].cpu().numpy(), s)
        step = np.where(np.abs(want) < 2 * s[:, None], 0.25, np.where(np.abs(want) < 4 * s[:, None], 0.5, 1.0)) * s[:, None]
        assert (np.abs(got - want) <= step + off + 2.0 ** -22 * np.abs(want)).all()
    else:   # the block's scale is e4m3: within 2^-4 of amax / 6; a code within half a step of 2 scales
        got = torch.empty((n, dim), dtype=torch.bfloat16, device="cuda")
        dsa.dsa_cache_read(pool, dsa.block_table(bt), ints(req), ints(pos), got)
        blk = np.repeat(np.max(np.abs(want).reshape(n, -1, 16), axis=-1), 16, axis=1)
        assert (np.abs(np64(got) - want) <= blk * (1 + 2.0 ** -4) / 6 + blk * 2.0 ** -4 + off).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4_block"])
def test_append_without_norm_has_the_bytes_of_the_compressors_window_insert(fmt):
    spec = synth.CaseSpec("append_like_compress", cached=[700, 1500, 3], new=[1, 37, 260], seed=5, main_dtype=fmt,
                          swa_dtype=fmt)
    step = LayerStep(synth.make_case(spec, "cuda"))
    step.compress_main()
    want = step.case["swa_data"].clone()
    want_scale = None if step.case["swa_scale"] is None else step.case["swa_scale"].clone()
    again = synth.make_case(spec, "cuda")
    swa = dsa.pool(again["swa_data"], 256, again["swa_scale"], fmt=fmt)
    dsa.dsa_cache_append(again["cu_new"], again["start_pos"], again["x_new"], dsa.rope(64, 10000.0), swa,
                         dsa.block_table(again["bt_swa"]))
    torch.cuda.synchronize()
    assert torch.equal(again["swa_data"].view(torch.uint8), want.view(torch.uint8))
    assert want_scale is None or torch.equal(again["swa_scale"], want_scale)


def test_append_bad_pages_and_strides():
    """Rows without a page raise DSA_ERR_DEVICE_FAULT and are left out, the others are written; rows of a wider buffer."""
    g = gen(21)
    starts, counts = [250, 10, -4, 1200], [20, 5, 6, 4]
    cu, req, pos = schedule(starts, counts)
    bt = ints([[0, -1, 2, -1, -1], [9, 3, 1, 1, 1], [3, 1, 1, 1, 1], [1, 1, 1, 1, 4]])   # 9: beyond the pool
    pool, data, _ = make_pool(5, 128, "bf16")
    before = data.clone()
    wide = randn(g, int(cu[-1]), 3 * 128).to(torch.bfloat16)
    x = wide[:, 128:256]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_append(ints(cu), ints(starts), x, dsa.rope(64, 10000.0), pool, dsa.block_table(bt), norm=True,
                         dev_status=status)
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    good = [j for j in range(len(pos)) if (req[j] == 0 and pos[j] < 256) or (req[j] == 3 and pos[j] < 1280)]
    rows = [0 * 256 + pos[j] if req[j] == 0 else 4 * 256 + pos[j] - 1024 for j in good]
    want = OP.append_rows(np64(x)[good], pos[good], None, EPS, True, 64)
    assert np.allclose(np64(data[rows]), want, rtol=BF16 * 1.01, atol=1e-5)
    left = np.setdiff1d(np.arange(5 * 256), rows)
    assert torch.equal(data[left].view(torch.uint8), before[left].view(torch.uint8))
