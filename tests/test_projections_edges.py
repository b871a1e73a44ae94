"""The operators around the attention where sizes are large or odd: offsets beyond 32 bits, many requests and empty ones,
outputs at every alignment, products in several forms side by side."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from oracle import projection as OP
from oracle.codecs import e4m3_decode
from _parity import np64
from _rows8 import half_step
from test_projections import (BF16, EPS, NORM_OFF, check_gemm, check_norm, gen, ints, make_pool, new_out, physical, randn, rows8,
                              run_norm, schedule, tables, weights8)

pytestmark = pytest.mark.gpu


def test_norm_rows_far_apart():
    """Rows 2^22 values apart: the last ones lie beyond 2^31 values (and 2^32 bytes)."""
    n, d, ld = 530, 272, 1 << 22
    g = gen(1)
    wide = torch.empty((n, ld), dtype=torch.bfloat16, device="cuda")
    x, total = wide[:, 64:64 + d], wide[:, 1024:1024 + d]
    x.copy_(randn(g, n, d))
    r = randn(g, n, d).to(torch.bfloat16)
    out, scale, total = run_norm(x, r, None, sum_out=total)
    check_norm(x, r, None, out, scale, total)


@pytest.mark.parametrize("m,n,k", [(530, 40, 128), (530, 4000, 128)])   # few rows' form, and pairs
def test_gemm_rows_far_apart(m, n, k):
    g = gen(2)
    m = m if n < 100 else 2 * m + 240
    ld = 1 << 22 if m < 1000 else 1 << 21
    form = dsa.dsa_gemm_q8_plan(m, n, k)[0]
    assert form == (128 if n < 100 else 256)
    a, a_scale = rows8(g, m, 1, k)
    far = torch.empty((m, 1, ld), dtype=torch.uint8, device="cuda")[:, :, 32:32 + k]
    far.copy_(a)
    w, w_scale = weights8(g, 1, n, k)
    out = torch.empty((m, 1, ld), dtype=torch.bfloat16, device="cuda")[:, :, 8:8 + n]
    dsa.dsa_gemm_q8(far, a_scale, w, w_scale, out)
    check_gemm(a, a_scale, w, w_scale, out, None)


@pytest.mark.parametrize("dim,fmt", [(512, "bf16"), (512, "fp8"), (512, "fp4_block"), (128, "bf16")])
def test_append_beyond_32_bits_of_a_pool(dim, fmt):
    """Blocks at both ends of a pool of more than 2^32 bytes."""
    row = {"bf16": 2 * dim, "fp8": dim, "fp4_block": dim // 16 * 9}[fmt]
    blocks = (1 << 32) // (256 * row) + 5
    rows = blocks * 256
    data = torch.empty((rows, dim if fmt == "bf16" else row), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")
    scale = None if fmt == "bf16" else torch.empty((rows,), device="cuda")
    pool = dsa.pool(data, 256, scale, fmt="fp4_block" if fmt == "fp4_block" else None)
    g = gen(3)
    bt = ints([[blocks - 1, 0], [blocks - 2, 1]])
    starts, counts = [250, 3], [20, 7]
    cu, req, pos = schedule(starts, counts)
    x = randn(g, int(cu[-1]), dim).to(torch.bfloat16)
    dsa.dsa_cache_append(ints(cu), ints(starts), x, dsa.rope(64), pool, dsa.block_table(bt), norm=True)
    got = torch.empty_like(x)
    dsa.dsa_cache_read(pool, dsa.block_table(bt), ints(req), ints(pos), got)
    want = OP.append_rows(np64(x), pos, None, EPS, True, 64)
    room = {"bf16": BF16, "fp8": 2.0 ** -4 + BF16, "fp4_block": 0.5}[fmt]
    assert (np.abs(np64(got) - want) <= room * np.abs(want) + (1e-5 if fmt == "bf16" else 2.0 ** -10 * 0.02 + (0.5 if fmt == "fp4_block" else 0.001))).all()


def test_append_many_requests_with_empty_ones():
    """3,000 requests of 0 to 3 rows, some thousand of them empty in a row."""
    g = gen(4)
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 4, 3000)
    counts[500:1700] = 0
    counts[-5:] = 0
    starts = rng.integers(0, 600, 3000)
    cu, req, pos = schedule(list(starts), list(counts))
    bt, blocks = tables(list(starts), list(counts), g)
    for fmt, dim in (("bf16", 512), ("fp8", 128)):
        pool, data, scale = make_pool(blocks, dim, fmt)
        x = randn(g, int(cu[-1]), dim).to(torch.bfloat16)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dsa.dsa_cache_append(ints(cu), ints(starts), x, dsa.rope(64), pool, dsa.block_table(bt), dev_status=status)
        assert int(status) == 0
        want = OP.append_rows(np64(x), pos, None, EPS, False, 64)
        rows = physical(bt, req, pos)
        if fmt == "bf16":
            assert (np.abs(np64(data[rows]) - want) <= BF16 * np.abs(want) + 1e-5).all()
        else:
            got = torch.empty_like(x)
            dsa.dsa_cache_read(pool, dsa.block_table(bt), ints(req), ints(pos), got)
            assert (np.abs(np64(got) - want) <= (2.0 ** -4 + BF16) * np.abs(want) + 0.001 * np.max(np.abs(want))).all()


@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4, 8, 16])
@pytest.mark.parametrize("m,n", [(9, 131), (2050, 2300)])
def test_gemm_outputs_at_every_alignment(fmt, shift, m, n):
    """Outputs that begin `shift` elements into a row, rows an odd or even number of elements apart."""
    k = 144
    g = gen(5 + shift)
    a, a_scale = rows8(g, m, 1, k)
    w, w_scale = weights8(g, 1, n, k)
    base, scale = new_out(m, 1, n, fmt)
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, base, out_scale=scale)
    for extra in (0, 5, 48 - n % 16):
        wide = torch.full((m, 1, n + 16 + extra), 3, dtype=base.dtype, device="cuda")
        out = wide[:, :, shift:shift + n]
        again = None if scale is None else torch.empty_like(scale)
        dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale=again)
        assert torch.equal(out.view(torch.uint8) if fmt == "fp8" else out, base)
        assert (wide[:, :, :shift] == 3).all() and (wide[:, :, shift + n:] == 3).all()
        assert scale is None or torch.equal(again, scale)


def test_gemm_scales_at_every_alignment():
    """Rows' scales that do not lie on 16 bytes (the pairs' form reads eight of them at once where they do)."""
    m, n, k = 2050, 2300, 1168   # ten blocks
    g = gen(6)
    a, a_scale = rows8(g, m, 1, k)
    w, w_scale = weights8(g, 1, n, k)
    base, _ = new_out(m, 1, n, "f32")
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, base)
    for pad, shift in ((2, 0), (2, 1), (6, 4), (0, 0)):
        wide = torch.zeros((m, 1, 10 + pad + shift), device="cuda")
        scale = wide[:, :, shift:shift + 10]
        scale.copy_(a_scale)
        out, _ = new_out(m, 1, n, "f32")
        dsa.dsa_gemm_q8(a, scale, w, w_scale, out)
        assert torch.equal(out, base)


def test_products_of_both_forms_at_once():
    """Products of few rows and of many on three streams at the same time, each as alone."""
    g = gen(7)
    shapes = [(32, 2048, 4096, 2), (2100, 2048, 528, 1), (300, 1000, 1040, 1)]
    data = [(*rows8(g, m, gr, k), *weights8(g, gr, n, k)) for m, n, k, gr in shapes]
    alone = [new_out(m, gr, n, "bf16")[0] for m, n, k, gr in shapes]
    for d, o in zip(data, alone):
        dsa.dsa_gemm_q8(*d, o)
        torch.cuda.synchronize()
    outs = [torch.empty_like(o) for o in alone]
    streams = [torch.cuda.Stream() for _ in shapes]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for d, o, s in zip(data, outs, streams):
            dsa.dsa_gemm_q8(*d, o, stream=s)
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o, want)


def test_no_rows_and_one_value():
    """Calls without rows leave everything as it was; the smallest sizes."""
    g = gen(8)
    w, w_scale = weights8(g, 1, 3, 16)
    out = torch.empty((0, 1, 3), device="cuda")
    dsa.dsa_gemm_q8(torch.empty((0, 1, 16), dtype=torch.uint8, device="cuda"), torch.empty((0, 1, 1), device="cuda"), w, w_scale, out)
    dsa.dsa_norm_q8(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), None, EPS, torch.empty((0, 64), dtype=torch.uint8, device="cuda"),
                    torch.empty((0, 1), device="cuda"))
    a, a_scale = rows8(g, 1, 16)
    one = torch.empty((1, 1), device="cuda")
    dsa.dsa_gemm_q8(a, a_scale, w[0, :1], w_scale[0, :1], one)     # no dimension for the groups
    check_gemm(a[:, None], a_scale[:, None], w[:, :1], w_scale, one[:, None], None)


def test_norm_of_one_row_is_the_row_of_many():
    """A row's result does not depend on the rows around it."""
    g = gen(9)
    for dim in (400, 2000, 4096, 8192):
        x = randn(g, 1000, dim).to(torch.bfloat16)
        r = randn(g, 1000, dim).to(torch.bfloat16)
        many = run_norm(x, r, None)
        one = run_norm(x[777:778], r[777:778], None)
        for a, b in zip(many, one):
            assert torch.equal(a[777:778], b)
        check_norm(x[777:778], r[777:778], None, *one)
    assert NORM_OFF < 1e-5


@pytest.mark.parametrize("fmt,dim", [("bf16", 512), ("fp8", 512), ("bf16", 128), ("fp8", 64)])
def test_append_norms_rows_of_huge_and_tiny_values(fmt, dim):
    """Rows whose squares leave fp32 at either end, of zeros, and with one value that outweighs the others."""
    g = gen(dim)
    x = randn(g, 9, dim).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** 70
    x[2] *= 2.0 ** 122
    x[3] *= 2.0 ** -100
    x[4, 5] = 3e38
    x[5, :] = -3.3e38
    x[6] *= 2.0 ** 60
    x[7] *= 2.0 ** -40
    gamma = 1 + 0.2 * randn(g, dim)
    cu, req, pos = schedule([250], [9])
    bt, blocks = tables([250], [9], g)
    pool, data, scale = make_pool(blocks, dim, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_cache_append(ints(cu), ints([250]), x, dsa.rope(64), pool, dsa.block_table(bt), norm=True, rms_gamma=gamma,
                         rms_eps=EPS, dev_status=status)
    assert int(status) == 0
    want = OP.append_rows(np64(x), pos, np64(gamma), EPS, True, 64)
    off = NORM_OFF * np.abs(want)
    tail = want[:, dim - 64:]
    off[:, dim - 64:] = (1e-6 + NORM_OFF) * np.repeat(np.hypot(tail[:, 0::2], tail[:, 1::2]), 2, axis=1)
    rows = physical(bt, req, pos)
    if fmt == "bf16":
        # Below 2^-126 the steps no longer shrink with the value: half of bf16's is 2^-134 there (row 4, whose large value makes
        # the others 2^-123 of theirs), of fp32's 2^-150, a few times
        tiny = np.where(np.abs(want) < 2.0 ** -125, 2.0 ** -134 + 2.0 ** -146, 0)
        err = np.abs(np64(data[rows]) - want) - (BF16 * np.abs(want) + off * (1 + BF16) + tiny)
        worst = np.unravel_index(np.argmax(err), err.shape)
        assert err[worst] <= 0, (worst, err[worst], want[worst])
    else:
        s = np64(scale[rows])[:, None]
        amax = np.max(np.abs(want), axis=1, keepdims=True)
        ideal = np.where(amax > 0, amax / 448, 1.0)
        assert (np.abs(s - ideal) <= np.max(off, axis=1, keepdims=True) / 448 + 2.0 ** -23 * ideal).all()
        q = np.clip(want / s, -448, 448)
        got = e4m3_decode(data[rows].cpu().numpy())
        assert (np.abs(got - q) <= half_step(q) + off / s + 2.0 ** -22 * np.abs(q)).all()


@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("m,n,k,groups", [(2050, 2100, 400, 1), (2050, 2177, 256, 1), (2304, 2304, 1040, 1), (520, 2432, 400, 3),
                                          (300, 900, 2576, 4)])
def test_gemm_last_tiles(m, n, k, groups, fmt):
    """Many rows: last tiles that have no second block of 128 outputs, or a part of either; more tiles than pairs of CTAs and
    fewer; chunks of scales that end early."""
    g = gen(m + n)
    a, a_scale = rows8(g, m, groups, k)
    w, w_scale = weights8(g, groups, n, k)
    out, out_scale = new_out(m, groups, n, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale, dev_status=status)
    assert int(status) == 0
    check_gemm(a, a_scale, w, w_scale, out, out_scale)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("m,n,k,groups", [(500, 2900, 8192, 1), (600, 2100, 4112, 1), (500, 1537, 4096, 2), (1000, 1153, 6160, 1),
                                          (2000, 700, 5120, 1)])
def test_gemm_blocks_shared_by_two_pairs(m, n, k, groups, fmt):
    """Few tiles of many blocks: two pairs of CTAs share a tile's blocks and exchange their sums; ragged rows, outputs and blocks;
    the same bits again."""
    g = gen(m + n)
    a, a_scale = rows8(g, m, groups, k)
    w, w_scale = weights8(g, groups, n, k)
    assert dsa.dsa_gemm_q8_plan(m, n, k, groups) == (256, 256, 4)
    outs = []
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out, out_scale = new_out(m, groups, n, fmt)
        dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale, dev_status=status)
        outs.append(out)
    assert int(status) == 0
    check_gemm(a, a_scale, w, w_scale, out, out_scale)
    assert all(torch.equal(o.view(torch.uint8), out.view(torch.uint8)) for o in outs)


def test_gemm_two_pairs_bounded_waits():
    g = gen(13)
    a, a_scale = rows8(g, 500, 1, 8192)
    w, w_scale = weights8(g, 1, 2900, 8192)
    assert dsa.dsa_gemm_q8_plan(500, 2900, 8192) == (256, 256, 4)
    out, _ = new_out(500, 1, 2900, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_debug_gemm_q8_stalled(a, a_scale, w, w_scale, out, 20_000_000, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_TIMEOUT and not out.any()
    status.zero_()
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, dev_status=status)
    check_gemm(a, a_scale, w, w_scale, out, None)
    assert int(status) == 0


@pytest.mark.parametrize("m,n,k,n2", [(2048, 4096, 2048, 512), (500, 4096, 8192, 1024), (33, 2048, 1024, 4096)])
def test_products_of_products_from_a_graph(m, n, k, n2):
    """8-bit outputs read by the next product, launched before the first has ended: the bits of calls with a wait in between."""
    g = gen(m)
    w, w_scale = weights8(g, 1, n, k)
    w2, w2_scale = weights8(g, 1, n2, n)
    inputs = [rows8(g, m, 1, k) for _ in range(3)]
    mid, mid_scale = new_out(m, 1, n, "fp8")
    outs = [new_out(m, 1, n2, "bf16")[0] for _ in inputs]

    def chain(i, wait=lambda: None):
        dsa.dsa_gemm_q8(*inputs[i], w, w_scale, mid, mid_scale)
        wait()
        dsa.dsa_gemm_q8(mid, mid_scale, w2, w2_scale, outs[i])
        wait()

    for i in range(3):
        chain(i, torch.cuda.synchronize)
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in list(range(3)) * 3:
            chain(i)
    for _ in range(10):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, x) for o, x in zip(outs, want))
