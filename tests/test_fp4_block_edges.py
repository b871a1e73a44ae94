"""Calls over 4-bit cache rows that their documentation allows and that meet the edges of the plan, of the block tables and of
the format: positions beyond a table, sizes planned for other lengths, refusals, waits that run out, signed zeros.

Tolerances are those of test_cache_fp4_block (derived there) unless a test states its own."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from compressed_sparse_attention_c4a_gb300 import synth
from oracle import codecs
from test_cache_fp4_block import (D, F, S, SM, _attn_case, _awkward_rows, _check, _expected, _on_gpu, _paged, _pools, _run,
                                  _schedule)
from _parity import np64

gpu = pytest.mark.gpu


# ---- positions beyond the block table ---------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("rows,heads,kind", [(90, 64, "c4a"), (170, 16, "c128a"), (3, 64, "c4a")])
def test_positions_beyond_the_block_table_cost_no_more_than_the_table(rows, heads, kind):
    """Attention over every visible entry: a position one block past the main table (its window mapped), and the largest
    position there is.  Both rows are zeros with the device status, the others right, and the call takes no longer than its
    planned tiles: 2^31 - 1 would be 536,870,904 entries of c4a, 11 million tiles, more than ten seconds."""
    spec = S("beyond", kind=kind, cached=[1000] * rows, new=[1] * rows, heads=heads, topk=0,
             idx_heads=0, seed=33, **F)
    case = _attn_case(spec, None, seed=3)
    mb = case["bt_main"].shape[1]
    case["bt_swa"] = torch.cat([case["bt_swa"], torch.zeros((rows, mb + 1 - case["bt_swa"].shape[1]), dtype=torch.int32)], 1)
    case["q_pos"][0] = 256 * mb + 255
    case["q_pos"][rows - 1] = 2 ** 31 - 1
    dev = _on_gpu(case)
    ok = dict(case, q_pos=torch.full_like(case["q_pos"], 900))
    _run(ok, _on_gpu(ok))                                            # loads the kernels
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    out, lse, status, _ = _run(case, dev)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 500.0
    assert int(status) == dsa.DSA_ERR_DEVICE_FAULT
    for j in (0, rows - 1):
        assert not np64(out[j]).any() and np.isneginf(np64(lse[j])).all(), j
    _check(out, lse, _expected(case, range(1, rows - 1, max(1, rows // 12))))


# ---- the workspace ------------------------------------------------------------------------------------------------------
def _need(rows, heads, keys, fmt):
    """Bytes of split partials that a call of exactly these sizes needs (its plan; 516 floats per row, split and head)."""
    _, _, splits, _ = dsa.dsa_attn_plan(rows, heads, keys, fmt)
    return rows * splits * heads * 516 * 4 if splits > 1 else 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4_block"])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_a_workspace_sized_for_more_keys_serves_fewer(fmt, heads):
    """dsa_attn_workspace_size covers every call of at most max_keys keys, whatever the pool's format: the split counts of the
    plans rise and fall with the key count (host arithmetic)."""
    for rows in (1, 2, 3, 4, 7, 8, 12, 16, 19, 37, 77, 153):
        most = 0
        for keys in sorted(set(range(1, 9000, 61)) | set(range(48, 9000, 96)) | set(range(47, 2400, 48))):
            most = max(most, _need(rows, heads, keys, fmt))
            size = dsa.dsa_attn_workspace_size(rows, heads, keys)
            assert size >= most, (rows, keys, size, most)
    # no more than the largest need of any format up to there
    for rows, keys in ((1, 700), (4, 1300), (19, 640), (200, 640)):
        largest = max(_need(rows, heads, k, f) for k in range(1, keys + 1) for f in ("bf16", "fp8", "fp4_block"))
        assert dsa.dsa_attn_workspace_size(rows, heads, keys) == largest


def test_workspace_size_of_the_longest_lengths():
    """Sizes near the largest int are answered at once and do not fall."""
    for rows in (1, 5, 36, 1000):
        size = dsa.dsa_attn_workspace_size(rows, 64, 8320)
        for keys in (10 ** 6, 2 ** 31 - 2048, 2 ** 31 - 1):
            assert dsa.dsa_attn_workspace_size(rows, 64, keys) >= size


# ---- waits that run out -------------------------------------------------------------------------------------------------
def test_stalled_attention_refuses_a_row_outside_the_call():
    import ctypes
    P, f = ctypes.c_void_p, dsa._lib.dsa_debug_sparse_attn_stalled
    bt, rope = dsa.DsaBlockTable(64, 2, 4), dsa.DsaRope(64, 10000.0)
    main, swa = dsa.DsaPool(256, 512, 4, 64, 512, dsa.DSA_FP4_BLOCK), dsa.DsaPool(256, 512, 4, 256, 512, dsa.DSA_FP4_BLOCK)
    for row in (-1, 2, 2 ** 31 - 1):
        assert f(2, 64, P(16), P(16), None, 0, P(16), 8, ctypes.byref(main), ctypes.byref(bt), ctypes.byref(swa),
                 ctypes.byref(bt), 128, 0.044, ctypes.byref(rope), P(16), None, None, 0, row, None, None) == \
            dsa.DSA_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("fmt,rows,heads,topk", [("fp4_block", 400, 64, 150), ("fp4_block", 330, 16, 1), ("fp4_block", 3, 64, 200),
                                                 ("fp4_block", 40, 64, 200), ("bf16", 3, 64, 500), ("bf16", 40, 64, 200),
                                                 ("fp8", 200, 32, 100)])
def test_rows_that_a_wait_kept_from_being_finished_are_zeros(fmt, rows, heads, topk):
    """A row whose queries never arrive in its last CTAs: the waits run out after two seconds, the kernel returns and records
    it, the row (of 4-bit rows taken one after another: and those that its CTA would have taken next) is zeros with lse -inf,
    whole clusters and splits of keys included; every other row has the bits of a normal call, and so has the next call."""
    spec = S("stalled", cached=[2500 + i for i in range(rows)], new=[1] * rows, heads=heads, topk=topk, window=100, seed=12,
             main_dtype=fmt, swa_dtype=fmt)
    case = _attn_case(spec, "random", seed=2)
    dev = _on_gpu(case)
    want, want_lse, status, ws = _run(case, dev)
    torch.cuda.synchronize()
    assert int(status) == 0 and bool(torch.isfinite(want_lse).all())
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _, cluster, splits, _ = dsa.dsa_attn_plan(rows, heads, topk + 100, fmt)
    in_turn = fmt == "fp4_block" and cluster == 1 and splits == 1
    stall = (sms + 3 if in_turn else rows // 2)
    lost = list(range(stall, rows, sms)) if in_turn else [stall]
    out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
    main, bt, swa, sbt = _pools(case, dev)
    dsa.dsa_debug_sparse_attn_stalled(dev["q"], dev["q_pos"], None, spec.kind, dev["topk"], topk, main, bt, swa, sbt, 100, SM,
                                      dsa.rope(64), out, stall, lse, ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == dsa.DSA_ERR_TIMEOUT
    keep = torch.ones(rows, dtype=torch.bool)
    keep[lost] = False
    assert not bool(out[lost].any()) and bool(torch.isneginf(lse[lost]).all())
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    again, again_lse, status, _ = _run(case, dev)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(again, want) and torch.equal(again_lse, want_lse)


# ---- refusals ---------------------------------------------------------------------------------------------------------------
@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: only where no launch can follow")
@pytest.mark.parametrize("dtype", [dsa.DSA_FP4_BLOCK, dsa.DSA_BF16])
def test_topk_and_attention_in_one_call_refuse_before_anything_is_launched(dtype):
    """Where the call is two launches, what the attention refuses is refused before the top-k runs: nothing is launched and no
    memory is touched (without a GPU a launch would answer DSA_ERR_CUDA instead)."""
    import ctypes
    P, f = ctypes.c_void_p, dsa._lib.dsa_topk_sparse_attn_decode
    bt, rope = dsa.DsaBlockTable(64, 2, 64), dsa.DsaRope(64, 10000.0)
    pool = lambda epb, dim=512, d=dtype: dsa.DsaPool(256, 512, 4, epb, dim, d)  # noqa: E731
    assert dsa.dsa_attn_plan(1, 16, 512 + 128, dtype)[2] > 1                    # needs a workspace

    def call(main=pool(64), swa=pool(256), q=P(16), out=P(16), sm=0.044, ws=P(256), ws_bytes=1 << 30):
        return f(1, 16, q, P(16), 0, P(16), 4096, P(16), 512, P(16), ctypes.byref(main), ctypes.byref(bt), ctypes.byref(swa),
                 ctypes.byref(bt), 128, sm, ctypes.byref(rope), out, None, ws, ws_bytes, None, None)

    INV, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    assert call(ws=None, ws_bytes=0) == INV and call(ws_bytes=16) == INV and call(ws=P(16)) == INV
    assert call(q=None) == INV and call(q=P(8)) == INV and call(out=None) == INV and call(sm=0.0) == INV
    assert call(swa=pool(128)) == INV and call(main=pool(64, dim=128)) == UNS
    other = dsa.DSA_FP8_E4M3
    assert call(swa=pool(256, d=other)) == UNS


def test_binding_block_table_takes_the_first_two_sizes():
    """A table may carry a trailing dimension of one; one dimension alone is no table."""
    t = torch.zeros((3, 5, 1), dtype=torch.int32)
    bt = dsa.block_table(t)
    assert (bt.batch, bt.max_blocks, bt.table) == (3, 5, t.data_ptr())
    with pytest.raises(IndexError):
        dsa.block_table(torch.zeros(5, dtype=torch.int32))


# ---- the sign of a zero ---------------------------------------------------------------------------------------------------
def _rows_around_zero(n, seed):
    """bf16 rows with negative values that round to zero, negative zeros, and blocks whose scale rounds to zero."""
    x = _awkward_rows(n, seed).float()
    x[:, ::5] = -x[:, ::5].abs() * 2.0 ** -9
    x[:, 1::7] = -0.0
    x[:, 3::11] = -x[:, 3::11].abs() * 2.0 ** -24
    x[1::2, 64:96] = -2.0 ** -120
    return x.to(torch.bfloat16)


def test_oracle_writes_zero_codes_without_a_sign():
    data, _ = codecs.fp4_block_quantize_rows(np64(_rows_around_zero(24, 4)))
    assert not ((data[:, :256] & 15) == 8).any() and not ((data[:, :256] >> 4) == 8).any()


@gpu
@pytest.mark.parametrize("n", [40, 10500])
def test_stored_bytes_are_the_oracles_zero_codes_included(n):
    """A row a warp and four rows a warp: every byte and scale equal the oracle's, where a code of magnitude zero is 0."""
    x = _rows_around_zero(n, 6)
    bt, blocks = _paged([n], [0], 64, 2)
    gd, gs = torch.full((blocks * 64, 288), 17, dtype=torch.uint8, device="cuda"), torch.zeros(blocks * 64, device="cuda")
    cu, start = _schedule([n], [0])
    table = bt.cuda()
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), dsa.pool(gd, 64, gs, fmt="fp4_block"), dsa.block_table(table))
    torch.cuda.synchronize()
    rows = (bt[0].long()[:, None] * 64 + torch.arange(64)).flatten()[:n].numpy()
    want, ws = codecs.fp4_block_quantize_rows(np64(x))
    assert np.array_equal(gd.cpu().numpy()[rows], want) and np.array_equal(np64(gs)[rows], ws)


@gpu
def test_compressor_stores_zero_codes_without_a_sign():
    from compressed_sparse_attention_c4a_gb300.step import LayerStep
    spec = S("zeros", cached=[1000, 6, 0], new=[1, 1, 40], queries="all", idx_heads=0, topk=0, seed=42, **F)
    case = synth.make_case(spec, "cpu")
    case["x_new"][:, ::3] = -case["x_new"][:, ::3].abs() * 2.0 ** -12
    for k in ("main_data", "swa_data"):
        case[k].zero_()                                     # what is not written holds no sign
    dev = _on_gpu(case)
    step = LayerStep(dev)
    step.compress_main()
    torch.cuda.synchronize()
    assert int(step.status) == 0
    for k in ("main_data", "swa_data"):
        codes = dev[k].cpu().numpy()[:, :256]
        assert (codes >> 4 > 8).any() and ((codes & 15) == 0).any()
        assert not ((codes & 15) == 8).any() and not ((codes >> 4) == 8).any()


# ---- the normaliser ---------------------------------------------------------------------------------------------------------
def _one_value_case(rows, heads):
    """Every key holds 1 in dims 0 .. 255; one entry, in a row's second tile, also holds 1 in dim 256, the only dim of the
    queries that is not zero: its logit is up to 7.9 powers of two above the others', within the lazy maximum's margin."""
    spec = S("one_value", cached=[1000] * rows, new=[1] * rows, heads=heads, topk=64, window=1, seed=3, **F)
    case = _attn_case(spec, "random", seed=1)
    for k in ("main", "swa"):
        case[k + "_data"][:] = 0
        case[k + "_data"][:, :128] = 0x22                   # two codes of 1
        case[k + "_data"][:, 256:] = 0x38                   # block scales of 1
        case[k + "_scale"][:] = 1.0
    tk = torch.full((rows, 64), -1, dtype=torch.int32)
    tk[:, 0], tk[:, 60] = 3, 200
    for j in range(rows):
        case["main_data"][int(case["bt_main"][j, 200 // 64]) * 64 + 200 % 64, 128] = 0x02
    case["topk"] = tk
    x = torch.linspace(0.1, 7.9, rows * heads)[torch.randperm(rows * heads, generator=torch.Generator().manual_seed(5))]
    q = torch.zeros((rows, heads, D))
    q[:, :, 256] = (x / (SM * np.log2(np.e))).view(rows, heads)
    case["q"] = q.to(torch.bfloat16)
    return case


@gpu
@pytest.mark.parametrize("rows,heads", [(160, 64), (330, 16)])
def test_weights_add_up_to_one_whatever_their_rounding(rows, heads):
    """Values that all keys share come out exactly: the probabilities are rounded to bf16 before they multiply the values, and
    the normaliser sums them as rounded.  In fp32 the three weights, their sum, its reciprocal and the product are off by a few
    2^-24, far less than 2^-9, half a bf16 step below 1.  (Summed before the rounding they differ by up to 2^-8.)  In e4m3 the
    value is 448 times the block's scale.  The log-sum-exp is that of the probabilities before the rounding."""
    case = _one_value_case(rows, heads)
    dev = _on_gpu(case)
    out, lse, status, ws = _run(case, dev)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert dsa.dsa_attn_plan(rows, heads, 65, "fp4_block")[1:3] == (1, 1)       # a row in one CTA: nothing is exchanged
    assert bool((out[:, :, :256] == 1.0).all())
    want = _expected(case, range(0, rows, 40))
    _check(out, lse, want)
    main, bt, swa, sbt = _pools(case, dev)
    o8 = torch.zeros((rows, heads, D), dtype=torch.uint8, device="cuda")
    s8 = torch.zeros((rows, heads, 4), device="cuda")
    dsa.dsa_sparse_attn_q8(dev["q"], dev["q_pos"], dev["q_req"], "c4a", dev["topk"], 64, main, bt, swa, sbt, 1, SM,
                           dsa.rope(64), o8, s8, lse, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and bool((o8[:, :, :256] == 0x7E).all())            # 448
    assert bool(((s8[:, :, :2] * 448.0 - 1.0).abs() <= 2.0 ** -20).all())


# ---- the ends of the range ------------------------------------------------------------------------------------------------
@gpu
def test_values_at_the_ends_of_the_range_read_back_rounded():
    """Rows of the smallest scales, whose values' lowest bits lie below bf16's smallest subnormal: rounded to nearest even, and
    exact where scale times block scale is at least 2^-129.  Rows of bf16's largest magnitudes: 2016 * 2^117 and below come
    back finite, above it as infinities (2112 * 2^117 is beyond fp32)."""
    g = np.random.default_rng(8)
    n = 64
    codes = g.integers(0, 256, (n, 256)).astype(np.uint8)
    codes[(codes & 15) == 8] &= 0xF0
    bs = np.where(g.random((n, 32)) < 0.5, g.integers(0, 16, (n, 32)), g.integers(0, 127, (n, 32))).astype(np.uint8)
    data, scale = np.concatenate([codes, bs], 1), 2.0 ** g.integers(-126, -115, n)
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    gd, gs = torch.tensor(data).cuda(), torch.tensor(scale, dtype=torch.float32).cuda()
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.empty((n, D), dtype=torch.bfloat16, device="cuda")
    pool = dsa.pool(gd, 64, gs, fmt="fp4_block")
    dsa.dsa_cache_read(pool, dsa.block_table(bt), torch.zeros_like(ids), ids, out)
    vals = codecs.fp4_block_dequantize_rows(data, scale)
    assert torch.equal(out.cpu().float(), torch.tensor(vals).to(torch.float32).to(torch.bfloat16).float())
    exact = np.repeat(scale[:, None] * codecs.e4m3_decode(bs) >= 2.0 ** -129, 16, axis=1)
    assert exact.any() and not exact.all() and np.array_equal(np64(out)[exact], vals[exact])
    assert not np.array_equal(np64(out), vals)
    # the largest
    tops = torch.tensor([0x7F7C, 0x7F7D, 0x7F7E, 0x7F7F], dtype=torch.int16).view(torch.bfloat16)   # 2016 2^117, then above
    x = torch.zeros((4, D), dtype=torch.bfloat16)
    x[:, 7] = tops
    cu, start = _schedule([4], [0])
    dsa.dsa_cache_write(cu.cuda(), start.cuda(), x.cuda(), pool, dsa.block_table(bt))
    dsa.dsa_cache_read(pool, dsa.block_table(bt), torch.zeros_like(ids), ids, out)
    got = out[:4].float().cpu()
    assert float(got[0, 7]) == 1920 * 2.0 ** 117 and bool(torch.isinf(got[1:, 7]).all())
    got[:, 7] = 0
    assert not bool(got.any())


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: only where no launch can follow")
@pytest.mark.parametrize("dtype", [dsa.DSA_FP4_BLOCK, dsa.DSA_BF16])
@pytest.mark.parametrize("max_blocks", [2 ** 25, 2 ** 26, 2 ** 31 - 1])
def test_a_table_of_more_entries_than_an_int_holds_is_planned_as_a_long_one(dtype, max_blocks):
    """Attention over every visible entry under a table of 2^31 entries or more: the plan is a long row's (its key splits need
    a workspace, and without one the call is refused), not that of what is left of the product modulo 2^32, whose few tiles
    would leave most keys out.  Without a GPU a launch would answer DSA_ERR_CUDA instead."""
    import ctypes
    P, rope = ctypes.c_void_p, dsa.DsaRope(64, 10000.0)
    bt, swa_bt = dsa.DsaBlockTable(64, 2, max_blocks), dsa.DsaBlockTable(64, 2, 64)
    main, swa = dsa.DsaPool(256, 512, 4, 64, 512, dtype), dsa.DsaPool(256, 512, 4, 256, 512, dtype)
    assert dsa.dsa_attn_workspace_size(1, 64, 2 ** 30) > 0
    got = dsa._lib.dsa_sparse_attn_decode(1, 64, P(16), P(16), 0, None, 0, ctypes.byref(main), ctypes.byref(bt),
                                          ctypes.byref(swa), ctypes.byref(swa_bt), 128, 0.044, ctypes.byref(rope), P(16), None,
                                          None, 0, None, None)
    assert got == dsa.DSA_ERR_INVALID_ARG
