"""Calls over 4-bit cache rows that their documentation allows and that meet the edges of the plan, of the block tables and of
the format: positions beyond a table, sizes planned for other lengths, refusals, waits that run out, signed zeros.

Tolerances are those of test_cache_fp4_block (derived there) unless a test states its own."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from test_cache_fp4_block import D, F, S, _attn_case, _check, _expected, _on_gpu, _run
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
