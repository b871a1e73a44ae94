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
