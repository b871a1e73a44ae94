"""dsa_gemm_q8, many rows: a pair of CTAs that takes tile after tile, each tile's outputs leaving shared memory by a bulk copy while
the next tile's are on their way there.  Few blocks along k make the tiles follow one another closely."""
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from test_projections import check_gemm, gen, new_out, rows8, weights8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,groups", [(4096, 8192, 16, 1), (4096, 8192, 128, 1), (4000, 8208, 128, 1), (3000, 1040, 144, 5)])
@pytest.mark.parametrize("fmt", ["fp8", "bf16", "f32"])
def test_gemm_tile_after_tile(m, n, k, groups, fmt):
    """Four to seven tiles a pair, alone and again beside a stream that keeps the memory busy: against float64, and the same bits
    every time."""
    g = gen(m + n + k)
    assert dsa.dsa_gemm_q8_plan(m, n, k, groups) == (256, 256, 2)
    a, a_scale = rows8(g, m, groups, k)
    w, w_scale = weights8(g, groups, n, k)
    first, first_scale = new_out(m, groups, n, fmt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_gemm_q8(a, a_scale, w, w_scale, first, first_scale, dev_status=status)
    check_gemm(a, a_scale, w, w_scale, first, first_scale)
    busy = torch.cuda.Stream()
    big = torch.zeros((2, 1 << 28), dtype=torch.uint8, device="cuda")
    busy.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        with torch.cuda.stream(busy):
            for _ in range(4):
                big[0].copy_(big[1])
        out, out_scale = new_out(m, groups, n, fmt)
        for _ in range(4):
            dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale, dev_status=status)
        assert torch.equal(out.view(torch.uint8), first.view(torch.uint8))
        assert out_scale is None or torch.equal(out_scale, first_scale)
    torch.cuda.synchronize()
    assert int(status) == 0
