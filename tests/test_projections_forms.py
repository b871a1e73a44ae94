"""The forms of the product that the tests reach, what a repeated call repeats, and the launches of the step between its projections."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa
from test_projected_step import SPECS, make
from test_projections import SHAPES, check_gemm, gen, new_out, rows8, weights8

pytestmark = pytest.mark.gpu

SHARED = [(500, 1537, 4096, 2), (600, 2100, 4112, 1)]   # two pairs of CTAs to a tile


def test_the_shapes_reach_every_form():
    plans = {dsa.dsa_gemm_q8_plan(*s) for s in SHAPES + SHARED}
    assert plans >= {(128, rows, share) for rows in (16, 32) for share in (1, 2, 4, 8)} | {(256, 256, 2), (256, 256, 4)}


@pytest.mark.parametrize("m,n,k,groups", SHARED + [(32, 1024, 4096, 8), (300, 640, 384, 1), (700, 300, 272, 16)])
@pytest.mark.parametrize("fmt", ["f32", "bf16", "fp8"])
def test_the_same_call_gives_the_same_codes_and_scales(m, n, k, groups, fmt):
    g = gen(m + n)
    a, a_scale = rows8(g, m, groups, k)
    w, w_scale = weights8(g, groups, n, k)
    outs = [new_out(m, groups, n, fmt) for _ in range(5)]
    for out, out_scale in outs:
        dsa.dsa_gemm_q8(a, a_scale, w, w_scale, out, out_scale)
    check_gemm(a, a_scale, w, w_scale, *outs[0])
    for out, out_scale in outs[1:]:
        assert torch.equal(out.view(torch.uint8), outs[0][0].view(torch.uint8))
        assert out_scale is None or torch.equal(out_scale, outs[0][1])


def kernel_nodes(run):
    """Kernels of what `run` launches on the current stream, counted in a captured graph."""
    rt = ctypes.CDLL("libcudart.so.13")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        run()
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    count = ctypes.c_size_t()
    assert rt.cudaGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert rt.cudaGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    kinds = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        assert rt.cudaGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    return kinds.count(0)   # cudaGraphNodeTypeKernel


@pytest.mark.parametrize("name", list(SPECS))
def test_projected_step_launches_what_it_says(name):
    step, x = make(name)
    step.run(x)
    torch.cuda.synchronize()
    assert kernel_nodes(lambda: step.run(x)) == step.launches_per_step()
