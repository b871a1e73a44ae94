"""The layer step between its projections, as a model runs it: each stage against the oracle over the stage's own inputs as
the GPU left them (an error of one stage does not hide in the next one's)."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import synth
from compressed_sparse_attention_c4a_gb300.step import LayerProjections, ProjectedStep, SM_SCALE
from oracle import attention as OA, layer as OL, projection as OP
from oracle.codecs import e4m3_decode
from _parity import attn_bound, np64, oracle_pool, pool_absmax
from _rows8 import assert_rows8
from test_projections import BF16, NORM_OFF, check_gemm, gen, randn

pytestmark = pytest.mark.gpu

SPECS = {
    "decode": synth.CaseSpec("p_decode", cached=[700, 1500, 8, 0, 4095], new=[1] * 5, heads=64, seed=61),
    "prefill": synth.CaseSpec("p_prefill", cached=[301, 0], new=[70, 40], queries="all", heads=16, seed=62),
    "dense": synth.CaseSpec("p_dense", kind="c128a", cached=[1279, 5000, 127], new=[1] * 3, heads=32, idx_heads=0, topk=0, seed=63),
    "fp8_caches": synth.CaseSpec("p_fp8", cached=[700, 1023], new=[1] * 2, heads=64, main_dtype="fp8", swa_dtype="fp8", seed=64),
}


def weights(g, *shape):
    """Codes [.. n][k] of N(0, 1 / k) values with a scale per 128 x 128."""
    n, k = shape[-2:]
    v = randn(g, *shape) / k ** 0.5
    nb, kb = -(-n // 128), -(-k // 128)
    scale = torch.rand((*shape[:-2], nb, kb), generator=g, device="cuda") * 0.5 / 448 / k ** 0.5 * 8 + 4.0 / 448 / k ** 0.5
    full = scale.repeat_interleave(128, -1)[..., :k].repeat_interleave(128, -2)[..., :n, :]
    return (v / full).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def make(name, hidden=400, rank=256):
    spec = SPECS[name]
    g = gen(spec.seed)
    groups = spec.heads // 8
    proj = LayerProjections(1 + 0.2 * randn(g, hidden), weights(g, spec.heads * 512, hidden), weights(g, 512, hidden),
                            weights(g, groups, rank, 8 * 512), weights(g, hidden, groups * rank), q_norm=1 + 0.2 * randn(g, 512),
                            kv_norm=1 + 0.2 * randn(g, 512))
    case = synth.make_case(spec, "cuda")
    residual = (2 * randn(g, case["nq"], hidden)).to(torch.bfloat16)
    x = randn(g, case["nq"], hidden).to(torch.bfloat16)
    return ProjectedStep(case, proj, residual), x


@pytest.mark.parametrize("name", list(SPECS))
def test_projected_step_matches_the_oracle_stage_by_stage(name):
    step, x = make(name)
    spec, c, p = step.spec, step.case, step.proj
    residual0 = step.residual.clone()
    step.run(x)
    torch.cuda.synchronize()
    assert int(step.status) == 0
    h = np64(x) + np64(residual0)
    v = OP.rms_norm(h, np64(p.norm), p.eps)
    assert_rows8(step.hidden8.cpu().numpy(), np64(step.hidden8_scale), v, NORM_OFF * np.abs(v))
    assert (np.abs(np64(step.residual) - h) <= (BF16 + 2.0 ** -24) * np.abs(h)).all()
    rows8 = (step.hidden8[:, None], step.hidden8_scale[:, None])
    check_gemm(*rows8, p.q[0][None], p.q[1][None], step.q_raw[:, None], None)
    check_gemm(*rows8, p.kv[0][None], p.kv[1][None], step.kv[:, None], None)
    q = OA.query_prep(np64(step.q_raw).reshape(c["nq"], spec.heads, 512), np64(c["q_pos"])[:, None], spec.rope_dim, np64(p.q_norm))
    assert (np.abs(np64(c["q"]) - q) <= BF16 * np.abs(q) + 2e-5 * np.max(np.abs(q))).all()
    # the appended rows
    pos, req = np64(c["q_pos"]), np64(c["q_req"])
    bt = np64(c["bt_swa"])
    rows = bt[req, pos // 256].astype(np.int64) * 256 + pos % 256
    want = OP.append_rows(np64(step.kv), pos, np64(p.kv_norm), p.eps, True, 64)
    if spec.swa_dtype == "bf16":
        assert (np.abs(np64(c["swa_data"][rows]) - want) <= BF16 * np.abs(want) + 1e-5 * np.max(np.abs(want))).all()
    else:
        got = e4m3_decode(c["swa_data"][rows].cpu().numpy()) * np64(c["swa_scale"][rows])[:, None]
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + np64(c["swa_scale"][rows])[:, None] * 2.0 ** -10
                + 1e-4 * np.max(np.abs(want))).all()
    # the attention over the caches and the queries as they are
    main, swa = oracle_pool(c["main_data"], c["main_scale"], c["epb"]), oracle_pool(c["swa_data"], c["swa_scale"], 256)
    o, _ = OL.sparse_attn(np64(c["q"]), pos, req, spec.kind, np64(step.topk) if step.has_index else None, main,
                          np64(c["bt_main"]), swa, bt, spec.window, SM_SCALE, spec.rope_dim)
    W = np.stack([o[i] for i in range(c["nq"])]).reshape(c["nq"], -1)
    scale = np64(step.out8_scale).reshape(c["nq"], -1)
    got = e4m3_decode(step.out8.cpu().numpy()).reshape(W.shape) * np.repeat(scale, 128, axis=1)
    vmax = pool_absmax((c["main_data"], c["main_scale"]), (c["swa_data"], c["swa_scale"]))
    assert (np.abs(got - W) <= np.abs(W) * 2.0 ** -4 + np.repeat(scale, 128, axis=1) * 2.0 ** -10 + attn_bound(W, vmax)).all()
    # the products behind it
    check_gemm(step.out8, step.out8_scale, *p.o, step.low8, step.low8_scale)
    low = step.low8.view(c["nq"], 1, -1), step.low8_scale.view(c["nq"], 1, -1)
    check_gemm(*low, p.out[0][None], p.out[1][None], step.delta[:, None], None)
    assert step.launches_per_step() >= 8


@pytest.mark.parametrize("name", ["decode", "dense"])
def test_projected_step_replayed_from_a_graph_on_another_stream(name):
    """Two runs of one step from a captured graph give the bits of the same two runs launched one by one."""
    a, x = make(name)
    b, _ = make(name)
    for _ in range(2):
        a.run(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.run(x)
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert int(a.status) == 0 and int(b.status) == 0
    for k in ("residual", "hidden8", "q_raw", "kv", "out8", "low8", "delta"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert torch.equal(a.case["swa_data"], b.case["swa_data"])


def test_two_layers_hand_the_residual_stream_on():
    """The second layer's norm adds the first one's output to the stream that the first one's norm left."""
    first, x = make("decode")
    second, _ = make("decode")
    second.residual = first.residual
    first.run(x)
    before = np64(first.residual)
    second.run(first.delta)
    torch.cuda.synchronize()
    want = before + np64(first.delta)
    assert (np.abs(np64(first.residual) - want) <= (BF16 + 2.0 ** -24) * np.abs(want)).all()
    assert torch.isfinite(second.delta.float()).all()


def test_projected_step_needs_a_query_for_each_new_token():
    spec = synth.CaseSpec("p_last", cached=[5], new=[3], seed=1)
    case = synth.make_case(spec, "cuda")
    with pytest.raises(ValueError):
        ProjectedStep(case, None, torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda"))
