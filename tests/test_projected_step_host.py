"""ProjectedStep's refusals: sizes that the attention, the query job or the grouped product would run past or misread."""
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import synth
from compressed_sparse_attention_c4a_gb300.step import LayerProjections, ProjectedStep


def codes(*shape):
    blocks = [-(-n // 128) for n in shape[-2:]]
    return torch.zeros(shape, dtype=torch.uint8), torch.ones((*shape[:-2], *blocks))


def make(heads=16, groups=2, rank=128, inner=None, q_norm=None, **case):
    hidden = 144
    spec = synth.CaseSpec("p", **{"cached": [5, 300], "new": [1, 1], "heads": heads, "seed": 3, **case})
    inner = heads // groups * 512 if inner is None else inner
    proj = LayerProjections(torch.ones(hidden), codes(heads * 512, hidden), codes(512, hidden), codes(groups, rank, inner),
                            codes(hidden, groups * rank), q_norm=q_norm)
    data = synth.make_case(spec, "cpu")
    return ProjectedStep(data, proj, torch.zeros((data["nq"], hidden), dtype=torch.bfloat16))


def test_buffers_fit_the_attention():
    for heads, groups, rank in ((16, 1, 128), (16, 2, 256), (64, 8, 128), (16, 1, 400)):
        step = make(heads, groups, rank, q_norm=torch.ones(512))
        assert step.out8.numel() == 2 * heads * 512 and step.out8_scale.numel() == 2 * heads * 4
        assert step.low8_scale.view(2, -1).shape[1] == -(-groups * rank // 128)
    make(16, 2, new=[3, 2], queries="all")


@pytest.mark.parametrize("args", [
    dict(heads=64, groups=3),                              # 63 heads of 64 would fit
    dict(heads=16, groups=32, inner=512), dict(inner=4096 - 512), dict(inner=8192),
    dict(rank=200),                                        # 2 ceil(200 / 128) is ceil(400 / 128): no shape gives it away
    dict(rank=64), dict(q_norm=torch.ones(256)), dict(q_norm=torch.ones(512, dtype=torch.bfloat16)),
    dict(q_norm=torch.ones(1024)[::2]),
    dict(new=[2, 0]), dict(new=[0, 2]), dict(new=[3, 1])])  # the last token's query of each request only
def test_refusals(args):
    with pytest.raises(ValueError):
        make(**args)
