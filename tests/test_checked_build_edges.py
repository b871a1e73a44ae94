"""The bounds-checked build of the operators around the attention, in the cases that the parametrised files beside the first hold: products
whose blocks two pairs share, last tiles, tile after tile; far offsets, alignments, many requests; values at the ends of the range
(test_checked_build.py says what a failed check does; dsa_norm_q8 has no status word, its values show a skipped access)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ["test_projections_edges.py", "test_gemm_outputs_in_turn.py", "test_projections_forms.py", "test_norm_span.py", "test_append_span.py"]


def test_the_norm_carries_index_checks():
    text = open(os.path.join(ROOT, "compressed_sparse_attention_c4a_gb300", "csrc", "norm.cu")).read()
    assert text.count("DSA_IDX_OK(") >= 3


@pytest.mark.gpu
@pytest.mark.parametrize("name", FILES)
def test_checked_build_passes_the_edge_cases(name):
    from compressed_sparse_attention_c4a_gb300 import build
    build.build(checked=True)
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.join("tests", name), "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=dict(os.environ, DSA_CHECKED="1"), capture_output=True, text=True, timeout=1200)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
    assert " passed" in res.stdout and " failed" not in res.stdout
