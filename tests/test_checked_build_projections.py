"""The bounds-checked build of the operators around the attention (test_checked_build.py says what a failed check does): their
cases pass through it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("source,checks", [("gemm.cu", 4), ("cache.cu", 8)])
def test_the_kernels_carry_index_checks(source, checks):
    text = open(os.path.join(ROOT, "compressed_sparse_attention_c4a_gb300", "csrc", source)).read()
    assert text.count("DSA_IDX_OK(") >= checks


@pytest.mark.gpu
def test_checked_build_passes_the_projection_cases():
    from compressed_sparse_attention_c4a_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, DSA_CHECKED="1")
    files = [os.path.join("tests", f) for f in ("test_projections.py", "test_projected_step.py")]
    res = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
    assert " passed" in res.stdout and " failed" not in res.stdout
