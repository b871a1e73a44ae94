"""The bounds-checked build over 4-bit rows: the kernels that store, read and attend to them check their computed table, ring and
row indexes there (test_checked_build.py says what a failed check does), and their cases pass through it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("source", ["attention_fp4.cu", "cache.cu"])
def test_the_kernels_carry_index_checks(source):
    text = open(os.path.join(ROOT, "compressed_sparse_attention_c4a_gb300", "csrc", source)).read()
    assert text.count("DSA_IDX_OK(") >= 4


@pytest.mark.gpu
def test_checked_build_passes_the_block_row_cases():
    from compressed_sparse_attention_c4a_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, DSA_CHECKED="1")
    sel = ("test_write_then_read or test_write_and_read or test_bad_rows or test_compressor_stores or test_many_rows_at or "
           "(test_attention and not entry_points) or test_many_rows_of or test_tiles_without or test_positions_beyond")
    files = [os.path.join("tests", f) for f in ("test_cache_fp4_block.py", "test_fp4_block_edges.py")]
    res = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k", sel],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
    assert " passed" in res.stdout and " failed" not in res.stdout
