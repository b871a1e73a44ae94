"""The staleness key of the committed kernel summaries: it covers every header that a kernel's source includes."""
import os
import shutil

import bench

CSRC = os.path.join("compressed_sparse_attention_c4a_gb300", "csrc")


def test_a_change_in_any_included_header_changes_the_digest(tmp_path, monkeypatch):
    """Against the includes read from the sources: a kernel's digest moves with each header that it includes, directly or
    through another, and with no other file."""
    names = sorted(os.listdir(os.path.join(bench.ROOT, CSRC)))
    text = {n: open(os.path.join(bench.ROOT, CSRC, n)).read() for n in names}

    def reach(n, seen):
        for line in text[n].splitlines():
            if line.startswith('#include "') and line.split('"')[1] in text:
                inc = line.split('"')[1]
                if inc not in seen:
                    seen.add(inc)
                    reach(inc, seen)
        return seen

    root = tmp_path / "tree"
    shutil.copytree(os.path.join(bench.ROOT, CSRC), root / CSRC)
    before = {k: bench.kernel_source_digest(k) for k in bench.KERNEL_SOURCES}
    monkeypatch.setattr(bench, "ROOT", str(root))
    assert {k: bench.kernel_source_digest(k) for k in bench.KERNEL_SOURCES} == before
    for n in names:
        (root / CSRC / n).write_text(text[n] + "\n// changed\n")
        for k, src in bench.KERNEL_SOURCES.items():
            # every digest also holds the two headers that every kernel included at first
            covered = n == src or n in reach(src, set()) or n in ("common.cuh", "topk_cluster.cuh")
            assert (bench.kernel_source_digest(k) != before[k]) == covered, (k, n)
        (root / CSRC / n).write_text(text[n])


def test_every_kernel_summary_names_its_sources_digest():
    """A summary without the line could never be told from a current one."""
    folder = os.path.join(bench.ROOT, "profiles")
    for name in sorted(os.listdir(folder)):
        if any(name.startswith(k + "_") for k in bench.KERNEL_SOURCES):
            lines = open(os.path.join(folder, name)).read().splitlines()
            assert sum(line.startswith("source_sha256_16: ") for line in lines) == 1, name
            assert sum(line.startswith("dram_bytes_per_launch: ") for line in lines) == 1, name
