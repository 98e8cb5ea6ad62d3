"""The recorded DRAM traffic counts only for the very sources it was taken on, the shared header
among them (host only)."""
import hashlib
import os
import shutil

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join("decode_step_kv_gb300", "csrc")
FILES = ["fa_decode.cu", "fa_common.cuh"]


@pytest.fixture
def tree(tmp_path, monkeypatch):
    os.makedirs(tmp_path / CSRC)
    os.makedirs(tmp_path / "profiles")
    sha = {}
    for f in FILES:
        shutil.copy(os.path.join(ROOT, CSRC, f), tmp_path / CSRC / f)
        sha[f] = hashlib.sha256((tmp_path / CSRC / f).read_bytes()).hexdigest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    summary = tmp_path / "profiles" / "k_w.md"
    summary.write_text(f"Kernel source: x, source sha256: {sha['fa_decode.cu']}\n"
                       f"fa_common.cuh sha256: {sha['fa_common.cuh']}\n"
                       "- traffic_bytes_per_launch: 4295000000 (scaled)\n")
    return tmp_path, summary


def test_read_for_its_own_sources(tree):
    assert bench.recorded_traffic("k", "w") == 4295000000


@pytest.mark.parametrize("changed", FILES)
def test_not_for_a_changed_file(tree, changed):
    with open(tree[0] / CSRC / changed, "ab") as f:
        f.write(b"\n")
    assert bench.recorded_traffic("k", "w") is None


@pytest.mark.parametrize("line", ["source sha256", "fa_common.cuh sha256", "traffic_bytes_per_launch"])
def test_not_from_a_summary_without_a_line(tree, line):
    text = tree[1].read_text()
    assert line in text
    tree[1].write_text(text.replace(line, "something else"))
    assert bench.recorded_traffic("k", "w") is None
