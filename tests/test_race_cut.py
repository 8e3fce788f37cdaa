"""The bytes that the race's wide loads touch, for every alignment and short
vocabulary, without a GPU: tests/race_cut_check.cpp against csrc/race_cut.h."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_loads_lie_inside_their_rows(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "race_cut_check")
    r = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror",
                        "-I", os.path.join(ROOT, "zero_sharded_optimizer_shard_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "race_cut_check.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_kernels_use_it():
    """Both races cut their rows there, and words are read whole only where they lie in
    the row."""
    src = open(os.path.join(ROOT, "zero_sharded_optimizer_shard_gb300", "csrc", "verify.cu")).read()
    assert src.count("= race_cut(") == 2 and src.count("end_token(") == 2
    assert "word_in_row(" in src and "edge_element(" not in src
