"""The arithmetic by which the dense attention kernels divide a batch, compiled
for the host."""
import os
import shutil
import subprocess

import pytest


def test_steps_in_closed_form(tmp_path):
    """The steps of a request's first row tiles, whatever the heads and the row tile's size."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(here), "deepseek_sparse_attention_fp8_gb300", "csrc")
    exe = str(tmp_path / "dense_steps_check")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                        "-fno-sanitize-recover=undefined", "-I", csrc, os.path.join(here, "dense_steps_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "steps ok" in r.stdout, (r.returncode, r.stdout, r.stderr)
