"""How chunks' work is found: ``tests/chunk_cost_check.cpp`` is compiled against the
library's closed forms and run. Plain C++, no GPU needed."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_closed_forms_and_the_search(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "chunk_cost_check"
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "turboquant_paged_kv_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "chunk_cost_check.cpp"), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert run.returncode == 0, run.stdout
    assert "places" in run.stdout and "sums" in run.stdout
