"""The library's memory between calls (csrc/workspace.h) on a stand-in for the
CUDA runtime: a buffer that a graph or another thread's call uses is not freed
nor shared."""
import os
import shutil
import subprocess

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_api", "workspace_test.cpp")


def test_buffers_of_streams_graphs_and_threads(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "workspace_test")
    subprocess.run([cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-pthread", SOURCE, "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout + run.stderr
    assert run.stdout.split("\n")[:4] == ["ok growth", "ok graphs", "ok products_in_captures", "ok threads"]
