"""The language-model operators on the bounds-checked debug build: the tests
of layer norm and of the vocabulary loss, in a child process whose library
records an index outside an array (sites 16-22) in the error word that they
read through gemm_f32_status()."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_reports_no_out_of_extent_access():
    from accelerator_row_major_gb300 import build as build_mod
    env = dict(os.environ, GEMM_F32_LIBRARY=build_mod.build(checked=True))
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                          "tests/test_gpu_layer_norm.py", "tests/test_gpu_vocab_loss.py",
                          "-k", "against_64_bits or streamed or many_rows or strided or pieces"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    tail = "\n".join((run.stdout + run.stderr).splitlines()[-30:])
    assert run.returncode == 0, tail
    assert " passed" in run.stdout and "failed" not in run.stdout, tail
