"""The norms at a block's ends and the checkpoints on the bounds-checked debug
build, in a child process whose library records an index outside an array in
the error word that the tests read through gemm_f32_status()."""
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
                          "tests/test_gpu_block_norm.py", "tests/test_gpu_checkpoint.py",
                          "-k", "widths or forms or strides or many_rows or start_anywhere or values or weight_gradient"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    tail = "\n".join((run.stdout + run.stderr).splitlines()[-30:])
    assert run.returncode == 0, tail
    assert " passed" in run.stdout and "failed" not in run.stdout, tail
