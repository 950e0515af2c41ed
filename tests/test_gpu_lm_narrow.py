"""Many rows shorter than a 16-byte block: norms of 1 to 9 columns, dense and
spread, at every distance from a boundary; and the newer tests of the norms on
the bounds-checked library, which checks the blocks that bulk copies read."""
import os
import subprocess
import sys

import pytest

from tests._gpu import lib
from tests.test_gpu_layer_norm import _check_forward, _check_grad, _inputs, _torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width,stride", [(1, 1), (1, 3), (2, 2), (3, 3), (4, 4), (5, 5), (6, 7), (7, 7), (8, 8), (9, 9), (2, 12)])
def test_narrow_rows(width, stride, kind):
    torch, types = _torch()
    g = lib()
    rows = 10002
    x, dy, w, b = _inputs(rows, width, kind, "f32", width + stride)

    def placed(t, first):
        """t's rows `stride` apart in a buffer of NaN that ends with the last of them."""
        buf = torch.full((first + (rows - 1) * stride + width,), float("nan"), device="cuda", dtype=types[kind])
        view = torch.as_strided(buf, (rows, width), (stride, 1), first)
        view.copy_(t)
        return view

    for first in range(8 if kind == "bf16" else 4):
        xs, ds = placed(x, first), placed(dy, first)
        y, mean, rstd = g.layer_norm(xs, w, b, out=placed(x, first))
        assert g.gemm_f32_last_kernel() == "layer_norm_stream_kernel"
        _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
        dx, dw, db = g.layer_norm_grad(ds, xs, w, mean, rstd, out=placed(x, first))
        _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, "f32")
        assert g.gemm_f32_status(None) == (0, 0)


def test_on_the_bounds_checked_library():
    from accelerator_row_major_gb300 import build as build_mod
    env = dict(os.environ, GEMM_F32_LIBRARY=build_mod.build(checked=True))
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                          "tests/test_gpu_lm_narrow.py", "tests/test_gpu_layer_norm_slices.py", "-k", "not bounds_checked"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    tail = "\n".join((run.stdout + run.stderr).splitlines()[-30:])
    assert run.returncode == 0, tail
    assert " passed" in run.stdout and "failed" not in run.stdout, tail
