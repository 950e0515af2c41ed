"""Gradient of norms of many rows whose values are near the end of the range:
rows all but constant at 2e36, whose mean times 1 / sqrt(eps) overflows."""
import pytest

from tests._gpu import lib
from tests.test_gpu_layer_norm import _check_grad, _inputs, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(10, 16), (10000, 16), (10000, 17), (10000, 3), (10000, 100), (10000, 101)])
def test_constant_rows_of_large_values(rows, width, kind):
    """hat is 0 there, so dx is rstd (g - mean of g), and the columns' sums are those of the other rows."""
    torch, types = _torch()
    g = lib()
    x, dy, w, b = _inputs(rows, width, kind, "f32", width)
    x[::5] = torch.tensor(2e36).to(types[kind])
    mean, rstd = x.double().mean(1).float(), torch.full((rows,), 316.0, device="cuda")
    mean[::5] = x[::5, 0].float()
    live = torch.arange(rows, device="cuda") % 5 != 0
    rstd[live] = 1.0
    dx, dw, db = g.layer_norm_grad(dy, x, w, mean, rstd)
    _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, "f32")
