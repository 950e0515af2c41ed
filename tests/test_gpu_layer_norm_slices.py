"""Gradient of wide norms whose rows a cluster shares: rows off 16-byte
boundaries at the widths where a slice fills the threads that hold it; and
many rows at the widths of every streaming group.  Inputs, tolerances and the
64-bit forms are those of test_gpu_layer_norm.py."""
import pytest

from tests._gpu import lib
from tests.test_gpu_layer_norm import _check_forward, _check_grad, _inputs, _torch

pytestmark = pytest.mark.gpu

ROWS = 330          # above four rows for each cluster of two CTAs (76 of them)


def _at(t, first):
    """t's values in a dense matrix that starts `first` elements above a boundary, between sevens."""
    torch, _ = _torch()
    buf = torch.full((t.numel() + first + 16,), 7.0, device="cuda", dtype=t.dtype)
    view = buf[first:first + t.numel()].view(t.shape)
    view.copy_(t)
    return buf, view


def _gradient(x, dy, w, mean, rstd, first, kind, wkind):
    """layer_norm_grad on copies `first` elements above a boundary; nothing outside dx is written."""
    g = lib()
    (_, xs), (_, ds), (buf, out) = _at(x, first), _at(dy, first), _at(x * 0 + 5, first)
    dx, dw, db = g.layer_norm_grad(ds, xs, w, mean, rstd, out=out)
    _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, wkind)
    assert (buf[:first] == 7).all() and (buf[first + out.numel():] == 7).all()
    assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width", [12273, 12277, 12280, 12281, 12285, 12288, 16369, 16376, 16377, 16381, 16384,
                                   32737, 32744, 32761, 32765, 32768])
def test_full_slices_at_every_alignment(width, kind):
    x, dy, w, b = _inputs(ROWS, width, kind, "f32", width)
    _, mean, rstd = lib().layer_norm(x, w, b)
    for first in (0, 1, 2, 3) if kind == "f32" else (0, 1, 3, 4, 7):
        _gradient(x, dy, w, mean, rstd, first, kind, "f32")


@pytest.mark.parametrize("kind,wkind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,width", [(10000, 513), (10000, 600), (10000, 761), (10000, 768), (5000, 1281), (5000, 1535),
                                        (2500, 2049), (2500, 2500), (2500, 2503), (2500, 3065), (1300, 4603), (1300, 6136),
                                        (1300, 8185), (ROWS, 9001), (ROWS, 12001), (ROWS, 12293), (ROWS, 14000),
                                        (ROWS, 14001), (1300, 12293), (1300, 16001)])
def test_many_rows_of_every_group(rows, width, kind, wkind):
    """Forward and backward, rows on boundaries and off them."""
    g = lib()
    x, dy, w, b = _inputs(rows, width, kind, wkind, width)
    for first in (0, 3):
        (_, xs), (buf, out) = _at(x, first), _at(x * 0 + 5, first)
        y, mean, rstd = g.layer_norm(xs, w, b, out=out)
        _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
        assert (buf[:first] == 7).all() and (buf[first + out.numel():] == 7).all()
        _gradient(x, dy, w, mean, rstd, first, kind, wkind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(10000, 256), (10000, 257), (10000, 5), (2500, 2049), (1300, 8192), (ROWS, 12281),
                                        (ROWS, 16384), (ROWS, 20001)])
def test_in_place_streamed(rows, width, kind):
    """Results over x or dy, rows of which one group reads while another writes their neighbours."""
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(rows, width, kind, "f32", rows + width)
    y, mean, rstd = g.layer_norm(x, w, b)
    want = g.layer_norm_grad(dy, x, w, mean, rstd)
    xc = x.clone()
    got = g.layer_norm(xc, w, b, out=xc)
    assert got[0] is xc and all(torch.equal(p, q) for p, q in zip(got, (y, mean, rstd)))
    over = dy.clone()
    assert all(torch.equal(p, q) for p, q in zip(g.layer_norm_grad(over, x, w, mean, rstd, out=over), want))
    over = x.clone()
    assert all(torch.equal(p, q) for p, q in zip(g.layer_norm_grad(dy, over, w, mean, rstd, out=over), want))
    assert g.gemm_f32_status(None) == (0, 0)
