"""Gradients of rows that are almost certain of their target: g at the target
is -(1 - p), small, and keeps its relative precision.

x has one element of 1 in each row, in a column of the row's own, so column t
of dw is row t of g alone.  In bfloat16 g is rounded once (2^-8 of it at most)
and the result once more; 1 - p carries the rounding of the powers (2^-22) and
of their sum (below 2^-20) relative to 1."""
import pytest

from tests._gpu import lib
from tests.test_gpu_vocab_loss import _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [20, 100, 300])
@pytest.mark.parametrize("base", [0.0, -300.0])
def test_gradient_at_an_almost_certain_target(base, rows, kind):
    torch, types = _torch()
    g = lib()
    vocab, width = 700, rows
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.eye(rows, device="cuda", dtype=types[kind])
    w = base + torch.randn((vocab, width), generator=gen, device="cuda")
    y = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    w[y, torch.arange(rows, device="cuda")] = base + torch.linspace(6.0, 20.0, rows, device="cuda")
    w = w.to(types[kind])
    dw = g.vocab_loss_grad(x, w, y, reduction="sum")[4].double()
    want = torch.softmax(w.double().t(), 1)
    at = torch.arange(rows, device="cuda")
    rest = want.clone()
    rest[at, y] = 0.0
    want[at, y] = -rest.sum(1)
    off = (dw.t() - want).abs()[at, y]
    once = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    assert (off <= 2.02 * once * want[at, y].abs() + 2.0 ** -19).all(), float((off / want[at, y].abs()).max())
