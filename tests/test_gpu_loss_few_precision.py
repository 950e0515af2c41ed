"""bfloat16 gradients of few rows: dx and dw carry one rounding of bfloat16,
the result's own (2^-8 of it at most: 1 + 2^-8 lies half way between two bfloat16
values), since few terms make up an element and a second rounding, of g, would
show.

Of one row an element of dw is one product: g, whose exponential is held in
fp16 (2^-12), times x.  Besides that the logits' own error (test_gpu_vocab_loss
derives it) moves every probability by the same small factor; 2^-11 covers it
at this width.  Of several rows, and for dx, the terms' sizes count."""
import pytest

from tests._gpu import lib
from tests.test_gpu_vocab_loss import _inputs, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 2, 7, 16, 17, 32])
@pytest.mark.parametrize("width,vocab", [(64, 3000), (136, 777), (77, 1001)])
def test_one_rounding(width, vocab, rows):
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(rows, width, vocab, "bf16", rows + width, ignored=0.0)
    _, _, _, dx, dw = g.vocab_loss_grad(x, w, y, reduction="sum", grad_scale=0.5)
    assert g.gemm_f32_last_kernel() == "few_gemm_kernel"
    xd, wd = x.double(), w.double()
    p = torch.softmax(xd @ wd.t(), 1)
    p[torch.arange(rows, device="cuda"), y] -= 1.0
    for got, want, size in ((dw, 0.5 * p.t() @ xd, 0.5 * p.abs().t() @ xd.abs()), (dx, 0.5 * p @ wd, 0.5 * p.abs() @ wd.abs())):
        off = (got.double() - want).abs() - 2.0 ** -8 * want.abs()
        assert (off <= 2.0 ** -11 * size + 2.0 ** -40).all(), float((off / size.clamp(min=1e-30)).max())
    assert g.gemm_f32_status(None) == (0, 0)
