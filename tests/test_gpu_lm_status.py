"""What gemm_f32_status() says when a loss has met a target outside the
vocabulary and a wait has run out on the same device: both, the failure first."""
import pytest

import workloads
from tests._gpu import lib

pytestmark = pytest.mark.gpu


def _bad_target(g, torch):
    x, w = torch.randn(8, 16, device="cuda"), torch.randn(40, 16, device="cuda")
    g.vocab_loss(x, w, torch.tensor([1, 2, 40, 3, -7, 4, 5, -100], device="cuda"))


@pytest.mark.parametrize("target_first", [True, False])
def test_a_target_does_not_hide_a_wait_that_ran_out(target_first):
    import torch
    g = lib()
    A, B = (torch.from_numpy(t).cuda() for t in workloads.make_inputs(256, 64, 256, "uniform", 8))
    C = torch.empty((256, 256), device="cuda")
    s = torch.cuda.current_stream()
    if target_first:
        _bad_target(g, torch)
    assert g.gemm_f32_ex(A, B, C, 256, 256, 64, "tc3x", g.FLAG_TEST_DROP_COPY, s) == g.GEMM_F32_OK
    if not target_first:
        _bad_target(g, torch)
    code, site = g.gemm_f32_status(s)
    assert code == g.GEMM_F32_ETIMEOUT and 1 <= site <= 8
    assert g.gemm_f32_status(s)[0] == g.GEMM_F32_ETARGET
    assert g.gemm_f32_status(s) == (g.GEMM_F32_OK, 0)
    assert bool(torch.isfinite(g.matmul(A, B)).all()) and g.gemm_f32_status(s) == (g.GEMM_F32_OK, 0)
