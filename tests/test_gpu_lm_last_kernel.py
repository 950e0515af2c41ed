"""gemm_f32_last_kernel() after the language-model operators: which path a
call took, by the sizes at which the paths are known to be different ones."""
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,first,kernel", [
    (1, 4096, 0, "layer_norm%s_kernel"), (500, 777, 0, "layer_norm%s_kernel"), (65536, 1024, 0, "layer_norm%s_stream_kernel"),
    (20000, 1001, 1, "layer_norm%s_stream_kernel"), (40, 40000, 0, "layer_norm%s_kernel"), (1000, 40000, 0, "layer_norm%s_kernel")])
def test_norms(rows, width, first, kernel):
    import torch
    g = lib()
    x = torch.randn(rows * width + first, device="cuda").bfloat16()[first:].view(rows, width)
    out = torch.empty(rows * width + first, device="cuda", dtype=torch.bfloat16)[first:].view(rows, width)
    _, mean, rstd = g.layer_norm(x, out=out)
    assert g.gemm_f32_last_kernel() == kernel % ""
    g.layer_norm_grad(x, x, None, mean, rstd, out=out)
    assert g.gemm_f32_last_kernel() == kernel % "_grad"
    g.layer_norm_grad(x[:0], x[:0], None, mean[:0], rstd[:0])
    assert g.gemm_f32_last_kernel() == "norm_columns_kernel" and g.gemm_f32_last_launches() == 1


@pytest.mark.parametrize("kind,rows,kernel", [("bfloat16", 1, "few_gemm_kernel"), ("bfloat16", 32, "few_gemm_kernel"),
                                              ("bfloat16", 500, "half_gemm_kernel"), ("float32", 100, "few_gemm_kernel"),
                                              ("float32", 500, "half_gemm_kernel"), ("float32", 0, "memset")])
def test_losses(kind, rows, kernel):
    import torch
    g = lib()
    x, w = (torch.randn(n, 64, device="cuda").to(getattr(torch, kind)) for n in (rows, 300))
    y = torch.zeros(rows, dtype=torch.int64, device="cuda")
    for call in (g.vocab_loss, g.vocab_loss_grad):
        call(x, w, y)
        assert g.gemm_f32_last_kernel() == kernel
