"""Which kernel rows of more than 32768 columns take, by type and form, as the header says; and that both are right."""
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,norm,gate,post,bias,width,forward,gradient", [
    ("bf16", "rms", "none", False, False, 131072, "", "_wide"), ("f32", "rms", "none", False, False, 86016, "", "_wide"),
    ("f32", "rms", "none", False, False, 131072, "_wide", "_wide"), ("f32", "layer", "element", True, True, 40960, "", "_wide"),
    ("f32", "layer", "element", True, True, 40968, "_wide", "_wide"), ("bf16", "rms", "none", True, False, 65536, "", ""),
    ("bf16", "rms", "none", True, False, 65544, "", "_wide"), ("f32", "rms", "element", True, False, 36864, "", ""),
    ("f32", "rms", "element", True, False, 36872, "", "_wide"), ("bf16", "rms", "channel", True, False, 40000, "", "_wide"),
    ("bf16", "layer", "none", True, True, 32768, "", ""), ("bf16", "layer", "none", True, True, 32776, "", "_wide")])
def test_kernel_of_wide_rows(kind, norm, gate, post, bias, width, forward, gradient):
    from tests import _block as b
    g = lib()
    s = b.inputs(3, width, kind, "f32", norm, gate, post, width, bias=bias)
    got = b.call(g, s)
    assert g.gemm_f32_last_kernel() == "block_norm%s_kernel" % forward and g.gemm_f32_last_launches() == 1
    b.check(got, b.forward(s))
    grads = b.call_grad(g, s, got["h"], s["branch"], got["stats"])
    assert g.gemm_f32_last_kernel() == "block_norm_grad%s_kernel" % gradient and g.gemm_f32_last_launches() == 2
    b.check(grads, b.gradients(s, got["h"], s["branch"], got["stats"]))
    assert g.gemm_f32_status(None) == (0, 0)
