"""The scratch of the language-model operators: what it held before a call
does not matter."""
import ctypes

import pytest

from tests._gpu import lib
from tests.test_gpu_vocab_loss import _check, _exact, _inputs, _torch

pytestmark = pytest.mark.gpu


def _scratch(stream, nbytes):
    """Address of the library's scratch for calls on a stream, by its internal function."""
    from accelerator_row_major_gb300 import _binding
    f = _binding.lib()._ZN13gemm_f32_impl15acquire_scratchEiP11CUstream_stm
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t], ctypes.c_void_p
    return f(0, stream, nbytes)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [9, 200, 600])
def test_a_scratch_that_holds_anything(rows, kind):
    """Memory that an allocation returns is not zero: every word of the scratch holds 3.0 before the call."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(rows, 100, 1200, kind, rows)
    want = _exact(x, w, y, kind)
    one, threes = torch.ones((1, 1), device="cuda"), torch.full((1, 1 << 18), 3.0, device="cuda")
    for call in (g.vocab_loss, g.vocab_loss_grad):
        call(x, w, y)                                   # sizes it
        at = _scratch(0, 1 << 18)
        g.check(g.gemm_f32(one, threes, at, 1, 1 << 16, 1))
        _check(call(x, w, y), want)
