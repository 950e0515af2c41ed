"""Host-side checks of the language-model operators' C ABI that need no GPU:
the header compiles as C and C++, every function it declares is exported, and
malformed requests are rejected on the host before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest

from accelerator_row_major_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["gemm_f32_layer_norm", "gemm_f32_layer_norm_grad", "gemm_f32_vocab_loss", "gemm_f32_vocab_loss_grad"]
P = 0x10000000                      # addresses far apart, never touched
X, W, Y, DX, DW, S, T = (P + i * 0x10000000 for i in range(7))


@pytest.fixture(scope="module")
def g():
    build_mod.build()
    import accelerator_row_major_gb300 as pkg
    return pkg


def test_header_compiles_and_its_functions_are_exported(g, tmp_path):
    from accelerator_row_major_gb300 import _binding
    assert g.declared_symbols(_binding.LM_HEADER) == NAMES
    lib = ctypes.CDLL(build_mod.LIB)
    assert all(hasattr(lib, name) for name in NAMES)
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_f32_lm.h"\nint (*entry)(int, int, long long, int, const void*, long long, const void*, '
                   'const void*, float, void*, long long, float*, float*, gemm_f32_stream_t) = gemm_f32_layer_norm;\n'
                   'int main(void) { return entry == 0 ? (int)GEMM_F32_MEAN : (int)GEMM_F32_TYPE_F32; }\n')
    for cc, std in (("gcc", "-std=c99"), ("g++", "-std=c++17")):
        if shutil.which(cc):
            subprocess.run([cc, std, "-x", "c" if cc == "gcc" else "c++", "-Wall", "-Wextra", "-Werror", "-I",
                            os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "h.o")], check=True)


def _norm(lib, **kw):
    a = dict(type=0, wtype=0, rows=4, width=8, x=X, ldx=8, weight=W, bias=0, eps=1e-5, y=Y, ldy=8, mean=S, rstd=S + 64)
    a.update(kw)
    return lib.gemm_f32_layer_norm(a["type"], a["wtype"], a["rows"], a["width"], a["x"], a["ldx"], a["weight"], a["bias"],
                                   a["eps"], a["y"], a["ldy"], a["mean"], a["rstd"], 0)


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(wtype=1), dict(type=1, wtype=3), dict(rows=-1), dict(width=0), dict(x=0), dict(y=0), dict(ldx=7),
    dict(ldy=7), dict(x=X + 2), dict(weight=W + 1), dict(bias=W + 2), dict(mean=S + 2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(y=X + 4), dict(y=X, ldy=16), dict(y=X - 16),
])
def test_layer_norm_rejects(g, kw):
    from accelerator_row_major_gb300 import _binding
    assert _norm(_binding.lib(), **kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0 and g.gemm_f32_last_kernel() == "none"


def _norm_grad(lib, **kw):
    a = dict(type=0, wtype=0, rows=4, width=8, dy=Y, lddy=8, x=X, ldx=8, weight=W, mean=S, rstd=S + 64, dx=DX, lddx=8,
             dw=DW, db=DW + 64)
    a.update(kw)
    return lib.gemm_f32_layer_norm_grad(a["type"], a["wtype"], a["rows"], a["width"], a["dy"], a["lddy"], a["x"],
                                        a["ldx"], a["weight"], a["mean"], a["rstd"], a["dx"], a["lddx"], a["dw"],
                                        a["db"], 0)


@pytest.mark.parametrize("kw", [
    dict(type=-1), dict(wtype=1), dict(rows=-2), dict(width=0), dict(dy=0), dict(x=0), dict(lddy=7), dict(ldx=1),
    dict(lddx=7), dict(mean=0), dict(rstd=0), dict(mean=S + 1), dict(dw=DW + 2), dict(db=DW + 3), dict(dx=X + 8),
    dict(dx=Y, lddx=9), dict(type=1, dx=DX + 1),
])
def test_layer_norm_grad_rejects(g, kw):
    from accelerator_row_major_gb300 import _binding
    assert _norm_grad(_binding.lib(), **kw) == g.GEMM_F32_EINVAL


def _loss(lib, grad, **kw):
    a = dict(type=1, rows=4, width=8, vocab=32, x=X, ldx=8, w=W, ldw=8, targets=T, bits=64, ignore=-100, reduction=1,
             scale=1.0, loss=S, lse=S + 64, total=S + 128, dx=DX, lddx=8, dw=DW, lddw=8, piece=0)
    a.update(kw)
    head = [a[k] for k in ("type", "rows", "width", "vocab", "x", "ldx", "w", "ldw", "targets", "bits", "ignore",
                           "reduction")]
    if not grad:
        return lib.gemm_f32_vocab_loss(*head, a["loss"], a["lse"], a["total"], 0)
    return lib.gemm_f32_vocab_loss_grad(*head, a["scale"], a["loss"], a["lse"], a["total"], a["dx"], a["lddx"], a["dw"],
                                        a["lddw"], a["piece"], 0)


BAD = [dict(type=2), dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(vocab=0), dict(vocab=2 ** 31 - 1), dict(x=0),
       dict(w=0), dict(ldx=7), dict(ldw=7), dict(targets=0), dict(targets=T + 4), dict(bits=16), dict(reduction=2),
       dict(loss=S + 1), dict(lse=S + 2), dict(total=S + 3), dict(x=X + 1)]


@pytest.mark.parametrize("kw", BAD)
def test_vocab_loss_rejects(g, kw):
    from accelerator_row_major_gb300 import _binding
    for grad in (False, True):
        assert _loss(_binding.lib(), grad, **kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0


@pytest.mark.parametrize("kw", [dict(scale=float("nan")), dict(lddx=7), dict(lddw=7), dict(dx=DX + 1), dict(dw=DW + 1),
                                dict(dx=X), dict(dw=W + 16), dict(dx=W), dict(dw=X - 16), dict(dx=DW + 32)])
def test_vocab_loss_grad_rejects(g, kw):
    from accelerator_row_major_gb300 import _binding
    assert _loss(_binding.lib(), True, **kw) == g.GEMM_F32_EINVAL


def test_nothing_to_do_and_no_gpu(g):
    torch = pytest.importorskip("torch")
    from accelerator_row_major_gb300 import _binding
    lib = _binding.lib()
    assert _norm(lib, rows=0, x=0, y=0) == g.GEMM_F32_OK
    assert _norm_grad(lib, rows=0, dw=0, db=0, x=0, dy=0) == g.GEMM_F32_OK
    assert _norm_grad(lib, dx=0, dw=0, db=0) == g.GEMM_F32_OK
    assert _loss(lib, False, rows=0, x=0, targets=0, total=0) == g.GEMM_F32_OK
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _norm(lib) == g.GEMM_F32_EDEVICE
    assert _norm(lib, y=X) == g.GEMM_F32_EDEVICE          # in place is allowed
    assert _norm_grad(lib, dx=Y) == g.GEMM_F32_EDEVICE
    assert _loss(lib, False) == g.GEMM_F32_EDEVICE
    assert _loss(lib, True, bits=32, type=0) == g.GEMM_F32_EDEVICE


def test_operators_need_cuda_tensors(g):
    torch = pytest.importorskip("torch")
    x, w, y = torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: g.layer_norm(x), lambda: g.layer_norm_grad(x, x, None, y, y), lambda: g.vocab_loss(x, w, y),
                 lambda: g.vocab_loss_grad(x, w, y)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        g.no_such_operator
