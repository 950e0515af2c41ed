"""Host-side checks of gemm_f32_block.h that need no GPU: the header compiles
as C and C++ and its structures are the binding's, every function it declares
is exported, and malformed requests are rejected before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest

from accelerator_row_major_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["gemm_f32_block_norm", "gemm_f32_block_norm_grad", "gemm_f32_checkpoint", "gemm_f32_restore", "gemm_f32_weight_grad"]
P = 0x10000000                      # addresses far apart, never touched
A = [P * i for i in range(1, 40)]


@pytest.fixture(scope="module")
def g():
    build_mod.build()
    import accelerator_row_major_gb300 as pkg
    return pkg


def test_header_compiles_and_its_functions_are_exported(g, tmp_path):
    from accelerator_row_major_gb300 import _binding
    assert g.declared_symbols(_binding.BLOCK_HEADER) == NAMES
    lib = ctypes.CDLL(build_mod.LIB)
    assert all(hasattr(lib, name) for name in NAMES)
    fields = {"gemm_f32_block_t": _binding.Block, "gemm_f32_rows_t": _binding.Rows}
    lines = ['  printf("%%zu\\n", sizeof(%s));' % t for t in fields]
    lines += ['  printf("%%zu\\n", offsetof(%s, %s));' % (t, name) for t, c in fields.items() for name, _ in c._fields_]
    src = tmp_path / "h.c"
    src.write_text('#include <stdio.h>\n#include "gemm_f32_block.h"\n'
                   'int (*entry)(int, long long, int, const void*, long long, unsigned char*, long long, unsigned char*, long long, '
                   'gemm_f32_stream_t);\nint main(void) {\n%s\n  return entry != 0 || GEMM_F32_NORM_RMS != 1 || '
                   'GEMM_F32_SAVED_BLOCK != 32;\n}\n' % "\n".join(lines))
    for cc, std in (("gcc", "-std=c99"), ("g++", "-std=c++17")):
        if not shutil.which(cc):
            continue
        subprocess.run([cc, std, "-x", "c" if cc == "gcc" else "c++", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "h")], check=True)
        got = [int(v) for v in subprocess.run([str(tmp_path / "h")], check=True, capture_output=True, text=True).stdout.split()]
        want = [ctypes.sizeof(c) for c in fields.values()]
        want += [getattr(c, name).offset for c in fields.values() for name, _ in c._fields_]
        assert got == want


def _block(kw):
    from accelerator_row_major_gb300 import _binding
    f = dict(type=0, weight_type=0, norm=0, post=1, rows=4, width=40, eps=1e-5, residual_scale=1.0, branch_scale=1.0, weight=A[0],
             bias=A[1], post_weight=A[2], post_bias=A[3], gate=A[4], ld_gate=40)
    f.update({k: v for k, v in kw.items() if k in f})
    b = _binding.Block()
    for k, v in f.items():
        setattr(b, k, v)
    return b


def _norm(**kw):
    from accelerator_row_major_gb300 import _binding
    a = dict(branch=A[5], ldb=40, residual=A[6], ldr=40, y=A[7], ldy=40, h=A[8], ldh=40, stats=A[9])
    a.update({k: v for k, v in kw.items() if k in a})
    return _binding.lib().gemm_f32_block_norm(ctypes.byref(_block(kw)), a["branch"], a["ldb"], a["residual"], a["ldr"], a["y"],
                                              a["ldy"], a["h"], a["ldh"], a["stats"], 0)


BAD_BLOCK = [dict(type=2), dict(weight_type=1), dict(type=1, weight_type=3), dict(norm=2), dict(norm=-1), dict(post=2), dict(rows=-1),
             dict(width=0), dict(residual_scale=float("nan")), dict(branch_scale=float("inf")), dict(weight=A[0] + 2),
             dict(bias=A[1] + 1), dict(post_weight=A[2] + 2), dict(post_bias=A[3] + 1), dict(gate=A[4] + 2),
             dict(gate=A[4] + 2, ld_gate=0), dict(ld_gate=39), dict(ld_gate=-40), dict(norm=1), dict(norm=1, bias=0),
             dict(norm=1, post_bias=0), dict(post=0), dict(post=0, post_bias=0), dict(rows=1 << 62, ld_gate=1 << 40), dict(width=2 ** 31 - 1, ld_gate=0)]


@pytest.mark.parametrize("kw", BAD_BLOCK + [
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(branch=0), dict(residual=0), dict(y=0), dict(ldb=39),
    dict(ldr=0), dict(ldy=-40), dict(ldh=39), dict(branch=A[5] + 2), dict(y=A[7] + 1), dict(h=A[8] + 2), dict(stats=A[9] + 2),
    dict(y=A[5] + 4), dict(y=A[5], ldy=48), dict(y=A[5], ldb=48), dict(y=A[6] - 16), dict(h=A[7]), dict(h=A[7] + 40), dict(y=A[4] + 8),
    dict(h=A[6] + 4 * 40 * 3)])
def test_block_norm_rejects(g, kw):
    assert _norm(**kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0 and g.gemm_f32_last_kernel() == "none"


def _grad(**kw):
    from accelerator_row_major_gb300 import _binding
    a = dict(dy=A[5], lddy=40, dh=A[6], lddh=40, h=A[7], ldh=40, h_codes=0, ldhc=64, h_exponents=0, ldhe=16, branch=A[8], ldb=40,
             b_codes=0, ldbc=64, b_exponents=0, ldbe=16, stats=A[9], dbranch=A[10], lddb=40, dresidual=A[11], lddr=40, dgate=A[12],
             lddg=40, dweight=A[13], dbias=A[14], dpost_weight=A[15], dpost_bias=A[16], no_h=False, no_branch=False)
    a.update({k: v for k, v in kw.items() if k in a})
    h, b = _binding.Rows(), _binding.Rows()
    for r, p, d in ((h, "h", "ldh"), (b, "b", "ldb")):
        r.data, r.ld = a["h" if p == "h" else "branch"], a[d]
        r.codes, r.ld_codes = a[p + "_codes"], a["ld%sc" % p]
        r.exponents, r.ld_exponents = a[p + "_exponents"], a["ld%se" % p]
    return _binding.lib().gemm_f32_block_norm_grad(
        ctypes.byref(_block(kw)), a["dy"], a["lddy"], a["dh"], a["lddh"], None if a["no_h"] else ctypes.byref(h),
        None if a["no_branch"] else ctypes.byref(b), a["stats"], a["dbranch"], a["lddb"], a["dresidual"], a["lddr"], a["dgate"],
        a["lddg"], a["dweight"], a["dbias"], a["dpost_weight"], a["dpost_bias"], 0)


KEPT = dict(h_codes=A[17], h_exponents=A[18])


@pytest.mark.parametrize("kw", BAD_BLOCK + [
    dict(dy=0), dict(lddy=39), dict(dy=A[5] + 1), dict(dh=A[6] + 2), dict(lddh=39), dict(no_h=True), dict(h=0), dict(ldh=3),
    dict(no_branch=True), dict(branch=0), dict(ldb=39), dict(stats=0), dict(stats=A[9] + 1), dict(dbranch=A[10] + 2), dict(lddb=39),
    dict(lddr=8), dict(lddg=39), dict(dgate=A[12] + 1), dict(dweight=A[13] + 2), dict(dbias=A[14] + 1), dict(dpost_weight=A[15] + 3),
    dict(dbranch=A[11]), dict(dbranch=A[11] + 16), dict(dgate=A[10]), dict(dresidual=A[5] + 8), dict(dresidual=A[5], lddr=44),
    dict(dresidual=A[7] - 4), dict(dbranch=A[8] + 40),
    dict(KEPT, h_codes=A[17] + 8), dict(KEPT, h_exponents=A[18] + 1), dict(KEPT, h_exponents=0), dict(KEPT, ldhc=32),
    dict(KEPT, ldhc=72), dict(KEPT, ldhe=8), dict(KEPT, ldhe=0), dict(KEPT, dresidual=A[17]), dict(KEPT, dbranch=A[18] - 4),
    dict(norm=1, bias=0, post_bias=0, dbias=A[14], dpost_bias=0), dict(norm=1, bias=0, post_bias=0, dbias=0),
    dict(post=0, post_weight=0, post_bias=0, dpost_weight=0), dict(gate=0, ld_gate=0)])
def test_block_norm_grad_rejects(g, kw):
    assert _grad(**kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0 and g.gemm_f32_last_kernel() == "none"


def _keep(restore=False, **kw):
    from accelerator_row_major_gb300 import _binding
    a = dict(type=0, rows=4, width=40, x=A[0], ldx=40, codes=A[1], ldc=64, exponents=A[2], lde=16)
    a.update(kw)
    lib = _binding.lib()
    if restore:
        return lib.gemm_f32_restore(a["type"], a["rows"], a["width"], a["codes"], a["ldc"], a["exponents"], a["lde"], a["x"], a["ldx"], 0)
    return lib.gemm_f32_checkpoint(a["type"], a["rows"], a["width"], a["x"], a["ldx"], a["codes"], a["ldc"], a["exponents"], a["lde"], 0)


@pytest.mark.parametrize("restore", [False, True])
@pytest.mark.parametrize("kw", [dict(type=2), dict(rows=-1), dict(width=0), dict(x=0), dict(ldx=39), dict(x=A[0] + 2), dict(codes=0),
                                dict(codes=A[1] + 8), dict(ldc=40), dict(ldc=48), dict(ldc=72), dict(exponents=0),
                                dict(exponents=A[2] + 4), dict(lde=2), dict(lde=0), dict(width=1000, ldx=1000, ldc=1024),
                                dict(codes=A[0]), dict(codes=A[0] + 16 * 39), dict(exponents=A[0] - 16), dict(rows=1 << 60, ldc=1 << 30),
                                dict(width=2 ** 31 - 1000, ldx=1 << 31, ldc=1 << 31, lde=1 << 26)])
def test_checkpoint_and_restore_reject(g, kw, restore):
    assert _keep(restore, **kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0 and g.gemm_f32_last_kernel() == "none"


def test_codes_and_exponents_apart(g):
    assert _keep(exponents=A[1] + 16) == g.GEMM_F32_EINVAL


def _dw(**kw):
    from accelerator_row_major_gb300 import _binding
    a = dict(type=0, rows=4, width=40, out=24, dy=A[0], lddy=24, codes=A[1], ldc=64, exponents=A[2], lde=16, dw_type=0, dw=A[3], lddw=40,
             accumulate=0)
    a.update(kw)
    return _binding.lib().gemm_f32_weight_grad(*[a[k] for k in ("type", "rows", "width", "out", "dy", "lddy", "codes", "ldc",
                                                                "exponents", "lde", "dw_type", "dw", "lddw", "accumulate")], 0)


@pytest.mark.parametrize("kw", [dict(type=3), dict(dw_type=1), dict(dw_type=2), dict(rows=-1), dict(rows=2 ** 31 - 1024), dict(width=0),
                                dict(out=0), dict(out=2 ** 31 - 1, lddy=2 ** 31), dict(dy=0), dict(dy=A[0] + 1), dict(lddy=23),
                                dict(codes=0), dict(ldc=32), dict(exponents=0), dict(dw=0), dict(dw=A[3] + 2), dict(lddw=39),
                                dict(accumulate=2), dict(type=1, dw_type=1, accumulate=1), dict(dw=A[0]), dict(dw=A[0] + 4 * 24 * 4 - 4),
                                dict(dw=A[1] - 16), dict(dw=A[2] + 12)])
def test_weight_grad_rejects(g, kw):
    assert _dw(**kw) == g.GEMM_F32_EINVAL
    assert g.gemm_f32_last_launches() == 0 and g.gemm_f32_last_kernel() == "none"


def test_nothing_to_do_and_no_gpu(g):
    torch = pytest.importorskip("torch")
    from accelerator_row_major_gb300 import _binding
    none = dict(dbranch=0, dresidual=0, dgate=0, dweight=0, dbias=0, dpost_weight=0, dpost_bias=0)
    assert _norm(rows=0, branch=0, residual=0, y=0) == g.GEMM_F32_OK
    assert _grad(**none) == g.GEMM_F32_OK
    assert _grad(rows=0, dy=0, no_h=True, dweight=0, dbias=0, dpost_weight=0, dpost_bias=0) == g.GEMM_F32_OK
    assert _keep(rows=0, x=0, codes=0) == g.GEMM_F32_OK and _keep(True, rows=0, x=0, codes=0) == g.GEMM_F32_OK
    assert _dw(rows=0, accumulate=1, dy=0, codes=0) == g.GEMM_F32_OK
    assert _binding.lib().gemm_f32_block_norm(None, A[0], 8, A[1], 8, A[2], 8, A[3], 8, A[4], 0) == g.GEMM_F32_EINVAL
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (lambda: _norm(), lambda: _norm(h=0, stats=0), lambda: _norm(y=A[5], h=A[6]), lambda: _norm(y=A[4], h=A[5]),
                 lambda: _norm(norm=1, bias=0, post_bias=0, weight=0), lambda: _norm(ld_gate=0), lambda: _grad(),
                 lambda: _grad(dresidual=A[5], dbranch=A[8], dgate=A[4]), lambda: _grad(dh=0, **dict(KEPT, h=0)), lambda: _keep(),
                 lambda: _keep(True), lambda: _dw(), lambda: _dw(accumulate=1), lambda: _dw(type=1, dw_type=0),
                 lambda: _grad(gate=0, ld_gate=0, post=0, post_weight=0, post_bias=0, no_branch=True, dgate=0, dpost_weight=0, dpost_bias=0)):
        assert call() == g.GEMM_F32_EDEVICE


def test_operators_need_cuda_tensors(g):
    torch = pytest.importorskip("torch")
    x, s = torch.zeros(2, 8), torch.zeros(2, 2)
    kept = g.Checkpoint(torch.zeros(2, 32).to(torch.float8_e4m3fn), torch.zeros(2, 16, dtype=torch.uint8), 8, torch.float32)
    assert kept.shape == (2, 8) and kept.device == torch.device("cpu")
    for call in (lambda: g.block_norm(x, x), lambda: g.block_norm_grad(x, x, x, x, s), lambda: g.checkpoint(x), lambda: g.restore(kept),
                 lambda: g.weight_grad(x, kept)):
        with pytest.raises(ValueError):
            call()
