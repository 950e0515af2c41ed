"""The norms at a block's ends and their gradients against a plain
implementation in 64 bits (tests/_block.py has the bounds and their reasons)."""
import itertools

import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu

# one element, odd ones, each number of warps a row, slices, and the kernels that read a row again
WIDTHS = [1, 2, 7, 8, 33, 64, 129, 256, 264, 513, 777, 1024, 1032, 2048, 2056, 4096, 4100, 5000, 8192, 8200, 12296, 16384, 20001,
          32768, 32776, 40000, 140000]
FORMS = list(itertools.product(("layer", "rms"), ("none", "channel", "element"), (False, True)))


@pytest.mark.parametrize("kind,wkind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, kind, wkind):
    from tests import _block as b
    g = lib()
    for i, rows in enumerate((1, 3, 37) if width > 64 else (1, 700)):
        norm, gate, post = FORMS[(width + 5 * i + len(kind + wkind)) % len(FORMS)]
        b.both(g, b.inputs(rows, width, kind, wkind, norm, gate, post, width + rows, (1.25, 0.5)))
    b.both(g, b.inputs(2, width, kind, wkind, "layer", "channel", True, width, (1.0, 0.25)), saved=True)


@pytest.mark.parametrize("norm,gate,post", FORMS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width", [264, 1001, 4096])
def test_forms(width, kind, norm, gate, post):
    from tests import _block as b
    g = lib()
    for saved, scales in ((False, (1.0, 1.0)), (True, (1.25, 0.5))):
        s = b.inputs(50, width, kind, "f32", norm, gate, post, 3, scales)
        got, grads = b.both(g, s, saved)
        assert (grads["dbranch"] is grads["dresidual"]) == (not post and gate == "none" and scales[0] == scales[1])


@pytest.mark.parametrize("rows,width,kind,norm,gate,post,saved", [
    (5000, 1024, "bf16", "rms", "none", True, False), (4999, 777, "f32", "layer", "channel", False, False),
    (3001, 2048, "f32", "layer", "channel", True, False), (2500, 333, "bf16", "layer", "element", True, True),
    (20000, 64, "bf16", "rms", "channel", True, False), (20003, 129, "f32", "layer", "element", False, True),
    (1700, 4096, "bf16", "layer", "element", False, True), (1601, 8192, "f32", "layer", "channel", True, True),
    (1500, 8192, "bf16", "rms", "none", False, False), (1203, 12288, "bf16", "layer", "none", True, False),
    (800, 16384, "bf16", "rms", "element", True, True), (401, 32768, "f32", "layer", "none", False, False),
    (333, 40000, "bf16", "layer", "channel", True, True)])
def test_many_rows(rows, width, kind, norm, gate, post, saved):
    """More rows than the GPU works on at a time: rings that go round, threads that sum several rows, last turns that
    have a row for some groups only; and the same bits again."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(rows, width, kind, "f32", norm, gate, post, rows, (1.0, 0.5))
    got, grads = b.both(g, s, saved)
    again = b.call(g, s)
    assert all(torch.equal(got[k], again[k]) for k in got)
    kept = (g.checkpoint(got["h"]), g.checkpoint(s["branch"])) if saved else (got["h"], s["branch"])
    again = b.call_grad(g, s, *kept, got["stats"])
    assert all(torch.equal(v, again[k]) for k, v in grads.items() if v is not None)


@pytest.mark.parametrize("rows", [151, 152, 153, 303, 304, 305, 607, 608, 609, 1217])
@pytest.mark.parametrize("post", [False, True])
def test_rows_around_whole_turns(rows, post):
    """A row more or less than the SMs, or pairs of rows, take at a time."""
    from tests import _block as b
    g = lib()
    for width, kind in ((4096, "bf16"), (1040, "f32")):
        b.both(g, b.inputs(rows, width, kind, "f32", "layer", "none", post, rows))
        b.both(g, b.inputs(rows, width, kind, "f32", "rms", "channel", post, rows))


@pytest.mark.parametrize("rows", [1, 2, 151, 153, 305, 607, 1217])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
def test_rows_of_two_layer_norms(rows, gate):
    """Sums of a row that go with the next one's, rows in pairs: a row more or less than whole turns, clusters."""
    from tests import _block as b
    g = lib()
    for width, kind in ((512, "bf16"), (1001, "f32"), (4096, "bf16"), (8192, "f32"), (9000, "bf16")):
        b.both(g, b.inputs(rows, width, kind, "f32", "layer", gate, True, rows, (1.25, 0.5)))


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("rows,width,kind", [(1, 40, "f32"), (900, 1024, "bf16"), (700, 1001, "f32"), (500, 8192, "f32")])
def test_vectors_with_zeros(rows, width, kind, norm):
    """Columns whose gate or weight is 0: the gradients of either come from the sums all the same."""
    from tests import _block as b
    g = lib()
    for gate in ("channel", "none"):
        s = b.inputs(rows, width, kind, "f32", norm, gate, True, width, (1.0, -0.5))
        if gate == "channel":
            s["how"]["gate"][::3] = 0
        s["how"]["post_weight"][1::4] = 0
        s["weight"][2::5] = 0
        if norm == "layer":
            s["how"]["post_bias"] *= 8
        _, grads = b.both(g, s)
        if gate == "channel":
            assert (grads["dpost_weight"][::3] == 0).all() and grads["dpost_weight"][1::3].abs().min() > 0
            unweighted = grads["dgate"][1::4]          # the bias alone is left of the branch there
            assert unweighted.abs().min() > 0 if norm == "layer" else (unweighted == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width,ld,first", [(1000, 1003, 1), (1000, 1008, 8), (1000, 1008, 3), (5000, 5120, 0), (64, 65, 5),
                                            (9, 10, 1), (3, 3, 1), (1, 5, 2), (33000, 33001, 1), (140000, 140004, 3)])
def test_strides(kind, width, ld, first):
    """Column slices, rows that start anywhere, each matrix differently; what lies around stays as it was."""
    import torch
    from tests import _block as b
    g = lib()
    rows = 40 if width < 40000 else 6
    s = b.inputs(rows, width, kind, "f32", "layer", "element", True, ld, (1.25, 0.5))
    t = b.TYPES[kind]

    def strided(x, shift):
        room = torch.full((rows * (ld + shift) + first + 64,), 7.0, device="cuda", dtype=t)
        view = room[first + shift:first + shift + rows * (ld + shift)].view(rows, ld + shift)[:, :width]
        if x is not None:
            view.copy_(x)
        return view, room

    for i, k in enumerate(("branch", "residual", "dy", "dh")):
        s[k] = strided(s[k], i)[0]
    s["how"]["gate"] = strided(s["how"]["gate"], 4)[0]
    (y, y_room), (h, h_room) = strided(None, 1), strided(None, 2)
    got = b.call(g, s, out=y, out_h=h)
    b.check(got, b.forward(s))
    d, d_room = strided(None, 3)
    grads = b.call_grad(g, s, h, s["branch"], got["stats"], out=d)
    b.check(grads, b.gradients(s, h, s["branch"], got["stats"]))
    for view, room in ((y, y_room), (h, h_room), (d, d_room)):
        assert view.data_ptr() >= room.data_ptr()
        view.fill_(7.0)
        assert (room == 7.0).all()
    assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(700, 1024), (700, 1001), (30, 9000), (300, 8192), (20, 40000), (3, 140000)])
def test_in_place(rows, width, kind):
    """Outputs that are inputs: the stream in place, gradients over what they came from."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(rows, width, kind, "f32", "layer", "element", True, width)
    want = b.call(g, s)
    grads = b.call_grad(g, s, want["h"], s["branch"], want["stats"])
    for y, h in (("branch", "residual"), ("residual", "branch"), ("gate", "residual")):
        c = {k: v.clone() if torch.is_tensor(v) else v for k, v in s.items()}
        c["how"] = dict(s["how"], gate=s["how"]["gate"].clone())
        at = dict(c, gate=c["how"]["gate"])
        got = b.call(g, c, out=at[y], out_h=at[h])
        assert got["y"] is at[y] and got["h"] is at[h]
        assert all(torch.equal(got[k], want[k]) for k in want)
    for name in ("dy", "dh", "h", "branch", "gate"):
        c = {k: v.clone() if torch.is_tensor(v) else v for k, v in dict(s, h=want["h"]).items()}
        c["how"] = dict(s["how"], gate=s["how"]["gate"].clone())
        out = dict(c, gate=c["how"]["gate"])[name]
        got = b.call_grad(g, c, c["h"], c["branch"], want["stats"], out=out)
        assert got["dresidual"] is out
        assert all(torch.equal(got[k], v) for k, v in grads.items() if v is not None)


@pytest.mark.parametrize("rows,width,kind", [(700, 1024, "bf16"), (1500, 1001, "f32"), (300, 8192, "f32"), (20, 40000, "bf16")])
def test_branch_gradient_in_place(rows, width, kind):
    """dbranch over what it came from, by the C call: rows that are written behind the next one's sums included."""
    import ctypes
    from accelerator_row_major_gb300 import _binding, _block, _lm
    import torch
    from tests import _block as b
    g = lib()
    for gate in ("none", "channel", "element"):
        s = b.inputs(rows, width, kind, "f32", "layer", gate, True, width, (1.25, 0.5))
        fwd = b.call(g, s)
        want = b.call_grad(g, s, fwd["h"], s["branch"], fwd["stats"])["dbranch"]
        for name in ("dy", "dh", "h", "branch") + (("gate",) if gate == "element" else ()):
            c = {k: v.clone() if torch.is_tensor(v) else v for k, v in dict(s, h=fwd["h"]).items()}
            c["gate"] = None if gate == "none" else s["how"]["gate"].clone()
            how, out = dict(c["how"], gate=c["gate"]), c[name]
            block, _ = _block._block(c["dy"], _lm._matrix("dy", c["dy"]), how["kind"], 0.0, c["weight"], None, True,
                                     how["post_weight"], how["post_bias"], how["gate"], how["residual_scale"], how["branch_scale"])
            at = [ctypes.byref(_binding.Rows(c[k].data_ptr(), width)) for k in ("h", "branch")]
            g.check(_binding.lib().gemm_f32_block_norm_grad(
                ctypes.byref(block), c["dy"].data_ptr(), width, c["dh"].data_ptr(), width, *at, fwd["stats"].data_ptr(),
                out.data_ptr(), width, None, 0, None, 0, None, None, None, None, torch.cuda.current_stream().cuda_stream))
            assert torch.equal(out, want), (gate, name)


def test_what_is_not_there():
    """No weights, no biases, no dh; no rows."""
    import torch
    from tests import _block as b
    g = lib()
    for norm, post, gate in (("layer", True, "element"), ("rms", True, "channel"), ("layer", False, "none"), ("layer", True, "channel")):
        s = b.inputs(70, 520, "bf16", "bf16", norm, gate, post, 5, bias=False)
        s["weight"] = s["how"]["post_weight"] = None
        got = b.call(g, s)
        b.check(got, b.forward(s))
        grads = b.call_grad(g, s, got["h"], s["branch"], got["stats"], dh=False)
        b.check(grads, b.gradients(s, got["h"], s["branch"], got["stats"], dh=False))
        assert grads["dweight"].dtype == (torch.bfloat16 if gate == "channel" else torch.float32)
        e = b.inputs(0, 520, "bf16", "f32", norm, gate, post, 5)
        got = b.call(g, e)
        assert got["y"].shape == (0, 520) and got["stats"].shape == (4 if post else 2, 0)
        grads = b.call_grad(g, e, got["h"], e["branch"], got["stats"])
        for k in ("dweight", "dbias", "dpost_weight", "dpost_bias"):
            assert grads[k] is None or not grads[k].any()
        assert g.gemm_f32_last_kernel() == "block_columns_kernel"
    plain = torch.randn(5, 64, device="cuda")
    y, h, stats = g.block_norm(plain, plain, kind="rms")
    assert torch.equal(h, plain + plain)
    grads = g.block_norm_grad(plain, None, h, None, stats, kind="rms")
    assert grads.dbranch is grads.dresidual and grads.dbias is None and grads.dgate is None


@pytest.mark.parametrize("width", [1024, 1001, 8192, 40000])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_rows_that_are_not_finite_stay_by_themselves(norm, width):
    """A row with NaN or infinities spoils its own results alone; a row of zeros is one of zeros."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(41, width, "f32", "f32", norm, "element", True, 9)
    for t, row, v in ((s["branch"], 3, float("nan")), (s["residual"], 17, float("inf")), (s["how"]["gate"], 29, float("nan"))):
        t[row, width // 2] = v
    s["branch"][35] = s["residual"][35] = 0.0
    got = b.call(g, s)
    fine = torch.ones(41, dtype=torch.bool, device="cuda")
    fine[[3, 17, 29]] = False
    want = b.forward(s)
    for k in ("y", "h"):
        assert ((got[k].double() - want[k][0]).abs() <= want[k][1])[fine].all()
        assert not torch.isfinite(got["y"][~fine]).all(1).any()
    grads = b.call_grad(g, s, got["h"], s["branch"], got["stats"])
    want = b.gradients(s, got["h"], s["branch"], got["stats"])
    for k in ("dresidual", "dbranch", "dgate"):
        assert torch.isfinite(grads[k][fine]).all()
        assert ((grads[k].double() - want[k][0]).abs() <= want[k][1])[fine].all()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e15, 1e25])
def test_small_and_large_rows(scale):
    """Squares that vanish beside eps or overflow: as the formula in fp32 has it, and finite gradients."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(20, 1000, "f32", "f32", "layer", "none", True, 1)
    s["branch"] *= scale
    s["residual"] *= scale
    got = b.call(g, s)
    assert torch.isfinite(got["h"]).all() and torch.isfinite(got["y"]).all()
    if scale < 1e20:
        b.check(got, b.forward(s))
    grads = b.call_grad(g, s, got["h"], s["branch"], got["stats"])
    assert all(torch.isfinite(v).all() for v in grads.values() if v is not None)


@pytest.mark.parametrize("width,forward,gradient", [(1, "", ""), (1024, "", ""), (32768, "", ""), (32769, "", "_wide"),
                                                    (131073, "_wide", "_wide")])
def test_last_kernel(width, forward, gradient):
    from tests import _block as b
    g = lib()
    s = b.inputs(3, width, "bf16")
    got = b.call(g, s)
    assert g.gemm_f32_last_kernel() == "block_norm%s_kernel" % forward and g.gemm_f32_last_launches() == 1
    b.call_grad(g, s, got["h"], None, got["stats"])
    assert g.gemm_f32_last_kernel() == "block_norm_grad%s_kernel" % gradient and g.gemm_f32_last_launches() == 2


def test_gradients_against_differences():
    """(f(x + t v) - f(x - t v)) / 2 t of a scalar of the call's outputs, along random directions of every input, in 64
    bits on the formula and, to fp32's own noise, on the kernels."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(6, 96, "f32", "f32", "layer", "element", True, 2, (1.25, 0.5))
    got = b.call(g, s)
    grads = b.call_grad(g, s, got["h"], s["branch"], got["stats"])
    names = {"branch": "dbranch", "residual": "dresidual", "weight": "dweight", "bias": "dbias", "gate": "dgate",
             "post_weight": "dpost_weight", "post_bias": "dpost_bias"}
    dy, dh = s["dy"].double(), s["dh"].double()

    def value(c):
        w = b.forward(c)
        return float((w["y"][0] * dy).sum() + (w["h"][0] * dh).sum())

    def moved(name, v, t):
        c = {k: x.double() if torch.is_tensor(x) else x for k, x in s.items()}
        c["how"] = {k: x.double() if torch.is_tensor(x) else x for k, x in s["how"].items()}
        to = c if name in c else c["how"]
        to[name] = to[name] + t * v
        return c

    b.ROUND[torch.float64] = 0.0
    for name, grad in names.items():
        x = s.get(name, s["how"].get(name))
        v = torch.randn(x.shape, device="cuda", dtype=torch.float64)
        t = 1e-6                                        # differences are off by t^2 and by 2^-52 value / t: 1e-9
        slope = (value(moved(name, v, t)) - value(moved(name, v, -t))) / (2 * t)
        along = float((grads[grad].double() * v).sum())
        assert abs(slope - along) <= 1e-4 * float((grads[grad].double() * v).abs().sum()) + 1e-6, name
