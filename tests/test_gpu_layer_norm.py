"""Layer norm and its gradient against a plain implementation in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24 for an fp32 value, 2^-9
for a result rounded to bfloat16):
  - a row's mean is a sum of D terms in a tree of depth at most about
    D / 1024 + 24: its error is below 64 u mean|x| for every width here;
  - hat = (x - mean) rstd: the subtraction is exact to u (|x| + |mean|), so
    hat is off by at most (64 + 4) u (max|x|) rstd, and by the relative error
    of rstd (below 64 u), and y by that times |weight|, plus one rounding;
  - dx is rstd times a difference of terms of size |g|, mean|g| and
    |hat| mean|g hat|, each off by at most 128 u of its size;
  - a column sum over R rows is a tree of depth below R / 16 + 64 whose
    terms are off by 80 u.
"""
import numpy as np
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}     # one rounding, relative (a full unit for bf16's half way)


def _torch():
    import torch
    return torch, {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(rows, width, kind, wkind, seed, offset=0.5):
    torch, types = _torch()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = (rnd(rows, width) + offset * rnd(rows, 1)).to(types[kind])
    dy = rnd(rows, width).to(types[kind])
    w = (1 + 0.1 * rnd(width)).to(types[wkind])
    b = (0.1 * rnd(width)).to(types[wkind])
    return x, dy, w, b


def _exact(x, w, b, eps):
    x, w, b = x.double(), w.double(), b.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    return (x - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]


def _check_forward(x, w, b, eps, y, mean, rstd, kind):
    ye, me, re = _exact(x, w, b, eps)
    xd = x.double()
    assert ((mean.double() - me).abs() <= 64 * U * xd.abs().mean(1)).all()
    # rstd: the centred squares carry the mean's error
    assert ((rstd.double() - re).abs() <= 64 * U * re * (1 + xd.abs().amax(1) * re)).all()
    big = xd.abs().amax(1, keepdim=True) * re[:, None]
    hat = (xd - me[:, None]) * re[:, None]
    tol = (68 * U * big + 64 * U * (1 + big) * hat.abs()) * w.double().abs() + 4 * U * (ye.abs() + b.double().abs())
    assert ((y.double() - ye).abs() <= tol + ROUND[kind] * ye.abs()).all()


def _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, wkind):
    xd, g0, wd = x.double(), dy.double(), w.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    hat, D, R = (xd - m) * r, x.shape[1], x.shape[0]
    g = g0 * wd
    dxe = r * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + hat.abs() * (g * hat).abs().mean(1, keepdim=True)
                + (xd.abs() + m.abs()) * r * (g * hat).abs().mean(1, keepdim=True))
    assert ((dx.double() - dxe).abs() <= 128 * U * size + ROUND[kind] * dxe.abs()).all()
    depth = (R / 16 + 144) * U
    terms = (g0.abs() * (hat.abs() + (xd.abs() + m.abs()) * r)).sum(0)
    dwe, dbe = (g0 * hat).sum(0), g0.sum(0)
    assert ((dw.double() - dwe).abs() <= depth * terms + ROUND[wkind] * dwe.abs()).all()
    assert ((db.double() - dbe).abs() <= depth * g0.abs().sum(0) + ROUND[wkind] * dbe.abs()).all()


# widths: one element, odd ones, every register layout's last and first width, and the wide kernels
WIDTHS = [1, 2, 7, 64, 129, 256, 264, 513, 777, 1024, 1032, 2048, 2056, 4096, 4100, 5000, 8192, 8200, 9001,
          16384, 16392, 32768, 40000]


@pytest.mark.parametrize("kind,wkind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width", WIDTHS)
def test_against_64_bits(width, kind, wkind):
    g = lib()
    for rows in (1, 3, 37) if width > 64 else (1, 1000):
        x, dy, w, b = _inputs(rows, width, kind, wkind, width + rows)
        y, mean, rstd = g.layer_norm(x, w, b, eps=1e-5)
        assert g.gemm_f32_last_kernel() == "layer_norm_kernel"
        _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
        dx, dw, db = g.layer_norm_grad(dy, x, w, mean, rstd)
        assert dw.dtype == w.dtype and dx.dtype == x.dtype
        _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, wkind)
        assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("rows,width,kind", [(5000, 1024, "bf16"), (4999, 777, "f32"), (3001, 2048, "f32"),
                                             (2500, 333, "bf16"), (700, 8192, "bf16")])
def test_many_rows(rows, width, kind):
    """More rows than the persistent grid has groups: each thread sums several rows."""
    g = lib()
    x, dy, w, b = _inputs(rows, width, kind, "f32", rows)
    y, mean, rstd = g.layer_norm(x, w, b)
    _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
    dx, dw, db = g.layer_norm_grad(dy, x, w, mean, rstd)
    _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, "f32")
    again = g.layer_norm_grad(dy, x, w, mean, rstd)
    torch, _ = _torch()
    assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again))   # a fixed order of sums


@pytest.mark.parametrize("kind,wkind", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_streamed_rows_of_every_width(kind, wkind):
    """Enough rows for the streaming kernels at each of their widths, on 16-byte rows and others, in one
    process and in this order: every kernel sets up its own shared memory."""
    g = lib()
    for width in (1024, 256, 8, 512, 264, 2048, 1032, 4096, 8192, 4104, 16384, 8200, 20000,
                  1023, 255, 3, 511, 259, 2047, 1025, 4095, 8190, 4097, 16383, 8201, 20001):
        rows = 10000 if width <= 1024 else 5000 if width <= 2048 else 2500 if width <= 4096 else 1300
        x, dy, w, b = _inputs(rows, width, kind, wkind, width)
        y, mean, rstd = g.layer_norm(x, w, b)
        _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
        dx, dw, db = g.layer_norm_grad(dy, x, w, mean, rstd)
        _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, wkind)
        assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("width,offset", [(777, 1), (777, 3), (1024, 5), (100, 7), (33, 2), (258, 4)])
def test_streamed_rows_at_every_alignment(width, offset, apart, kind):
    """Dense rows of which the first starts off a 16-byte boundary, equally far in x, dy and the results
    (streamed) or not (loaded by the threads)."""
    torch, types = _torch()
    g = lib()
    rows = 10000
    x, dy, w, b = _inputs(rows, width, kind, "f32", width + offset)

    def shifted(t, by):
        buf = torch.full((rows * width + 32,), 7.0, device="cuda", dtype=types[kind])
        view = buf[by:by + rows * width].view(rows, width)
        if t is not None:
            view.copy_(t)
        return buf, view

    (_, xs), (_, ds) = shifted(x, offset), shifted(dy, (offset + apart) % 8)
    buf, out = shifted(None, (offset + 2 * apart) % 8)
    y, mean, rstd = g.layer_norm(xs, w, b, out=out)
    _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
    dbuf, dout = shifted(None, (offset + 4 * apart) % 8)
    dx, dw, db = g.layer_norm_grad(ds, xs, w, mean, rstd, out=dout)
    _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, "f32")
    for t, by in ((buf, (offset + 2 * apart) % 8), (dbuf, (offset + 4 * apart) % 8)):
        assert (t[:by] == 7).all() and (t[by + rows * width:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width,pad,first", [(256, 8, 0), (256, 1, 0), (96, 5, 3), (1000, 16, 8), (9000, 7, 1)])
def test_strided_rows(width, pad, first, kind):
    """Column slices of a wider matrix: strides and bases that do and do not keep 16-byte alignment."""
    torch, types = _torch()
    g = lib()
    x, dy, w, b = _inputs(23, width, kind, "f32", pad)

    def wide(t):
        out = torch.full((23, first + width + pad), 7.0, device="cuda", dtype=types[kind])
        out[:, first:first + width] = t
        return out, out[:, first:first + width]

    (_, xs), (_, ds) = wide(x), wide(dy)
    buf, ys = wide(torch.zeros_like(x))
    y, mean, rstd = g.layer_norm(xs, w, b, out=ys)
    _check_forward(x, w, b, 1e-5, y, mean, rstd, kind)
    dbuf, os_ = wide(torch.zeros_like(x))
    dx, dw, db = g.layer_norm_grad(ds, xs, w, mean, rstd, out=os_)
    _check_grad(x, dy, w, mean, rstd, dx, dw, db, kind, "f32")
    for t in (buf, dbuf):                            # nothing outside the window is written
        assert (t[:, :first] == 7).all() and (t[:, first + width:] == 7).all()


@pytest.mark.parametrize("width", [512, 777, 20001])
def test_in_place(width):
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(65, width, "f32", "f32", 5)
    y, mean, rstd = g.layer_norm(x, w, b)
    want = g.layer_norm_grad(dy, x, w, mean, rstd)
    over_dy, over_x, xc = dy.clone(), x.clone(), x.clone()
    assert torch.equal(g.layer_norm(xc, w, b, out=xc)[0], y)
    for out, other in ((over_dy, x), (over_x, dy)):
        got = g.layer_norm_grad(out, other, w, mean, rstd, out=out) if out is over_dy else \
            g.layer_norm_grad(other, out, w, mean, rstd, out=out)
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_without_weights_and_without_rows():
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(40, 300, "f32", "f32", 9)
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    assert torch.equal(g.layer_norm(x)[0], g.layer_norm(x, one, zero)[0])
    y, mean, rstd = g.layer_norm(x)
    assert all(torch.equal(a, c) for a, c in zip(g.layer_norm_grad(dy, x, None, mean, rstd),
                                                 g.layer_norm_grad(dy, x, one, mean, rstd)))
    y, mean, rstd = g.layer_norm(x[:0], w, b)
    assert y.shape == (0, 300) and mean.shape == (0,)
    dx, dw, db = g.layer_norm_grad(dy[:0], x[:0], w, mean, rstd)
    assert dx.shape == (0, 300) and (dw == 0).all() and (db == 0).all()


def test_constant_rows_and_values_that_are_not_finite():
    """A constant row has variance 0: hat is 0 and rstd 1 / sqrt(eps).  Infinities and NaN stay in their row."""
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(6, 512, "f32", "f32", 11)
    x[1] = 3.0
    x[2, 7] = float("inf")
    x[3, 0] = float("nan")
    y, mean, rstd = g.layer_norm(x, w, b, eps=1e-5)
    assert torch.equal(y[1], b) and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    rows = torch.tensor([0, 1, 4, 5], device="cuda")
    _check_forward(x[rows], w, b, 1e-5, y[rows], mean[rows], rstd[rows], "f32")
    large = torch.full((2, 64), 1e20, device="cuda")
    large[:, ::2] = -1e20                            # the squares overflow in fp32: rstd 0, as the formula gives
    y, mean, rstd = g.layer_norm(large, eps=1e-5)
    assert (rstd == 0).all() and (y == 0).all()


@pytest.mark.parametrize("width", [48, 777])
def test_gradient_against_differences(width):
    """Central differences of sum(dy * y) in 64 bits along random directions of x, weight and bias.

    The loss is smooth with curvature of order 1 per direction of unit norm;
    at step 1e-4 the difference is off by about 1e-8 of the gradient's scale,
    far below the kernels' fp32 error, for which 1e-4 of the scale is ample."""
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(9, width, "f32", "f32", width)
    y, mean, rstd = g.layer_norm(x, w, b, eps=1e-3)
    dx, dw, db = g.layer_norm_grad(dy, x, w, mean, rstd)
    gen = torch.Generator(device="cuda").manual_seed(1)
    f = lambda xx, ww, bb: (dy.double() * _exact(xx, ww, bb, 1e-3)[0]).sum()  # noqa: E731
    at = [x.double(), w.double(), b.double()]
    for k, grad in enumerate((dx, dw, db)):
        for _ in range(3):
            v = torch.randn(at[k].shape, generator=gen, device="cuda", dtype=torch.float64)
            v /= v.norm()
            up, down = list(at), list(at)
            up[k], down[k] = at[k] + 1e-4 * v, at[k] - 1e-4 * v
            diff = (f(*up) - f(*down)) / 2e-4
            assert abs(float(diff - (grad.double() * v).sum())) <= 1e-4 * float(grad.double().norm())


def test_another_stream_and_graph_capture():
    torch, _ = _torch()
    g = lib()
    x, dy, w, b = _inputs(300, 1000, "bf16", "f32", 3)
    want = g.layer_norm(x, w, b)
    want_g = g.layer_norm_grad(dy, x, w, want[1], want[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g.layer_norm_grad(dy, x, w, *g.layer_norm(x, w, b)[1:])       # sizes this stream's scratch
        graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = g.layer_norm(x, w, b)
        got_g = g.layer_norm_grad(dy, x, w, got[1], got[2])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got + got_g, want + want_g))


def test_refusals():
    torch, _ = _torch()
    g = lib()
    x = torch.zeros((4, 8), device="cuda")
    w = torch.ones(8, device="cuda")
    stat = torch.zeros(4, device="cuda")
    for bad in (lambda: g.layer_norm(x.cpu(), w), lambda: g.layer_norm(x.half(), w), lambda: g.layer_norm(x[0], w),
                lambda: g.layer_norm(x, w[:7]), lambda: g.layer_norm(x, w.bfloat16()),
                lambda: g.layer_norm(x.t(), w[:4]), lambda: g.layer_norm(x, w, out=x[:3]),
                lambda: g.layer_norm(x[:, :0]), lambda: g.layer_norm(x[:1].expand(4, 8), w),
                lambda: g.layer_norm(x.bfloat16(), w, w.bfloat16()),
                lambda: g.layer_norm_grad(x[:2], x, w, stat, stat),
                lambda: g.layer_norm_grad(x, x, w, stat[:3], stat)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g.GemmError):
        g.layer_norm(x, w, eps=-1.0)
    base = torch.zeros(64, device="cuda")
    with pytest.raises(g.GemmError):                 # y starts inside x
        g.layer_norm(base[:32].view(4, 8), w, out=base[8:40].view(4, 8))
    assert np.isfinite(g.layer_norm(x, w)[0].cpu().numpy()).all()
