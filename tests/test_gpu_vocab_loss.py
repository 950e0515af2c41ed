"""The vocabulary loss and its gradients against a plain implementation in 64 bits.

Tolerances, derived from the arithmetic (A_t is the largest sum |x||w| of row
t's logits, K the width, U = 2^-24):
  logits    bfloat16 operands have exact products; the tensor core adds 16 of
            them at a time into an fp32 sum, truncating by at most one unit in
            the last place of the largest partial sum: d_t = (K/16 + 16) 2U A_t.
            fp32 operands: 256 of K at a time, of which the 16 steps of the
            largest products count (the others are below 2^-7 of them), the
            dropped products, and K/256 additions to nearest:
            d_t = (20 * 2 + 8 + K/256 + 8) U A_t.
  lse       d_t, and the exponent's rounding: 4U max|z| + 16U |lse|
  loss      twice that
  g         relative error r_t = 2 d_t + 8U max|z| + 64U of each probability;
            with bfloat16 operands 2^-11 more for e held in fp16 and half a unit
            in the last place of bfloat16 (8 significant bits: 2^-8) of g itself
  dx, dw    those errors through the products, the products' own sums
            (over the vocabulary, or the rows) as for the logits, and one
            rounding of the result.
"""
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch():
    import torch
    return torch, {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(rows, width, vocab, kind, seed, scale=1.5, ignored=0.15):
    torch, types = _torch()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rnd(rows, width).to(types[kind])
    w = (scale / width ** 0.5 * rnd(vocab, width)).to(types[kind])
    y = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    if rows > 2:
        y[torch.rand(rows, generator=gen, device="cuda") < ignored] = -100
    return x, w, y


def _sum_error(k, kind):
    """Error of a sum of k products relative to the sum of their sizes."""
    return (k / 16 + 16) * 2 * U if kind == "bf16" else (20 * 2 + 8 + k / 256 + 8) * U


def _exact(x, w, y, kind, mean=True, grad_scale=1.0, ignore=-100):
    """Values and tolerances of everything the calls return, in 64 bits."""
    torch, _ = _torch()
    xd, wd = x.double(), w.double()
    z, sizes = xd @ wd.t(), xd.abs() @ wd.abs().t()
    d = _sum_error(x.shape[1], kind) * sizes.amax(1)
    lse = torch.logsumexp(z, 1)
    counts = (y != ignore) & (y >= 0) & (y < w.shape[0])
    at = torch.where(counts, y.long(), 0)[:, None]
    loss = torch.where(counts, lse - z.gather(1, at)[:, 0], 0.0)
    n = max(1, int(counts.sum())) if mean else 1
    zmax = z.abs().amax(1)
    lse_tol = d + 4 * U * zmax + 16 * U * lse.abs() + 4 * U
    p = torch.softmax(z, 1)
    g = p.clone().scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype)) * counts[:, None]
    r = 2 * d + 8 * U * zmax + 64 * U
    g_tol = r[:, None] * p * counts[:, None]
    if kind == "bf16":
        # e is kept to 2^-12 of it, at least to 2^-25 of its tile's maximum times 2^-15
        g_tol = g_tol + (2.0 ** -11 * p + 2.0 ** -39) * counts[:, None] + 2.0 ** -8 * g.abs()
    s = grad_scale / n
    out = {"loss": loss, "lse": lse, "total": loss.sum() / n, "dx": s * (g @ wd), "dw": s * (g.t() @ xd)}
    one = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    tol = {"lse": lse_tol, "loss": 2 * lse_tol + 4 * U * loss,
           "total": (2 * lse_tol + 4 * U * loss).sum() / n + 4 * U * out["total"].abs(),
           "dx": abs(s) * (g_tol @ wd.abs() + _sum_error(w.shape[0], kind) * (g.abs() @ wd.abs())) + 1.01 * one * out["dx"].abs(),
           "dw": abs(s) * (g_tol.t() @ xd.abs() + _sum_error(x.shape[0], kind) * (g.abs().t() @ xd.abs()))
           + 1.01 * one * out["dw"].abs()}
    for k in ("dx", "dw"):          # fp32: the scale's own rounding; both: what underflows
        tol[k] = tol[k] + 4 * U * out[k].abs() + 1e-38
    return out, tol


def _check(got, exact, names=("total", "loss", "lse", "dx", "dw")):
    out, tol = exact
    for name, t in zip(names, got):
        if t is None:
            continue
        off = (t.double() - out[name]).abs()
        worst = float((off / tol[name].clamp(min=1e-300)).max()) if off.numel() else 0.0
        assert worst <= 1.0, (name, worst)


SHAPES = [(1, 1, 1), (1, 8, 2), (2, 64, 100), (3, 100, 257), (1, 4096, 1000), (37, 777, 1001), (129, 64, 128),
          (256, 256, 256), (257, 72, 513), (300, 520, 5003), (64, 4096, 2048), (513, 33, 3001), (1000, 1024, 2000),
          (128, 200, 1000), (200, 2500, 1111), (17, 5000, 700), (129, 8, 5), (2049, 16, 40)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width,vocab", SHAPES)
def test_against_64_bits(rows, width, vocab, kind):
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(rows, width, vocab, kind, rows + width + vocab)
    exact = _exact(x, w, y, kind)
    got = g.vocab_loss(x, w, y)
    assert g.gemm_f32_last_launches() >= 2
    _check(got, exact)
    full = g.vocab_loss_grad(x, w, y)
    assert g.gemm_f32_status(None) == (0, 0)
    _check(full, exact)
    assert full[3].dtype == x.dtype and full[4].dtype == w.dtype
    assert all(torch.equal(a, b) for a, b in zip(full, g.vocab_loss_grad(x, w, y)))   # a fixed order of sums


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width,vocab,piece", [(700, 136, 1003, 1), (1025, 64, 2500, 3 << 20), (513, 257, 700, 1)])
def test_pieces_of_the_rows(rows, width, vocab, piece, kind):
    """A small bound on the scratch: the rows go in pieces of 256 and more, and dw is summed over them."""
    g = lib()
    x, w, y = _inputs(rows, width, vocab, kind, rows)
    exact = _exact(x, w, y, kind, mean=False, grad_scale=0.25)
    _check(g.vocab_loss_grad(x, w, y, reduction="sum", grad_scale=0.25, piece_bytes=piece), exact)
    assert g.gemm_f32_last_launches() > 10
    only = g.vocab_loss_grad(x, w, y, reduction="sum", grad_scale=0.25, piece_bytes=piece, need_dw=False)
    assert only[4] is None
    _check(only, exact)
    only = g.vocab_loss_grad(x, w, y, reduction="sum", grad_scale=0.25, piece_bytes=piece, need_dx=False)
    assert only[3] is None
    _check(only, exact)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad,first", [(8, 0), (5, 0), (16, 8), (3, 1)])
def test_strided_operands(pad, first, kind):
    """Column slices of wider matrices: rows that TMA can read and rows that are packed first."""
    torch, types = _torch()
    g = lib()
    x, w, y = _inputs(200, 128, 900, kind, pad)

    def wide(t):
        out = torch.full((t.shape[0], first + 128 + pad), float("nan"), device="cuda", dtype=types[kind])
        out[:, first:first + 128] = t
        return out[:, first:first + 128]

    want = g.vocab_loss_grad(x, w, y)
    got = g.vocab_loss_grad(wide(x), wide(w), y)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _check(got, _exact(x, w, y, kind))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width,vocab", [(1, 1, 8), (1, 7, 9), (2, 63, 5), (16, 65, 300), (33, 1023, 2051),
                                              (31, 1022, 2049), (65, 1020, 1000), (128, 509, 1777), (129, 509, 1777),
                                              (5, 2049, 5001), (8, 121, 40000), (3, 60, 8)])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_strided_few_rows_off_boundaries(rows, width, vocab, first, kind):
    """Rows of w at every distance from a 16-byte boundary, between NaN; every class of them has a label."""
    torch, types = _torch()
    g = lib()
    x, w, y = _inputs(rows, width, vocab, kind, width + first, ignored=0.0)
    if rows > 8:
        y[:8] = torch.arange(vocab - 8, vocab, device="cuda").clamp(min=0)
    flat = torch.full((first + vocab * width + 16,), float("nan"), device="cuda", dtype=types[kind])
    wide = flat[first:first + vocab * width].view(vocab, width)
    wide.copy_(w)
    _check(g.vocab_loss(x, wide, y), _exact(x, w, y, kind))
    pitch = width + 1 + first
    flat = torch.full((first + vocab * pitch + 16,), float("nan"), device="cuda", dtype=types[kind])
    wide = flat[first:first + vocab * pitch].view(vocab, pitch)[:, :width]
    wide.copy_(w)
    got = g.vocab_loss(x, wide, y)
    _check(got, _exact(x, w, y, kind))
    assert all(torch.equal(a, b) for a, b in zip(got, g.vocab_loss(x, wide, y)))
    assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("width", [67, 130])
def test_an_infinite_row_of_w_off_boundaries(width):
    """One row of w gives a logit of -inf (a vocabulary entry that is never taken); its neighbours keep theirs.
    In bfloat16, whose products are single ones (an infinite operand in parts gives NaN)."""
    torch, _ = _torch()
    g = lib()
    kind = "bf16"
    x, w, y = _inputs(6, width, 400, kind, 5, ignored=0.0)
    x, y = x.abs() + 0.25, y.clamp(max=300)
    keep = torch.arange(400, device="cuda") != 333
    want = _exact(x, w[keep], torch.where(y > 333, y - 1, y), kind)
    w[333] = float("-inf")
    _check(g.vocab_loss(x, w, y), want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_that_do_not_count(kind):
    """No row, one row and no counted row; int32 targets; another ignore_index; a target outside the vocabulary."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(70, 96, 300, kind, 1)
    none = torch.full_like(y, -100)
    total, loss, lse, dx, dw = g.vocab_loss_grad(x, w, none)
    assert float(total) == 0 and (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    _check((None, None, lse), _exact(x, w, none, kind))
    got = g.vocab_loss_grad(x, w, y.int())
    assert all(torch.equal(a, b) for a, b in zip(got, g.vocab_loss_grad(x, w, y)))
    y2 = torch.where(y == -100, torch.full_like(y, 7), y)
    _check(g.vocab_loss_grad(x, w, y2, ignore_index=7), _exact(x, w, y2, kind, ignore=7))
    assert g.gemm_f32_status(None) == (0, 0)
    y3 = y.clone()
    y3[5], y3[6] = 300, -3
    got = g.vocab_loss_grad(x, w, y3)
    assert g.gemm_f32_status(None)[0] == g.GEMM_F32_ETARGET
    assert g.gemm_f32_status(None) == (0, 0)
    _check(got, _exact(x, w, y3, kind))
    total, loss, lse, dx, dw = g.vocab_loss_grad(x[:0], w, y[:0])
    assert float(total) == 0 and loss.shape == (0,) and dx.shape == (0, 96) and (dw == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_large_logits(kind):
    """Logits of several hundred: exponentials relative to each tile's maximum, joined over far apart tiles."""
    torch, types = _torch()
    g = lib()
    x, w, y = _inputs(40, 64, 1500, kind, 3, scale=1.0)
    x = (x.float() * 64).to(types[kind])
    w[700:] = (w[700:].float() * 4).to(types[kind])
    y[:20] = torch.arange(20, device="cuda")           # targets with losses in the hundreds
    _check(g.vocab_loss_grad(x, w, y), _exact(x, w, y, kind))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_that_are_not_finite(kind):
    """A NaN or an infinite row of x spoils its own row (and dw, which sums over the rows), as the formula does."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(12, 64, 400, kind, 4, ignored=0.0)
    x[3, 5] = float("nan")
    x[7, 0] = float("inf")
    total, loss, lse, dx, dw = g.vocab_loss_grad(x, w, y)
    keep = torch.tensor([i not in (3, 7) for i in range(12)], device="cuda")
    assert torch.isnan(total) and torch.isnan(loss[3]) and torch.isnan(lse[7]) and torch.isnan(dx[3]).all()
    out, tol = _exact(x[keep], w, y[keep], kind)
    assert ((loss[keep].double() - out["loss"]).abs() <= tol["loss"]).all()
    assert ((lse[keep].double() - out["lse"]).abs() <= tol["lse"]).all()
    assert ((dx[keep].double() * 12 - out["dx"] * 10).abs() <= tol["dx"] * 10 + 2.0 ** -8 * out["dx"].abs() * 10).all()


def test_gradient_against_differences():
    """Central differences of the mean loss in 64 bits along random directions of x and w.

    With logits of scale 1.5 the third derivative along a unit direction is of
    order 1, so at step 1e-3 the difference is off by about 1e-7; the kernels'
    fp32 error is below 1e-5 of the gradient, and 1e-4 of it is allowed."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(33, 72, 301, "f32", 8)
    _, _, _, dx, dw = g.vocab_loss_grad(x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(2)
    f = lambda a, b: _exact(a, b, y, "f32")[0]["total"]  # noqa: E731
    for grad, at in ((dx, 0), (dw, 1)):
        for _ in range(3):
            v = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
            v /= v.norm()
            up, down = [x.double(), w.double()], [x.double(), w.double()]
            up[at], down[at] = up[at] + 1e-3 * v, down[at] - 1e-3 * v
            diff = (f(*up) - f(*down)) / 2e-3
            assert abs(float(diff - (grad.double() * v).sum())) <= 1e-4 * float(grad.double().norm()) + 1e-7


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_another_stream_and_graph_capture(kind):
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(300, 200, 2000, kind, 3)
    want = g.vocab_loss_grad(x, w, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g.vocab_loss_grad(x, w, y, stream=s)               # sizes this stream's scratch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = g.vocab_loss_grad(x, w, y)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.gemm_f32_status(s) == (0, 0)


def test_refusals():
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(6, 16, 20, "f32", 1)
    for bad in (lambda: g.vocab_loss(x, w[:, :8], y), lambda: g.vocab_loss(x, w.bfloat16(), y),
                lambda: g.vocab_loss(x, w, y[:5]), lambda: g.vocab_loss(x, w, y.float()),
                lambda: g.vocab_loss(x.cpu(), w, y), lambda: g.vocab_loss(x, w, y, reduction="none"),
                lambda: g.vocab_loss(x.t(), w, y), lambda: g.vocab_loss(x[0], w, y),
                lambda: g.vocab_loss(x.half(), w.half(), y), lambda: g.vocab_loss_grad(x, w[:0], y)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g.GemmError):
        g.vocab_loss_grad(x, w, y, grad_scale=float("inf"))
