"""8-bit checkpoints, exactly, and the weight gradient from them, against
64 bits."""
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


def _power(e):
    """2^e, from its bits."""
    import torch
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept(x):
    """(values, exponents + 127) by arithmetic in 64 bits; NaN where x is not finite."""
    import torch
    rows, width = x.shape
    blocks = -(-width // 32)
    v = torch.zeros(rows, blocks * 32, dtype=torch.float64, device=x.device)
    v[:, :width] = x
    v = v.view(rows, blocks, 32)
    finite = torch.where(v.isfinite(), v, 0.0)
    top = finite.abs().amax(2, keepdim=True)
    e = torch.frexp(torch.where(top > 0, top, 1.0)).exponent - 9
    e = torch.where(top > 448 * _power(e), e + 1, e)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    q = finite / _power(e)
    step = _power(torch.frexp(torch.where(q == 0, 1.0, q)).exponent.clamp(min=-5) - 4)
    q = torch.round(q / step) * step
    q = torch.where(e == 120, q.clamp(-240, 240), q)            # 256 would stand for 2^128
    q = torch.where(v.isfinite(), q * _power(e), float("nan"))
    return q.flatten(1)[:, :width], (e[:, :, 0] + 127).to(torch.uint8)


def _check(g, x):
    import torch
    saved = g.checkpoint(x)
    rows, width = x.shape
    blocks = -(-width // 32)
    values, exponents = _kept(x)
    assert saved.shape == (rows, width) and saved.dtype == x.dtype and saved.codes.shape == (rows, blocks * 32)
    assert torch.equal(saved.exponents[:, :blocks], exponents)
    codes = saved.codes.double()
    assert not codes[:, width:].any()
    got = codes.view(rows, blocks, 32) * _power(exponents.int() - 127)[:, :, None]
    got = got.flatten(1)[:, :width]
    assert torch.equal(got.isnan(), values.isnan())
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(values))
    back = g.restore(saved)
    assert back.dtype == x.dtype
    want = values.to(x.dtype)
    assert torch.equal(back.isnan(), want.isnan()) and torch.equal(torch.nan_to_num(back), torch.nan_to_num(want))
    assert g.gemm_f32_status(None) == (0, 0)
    return saved, back


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 31), (4, 32), (4, 33), (2, 255), (3, 256), (3, 257), (37, 777), (64, 1024),
                                        (9, 1001), (2, 40000), (5000, 40), (3000, 129), (700, 4096)])
def test_values(rows, width, kind):
    import torch
    g = lib()
    gen = torch.Generator(device="cuda").manual_seed(rows + width)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-12, 12, (rows, width), generator=gen, device="cuda").float())
    _check(g, x.to(getattr(torch, kind)))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_edges_of_the_formats(kind):
    """Powers of two and their neighbours, ties between codes, codes below the normal ones, the types' ends, zeros of
    both signs, what is not finite."""
    import torch
    g = lib()
    t = getattr(torch, kind)
    fi = torch.finfo(t)
    cases = [torch.tensor([448.0, 447.0, 449.0, 464.0, 1.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, -2.0 ** -10]),
             torch.tensor([fi.max, -fi.max, 1.0, fi.tiny, 0.0]), torch.tensor([fi.tiny, -fi.tiny / 4, fi.tiny / 64, 0.0, -0.0]),
             torch.tensor([fi.smallest_normal * 2 ** k for k in range(0, 30)]), torch.zeros(5), torch.tensor([-0.0, 0.0]),
             torch.tensor([float("nan"), 3.0, -1.0]), torch.tensor([float("inf"), -float("inf"), 5.0, 0.3]),
             torch.tensor([float("nan")] * 4), torch.tensor([1.0 + k / 32 for k in range(32)]),
             torch.tensor([448.0 * (1 + k / 64) for k in range(-16, 16)])]
    for scale in (1.0, 2.0 ** -20, 2.0 ** 40):
        x = torch.zeros(len(cases), 100)
        for i, c in enumerate(cases):
            x[i, 30:30 + len(c)] = c
            x[i, 96] = c[0]
        x = (x * scale).to(t).cuda()
        saved, back = _check(g, x)
        finite = x.isfinite()
        zero = (x == 0) & finite
        assert torch.equal(torch.signbit(back[zero]), torch.signbit(x[zero]))
        off = (back.double() - x.double()).abs()[finite]
        power = _power(saved.exponents[:, :4].int() - 127).repeat_interleave(32, 1)[:, :100][finite]
        assert (off <= torch.maximum(x.double().abs()[finite] / 16, power / 1024)).all()


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("first", range(0, 9))
@pytest.mark.parametrize("ld", [300, 301, 302, 304, 307])
def test_rows_that_start_anywhere(first, ld, kind):
    """The same codes from wherever the rows lie, and nothing written around them."""
    import torch
    g = lib()
    t, rows, width = getattr(torch, kind), 70, 300
    x = torch.randn(rows, width, device="cuda").to(t)
    room = torch.full((rows * ld + first + 16,), float("inf"), device="cuda", dtype=t)
    view = room[first:first + rows * ld].view(rows, ld)[:, :width]
    view.copy_(x)
    want, saved = g.checkpoint(x), g.checkpoint(view)
    assert torch.equal(saved.codes.view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(saved.exponents[:, :10], want.exponents[:, :10])
    view.fill_(3.0)
    g.restore(saved, out=view)
    assert torch.equal(view, g.restore(want))
    view.fill_(float("inf"))
    assert (room == float("inf")).all()
    tight = torch.full((width,), 5.0, device="cuda", dtype=t)      # nothing of the allocation around a single row
    s = g.checkpoint(tight[1:].view(1, -1))
    assert torch.equal(g.restore(s), tight[1:].view(1, -1))
    assert g.gemm_f32_status(None) == (0, 0)


def test_beyond_32_bits():
    """More than 2^31 elements: rows at the far end."""
    import torch
    g = lib()
    rows, width = 530000, 4096
    x = torch.zeros((rows, width), device="cuda", dtype=torch.bfloat16)
    far = torch.randn(100, width, device="cuda").bfloat16()
    x[-100:] = far
    saved = g.checkpoint(x)
    values, exponents = _kept(far)
    assert torch.equal(saved.exponents[-100:, :128], exponents)
    x.fill_(1.0)
    g.restore(saved, out=x)
    assert torch.equal(x[-100:].double(), values) and not x[:100].any() and not x[rows // 2].any()
    y, h, stats = g.block_norm(x, x, kind="rms", out=x, residual_scale=0.5, branch_scale=0.5)
    want = values / (values.square().mean(1, keepdim=True) + 1e-5).sqrt()
    assert ((x[-100:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    assert torch.equal(h[-100:].double(), values)


def _dw_check(dy, x, dw, add=None):
    """u = 2^-24; each product of bfloat16 values is exact, or, of an fp32 dy in three parts, off by 2^-23 of itself; the
    tensor cores add into their sums by truncation, up to 1024 of K, or all of a bfloat16 result's, one rounding for
    every 16: (K / 8 + 64) u of the terms' sizes; the rest is a rounding of the result."""
    import torch
    K = dy.shape[0]
    want = dy.double().t() @ x.double() + (add.double() if add is not None else 0)
    size = dy.double().abs().t() @ x.double().abs() + (add.double().abs() if add is not None else 0)
    chain = K if dw.dtype is torch.bfloat16 else min(K, 1024)
    bound = (chain / 8 + K / 256 + 80) * 2.0 ** -24 * size + (2.0 ** -8 if dw.dtype is torch.bfloat16 else 2.0 ** -24) * want.abs()
    assert dw.shape == want.shape and ((dw.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,width,out", [(1, 1, 1), (1, 64, 40), (7, 33, 5), (64, 256, 256), (65, 257, 255), (300, 777, 513),
                                            (1001, 1000, 64), (4096, 512, 320), (5000, 96, 2000), (16, 4096, 4096)])
def test_weight_gradient(rows, width, out, kind):
    import torch
    g = lib()
    t = getattr(torch, kind)
    dy, x = torch.randn(rows, out, device="cuda").to(t), torch.randn(rows, width, device="cuda").to(t)
    saved = g.checkpoint(x)
    values = _kept(x)[0]
    dw = g.weight_grad(dy, saved)
    assert dw.dtype == t and g.gemm_f32_last_kernel() == "half_gemm_kernel"
    _dw_check(dy, values, dw)
    assert torch.equal(dw, g.weight_grad(dy, saved))
    wide = torch.full((out, width), 2.0, device="cuda")
    _dw_check(dy, values, g.weight_grad(dy, saved, out=wide))
    before = wide.clone()
    assert g.weight_grad(dy, saved, out=wide, accumulate=True) is wide
    _dw_check(dy, values, wide, before)
    assert g.gemm_f32_status(None) == (0, 0)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_weight_gradient_of_slices(kind):
    """A dy and a dw that are column slices, on boundaries and off them; what lies around stays."""
    import torch
    g = lib()
    t, rows, width, out = getattr(torch, kind), 500, 200, 130
    x = torch.randn(rows, width, device="cuda").to(t)
    saved, values = g.checkpoint(x), _kept(x)[0]
    for first, ld in ((0, 136), (8, 144), (1, 133), (3, 200)):
        dy = torch.randn(rows * ld + first, device="cuda").to(t)[first:].view(rows, ld)[:, :out]
        room = torch.full((out * 210 + first,), 9.0, device="cuda", dtype=t)
        dw = room[first:].view(out, 210)[:, :width]
        g.weight_grad(dy, saved, out=dw)
        _dw_check(dy, values, dw)
        dw.fill_(9.0)
        assert (room == 9.0).all()


def test_no_rows():
    import torch
    g = lib()
    x = torch.zeros((0, 50), device="cuda")
    saved = g.checkpoint(x)
    assert saved.shape == (0, 50) and g.restore(saved).shape == (0, 50)
    dw = torch.full((7, 50), 3.0, device="cuda")
    g.weight_grad(torch.zeros((0, 7), device="cuda"), saved, out=dw, accumulate=True)
    assert (dw == 3.0).all()
    assert not g.weight_grad(torch.zeros((0, 7), device="cuda"), saved, out=dw).any()
    assert g.gemm_f32_last_kernel() == "memset"
