"""Losses at the ends of the range: vocabulary entries whose logit is the
type's lowest value, finite logits near the largest one, and rows that are
almost certain of their target.  Tolerances as in test_gpu_vocab_loss.py."""
import pytest

from tests._gpu import lib
from tests.test_gpu_vocab_loss import _check, _exact, _inputs, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 40, 300])
@pytest.mark.parametrize("low", [None, -1e4, -1e8, -3e10, -1e30])
def test_entries_masked_with_a_low_value(low, rows, kind):
    """A column of x that is 1 and a low value (None: the type's lowest) in that column of w takes entries out of the
    vocabulary: here a band of them that fills whole tiles, and single ones."""
    torch, types = _torch()
    g = lib()
    x, w, y = _inputs(rows, 64, 1300, kind, rows)
    x[:, 0], w[:, 0] = 1.0, 0.0
    masked = torch.zeros(1300, dtype=torch.bool, device="cuda")
    masked[250:1024] = True
    masked[::7] = True
    w[masked, 0] = torch.finfo(types[kind]).min if low is None else low
    y = torch.where(y >= 0, (~masked).nonzero()[:, 0][y % int((~masked).sum())], y)
    got = g.vocab_loss_grad(x, w, y)
    kept, row = w[~masked], torch.cumsum(~masked, 0) - 1
    want, tol = _exact(x, kept, torch.where(y >= 0, row[y.clamp(min=0)], y), kind)
    _check(got[:3], (want, tol))
    _check(g.vocab_loss(x, w, y), (want, tol))
    # dx holds the masked rows of w times 0; dw of the masked entries is 0
    assert ((got[3].double() - want["dx"]).abs() <= tol["dx"]).all()
    assert ((got[4][~masked].double() - want["dw"]).abs() <= tol["dw"]).all() and (got[4][masked] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 200])
def test_rows_of_the_lowest_value_and_of_the_largest(rows, kind):
    """Every logit of some rows is the lowest finite value (equal ones: lse is that value to its last place, the loss
    log(vocab) below its rounding), and others have one logit near the largest."""
    torch, types = _torch()
    g = lib()
    vocab = 700
    x = torch.zeros((rows, 16), device="cuda", dtype=types[kind])
    w = torch.zeros((vocab, 16), device="cuda", dtype=types[kind])
    info = torch.finfo(types[kind])
    x[0, 0], x[1, 1], x[2, 2] = 1.0, 1.0, 1.0
    w[:, 0] = info.min
    w[123, 1] = info.max
    w[456, 2] = info.max / 2
    y = torch.full((rows,), 123, device="cuda")
    total, loss, lse, dx, dw = g.vocab_loss_grad(x, w, y)
    _, loss2, lse2 = g.vocab_loss(x, w, y)
    for l, z in ((loss, lse), (loss2, lse2)):
        assert abs(float(z[0]) / info.min - 1) < 1e-6 and abs(float(z[1]) / info.max - 1) < 1e-6
        assert abs(float(z[2]) / (info.max / 2) - 1) < 1e-6
        assert abs(float(l[0])) < 1e-6 * info.max and abs(float(l[1])) < 1e-6 * info.max
        assert abs(float(l[2]) / (info.max / 2) - 1) < 1e-6
    if rows > 3:                                     # the logits of the others are 0
        assert ((loss[3:] - torch.tensor(float(vocab)).log()).abs() < 1e-5).all()
    assert bool(torch.isfinite(dw[:, 3:]).all())


@pytest.mark.parametrize("rows", [5, 300])
def test_tiles_of_nothing_beside_low_logits(rows):
    """Entries of w that give logits of -inf fill whole tiles, and the others' logits lie far below 0: the gradient of
    w is 0 for the former and the formula's for the latter.  (dx multiplies 0 by the infinity.)"""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(rows, 64, 1300, "bf16", rows, ignored=0.0)
    x[:, 0], w[:, 0] = 1.0, -400.0
    none = torch.zeros(1300, dtype=torch.bool, device="cuda")
    none[200:800] = True
    w[none] = 0.0
    w[none, 0] = float("-inf")
    y = 800 + y % 500
    row = torch.cumsum(~none, 0) - 1
    want, tol = _exact(x, w[~none], row[y], "bf16")
    total, loss, lse, _, dw = g.vocab_loss_grad(x, w, y)
    _check((total, loss, lse), (want, tol))
    assert ((dw[~none].double() - want["dw"]).abs() <= tol["dw"]).all() and (dw[none] == 0).all()
