"""Sizes beyond the C calls' ints, on the stand-ins of
tests/test_lm_placement_cpu.py: refused, where ctypes would pass on their lower
32 bits and a call would work on a few of the columns."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_lm_placement_cpu import Tensor, world  # noqa: E402,F401

WRAPS = 2 ** 32 + 8                   # 8 as an int


@pytest.mark.parametrize("width", [2 ** 31, WRAPS])
def test_operators_refuse_what_an_int_does_not_hold(world, width):  # noqa: F811
    g = world.g
    x, y, s, t = Tensor((1, width)), Tensor((4, 8)), Tensor((2, 1)), Tensor((1,))
    blocks = -(-width // 32)
    kept = g.Checkpoint(Tensor((1, blocks * 32), torch.float8_e4m3fn), Tensor((1, -(-blocks // 16) * 16), torch.uint8), width,
                        torch.float32)
    small = g.Checkpoint(Tensor((1, 32), torch.float8_e4m3fn), Tensor((1, 16), torch.uint8), 8, torch.float32)
    for call in (lambda: g.block_norm(x, x), lambda: g.block_norm_grad(x, x, x, None, s), lambda: g.checkpoint(x), lambda: g.restore(kept),
                 lambda: g.weight_grad(Tensor((1, 4)), kept), lambda: g.weight_grad(x, small),
                 lambda: g.layer_norm(x), lambda: g.layer_norm_grad(x, x, None, t, t),
                 lambda: g.vocab_loss(y, Tensor((width, 8)), Tensor((4,), torch.int64)),
                 lambda: g.vocab_loss_grad(x, x, Tensor((1,), torch.int64)),
                 lambda: g.matmul(Tensor((width, 4)), Tensor((4, 4))), lambda: g.matmul(y, Tensor((8, width))),
                 lambda: g.matmul(x, Tensor((width, 2)))):
        with pytest.raises(ValueError):
            call()
    assert not world.calls


def test_the_largest_int_reaches_the_library(world):  # noqa: F811
    g, most = world.g, 2 ** 31 - 1
    g.checkpoint(Tensor((1, most)))
    g.vocab_loss(Tensor((4, 8)), Tensor((most, 8)), Tensor((4,), torch.int64))
    g.matmul(Tensor((most, 1)), Tensor((1, 1)))
    assert world.calls[0][3][2] == most and world.calls[1][3][3] == most and world.calls[2][3][3] == most
