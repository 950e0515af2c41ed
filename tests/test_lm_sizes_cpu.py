"""Sizes near the end of an int, on the host: refused where tiles rounded up
would pass it, and the bands of the rescaling pass cover the columns."""
import pytest

from tests.test_lm_abi_cpu import _loss, g  # noqa: F401


@pytest.mark.parametrize("kw", [dict(width=2 ** 31 - 1, ldx=2 ** 31, ldw=2 ** 31), dict(width=2 ** 31 - 256, ldx=2 ** 31, ldw=2 ** 31),
                                dict(vocab=2 ** 31 - 256)])
@pytest.mark.parametrize("grad", [False, True])
def test_losses_beyond_the_largest_sizes_are_refused(g, kw, grad):  # noqa: F811
    from accelerator_row_major_gb300 import _binding
    if grad:
        kw = dict(kw, dx=0, dw=0)
    assert _loss(_binding.lib(), grad, **kw) == g.GEMM_F32_EINVAL


@pytest.mark.parametrize("rows", [1, 3, 32, 5000])
@pytest.mark.parametrize("vocab", [1, 9, 2049, 32001, 131072, 2 ** 31 - 257, 2 ** 31 - 2049, 2 ** 30 + 1])
def test_bands_of_the_rescaling_pass(rows, vocab):
    """The host's choice of bands and the kernel's walk through one, in 32-bit unsigned arithmetic."""
    sms, step, mask = 152, 2048, 0xFFFFFFFF
    groups, cols = (rows + 3) // 4, (vocab + 7) // 8 * 8
    bands = 8 * sms // groups + 1
    band = ((cols - 1) // bands + 1 + step - 1) // step * step
    grid = (cols - 1) // band + 1
    assert band <= mask and grid <= 65535
    end = 0
    for by in range(grid):
        first, last = by * band & mask, min(cols, (by + 1) * band & mask)
        assert first == end and last > first                 # thread 0 begins where the band before ended
        end = last
        for thread in (0, 255):
            c = first + thread * 8
            assert c <= mask
            if c < last:
                steps = (last - 1 - c) // step
                assert c + (steps + 1) * step <= mask         # the step that leaves the band does not wrap
    assert end == cols
