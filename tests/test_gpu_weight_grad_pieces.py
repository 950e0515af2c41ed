"""The weight gradient over many rows: what the tensor cores' truncating sums
take from it stays that of 1024 rows, in either type of result."""
import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("into", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows", [8192, 32768])
def test_no_drift_with_the_rows(rows, into):
    """Positive operands, tiles enough that each is summed over all rows by one pair of SMs: the mean of the relative
    errors, u = 2^-24.  The tensor cores round 64 times in a sum of 1024, each time towards zero by at most 2 u of what has
    come together, a 64th more each time: 64 u of the sum.  These sums are added to nearest, rows / 1024 u at most.  The
    roundings of the results, at most 2^-8 of each and as often up as down, leave 2^-8 / sqrt(count) standard deviations
    or less in the mean of count of them, of which six are allowed."""
    import torch
    g = lib()
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    out, width = 512, 256 * pairs
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dy = (torch.rand(rows, out, generator=gen, device="cuda") * (1 + torch.rand(out, generator=gen, device="cuda"))).bfloat16()
    x = torch.rand(rows, width, generator=gen, device="cuda").bfloat16()
    saved = g.checkpoint(x)
    x = g.restore(saved)
    dw = g.weight_grad(dy, saved, out=torch.empty(out, width, device="cuda", dtype=getattr(torch, into)))
    total, count = 0.0, out * width
    for c in range(0, width, 2048):
        want = dy.double().t() @ x[:, c:c + 2048].double()
        total += float(((dw[:, c:c + 2048].double() - want) / want).sum())
    u = 2.0 ** -24
    assert abs(total / count) <= (64 + rows / 1024) * u + 6 * 2.0 ** -8 / count ** 0.5
    assert g.gemm_f32_status(None) == (0, 0)
