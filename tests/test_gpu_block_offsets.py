"""Gradients of the norms at a block's ends for rows whose mean is far from 0:
hat is off by its own roundings, not by those of the mean.

The bounds are those of tests/_block.py for rows around 0: it is given h and
the branch without their means in 64 bits, and statistics whose means are 0,
so that hat's size takes the place of (|x| + |mean|) rstd; the difference of
two fp32 values is off by u of itself, the product by as much again."""
import itertools

import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


def _stats(*rows):
    """fp32 means and reciprocal deviations of rows, from 64 bits."""
    import torch
    out = []
    for x in rows:
        x = x.double()
        mean = x.mean(1)
        out += [mean.float(), (1 / ((x - mean[:, None]).square().mean(1) + 1e-5).sqrt()).float()]
    return torch.stack(out)


def _check(g, b, s, h, branch, kept=None):
    import torch
    stats = _stats(h, branch) if s["how"]["post"] else _stats(h)
    grads = b.call_grad(g, s, *(kept or (h, branch)), stats)
    for k, v in grads.items():
        assert v is None or torch.isfinite(v).all(), k
    if kept:
        h, branch = (g.restore(t) for t in kept)
    centred = stats.clone()
    centred[::2] = 0
    h = h.double() - stats[0].double()[:, None]
    if s["how"]["post"]:
        branch = branch.double() - stats[2].double()[:, None]
    b.check(grads, b.gradients(s, h, branch, centred))
    assert g.gemm_f32_status(None) == (0, 0)


FORMS = list(itertools.product(("none", "channel", "element"), (False, True)))


@pytest.mark.parametrize("gate,post", FORMS)
@pytest.mark.parametrize("offset", [10.0, 1e3, 1e4])
@pytest.mark.parametrize("rows,width,kind", [(700, 1024, "f32"), (700, 1001, "f32"), (40, 60, "f32"), (300, 8192, "f32"), (9, 40000, "f32"),
                                             (700, 1024, "bf16"), (150, 4096, "bf16")])
def test_rows_with_an_offset(rows, width, kind, offset, gate, post):
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(rows, width, kind, "f32", "layer", gate, post, width, (1.25, 0.5))
    gen = torch.Generator(device="cuda").manual_seed(width)
    shift = offset * (1 + torch.rand(rows, 1, generator=gen, device="cuda"))
    h = (s["residual"].float() + shift).to(b.TYPES[kind])
    s["branch"] = (s["branch"].float() - shift).to(b.TYPES[kind])
    _check(g, b, s, h, s["branch"])


@pytest.mark.parametrize("gate,post", FORMS)
@pytest.mark.parametrize("rows,width,kind", [(300, 1024, "bf16"), (300, 1001, "f32"), (40, 40000, "f32")])
def test_kept_rows_with_an_offset(rows, width, kind, gate, post):
    from tests import _block as b
    g = lib()
    s = b.inputs(rows, width, kind, "f32", "layer", gate, post, width, (1.25, 0.5))
    h = (s["residual"].float() + 100).to(b.TYPES[kind])
    s["branch"] = (s["branch"].float() * 30 - 200).to(b.TYPES[kind])
    _check(g, b, s, h, s["branch"], (g.checkpoint(h), g.checkpoint(s["branch"])))


@pytest.mark.parametrize("gate,post", FORMS)
@pytest.mark.parametrize("width,kind", [(64, "f32"), (61, "f32"), (40, "bf16"), (1032, "f32"), (1001, "bf16"), (9000, "f32"), (40000, "f32")])
def test_large_rows_of_one_value(width, kind, gate, post):
    """A row of 2^120 has hat 0, although its mean over its deviation (of eps alone) leaves the range; elements outside
    rows that fill no whole thread count for nothing."""
    from tests import _block as b
    g = lib()
    s = b.inputs(12, width, kind, "f32", "layer", gate, post, width)
    h = s["residual"].clone()
    h[5] = 2.0 ** 120
    s["branch"][7] = -2.0 ** 120 if post else s["branch"][7]
    _check(g, b, s, h, s["branch"])
