"""The example examples/train_head.py: its gradients against automatic
differentiation of the same model in 64 bits, and its loss over some steps."""
import importlib.util
import math
import os

import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")


def _example():
    lib()
    spec = importlib.util.spec_from_file_location("train_head", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("vocab,width,rows", [(500, 64, 96), (1003, 77, 300)])
def test_gradients_of_the_whole_model(vocab, width, rows):
    """The products hold 1e-5 of |A||B| and the other operators a few units of fp32; through the norm's
    division these stay of the order of 1e-5 of each gradient's largest entries, of which 1e-3 is allowed."""
    import torch
    ex = _example()
    model = ex.Model(vocab, width)
    gen = torch.Generator(device="cuda").manual_seed(3)
    followers = torch.randint(0, vocab, (vocab, ex.CHOICES), generator=gen, device="cuda")
    tokens, targets = ex.batch(followers, rows, gen)
    loss, grads = model.gradients(tokens, targets)
    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    x = p["embedding"][tokens] @ p["hidden"]
    y = torch.nn.functional.layer_norm(x, (width,), p["weight"], p["bias"], 1e-5)
    exact = torch.nn.functional.cross_entropy(y @ p["head"].t(), targets, ignore_index=-100)
    exact.backward()
    exact = float(exact.detach())
    assert abs(float(loss) - exact) <= 1e-5 * exact
    for k, d in grads.items():
        want = p[k].grad
        assert float((d.double() - want).norm()) <= 1e-3 * float(want.norm()), k


def test_loss_falls():
    """From log(vocab) before the first step to well under half of it."""
    ex = _example()
    losses = ex.train(120, 1000, 128, 1024, report=lambda s: None)
    assert abs(losses[0] - math.log(1000)) < 0.3
    assert losses[-1] < 0.55 * losses[0]
