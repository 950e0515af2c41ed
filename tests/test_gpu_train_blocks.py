"""The example examples/train_blocks.py: its gradients against automatic
differentiation of the same model in 64 bits, and that it runs."""
import importlib.util
import math
import os

import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_blocks.py")


def _example():
    lib()
    spec = importlib.util.spec_from_file_location("train_blocks", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _reference(g, model, tokens, targets):
    """Loss and gradients in 64 bits; where the model keeps activations in 8 bits, so does the backward pass here."""
    import torch

    def kept(x):
        return g.restore(g.checkpoint(x.float())).double() if model.saved else x

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(kept(x), w)
            return x @ w.t()

        @staticmethod
        def backward(ctx, dz):
            x, w = ctx.saved_tensors
            return dz @ w, dz.t() @ x

    class Relu(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            y = x.relu()
            ctx.save_for_backward(kept(y))
            return y

        @staticmethod
        def backward(ctx, dy):
            return dy * (ctx.saved_tensors[0] > 0)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            mean = x.mean(1, keepdim=True)
            rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
            ctx.save_for_backward((kept(x) - mean) * rstd, rstd, w)
            return (x - mean) * rstd * w + b

        @staticmethod
        def backward(ctx, dy):
            hat, rstd, w = ctx.saved_tensors
            g_ = dy * w
            return rstd * (g_ - g_.mean(1, keepdim=True) - hat * (g_ * hat).mean(1, keepdim=True)), (dy * hat).sum(0), dy.sum(0)

    class Scale(torch.autograd.Function):
        """scale times the branch's norm, which the backward pass takes from what was kept of the branch."""
        @staticmethod
        def forward(ctx, p, s, again):
            ctx.save_for_backward(again, s)
            return p * s

        @staticmethod
        def backward(ctx, d):
            again, s = ctx.saved_tensors
            return d * s, (d * again).sum(0), None

    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    h = p["embedding"][tokens]
    y = torch.nn.functional.layer_norm(h, h.shape[1:], p["first"], p["first_bias"], 1e-5)
    for i in range(model.blocks):
        branch = Linear.apply(Relu.apply(Linear.apply(y, p["up%d" % i])), p["down%d" % i])
        post = Norm.apply(branch, p["post%d" % i], p["post_bias%d" % i])
        with torch.no_grad():
            mean = branch.mean(1, keepdim=True)
            rstd = 1 / ((branch - mean).square().mean(1, keepdim=True) + 1e-5).sqrt()
            again = (kept(branch) - mean) * rstd * p["post%d" % i] + p["post_bias%d" % i]
        h = h + Scale.apply(post, p["scale%d" % i], again)
        y = Norm.apply(h, p["norm%d" % i], p["bias%d" % i])
    loss = torch.nn.functional.cross_entropy(y @ p["head"].t(), targets, ignore_index=-100)
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("vocab,width,blocks,rows", [(300, 64, 1, 96), (500, 77, 3, 300)])
def test_gradients_of_the_whole_model(vocab, width, blocks, rows, saved):
    """The products hold 1e-5 of |A||B| and the other operators a few units of fp32: through the norms' divisions these
    stay of the order of 1e-5 of each gradient's size, of which 1e-3 is allowed.  In 8 bits an activation that is off by
    1e-5 lies across a border between two codes, 2^-4 apart, 3 times in 10,000, and then a gradient's term is off by 2^-3:
    sqrt(3e-4) / 8 = 2e-3 of its size, of which 1e-2 is allowed."""
    import torch
    ex = _example()
    model = ex.Model(vocab, width, blocks, saved)
    gen = torch.Generator(device="cuda").manual_seed(3)
    followers = torch.randint(0, vocab, (vocab, ex.CHOICES), generator=gen, device="cuda")
    tokens, targets = ex.batch(followers, rows, gen)
    loss, grads = model.gradients(tokens, targets)
    exact, want = _reference(ex.g, model, tokens, targets)
    assert abs(float(loss) - exact) <= 1e-5 * exact
    assert set(grads) == set(want)
    for k, d in grads.items():
        assert float((d.double() - want[k]).norm()) <= (1e-2 if saved else 1e-3) * float(want[k].norm()), k


def test_it_runs():
    ex = _example()
    losses = ex.train(25, 500, 96, 2, 512, report=lambda s: None)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses) and abs(losses[0] - math.log(500)) < 0.5
