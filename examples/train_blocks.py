"""Trains a model of residual blocks whose activations are kept in 8 bits.

    python examples/train_blocks.py [--steps 200] [--vocab 2000] [--width 256] [--blocks 4] [--rows 2048] [--full]

The text is the Markov chain of train_head.py.  A block multiplies the normed
stream by a matrix, takes what is positive and multiplies by a second matrix
(gemm_f32_general); block_norm adds the result to the stream, through a norm
and a learned scale per channel, and norms the stream for the next block.
What the backward pass needs of each block, the two products' inputs, the
stream and the block's output, is kept by checkpoint: 1.03 bytes an element
where fp32 takes 4 (--full keeps them as they are).  The weights' gradients
come from weight_grad, those of the norms, scales and stream from
block_norm_grad, the head's from vocab_loss_grad.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import accelerator_row_major_gb300 as g  # noqa: E402
from train_head import CHOICES, batch, product  # noqa: E402


class Model:
    def __init__(self, vocab, width, blocks, saved=True, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.saved, self.blocks = saved, blocks
        self.params = {"embedding": rnd(vocab, width), "head": 0.02 * rnd(vocab, width), "first": torch.ones(width, device="cuda"),
                       "first_bias": torch.zeros(width, device="cuda")}
        for i in range(blocks):
            self.params.update({"up%d" % i: rnd(2 * width, width) / math.sqrt(width), "down%d" % i: rnd(width, 2 * width) / math.sqrt(width),
                                "scale%d" % i: torch.full((width,), 0.3, device="cuda"), "post%d" % i: torch.ones(width, device="cuda"),
                                "post_bias%d" % i: torch.zeros(width, device="cuda"), "norm%d" % i: torch.ones(width, device="cuda"),
                                "bias%d" % i: torch.zeros(width, device="cuda")})
        self.moments = {k: (torch.zeros_like(p), torch.zeros_like(p)) for k, p in self.params.items()}
        self.steps = 0

    def _keep(self, x):
        return g.checkpoint(x) if self.saved else x

    def _weight_grad(self, dz, kept):
        """dz^T x of a product x w^T."""
        return g.weight_grad(dz, kept) if self.saved else product(dz, kept, trans_a=1)

    def _block(self, i):
        p = self.params
        return dict(gate=p["scale%d" % i], post=True, post_weight=p["post%d" % i], post_bias=p["post_bias%d" % i])

    def gradients(self, tokens, targets):
        """(mean loss, {parameter: gradient}) of predicting targets from tokens."""
        p, kept = self.params, []
        h = p["embedding"][tokens]
        first = h
        y, mean, rstd = g.layer_norm(h, p["first"], p["first_bias"])
        for i in range(self.blocks):
            up = product(y, p["up%d" % i], trans_b=1).relu_()
            branch = product(up, p["down%d" % i], trans_b=1)
            kept_y = self._keep(y)
            y, h, stats = g.block_norm(branch, h, p["norm%d" % i], p["bias%d" % i], **self._block(i))
            kept.append((kept_y, self._keep(up), self._keep(branch), self._keep(h), stats))
        loss, _, _, dy, dhead = g.vocab_loss_grad(y, p["head"], targets)
        grads, dh = {"head": dhead}, None
        for i in reversed(range(self.blocks)):
            kept_y, kept_up, branch, h, stats = kept.pop()
            d = g.block_norm_grad(dy, dh, h, branch, stats, p["norm%d" % i], **self._block(i))
            dh = d.dresidual
            grads.update({"norm%d" % i: d.dweight, "bias%d" % i: d.dbias, "scale%d" % i: d.dgate, "post%d" % i: d.dpost_weight,
                          "post_bias%d" % i: d.dpost_bias, "down%d" % i: self._weight_grad(d.dbranch, kept_up)})
            up = g.restore(kept_up) if self.saved else kept_up
            dup = product(d.dbranch, p["down%d" % i]).mul_(up > 0)
            grads["up%d" % i] = self._weight_grad(dup, kept_y)
            dy = product(dup, p["up%d" % i])
        dx, grads["first"], grads["first_bias"] = g.layer_norm_grad(dy, first, p["first"], mean, rstd, out=dy)
        grads["embedding"] = torch.zeros_like(p["embedding"]).index_add_(0, tokens, dx + dh)
        return loss, grads

    def step(self, tokens, targets, lr=2e-3):
        """One Adam step; returns the loss before it, on the device."""
        loss, grads = self.gradients(tokens, targets)
        self.steps += 1
        for k, d in grads.items():
            m, v = self.moments[k]
            m.lerp_(d, 0.1)
            v.lerp_(d * d, 0.001)
            self.params[k] -= lr * (m / (1 - 0.9 ** self.steps)) / ((v / (1 - 0.999 ** self.steps)).sqrt() + 1e-8)
        return loss


def train(steps, vocab, width, blocks, rows, saved=True, report=print):
    """Losses every 20 steps, the last one included."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    followers = torch.randint(0, vocab, (vocab, CHOICES), generator=gen, device="cuda")
    model, losses = Model(vocab, width, blocks, saved), []
    for i in range(steps):
        loss = model.step(*batch(followers, rows, gen))
        if i % 20 == 0 or i == steps - 1:
            losses.append(float(loss))
            report("step %4d  loss %.4f" % (i, losses[-1]))
    code, site = g.gemm_f32_status(torch.cuda.current_stream())
    if code != 0:
        raise g.GemmError(code, "train (site %d)" % site)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--full", action="store_true", help="keep the activations as they are")
    a = ap.parse_args()
    train(a.steps, a.vocab, a.width, a.blocks, a.rows, not a.full)
