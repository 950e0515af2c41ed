"""Trains a next-token model whose every product, norm and loss is this library's.

    python examples/train_head.py [--steps 200] [--vocab 4000] [--width 256] [--rows 2048]

The text is a random Markov chain: each token is followed by one of eight
others.  The model looks a token up in an embedding table, multiplies it by a
square matrix (gemm_f32), normalises the rows (layer_norm) and scores the
vocabulary (vocab_loss_grad); the gradients go back through layer_norm_grad
and two products with stored transposes (gemm_f32_general) to every
parameter.  The loss starts at log(vocab) and falls towards the chain's
entropy, log(8) or less.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import accelerator_row_major_gb300 as g  # noqa: E402

CHOICES = 8


def product(A, B, trans_a=0, trans_b=0):
    """op(A) op(B) by gemm_f32_general."""
    M, K = (A.shape[1], A.shape[0]) if trans_a else A.shape
    N = B.shape[0] if trans_b else B.shape[1]
    C = torch.empty((M, N), device=A.device)
    g.check(g.gemm_f32_general(trans_a, trans_b, M, N, K, 1.0, A, A.shape[1], B, B.shape[1], 0.0, C, N,
                               stream=torch.cuda.current_stream()))
    return C


class Model:
    def __init__(self, vocab, width, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.params = {"embedding": rnd(vocab, width), "hidden": rnd(width, width) / math.sqrt(width),
                       "weight": torch.ones(width, device="cuda"), "bias": torch.zeros(width, device="cuda"),
                       "head": 0.02 * rnd(vocab, width)}
        self.moments = {k: (torch.zeros_like(p), torch.zeros_like(p)) for k, p in self.params.items()}
        self.steps = 0

    def gradients(self, tokens, targets):
        """(mean loss, {parameter: gradient}) of predicting targets from tokens."""
        p = self.params
        e = p["embedding"][tokens]
        x = g.matmul(e, p["hidden"])
        y, mean, rstd = g.layer_norm(x, p["weight"], p["bias"])
        loss, _, _, dy, dhead = g.vocab_loss_grad(y, p["head"], targets)
        dx, dweight, dbias = g.layer_norm_grad(dy, x, p["weight"], mean, rstd, out=dy)
        dhidden = product(e, dx, trans_a=1)
        de = product(dx, p["hidden"], trans_b=1)
        dembedding = torch.zeros_like(p["embedding"]).index_add_(0, tokens, de)
        return loss, {"embedding": dembedding, "hidden": dhidden, "weight": dweight, "bias": dbias, "head": dhead}

    def step(self, tokens, targets, lr=3e-3):
        """One Adam step; returns the loss before it, on the device."""
        loss, grads = self.gradients(tokens, targets)
        self.steps += 1
        for k, d in grads.items():
            m, v = self.moments[k]
            m.lerp_(d, 0.1)
            v.lerp_(d * d, 0.001)
            self.params[k] -= lr * (m / (1 - 0.9 ** self.steps)) / ((v / (1 - 0.999 ** self.steps)).sqrt() + 1e-8)
        return loss


def batch(followers, rows, gen):
    """`rows` tokens and what follows each; one pair in sixteen is padding."""
    tokens = torch.randint(0, followers.shape[0], (rows,), generator=gen, device="cuda")
    pick = torch.randint(0, CHOICES, (rows,), generator=gen, device="cuda")
    targets = followers[tokens, pick]
    targets[::16] = -100
    return tokens, targets


def train(steps, vocab, width, rows, report=print):
    """Losses every 20 steps, the last one included."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    followers = torch.randint(0, vocab, (vocab, CHOICES), generator=gen, device="cuda")
    model, losses = Model(vocab, width), []
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
    ap.add_argument("--vocab", type=int, default=4000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--rows", type=int, default=2048)
    a = ap.parse_args()
    train(a.steps, a.vocab, a.width, a.rows)
