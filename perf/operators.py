"""Layer norm and the vocabulary loss, each with its gradient: the cases their speed is measured on.

Four operators, named by the ``op`` of a case:

  norm       y = (x - mean) * rstd * weight + bias over the rows of x, with each row's mean and rstd
  norm_grad  its gradients dx, dweight, dbias from dy, x, weight and the rows' mean and rstd
  loss       z = x W^T; loss_t = log sum_v exp z_tv - z_ty for the target y of row t (0 where the
             target is ignored), and the mean over the rows that count
  loss_grad  the same with the mean's gradients dx and dW

``run`` computes them in plain torch operations in 32 bits where ``own`` is false, and calls this
library's entry points where it is true.  ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
IGNORED = -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
MOST_NORM = 65536 * 4096               # elements of x of the largest drawn norm
MOST_LOSS = 8192 * 4096 * 65536        # rows * width * vocabulary of the largest loss


def listed():
    return [
        # a single token of a serving step: latency alone
        {"name": "norm_one_row", "op": "norm", "type": "bf16", "weights": "bf16", "rows": 1, "width": 4096},
        # odd sizes: no row but the first starts on a 16-byte boundary
        {"name": "norm_ragged", "op": "norm", "type": "f32", "weights": "f32", "rows": 1001, "width": 777},
        # a training batch of a bf16 model that keeps its norms' weights in f32
        {"name": "norm_batch", "op": "norm", "type": "bf16", "weights": "f32", "rows": 65536, "width": 1024},
        # the backward pass of the ragged rows
        {"name": "norm_grad_ragged", "op": "norm_grad", "type": "f32", "weights": "f32", "rows": 1001, "width": 777},
        # a training batch, backward: the sum over 65,536 rows for each column
        {"name": "norm_grad_batch", "op": "norm_grad", "type": "bf16", "weights": "f32", "rows": 65536, "width": 1024},
        # a wide f32 model's batch, backward
        {"name": "norm_grad_wide", "op": "norm_grad", "type": "f32", "weights": "f32", "rows": 8192, "width": 8192},
        # scoring one token: the vocabulary's weights are read once
        {"name": "loss_one_row", "op": "loss", "type": "bf16", "rows": 1, "width": 4096, "vocab": 65536},
        # scoring a short prompt in f32
        {"name": "loss_prompt_f32", "op": "loss", "type": "f32", "rows": 64, "width": 4096, "vocab": 65536},
        # evaluation of a batch: compute bound
        {"name": "loss_batch", "op": "loss", "type": "bf16", "rows": 8192, "width": 1024, "vocab": 65536},
        # training on a ragged batch and vocabulary, width not a multiple of 8
        {"name": "loss_grad_ragged", "op": "loss_grad", "type": "bf16", "rows": 1001, "width": 777, "vocab": 32001},
        # training in f32
        {"name": "loss_grad_f32", "op": "loss_grad", "type": "f32", "rows": 4096, "width": 1024, "vocab": 32768},
        # training on a full batch: the largest case
        {"name": "loss_grad_batch", "op": "loss_grad", "type": "bf16", "rows": 8192, "width": 4096, "vocab": 65536},
    ]


def _between(rng, low, high):
    """A whole number spread over the logarithm; every other one a multiple of 8, as most models' sizes are."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5:
        v = max(low, v // 8 * 8)
    return v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "loss", "loss_grad"])
    kind = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_grad"):
        width = _between(rng, 32, 16384)
        rows = _between(rng, 1, min(65536, MOST_NORM // width))
        return {"op": op, "type": kind, "weights": "f32" if kind == "f32" else rng.choice(["f32", "bf16"]),
                "rows": rows, "width": width}
    width = _between(rng, 64, 8192)
    vocab = _between(rng, 1000, 131072)
    rows = _between(rng, 1, max(1, min(16384, MOST_LOSS // (width * vocab))))
    return {"op": op, "type": kind, "rows": rows, "width": width, "vocab": vocab}


def _normal(shape, gen, kind, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return v.mul_(scale).add_(shift).to(TYPES[kind])


def _statistics(x):
    """Each row's mean and 1 / sqrt(variance + EPS), in 32 bits."""
    x = x.float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    return mean, 1.0 / torch.sqrt((centred * centred).mean(1) + EPS)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    kind = case["type"]
    if case["op"] in ("norm", "norm_grad"):
        shape = (case["rows"], case["width"])
        # activations of a residual stream: unit scale, each row with an offset of its own
        s["x"] = (_normal(shape, gen, "f32") + _normal((shape[0], 1), gen, "f32", 0.5)).to(TYPES[kind])
        s["weight"] = _normal(shape[1:], gen, case["weights"], 0.1, 1.0)
        s["bias"] = _normal(shape[1:], gen, case["weights"], 0.1)
        if case["op"] == "norm_grad":
            s["dy"] = _normal(shape, gen, kind)
            s["mean"], s["rstd"] = _statistics(s["x"])
        return s
    rows, width, vocab = case["rows"], case["width"], case["vocab"]
    s["x"] = _normal((rows, width), gen, kind)                        # rows out of a layer norm
    s["w"] = _normal((vocab, width), gen, kind, 1.5 / math.sqrt(width))  # logits of scale 1.5
    s["targets"] = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    if rows > 1:  # one row in ten is padding
        s["targets"][torch.rand(rows, generator=gen, device="cuda") < 0.1] = IGNORED
    return s


def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm":
        mean, rstd = _statistics(s["x"])
        hat = (s["x"].float() - mean[:, None]) * rstd[:, None]
        return {"y": (hat * s["weight"].float() + s["bias"].float()).to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        hat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * hat).sum(0).to(s["weight"].dtype),
                "dbias": dy.sum(0).to(s["weight"].dtype)}
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    counts = targets != IGNORED
    at = torch.where(counts, targets, 0)[:, None]
    z = x @ w.t()
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    rows = torch.where(counts, lse - z.gather(1, at)[:, 0], 0.0)
    n = counts.sum().clamp(min=1)
    out = {"loss": rows.sum() / n, "rows": rows, "lse": lse}
    if s["op"] == "loss_grad":
        g = e / total
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=g.dtype))
        g *= (counts / n)[:, None]
        out["dx"] = (g @ w).to(s["x"].dtype)
        out["dw"] = (g.t() @ x).to(s["w"].dtype)
    return out


def _own(s):
    import accelerator_row_major_gb300 as lib

    if s["op"] == "norm":
        return dict(zip(("y", "mean", "rstd"), lib.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)))
    if s["op"] == "norm_grad":
        return dict(zip(("dx", "dweight", "dbias"),
                        lib.layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])))
    if s["op"] == "loss":
        return dict(zip(("loss", "rows", "lse"), lib.vocab_loss(s["x"], s["w"], s["targets"], ignore_index=IGNORED)))
    return dict(zip(("loss", "rows", "lse", "dx", "dw"),
                    lib.vocab_loss_grad(s["x"], s["w"], s["targets"], ignore_index=IGNORED)))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        # y = hat * weight + bias with hat = (x - mean) * rstd, for the mean and rstd that are given
        dy, rstd, width = s["dy"].double(), s["rstd"].double()[:, None], case["width"]
        hat = (s["x"].double() - s["mean"].double()[:, None]).mul_(rstd)
        dweight = torch.einsum("rd,rd->d", dy, hat)
        dhat = dy * s["weight"].double()
        along = torch.einsum("rd,rd->r", dhat, hat)[:, None] / width
        dx = (dhat - dhat.sum(1, keepdim=True) / width - along * hat).mul_(rstd)
        return {"dx": dx, "dweight": dweight, "dbias": dy.sum(0)}
    rows, width, vocab = case["rows"], case["width"], case["vocab"]
    grad = case["op"] == "loss_grad"
    if (6 if grad else 2) * rows * width * vocab > 1.6e13:  # seconds in 64 bits, at about 1 TFLOP/s
        return None
    x, w, targets = s["x"].double(), s["w"].double(), s["targets"]
    counts = targets.ne(IGNORED)
    n = max(1, int(counts.sum()))
    parts, lses = [], []
    dx, dw = torch.empty_like(x), torch.zeros_like(w)
    for a in range(0, rows, 1024):  # some rows at a time: their logits alone are held
        z = x[a:a + 1024] @ w.t()
        lse = torch.logsumexp(z, 1)
        lses.append(lse)
        here = counts[a:a + 1024].nonzero()[:, 0]
        y = targets[a:a + 1024][here]
        part = torch.zeros_like(lse)
        part[here] = lse[here] - z[here, y]
        parts.append(part)
        if grad:
            p = torch.zeros_like(z)
            p[here] = torch.softmax(z[here], 1)
            p[here, y] -= 1.0
            p /= n
            dx[a:a + 1024] = p @ w
            dw.addmm_(p.t(), x[a:a + 1024])
    parts = torch.cat(parts)
    out = {"loss": parts.sum() / n, "rows": parts, "lse": torch.cat(lses)}
    if grad:
        out["dx"], out["dw"] = dx, dw
    return out


def work(case):
    es = SIZE[case["type"]]
    rows, width = case["rows"], case["width"]
    if case["op"] in ("norm", "norm_grad"):
        ws = SIZE[case["weights"]]
        if case["op"] == "norm":  # x in, y out; weight, bias; mean, rstd
            return {"bytes": 2 * rows * width * es + 2 * width * ws + 8 * rows, "flops": 8 * rows * width}
        return {"bytes": 3 * rows * width * es + 3 * width * ws + 8 * rows, "flops": 14 * rows * width}
    vocab = case["vocab"]
    ends = (rows + vocab) * width * es
    if case["op"] == "loss":  # x, w and the targets in; the rows' losses and lse out
        return {"bytes": ends + 16 * rows, "flops": 2 * rows * width * vocab}
    return {"bytes": 2 * ends + 16 * rows, "flops": 6 * rows * width * vocab}
