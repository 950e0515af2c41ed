"""Norms at a block's ends, 8-bit activation checkpoints and what the backward pass makes of them: the cases their
speed is measured on.

Four operators, named by the ``op`` of a case:

  norm         the end of one block and the beginning of the next: h = a residual + b gate p, where p is the block's
               output or its norm, and y = the norm of h, with the rows' statistics
  norm_grad    its gradients, from h and the block's output or from 8-bit checkpoints of them
  checkpoint   a matrix kept in 8 bits and brought back: e4m3 codes, a power of two for every 32 columns of a row
  weight_grad  dw = dy^T x of a product y = x w^T whose x was kept in 8 bits

``run`` computes them in plain torch operations in 32 bits where ``own`` is false, and calls this library's entry
points where it is true.  ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32                              # columns that share a power of two
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
MOST_NORM = 49152 * 1024               # elements of the largest drawn matrix
MOST_GRAD = 8192 * 4096 * 4096          # rows * width * out of the largest weight gradient


def _norm(name, op, kind, rows, width, weights, norm, gate, post, scales, saved=False):
    return {"name": name, "op": op, "type": kind, "rows": rows, "width": width, "weights": weights, "norm": norm,
            "gate": gate, "post": post, "residual_scale": scales[0], "branch_scale": scales[1], "saved": saved}


def listed():
    return [
        # one token of a serving step, residual added and normed: latency alone
        _norm("norm_token", "norm", "bf16", 1, 4096, "bf16", "rms", "none", False, (1.0, 1.0)),
        # odd sizes: rows off 16-byte boundaries; a learned scale per channel on the block's output
        _norm("norm_ragged", "norm", "f32", 1001, 777, "f32", "layer", "channel", False, (1.0, 1.0)),
        # a training batch of a model with a norm on either side of its blocks
        _norm("norm_batch", "norm", "bf16", 65536, 1024, "f32", "rms", "none", True, (1.0, 1.0)),
        # the backward pass of the ragged rows
        _norm("norm_grad_ragged", "norm_grad", "f32", 1001, 777, "f32", "layer", "channel", False, (1.0, 1.0)),
        # the backward pass of the batch
        _norm("norm_grad_batch", "norm_grad", "bf16", 65536, 1024, "f32", "rms", "none", True, (1.0, 1.0)),
        # a batch whose activations were kept in 8 bits, its block's output gated element by element
        _norm("norm_grad_saved", "norm_grad", "bf16", 8192, 4096, "bf16", "layer", "element", False, (1.0, 0.5), True),
        # a wide f32 model with everything: both norms, a scale per channel, scaled residual
        _norm("norm_grad_wide", "norm_grad", "f32", 8192, 8192, "f32", "layer", "channel", True, (1.25, 0.5)),
        # a small activation of odd sizes, kept and brought back
        {"name": "checkpoint_ragged", "op": "checkpoint", "type": "f32", "rows": 1001, "width": 777},
        # a training batch's activation, kept and brought back
        {"name": "checkpoint_batch", "op": "checkpoint", "type": "bf16", "rows": 65536, "width": 1024},
        # weight gradient of a ragged batch and odd widths
        {"name": "weight_grad_ragged", "op": "weight_grad", "type": "bf16", "rows": 1001, "width": 777, "out": 513},
        # f32 training
        {"name": "weight_grad_f32", "op": "weight_grad", "type": "f32", "rows": 4096, "width": 1024, "out": 1024},
        # a full batch of a wide model: the largest case
        {"name": "weight_grad_batch", "op": "weight_grad", "type": "bf16", "rows": 8192, "width": 4096, "out": 4096},
    ]


def _between(rng, low, high):
    """A whole number spread over the logarithm; every other one a multiple of 8, as most models' sizes are."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5:
        v = max(low, v // 8 * 8)
    return v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_grad", "checkpoint", "weight_grad"])
    kind = rng.choice(["f32", "bf16"])
    if op == "weight_grad":
        width, out = _between(rng, 64, 8192), _between(rng, 64, 8192)
        rows = _between(rng, 1, max(1, min(16384, MOST_GRAD // (width * out))))
        return {"op": op, "type": kind, "rows": rows, "width": width, "out": out}
    width = _between(rng, 32, 16384)
    rows = _between(rng, 1, min(65536, MOST_NORM // width))
    if op == "checkpoint":
        return {"op": op, "type": kind, "rows": rows, "width": width}
    c = _norm("", op, kind, rows, width, "f32" if kind == "f32" else rng.choice(["f32", "bf16"]),
              rng.choice(["layer", "rms"]), rng.choice(["none", "channel", "element"]), rng.random() < 0.5,
              rng.choice([(1.0, 1.0), (1.25, 0.5), (1.0, 0.25)]), op == "norm_grad" and rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _normal(shape, gen, kind, scale=1.0, shift=0.0):
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return v.mul_(scale).add_(shift).to(TYPES[kind])


def _power(e):
    """2^e in 32 bits, for whole numbers e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x, fill=0.0):
    """x in 32 bits, its columns in blocks of 32, the last one filled up."""
    rows, width = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -width % BLOCK), value=fill)
    return x.view(rows, -1, BLOCK)


def _kept(x):
    """Codes (rows x whole blocks) and exponents (rows x blocks) of x: the least power of two that takes each block's
    largest magnitude to 448 or below, and x over it to the nearest e4m3 value."""
    v = _blocks(x)
    top = v.abs().amax(2)
    mantissa, e = torch.frexp(top)                       # top = mantissa 2^e, 0.5 <= mantissa < 1
    e = torch.where(top > 0, e - 9 + (mantissa > 0.875), -126).clamp(min=-126)
    codes = (v * _power(-e)[:, :, None]).to(torch.float8_e4m3fn)
    return codes.flatten(1), e


def _brought_back(codes, e, width):
    """What codes and exponents stand for, in 32 bits."""
    v = codes.float().view(codes.shape[0], -1, BLOCK) * _power(e)[:, :, None]
    return v.flatten(1)[:, :width]


def _statistics(x, norm):
    """Each row's mean (0 for rms) and 1 / sqrt(mean square around it + EPS), in 32 bits."""
    x = x.float()
    mean = x.mean(1) if norm == "layer" else torch.zeros(x.shape[0], device=x.device)
    x = x - mean[:, None]
    return mean, 1.0 / torch.sqrt((x * x).mean(1) + EPS)


def _keep(s, name, x):
    """A checkpoint as the library lays it out: codes in rows of whole blocks, exponents plus 127 as bytes in rows of
    a multiple of 16."""
    codes, e = _kept(x)
    s[name + "_codes"] = codes
    exponents = torch.zeros(e.shape[0], -(-e.shape[1] // 16) * 16, dtype=torch.uint8, device=x.device)
    exponents[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    s[name + "_exponents"] = exponents


def _kept_of(s, name):
    """The values of one of the state's checkpoints, in 32 bits."""
    blocks = -(-s["width"] // BLOCK)
    return _brought_back(s[name + "_codes"], s[name + "_exponents"][:, :blocks].int() - 127, s["width"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    kind, shape = case["type"], (case["rows"], case["width"])
    if case["op"] == "checkpoint":
        # activations of a residual stream: unit scale, a few channels much larger than the others
        s["x"] = _normal(shape, gen, "f32").mul_(1 + 30 * (torch.rand(shape[1], generator=gen, device="cuda") < 0.01)
                                                 ).to(TYPES[kind])
        return s
    if case["op"] == "weight_grad":
        s["dy"] = _normal((shape[0], case["out"]), gen, kind)
        _keep(s, "x", _normal(shape, gen, kind))
        return s
    s["weight"] = _normal(shape[1:], gen, case["weights"], 0.1, 1.0)
    s["bias"] = _normal(shape[1:], gen, case["weights"], 0.1) if case["norm"] == "layer" else None
    s["post_weight"] = _normal(shape[1:], gen, case["weights"], 0.1, 1.0) if case["post"] else None
    s["post_bias"] = _normal(shape[1:], gen, case["weights"], 0.1) if case["post"] and s["bias"] is not None else None
    s["gate"] = None
    if case["gate"] == "channel":
        s["gate"] = _normal(shape[1:], gen, case["weights"], 0.1, 0.5)
    elif case["gate"] == "element":     # sigmoids, as they come out of a projection
        s["gate"] = torch.sigmoid(_normal(shape, gen, "f32")).to(TYPES[kind])
    # the stream: unit scale, each row with an offset of its own; the block's output smaller
    stream = (_normal(shape, gen, "f32") + _normal((shape[0], 1), gen, "f32", 0.5)).to(TYPES[kind])
    branch = _normal(shape, gen, kind, 0.5)
    if case["op"] == "norm":
        s["residual"], s["branch"] = stream, branch
        return s
    s["dy"] = _normal(shape, gen, kind)
    s["dh"] = _normal(shape, gen, kind)
    s["stats"] = torch.stack(_statistics(stream, case["norm"]) +
                             (_statistics(branch, case["norm"]) if case["post"] else ()))
    uses_branch = case["post"] or case["gate"] != "none"
    if case["saved"]:
        _keep(s, "h", stream)
        if uses_branch:
            _keep(s, "branch", branch)
    else:
        s["h"], s["branch"] = stream, branch if uses_branch else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def run(s):
    if own:
        return _own(s)
    if s["op"] == "checkpoint":
        codes, e = _kept(s["x"])
        return {"x": _brought_back(codes, e, s["width"]).to(s["x"].dtype)}
    if s["op"] == "weight_grad":
        return {"dw": (s["dy"].float().t() @ _kept_of(s, "x")).to(s["dy"].dtype)}
    return _plain_norm(s) if s["op"] == "norm" else _plain_norm_grad(s)


def _scaled(x, weight, bias):
    if weight is not None:
        x = x * weight.float()
    return x + bias.float() if bias is not None else x


def _plain_norm(s):
    kind = s["residual"].dtype
    p = s["branch"].float()
    stats = []
    if s["post"]:
        stats = list(_statistics(p, s["norm"]))
        p = _scaled((p - stats[0][:, None]) * stats[1][:, None], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        p = p * s["gate"].float()
    h = s["residual_scale"] * s["residual"].float() + s["branch_scale"] * p
    mean, rstd = _statistics(h, s["norm"])
    y = _scaled((h - mean[:, None]) * rstd[:, None], s["weight"], s["bias"])
    return {"y": y.to(kind), "h": h.to(kind), "stats": torch.stack([mean, rstd] + stats)}


def _plain_norm_grad(s):
    kind, wkind, layer = s["dy"].dtype, s["weight"].dtype, s["norm"] == "layer"

    def back(g, hat, rstd):
        """Gradient of a norm's input from the gradient g of its normed rows."""
        d = g - hat * (g * hat).mean(1, keepdim=True)
        return rstd * (d - g.mean(1, keepdim=True) if layer else d)

    h = _kept_of(s, "h") if s["saved"] else s["h"].float()
    stats = s["stats"][:, :, None]
    dy = s["dy"].float()
    hat = (h - stats[0]) * stats[1]
    out = {"dweight": (dy * hat).sum(0).to(wkind)}
    if layer:
        out["dbias"] = dy.sum(0).to(wkind)
    d = s["dh"].float() + back(dy * s["weight"].float(), hat, stats[1])
    out["dresidual"] = (s["residual_scale"] * d).to(kind)
    if not s["post"] and s["gate"] is None:
        out["dbranch"] = out["dresidual"] if s["residual_scale"] == s["branch_scale"] else (s["branch_scale"] * d).to(kind)
        return out
    d = s["branch_scale"] * d
    p = b = _kept_of(s, "branch") if s["saved"] else s["branch"].float()
    if s["post"]:
        b = (b - stats[2]) * stats[3]
        p = _scaled(b, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        dgate = d * p
        out["dgate"] = dgate.to(kind) if s["gate"].dim() == 2 else dgate.sum(0).to(s["gate"].dtype)
        d = d * s["gate"].float()
    if s["post"]:
        out["dpost_weight"] = (d * b).sum(0).to(wkind)
        if layer:
            out["dpost_bias"] = d.sum(0).to(wkind)
        d = back(d * s["post_weight"].float(), b, stats[3])
    out["dbranch"] = d.to(kind)
    return out


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import accelerator_row_major_gb300 as lib

    if s["op"] == "checkpoint":
        return {"x": lib.restore(lib.checkpoint(s["x"]))}

    def saved(name):
        return lib.Checkpoint(s[name + "_codes"], s[name + "_exponents"], s["width"], TYPES[s["type"]])

    if s["op"] == "weight_grad":
        return {"dw": lib.weight_grad(s["dy"], saved("x"))}
    how = {"kind": s["norm"], "gate": s["gate"], "post": s["post"], "post_weight": s["post_weight"],
           "post_bias": s["post_bias"], "residual_scale": s["residual_scale"], "branch_scale": s["branch_scale"]}
    if s["op"] == "norm":
        return dict(zip(("y", "h", "stats"), lib.block_norm(s["branch"], s["residual"], s["weight"], s["bias"],
                                                             eps=EPS, **how)))
    uses_branch = s["post"] or s["gate"] is not None
    h = saved("h") if s["saved"] else s["h"]
    branch = None if not uses_branch else saved("branch") if s["saved"] else s["branch"]
    got = lib.block_norm_grad(s["dy"], s["dh"], h, branch, s["stats"], s["weight"], **how)._asdict()
    return {k: v for k, v in got.items() if v is not None}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exactly_kept(x):
    """The values an 8-bit checkpoint of x stands for, by arithmetic on whole powers of two."""
    rows, width = x.shape
    blocks = -(-width // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :width] = x
    v = v.view(rows, blocks, BLOCK)

    def power(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    top = v.abs().amax(2, keepdim=True)
    e = torch.frexp(torch.where(top > 0, top, 1.0)).exponent - 9     # top in [256, 512) 2^e
    e = torch.where(top > 448 * power(e), e + 1, e)
    e = torch.where(top > 0, e, -126).clamp(min=-126)
    v = v / power(e)
    # three bits behind the leading one; below 2^-6 steps of 2^-9
    step = power(torch.frexp(torch.where(v == 0, 1.0, v)).exponent.clamp(min=-5) - 4)
    return (torch.round(v / step) * step * power(e)).view(rows, -1)[:, :width]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return {"x": _exactly_kept(s["x"])}

    def kept(name):
        e = s[name + "_exponents"][:, :-(-case["width"] // BLOCK)].double() - 127
        v = s[name + "_codes"].double().unflatten(1, (-1, BLOCK)) * torch.ldexp(torch.ones_like(e), e)[:, :, None]
        return v.flatten(1)[:, :case["width"]]

    if case["op"] == "weight_grad":
        return {"dw": torch.einsum("ro,rd->od", s["dy"].double(), kept("x"))}
    alpha, beta, layer, width = case["residual_scale"], case["branch_scale"], case["norm"] == "layer", case["width"]
    weights = {k: v.double() for k, v in s.items() if k in ("weight", "bias", "post_weight", "post_bias", "gate")
               and v is not None}
    if case["op"] == "norm":
        def normed(x, weight, bias):
            mean = x.mean(1) if layer else torch.zeros(x.shape[0], dtype=x.dtype, device=x.device)
            centred = x - mean[:, None]
            rstd = torch.rsqrt(centred.square().mean(1) + EPS)
            return torch.addcmul(bias, centred.mul_(rstd[:, None]), weight), mean, rstd

        none = torch.zeros(width, dtype=torch.float64, device="cuda")
        p, stats = s["branch"].double(), ()
        if case["post"]:
            p, *stats = normed(p, weights["post_weight"], weights.get("post_bias", none))
        h = alpha * s["residual"].double() + beta * (p * weights["gate"] if "gate" in weights else p)
        y, *first = normed(h, weights["weight"], weights.get("bias", none))
        return {"y": y, "h": h, "stats": torch.stack([*first, *stats])}

    # gradients, with the statistics that are given
    stats = s["stats"].double()

    def through(grad, hat, rstd):
        along = torch.einsum("rd,rd->r", grad, hat)[:, None] / width
        d = torch.addcmul(grad, hat, along, value=-1)
        if layer:
            d -= grad.sum(1, keepdim=True) / width
        return d.mul_(rstd[:, None])

    hat = ((kept("h") if case["saved"] else s["h"].double()) - stats[0][:, None]).mul_(stats[1][:, None])
    dy = s["dy"].double()
    out = {"dweight": torch.einsum("rd,rd->d", dy, hat)}
    if layer:
        out["dbias"] = dy.sum(0)
    d = s["dh"].double() + through(dy * weights["weight"], hat, stats[1])
    del dy, hat
    out["dresidual"] = alpha * d
    d *= beta
    if case["post"] or case["gate"] != "none":
        b = kept("branch") if case["saved"] else s["branch"].double()
        if case["post"]:
            b = (b - stats[2][:, None]).mul_(stats[3][:, None])
        if "gate" in weights:
            p = b * weights["post_weight"] + weights.get("post_bias", 0.0) if case["post"] else b
            out["dgate"] = d * p if case["gate"] == "element" else torch.einsum("rd,rd->d", d, p)
            d = d * weights["gate"]
        if case["post"]:
            out["dpost_weight"] = torch.einsum("rd,rd->d", d, b)
            if layer:
                out["dpost_bias"] = d.sum(0)
            d = through(d * weights["post_weight"], b, stats[3])
    out["dbranch"] = d
    return out


def work(case):
    es, rows, width = SIZE[case["type"]], case["rows"], case["width"]
    n, kept = rows * width, rows * (width + -(-width // BLOCK))        # elements, bytes of a checkpoint
    if case["op"] == "checkpoint":  # in, kept, read again, out
        return {"bytes": 2 * n * es + 2 * kept, "flops": 4 * n}
    if case["op"] == "weight_grad":
        return {"bytes": rows * case["out"] * es + kept + case["out"] * width * es,
                "flops": 2 * n * case["out"]}
    ws = SIZE[case["weights"]]
    layer, gate, post = case["norm"] == "layer", case["gate"], case["post"]
    vectors = (1 + layer) * (1 + post) + (gate == "channel")
    statistics = 4 * rows * (4 if post else 2)
    if case["op"] == "norm":        # branch and residual in, h and y out
        return {"bytes": (4 + (gate == "element")) * n * es + vectors * width * ws + statistics,
                "flops": (8 + 6 * post + 2) * n}
    uses_branch = post or gate != "none"
    same = not uses_branch and case["residual_scale"] == case["branch_scale"]
    activations = (1 + uses_branch) * (kept if case["saved"] else n * es)
    matrices = 3 + (not same) + 2 * (gate == "element")                # dy, dh, dresidual, dbranch; gate, dgate
    return {"bytes": matrices * n * es + activations + (vectors + 1 + post + (gate == "channel")) * width * ws + statistics,
            "flops": (16 + 14 * post + 3 * (gate != "none")) * n}
