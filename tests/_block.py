"""Inputs and 64-bit results of the norms at a block's ends, with bounds on
what fp32 may be off by.

The bounds count, with u = 2^-24 and, for a result rounded to bfloat16, half a
step 2^-9 twice over (2^-8):
  - a sum over a row is a tree of depth at most 64 (+ width / 512 where a row
    is read again): it is off by that many u of the sum of its terms' sizes;
  - hat = x rstd - mean rstd: two roundings, 3 u (|x| + |mean|) rstd;
  - rstd from centred squares: 64 u (1 + max|x| rstd), and what the row's own
    errors E add, 2 rstd sqrt(mean E^2);
  - each further product or sum: u of its result, and its operands' errors.
"""
import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(rows, width, kind, wkind="f32", norm="layer", gate="none", post=False, seed=0, scales=(1.0, 1.0), bias=True):
    """A dict of what a forward call takes, and dy and dh."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, w = TYPES[kind], TYPES[wkind]

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"branch": (0.5 * rnd(rows, width)).to(t), "residual": (rnd(rows, width) + 0.5 * rnd(rows, 1)).to(t),
         "dy": rnd(rows, width).to(t), "dh": rnd(rows, width).to(t), "weight": (1 + 0.1 * rnd(width)).to(w),
         "bias": (0.1 * rnd(width)).to(w) if norm == "layer" and bias else None,
         "how": {"kind": norm, "post": post, "residual_scale": scales[0], "branch_scale": scales[1], "gate": None,
                 "post_weight": (1 + 0.1 * rnd(width)).to(w) if post else None,
                 "post_bias": (0.1 * rnd(width)).to(w) if post and norm == "layer" and bias else None}}
    if gate == "channel":
        s["how"]["gate"] = (0.5 + 0.1 * rnd(width)).to(w)
    elif gate == "element":
        s["how"]["gate"] = torch.sigmoid(rnd(rows, width)).to(t)
    return s


def _d(t):
    return None if t is None else t.double()


def _depth(width):
    return 64 + width / 512 if width > 32768 else 64


def _normed(x, E, norm, eps, depth):
    """(mean, rstd, hat) of rows x that are off by E, and what each is off by."""
    mean = x.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    big = (x.abs().amax(1, keepdim=True)) * rstd
    e_mean = (depth * U * x.abs().mean(1, keepdim=True) + E.mean(1, keepdim=True)) if norm == "layer" else torch.zeros_like(mean)
    e_rel = depth * U * (1 + big) + 2 * rstd * ((E + e_mean).square().mean(1, keepdim=True)).sqrt() + 8 * U
    hat = (x - mean) * rstd
    e_hat = (E + e_mean + 4 * U * (x.abs() + mean.abs())) * rstd + hat.abs() * e_rel
    return mean, rstd, hat, e_mean, e_rel * rstd, e_hat


def _affine(hat, e_hat, w, b):
    out = hat * w if w is not None else hat
    e = e_hat * (w.abs() if w is not None else 1) + 3 * U * (out.abs() + (b.abs() if b is not None else 0))
    return (out + b if b is not None else out), e


def forward(s, eps=1e-5):
    """{name: (exact, bound)} of y, h and stats."""
    how, t = s["how"], s["branch"].dtype
    b, r = s["branch"].double(), s["residual"].double()
    depth = _depth(b.shape[1])
    p, E, stats = b, torch.zeros_like(b), []
    if how["post"]:
        mean, rstd, hat, e_mean, e_rstd, e_hat = _normed(b, E, how["kind"], eps, depth)
        p, E = _affine(hat, e_hat, _d(how["post_weight"]), _d(how["post_bias"]))
        stats = [(mean, e_mean), (rstd, e_rstd)]
    if how["gate"] is not None:
        g = how["gate"].double()
        p, E = p * g, E * g.abs() + U * (p * g).abs()
    alpha, beta = how["residual_scale"], how["branch_scale"]
    h = alpha * r + beta * p
    E = abs(beta) * E + 3 * U * ((alpha * r).abs() + (beta * p).abs())
    mean, rstd, hat, e_mean, e_rstd, e_hat = _normed(h, E, how["kind"], eps, depth)
    y, Ey = _affine(hat, e_hat, _d(s["weight"]), _d(s["bias"]))
    stats = [(mean, e_mean), (rstd, e_rstd)] + stats
    return {"y": (y, Ey + ROUND[t] * y.abs()), "h": (h, E + ROUND[t] * h.abs()),
            "stats": (torch.stack([v[:, 0] for v, _ in stats]), torch.stack([e[:, 0] + U * v[:, 0].abs() for v, e in stats]))}


def gradients(s, h, branch, stats, dh=True):
    """{name: (exact, bound)} of the gradients for the h, branch (their values, in any type) and stats that are given."""
    how, t = s["how"], s["dy"].dtype
    layer, w = how["kind"] == "layer", _d(s["weight"])
    wtype = next((v.dtype for v in (s["weight"], s["bias"], how["post_weight"], how["post_bias"]) if v is not None),
                 how["gate"].dtype if how["gate"] is not None and how["gate"].dim() == 1 else torch.float32)
    dy, x = s["dy"].double(), h.double()
    R, D = dy.shape
    depth = _depth(D) + 96
    st = stats.double()[:, :, None]
    out = {}

    def column(name, terms, E, vector_type=wtype):
        v = terms.sum(0)
        out[name] = (v, (E + (R / 16 + 176) * U * terms.abs()).sum(0) + ROUND[vector_type] * v.abs())

    def back(g, E, hat, H, rstd):
        """Through a norm: g off by E, hat of size at most H."""
        mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
        v = rstd * (g - hat * mean(g * hat) - (mean(g) if layer else 0))
        size = rstd * (g.abs() + H * mean(g.abs() * H) + (mean(g.abs()) if layer else 0))
        return v, rstd * (E + H * mean(E * H) + (mean(E) if layer else 0)) + depth * U * size

    mean, rstd = (st[0] if layer else 0), st[1]
    hat = (x - mean) * rstd
    H = (x.abs() + (mean.abs() if layer else 0)) * rstd
    column("dweight", dy * hat, 4 * U * dy.abs() * H)
    if layer:
        column("dbias", dy, torch.zeros_like(dy))
    g = dy * w if w is not None else dy
    d, E = back(g, U * g.abs(), hat, H, rstd)
    if dh:
        d = d + s["dh"].double()
        E = E + 2 * U * (d.abs() + s["dh"].double().abs())
    alpha, beta = how["residual_scale"], how["branch_scale"]
    out["dresidual"] = (alpha * d, abs(alpha) * E + (U + ROUND[t]) * (alpha * d).abs())
    d, E = beta * d, abs(beta) * E + U * (beta * d).abs()
    gate = how["gate"]
    if how["post"] or gate is not None:
        b = branch.double()
        if how["post"]:
            mean, rstd = (st[2] if layer else 0), st[3]
            B = (b.abs() + (mean.abs() if layer else 0)) * rstd
            b = (b - mean) * rstd
            pw, pb = _d(how["post_weight"]), _d(how["post_bias"])
            pw = torch.ones_like(b[0]) if pw is None else pw
            p = b * pw + (pb if pb is not None else 0)
            Ep = 6 * U * (B * pw.abs() + (pb.abs() if pb is not None else 0))
        else:
            p, Ep = b, torch.zeros_like(b)
        if gate is not None:
            dgate = d * p
            e = E * p.abs() + d.abs() * Ep + 3 * U * dgate.abs()
            if gate.dim() == 2:
                out["dgate"] = (dgate, e + ROUND[t] * dgate.abs())
            else:
                column("dgate", dgate, e, gate.dtype)
            gd = gate.double()
            d, E = d * gd, E * gd.abs() + 2 * U * (d * gd).abs()
        if how["post"]:
            column("dpost_weight", d * b, E * B + 4 * U * d.abs() * B)
            if layer:
                column("dpost_bias", d, E)
            dw = d * pw
            d, E = back(dw, E * pw.abs() + U * dw.abs(), b, B, rstd)
    out["dbranch"] = (d, E + 2 * U * d.abs() + ROUND[t] * d.abs())
    return out


def check(got, want):
    """Every result is there, of the right shape, and within its bound."""
    names = {k for k, v in got.items() if v is not None}
    assert names == set(want), names ^ set(want)
    for k, (v, bound) in want.items():
        g = got[k].double()
        assert g.shape == v.shape, k
        off = (g - v).abs()
        assert (off <= bound + 1e-30).all(), "%s: off by %.3g where %.3g is allowed" % (
            k, float(off[~(off <= bound)][0]), float(bound.expand_as(off)[~(off <= bound)][0]))


def call(g, s, eps=1e-5, **more):
    return dict(zip(("y", "h", "stats"), g.block_norm(s["branch"], s["residual"], s["weight"], s["bias"], eps=eps, **s["how"], **more)))


def call_grad(g, s, h, branch, stats, dh=True, **more):
    return g.block_norm_grad(s["dy"], s["dh"] if dh else None, h, branch, stats, s["weight"], **s["how"], **more)._asdict()


def both(g, s, saved=False, eps=1e-5):
    """Forward and gradient checked against 64 bits."""
    got = call(g, s, eps)
    check(got, forward(s, eps))
    h, branch = got["h"], s["branch"]
    kept = (g.checkpoint(h), g.checkpoint(branch)) if saved else (h, branch)
    values = (g.restore(kept[0]).double(), g.restore(kept[1]).double()) if saved else (h, branch)
    grads = call_grad(g, s, *kept, got["stats"])
    check(grads, gradients(s, *values, got["stats"]))
    assert g.gemm_f32_status(None) == (0, 0)
    return got, grads
