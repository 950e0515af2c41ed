"""Norms at a block's ends, 8-bit checkpoints and the gradients computed from
them, on torch tensors: checks of arguments, allocation of outputs, and the
call into libgemm_f32.so (include/gemm_f32_block.h).

Matrices, streams, devices and scratch are as in _lm: 2-D CUDA tensors of
float32 or bfloat16 with contiguous rows, calls queued on `stream` or on
torch's current stream of the tensors' device, which owns what they allocate.
"""
from __future__ import annotations

import ctypes
import typing

import torch

from . import _lm
from ._binding import Block, MOST_INT, NORMS, Rows, check, elsewhere
from ._lm import _F32, _TYPES, _call, _like, _matrix, _vector, _weight_type

BLOCK = 32                                            # columns that share an exponent
_byref = ctypes.byref


class Checkpoint:
    """A matrix kept in 8 bits: what checkpoint() returns.

    codes      torch.float8_e4m3fn, rows x width rounded up to 32
    exponents  torch.uint8, rows x ceil(width / 32) rounded up to 16
    width, dtype   of the matrix

    Element (t, d) stands for codes[t, d] * 2 ** (exponents[t, d // 32] - 127).
    """
    __slots__ = ("codes", "exponents", "width", "dtype")

    def __init__(self, codes, exponents, width, dtype):
        self.codes, self.exponents, self.width, self.dtype = codes, exponents, width, dtype

    @property
    def shape(self):
        return self.codes.shape[0], self.width

    @property
    def device(self):
        return self.codes.device

    def get_device(self):
        return self.codes.get_device()


def _padded(width):
    """(bytes of a row of codes, of exponents)."""
    blocks = -(-width // BLOCK)
    return blocks * BLOCK, -(-blocks // 16) * 16


def _saved(name, saved):
    """(type, device index, rows, width) of a checkpoint whose tensors are as checkpoint() makes them."""
    kind, width = _TYPES.get(saved.dtype), saved.width
    if kind is None or type(width) is not int or not 1 <= width <= MOST_INT:
        raise ValueError("%s must hold a float32 or bfloat16 matrix of at most %d columns" % (name, MOST_INT))
    codes, exponents = saved.codes, saved.exponents
    rows, dev = codes.shape[0], codes.get_device()
    ldc, lde = _padded(width)
    if (not codes.is_cuda or exponents.get_device() != dev or codes.shape != (rows, ldc) or exponents.shape != (rows, lde)
            or codes.dtype is not torch.float8_e4m3fn or exponents.dtype is not torch.uint8
            or not codes.is_contiguous() or not exponents.is_contiguous()):
        raise ValueError("%s must have contiguous codes (float8_e4m3fn, %d columns) and exponents (uint8, %d columns) on "
                         "one CUDA device" % (name, ldc, lde))
    return kind, dev, rows, width


def _rows(name, t, x):
    """The C description of a matrix of x's shape, type and device, or of a checkpoint of such a one."""
    if not isinstance(t, Checkpoint):
        return Rows(t.data_ptr(), _like(name, t, x))
    kind, dev, rows, width = _saved(name, t)
    if (rows, width) != tuple(x.shape) or t.dtype is not x.dtype or dev != x.get_device():
        raise ValueError("%s must be kept from a %s matrix of shape %s on %s" % (name, x.dtype, tuple(x.shape), x.device))
    return Rows(None, 0, t.codes.data_ptr(), t.codes.shape[1], t.exponents.data_ptr(), t.exponents.shape[1])


def _block(x, matrix, kind, eps, weight, bias, post, post_weight, post_bias, gate, residual_scale, branch_scale):
    """(the C description, the vectors' type) of a block's end on matrices like x."""
    code, dev, rows, width, _ = matrix
    norm = NORMS.get(kind)
    if norm is None:
        raise ValueError("kind must be one of %s" % ", ".join(sorted(NORMS)))
    if not post and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias belong to post=True")
    if norm and (bias is not None or post_bias is not None):
        raise ValueError("an rms norm has no bias")
    wtype = types = None
    pw = pb = ppw = ppb = pg = ldg = 0
    if weight is not None:
        types = (wtype := _weight_type(x, weight),)
        pw = _vector("weight", weight, width, dev, types)
    if bias is not None:
        types = types or (wtype := _weight_type(x, bias),)
        pb = _vector("bias", bias, width, dev, types)
    if post_weight is not None:
        types = types or (wtype := _weight_type(x, post_weight),)
        ppw = _vector("post_weight", post_weight, width, dev, types)
    if post_bias is not None:
        types = types or (wtype := _weight_type(x, post_bias),)
        ppb = _vector("post_bias", post_bias, width, dev, types)
    if gate is not None:
        if gate.dim() == 2:
            pg, ldg = gate.data_ptr(), _like("gate", gate, x)
        else:
            types = types or (wtype := _weight_type(x, gate),)
            pg = _vector("gate", gate, width, dev, types)
    if wtype is None:
        wtype = _F32
    return Block(code, _TYPES[wtype], norm, 1 if post else 0, rows, width, eps, residual_scale, branch_scale, pw, pb, ppw, ppb, pg,
                 ldg), wtype


def block_norm(branch, residual, weight=None, bias=None, kind="layer", eps=1e-5, gate=None, post=False, post_weight=None,
               post_bias=None, residual_scale=1.0, branch_scale=1.0, out=None, out_h=None, stream=None):
    """(y, h, stats) at the end of a block whose output is `branch`:

        p = branch, or with post=True its norm (post_weight, post_bias)
        h = residual_scale * residual + branch_scale * gate * p
        y = the norm of h (weight, bias)

    kind: "layer" (around the rows' mean) or "rms" (no mean, no bias).  gate:
    None, one value per column, or a matrix of branch's shape and type.  The
    vectors all hold branch's type or all float32; a weight that is None is
    1, a bias 0.  stats is float32 with a row of `rows` values for each of
    mean and rstd of h and, with post, of branch; block_norm_grad takes it.
    `out` and `out_h`, the tensors for y and h, may each be branch, residual
    or a gate matrix."""
    matrix = _matrix("branch", branch)
    kind_, dev, rows, width, ldb = matrix
    if stream is not None or _lm._current_device() != dev:
        with elsewhere(dev, stream):
            return block_norm(branch, residual, weight, bias, kind, eps, gate, post, post_weight, post_bias, residual_scale,
                              branch_scale, out, out_h)
    ldr = _like("residual", residual, branch)
    b, _ = _block(branch, matrix, kind, eps, weight, bias, post, post_weight, post_bias, gate, residual_scale, branch_scale)
    if out is None:
        out = torch.empty_like(branch, memory_format=torch.contiguous_format)
        ldy = width
    else:
        ldy = _like("out", out, branch)
    if out_h is None:
        out_h = torch.empty_like(branch, memory_format=torch.contiguous_format)
        ldh = width
    else:
        ldh = _like("out_h", out_h, branch)
    stats = torch.empty((4 if post else 2, rows), dtype=_F32, device=branch.device)
    check(_lm.lib().gemm_f32_block_norm(_byref(b), branch.data_ptr(), ldb, residual.data_ptr(), ldr, out.data_ptr(), ldy,
                                        out_h.data_ptr(), ldh, stats.data_ptr(), _lm._raw_stream(dev)), "block_norm")
    return out, out_h, stats


class BlockNormGrads(typing.NamedTuple):
    """What block_norm_grad returns; None for what the block does not have."""
    dbranch: torch.Tensor
    dresidual: torch.Tensor
    dweight: torch.Tensor
    dbias: typing.Optional[torch.Tensor]
    dgate: typing.Optional[torch.Tensor]
    dpost_weight: typing.Optional[torch.Tensor]
    dpost_bias: typing.Optional[torch.Tensor]


def block_norm_grad(dy, dh, h, branch, stats, weight=None, kind="layer", gate=None, post=False, post_weight=None,
                    post_bias=None, residual_scale=1.0, branch_scale=1.0, out=None, stream=None):
    """Gradients of block_norm for dy, the gradient of y, and dh, the one that
    reaches h from further on (None: 0).

    h is the forward call's result and branch its input, each as it was or a
    Checkpoint of it (branch is read with post or a gate only, and may be None
    otherwise); stats and the other arguments are the forward call's
    (post_bias matters with both post and a gate).  dbranch, dresidual and the
    dgate of a matrix hold dy's type, the vectors' gradients the vectors' type
    (float32 where there is none).  An rms norm has no dbias or dpost_bias.
    Where nothing stands between branch and h and both scales are equal,
    dbranch and dresidual are one tensor.  `out`, the tensor for dresidual,
    may be dy, dh, h, branch or a gate matrix."""
    matrix = _matrix("dy", dy)
    code, dev, rows, width, lddy = matrix
    if stream is not None or _lm._current_device() != dev:
        with elsewhere(dev, stream):
            return block_norm_grad(dy, dh, h, branch, stats, weight, kind, gate, post, post_weight, post_bias,
                                   residual_scale, branch_scale, out)
    b, wtype = _block(dy, matrix, kind, 0.0, weight, None, post, post_weight, post_bias, gate, residual_scale, branch_scale)
    lddh = _like("dh", dh, dy) if dh is not None else 0
    c_h = _rows("h", h, dy)
    uses_branch = post or gate is not None
    if uses_branch and branch is None:
        raise ValueError("branch is needed with post or a gate")
    c_branch = _rows("branch", branch, dy) if uses_branch else None
    n_stats = 4 if post else 2
    if stats.dtype is not _F32 or stats.shape != (n_stats, rows) or stats.get_device() != dev or not stats.is_contiguous():
        raise ValueError("stats must be a contiguous float32 tensor of shape (%d, %d) on device %d" % (n_stats, rows, dev))
    if out is None:
        dresidual = torch.empty_like(dy, memory_format=torch.contiguous_format)
        ldr = width
    else:
        dresidual, ldr = out, _like("out", out, dy)
    same = not uses_branch and residual_scale == branch_scale
    dbranch = dresidual if same else torch.empty_like(dy, memory_format=torch.contiguous_format)
    layer, channel = kind == "layer", gate is not None and gate.dim() == 1
    device = dy.device
    dweight = torch.empty(width, dtype=wtype, device=device)
    dbias = torch.empty_like(dweight) if layer else None
    dpost_weight = torch.empty_like(dweight) if post else None
    dpost_bias = torch.empty_like(dweight) if post and layer else None
    dgate = torch.empty_like(dweight) if channel else None
    if gate is not None and not channel:
        dgate = torch.empty_like(dy, memory_format=torch.contiguous_format)
    _call("gemm_f32_block_norm_grad", _byref(b), dy.data_ptr(), lddy, 0 if dh is None else dh.data_ptr(), lddh, _byref(c_h),
          _byref(c_branch) if uses_branch else None, stats.data_ptr(), 0 if same else dbranch.data_ptr(), width,
          dresidual.data_ptr(), ldr, 0 if dgate is None else dgate.data_ptr(), width, dweight.data_ptr(),
          dbias.data_ptr() if layer else 0, dpost_weight.data_ptr() if post else 0, dpost_bias.data_ptr() if post and layer else 0,
          _lm._raw_stream(dev))
    return BlockNormGrads(dbranch, dresidual, dweight, dbias, dgate, dpost_weight, dpost_bias)


def checkpoint(x, stream=None):
    """x kept in 8 bits for the backward pass: a Checkpoint.

    Every 32 columns of a row share the least power of two that takes their
    largest magnitude to 448 or below; each element over it is rounded to the
    nearest e4m3 value (to within 2^-4 of itself, or 2^-10 of the power).
    Infinities and NaN are kept as NaN."""
    kind, dev, rows, width, ldx = _matrix("x", x)
    if stream is not None or _lm._current_device() != dev:
        with elsewhere(dev, stream):
            return checkpoint(x)
    ldc, lde = _padded(width)
    codes = torch.empty((rows, ldc), dtype=torch.float8_e4m3fn, device=x.device)
    exponents = torch.empty((rows, lde), dtype=torch.uint8, device=x.device)
    check(_lm.lib().gemm_f32_checkpoint(kind, rows, width, x.data_ptr(), ldx, codes.data_ptr(), ldc, exponents.data_ptr(), lde,
                                        _lm._raw_stream(dev)), "checkpoint")
    return Checkpoint(codes, exponents, width, x.dtype)


def restore(saved, out=None, stream=None):
    """The matrix that a Checkpoint stands for, in its dtype."""
    kind, dev, rows, width = _saved("saved", saved)
    if stream is not None or _lm._current_device() != dev:
        with elsewhere(dev, stream):
            return restore(saved, out)
    if out is None:
        out = torch.empty((rows, width), dtype=saved.dtype, device=saved.device)
        ldo = width
    else:
        ldo = _like("out", out, saved)
    check(_lm.lib().gemm_f32_restore(kind, rows, width, saved.codes.data_ptr(), saved.codes.shape[1],
                                     saved.exponents.data_ptr(), saved.exponents.shape[1], out.data_ptr(), ldo,
                                     _lm._raw_stream(dev)), "restore")
    return out


def weight_grad(dy, saved, out=None, accumulate=False, stream=None):
    """dw = dy.T @ x, the weight gradient of y = x @ w.T, whose x is a Checkpoint.

    `out`, the tensor for dw, holds dy's type or float32; a float32 one can be
    added to (accumulate=True).  dy has the checkpoint's dtype."""
    kind, dev, rows, width, lddy = _matrix("dy", dy)
    if stream is not None or _lm._current_device() != dev:
        with elsewhere(dev, stream):
            return weight_grad(dy, saved, out, accumulate)
    skind, sdev, srows, swidth = _saved("saved", saved)
    if skind != kind or sdev != dev or srows != rows:
        raise ValueError("saved must be kept from a %s matrix of %d rows on %s" % (dy.dtype, rows, dy.device))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out")
        out = torch.empty((width, swidth), dtype=dy.dtype, device=dy.device)
        ldw = swidth
    else:
        if out.dtype is not _F32 and (out.dtype is not dy.dtype or accumulate):
            raise ValueError("out must hold float32%s" % ("" if accumulate else " or dy's type"))
        _, odev, orows, owidth, ldw = _matrix("out", out)
        if (odev, orows, owidth) != (dev, width, swidth):
            raise ValueError("out must have shape (%d, %d), on %s" % (width, swidth, dy.device))
    _call("gemm_f32_weight_grad", kind, rows, swidth, width, dy.data_ptr(), lddy, saved.codes.data_ptr(),
          saved.codes.shape[1], saved.exponents.data_ptr(), saved.exponents.shape[1], _TYPES[out.dtype], out.data_ptr(), ldw,
          int(accumulate), _lm._raw_stream(dev))
    return out
