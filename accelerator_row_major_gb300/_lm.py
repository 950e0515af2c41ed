"""Layer norm and the vocabulary loss on torch tensors: checks of arguments,
allocation of outputs, and the call into libgemm_f32.so (include/gemm_f32_lm.h).

Matrices are 2-D CUDA tensors of float32 or bfloat16 with contiguous rows
(stride(1) == 1; stride(0) may exceed the width, as in a column slice).
Calls are queued on `stream`, or on torch's current stream of the tensors'
device, and return without waiting for it.
"""
from __future__ import annotations

import torch

from ._binding import REDUCTIONS, TYPE_BF16, TYPE_F32, _stream, check, lib

_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16}


def _type(name, t):
    if not t.is_cuda or t.dtype not in _TYPES:
        raise ValueError("%s must be a float32 or bfloat16 CUDA tensor" % name)
    return _TYPES[t.dtype]


def _matrix(name, t, like=None):
    """Row stride of a matrix operand, checked (against `like`: its shape, type and device)."""
    if like is None:
        _type(name, t)
    elif t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s must be a %s tensor on %s" % (name, like.dtype, like.device))
    if t.dim() != 2 or (like is not None and t.shape != like.shape):
        raise ValueError("%s must be a matrix%s" % (name, "" if like is None else " of shape %s" % (tuple(like.shape),)))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    width = max(1, t.shape[1])
    if t.shape[0] <= 1:
        return width
    if t.stride(0) < width:
        raise ValueError("%s must not have overlapping rows" % name)
    return t.stride(0)


def _vector(name, t, n, device, dtypes):
    if t.dim() != 1 or t.shape[0] != n or t.dtype not in dtypes or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d elements on %s"
                         % (name, " or ".join(str(d) for d in dtypes), n, device))
    return t.data_ptr()


def _queue(stream, device):
    return torch.cuda.current_stream(device).cuda_stream if stream is None else _stream(stream)


def _weights(x, named):
    """(their type, their addresses) of a norm's vectors: of one type, x's or float32; None gives address 0."""
    given = [t for _, t in named if t is not None]
    dtype = given[0].dtype if given else x.dtype
    allowed = (dtype,) if dtype in (x.dtype, torch.float32) else (x.dtype, torch.float32)
    at = [0 if t is None else _vector(n, t, x.shape[1], x.device, allowed) for n, t in named]
    return dtype, at


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """(y, mean, rstd): y = (x - mean) * rstd * weight + bias over each row of x.

    weight and bias hold x's type or float32 (None: 1 and 0); mean and rstd
    are float32, one value per row.  `out` may be x itself."""
    ldx = _matrix("x", x)
    if x.shape[1] < 1:
        raise ValueError("x must have at least one column")
    wtype, (pw, pb) = _weights(x, (("weight", weight), ("bias", bias)))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    ldo = _matrix("out", out, x)
    rows, width = x.shape
    mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    check(lib().gemm_f32_layer_norm(_TYPES[x.dtype], _TYPES[wtype], rows, width, x.data_ptr(), ldx, pw, pb, eps,
                                    out.data_ptr(), ldo, mean.data_ptr(), rstd.data_ptr(),
                                    _queue(stream, x.device)), "layer_norm")
    return out, mean, rstd


def layer_norm_grad(dy, x, weight, mean, rstd, out=None, stream=None):
    """(dx, dweight, dbias) of layer_norm for dy, the gradient of y, with the
    mean and rstd that layer_norm returned.

    dweight and dbias hold weight's type (float32 for weight None).  `out`,
    the tensor for dx, may be dy or x itself."""
    ldx = _matrix("x", x)
    if x.shape[1] < 1:
        raise ValueError("x must have at least one column")
    lddy = _matrix("dy", dy, x)
    rows, width = x.shape
    wtype, (pw,) = _weights(x, (("weight", weight),))
    if weight is None:
        wtype = torch.float32
    f32 = (torch.float32,)
    pm, pr = _vector("mean", mean, rows, x.device, f32), _vector("rstd", rstd, rows, x.device, f32)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    ldo = _matrix("out", out, x)
    dweight = torch.empty(width, dtype=wtype, device=x.device)
    dbias = torch.empty(width, dtype=wtype, device=x.device)
    check(lib().gemm_f32_layer_norm_grad(_TYPES[x.dtype], _TYPES[wtype], rows, width, dy.data_ptr(), lddy,
                                         x.data_ptr(), ldx, pw, pm, pr, out.data_ptr(), ldo, dweight.data_ptr(),
                                         dbias.data_ptr(), _queue(stream, x.device)), "layer_norm_grad")
    return out, dweight, dbias


def _loss_args(x, w, targets, reduction):
    ldx, ldw = _matrix("x", x), _matrix("w", w)
    if w.dtype != x.dtype or w.device != x.device or w.shape[1] != x.shape[1]:
        raise ValueError("w must be a %s matrix on %s with x's %d columns" % (x.dtype, x.device, x.shape[1]))
    if x.shape[1] < 1 or w.shape[0] < 1:
        raise ValueError("x and w must have at least one column and w one row")
    pt = _vector("targets", targets, x.shape[0], x.device, (torch.int64, torch.int32))
    if reduction not in REDUCTIONS:
        raise ValueError("reduction must be one of %s" % ", ".join(sorted(REDUCTIONS)))
    loss = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    lse = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    total = torch.empty((), dtype=torch.float32, device=x.device)
    return (_TYPES[x.dtype], x.shape[0], x.shape[1], w.shape[0], x.data_ptr(), ldx, w.data_ptr(), ldw, pt,
            64 if targets.dtype == torch.int64 else 32), loss, lse, total


def vocab_loss(x, w, targets, ignore_index=-100, reduction="mean", stream=None):
    """(total, loss, lse): softmax cross entropy of the logits x @ w.T, which are never stored.

    x: rows x width, w: vocab x width, of one type; targets: int64 or int32,
    one per row.  loss and lse are float32 per row (loss 0 where the target
    is ignore_index), total their sum, or mean over the rows that count.  A
    target outside the vocabulary counts as ignored and is reported by
    gemm_f32_status()."""
    args, loss, lse, total = _loss_args(x, w, targets, reduction)
    check(lib().gemm_f32_vocab_loss(*args, ignore_index, REDUCTIONS[reduction], loss.data_ptr(), lse.data_ptr(),
                                    total.data_ptr(), _queue(stream, x.device)), "vocab_loss")
    return total, loss, lse


def vocab_loss_grad(x, w, targets, ignore_index=-100, reduction="mean", grad_scale=1.0, need_dx=True, need_dw=True,
                    piece_bytes=0, stream=None):
    """(total, loss, lse, dx, dw): vocab_loss and the gradients of grad_scale * total.

    dx and dw hold x's type; need_dx / need_dw False leaves one out (None).
    piece_bytes bounds the scratch that holds a piece of the rows (0: the
    library's default)."""
    args, loss, lse, total = _loss_args(x, w, targets, reduction)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
    dw = torch.empty(w.shape, dtype=w.dtype, device=w.device) if need_dw else None
    check(lib().gemm_f32_vocab_loss_grad(*args, ignore_index, REDUCTIONS[reduction], grad_scale, loss.data_ptr(),
                                         lse.data_ptr(), total.data_ptr(), dx.data_ptr() if need_dx else 0,
                                         x.shape[1], dw.data_ptr() if need_dw else 0, x.shape[1], piece_bytes,
                                         _queue(stream, x.device)), "vocab_loss_grad")
    return total, loss, lse, dx, dw
