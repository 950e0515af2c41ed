"""Layer norm and the vocabulary loss on torch tensors: checks of arguments,
allocation of outputs, and the call into libgemm_f32.so (include/gemm_f32_lm.h).

Matrices are 2-D CUDA tensors of float32 or bfloat16 with contiguous rows
(stride(1) == 1; stride(0) may exceed the width, as in a column slice).
Calls are queued on `stream` (a torch stream or a handle), or on torch's
current stream of the tensors' device, and return without waiting for it.
They run on the tensors' device, and what they allocate belongs to the stream
they are queued on: a caller that goes on with it on another stream, or gives
a tensor of another stream's, orders the two and keeps the memory
(wait_stream, record_stream), as with torch's own operators.  Their scratch is
the library's, apart from torch's allocator, until gemm_f32_release().
"""
from __future__ import annotations

import torch

from ._binding import GEMM_F32_ESCRATCH, MOST_INT, REDUCTIONS, TYPE_BF16, TYPE_F32, check, elsewhere, lib

_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16}
_F32 = torch.float32
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream      # current_stream(i).cuda_stream, without the objects


def _stride(name, t, width):
    """Row stride of a matrix that is not contiguous."""
    if width > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if t.shape[0] <= 1:
        return width
    if t.stride(0) < width:
        raise ValueError("%s must not have overlapping rows" % name)
    return t.stride(0)


def _matrix(name, t):
    """(type, device index, rows, width, row stride) of an input matrix."""
    kind = _TYPES.get(t.dtype)
    if kind is None or not t.is_cuda:
        raise ValueError("%s must be a float32 or bfloat16 CUDA tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    rows, width = t.shape
    if width < 1:
        raise ValueError("%s must have at least one column" % name)
    if width > MOST_INT:
        raise ValueError("%s must have at most %d columns" % (name, MOST_INT))
    return kind, t.get_device(), rows, width, width if t.is_contiguous() else _stride(name, t, width)


def _like(name, t, x):
    """Row stride of a matrix of x's shape, type and device."""
    if t.dtype is not x.dtype or t.shape != x.shape or t.get_device() != x.get_device():
        raise ValueError("%s must be a %s matrix of shape %s on %s" % (name, x.dtype, tuple(x.shape), x.device))
    return t.shape[1] if t.is_contiguous() else _stride(name, t, t.shape[1])


def _vector(name, t, n, dev, dtypes):
    """Address of a contiguous vector of n elements."""
    if t.dtype not in dtypes or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d elements on device %d"
                         % (name, " or ".join(str(d) for d in dtypes), n, dev))
    return t.data_ptr()


def _call(name, *args):
    """A call that needs scratch.  Where the library finds no memory for it, torch's allocator may hold some that is
    free: it gives that back, once (but not during a capture)."""
    entry = getattr(lib(), name)
    code = entry(*args)
    if code == GEMM_F32_ESCRATCH and not torch.cuda.is_current_stream_capturing():
        torch.cuda.empty_cache()
        code = entry(*args)
    check(code, name)


def _weight_type(x, weight):
    dtype = weight.dtype
    if dtype is not x.dtype and dtype is not _F32:
        raise ValueError("weight and bias must hold x's type or float32")
    return dtype


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """(y, mean, rstd): y = (x - mean) * rstd * weight + bias over each row of x.

    weight and bias hold x's type or float32 (None: 1 and 0); mean and rstd
    are float32, one value per row.  `out` may be x itself."""
    kind, dev, rows, width, ldx = _matrix("x", x)
    if stream is not None or _current_device() != dev:
        with elsewhere(dev, stream):
            return layer_norm(x, weight, bias, eps, out)
    wtype, pw, pb = x.dtype, 0, 0
    if weight is not None:
        wtype = _weight_type(x, weight)
        pw = _vector("weight", weight, width, dev, (wtype,))
    if bias is not None:
        if weight is None:
            wtype = _weight_type(x, bias)
        pb = _vector("bias", bias, width, dev, (wtype,))
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldo = width
    else:
        ldo = _like("out", out, x)
    mean = torch.empty(rows, dtype=_F32, device=x.device)
    rstd = torch.empty_like(mean)
    check(lib().gemm_f32_layer_norm(kind, _TYPES[wtype], rows, width, x.data_ptr(), ldx, pw, pb, eps, out.data_ptr(),
                                    ldo, mean.data_ptr(), rstd.data_ptr(), _raw_stream(dev)), "layer_norm")
    return out, mean, rstd


def layer_norm_grad(dy, x, weight, mean, rstd, out=None, stream=None):
    """(dx, dweight, dbias) of layer_norm for dy, the gradient of y, with the
    mean and rstd that layer_norm returned.

    dweight and dbias hold weight's type (float32 for weight None).  `out`,
    the tensor for dx, may be dy or x itself."""
    kind, dev, rows, width, ldx = _matrix("x", x)
    if stream is not None or _current_device() != dev:
        with elsewhere(dev, stream):
            return layer_norm_grad(dy, x, weight, mean, rstd, out)
    lddy = _like("dy", dy, x)
    wtype, pw = _F32, 0
    if weight is not None:
        wtype = _weight_type(x, weight)
        pw = _vector("weight", weight, width, dev, (wtype,))
    pm, pr = _vector("mean", mean, rows, dev, (_F32,)), _vector("rstd", rstd, rows, dev, (_F32,))
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldo = width
    else:
        ldo = _like("out", out, x)
    dweight = torch.empty(width, dtype=wtype, device=x.device)
    dbias = torch.empty_like(dweight)
    _call("gemm_f32_layer_norm_grad", kind, _TYPES[wtype], rows, width, dy.data_ptr(), lddy, x.data_ptr(), ldx, pw,
          pm, pr, out.data_ptr(), ldo, dweight.data_ptr(), dbias.data_ptr(), _raw_stream(dev))
    return out, dweight, dbias


def _loss_args(x, w, targets, reduction, matrix):
    """The C call's arguments up to target_bits, the reduction's code and the outputs of both calls; `matrix` is x's."""
    kind, dev, rows, width, ldx = matrix
    wkind, wdev, vocab, wwidth, ldw = _matrix("w", w)
    if wkind != kind or wdev != dev or wwidth != width:
        raise ValueError("w must be a %s matrix on %s with x's %d columns" % (x.dtype, x.device, width))
    if not 1 <= vocab <= MOST_INT:
        raise ValueError("w must have at least one row, and at most %d" % MOST_INT)
    pt = _vector("targets", targets, rows, dev, (torch.int64, torch.int32))
    if reduction not in REDUCTIONS:
        raise ValueError("reduction must be one of %s" % ", ".join(sorted(REDUCTIONS)))
    loss = torch.empty(rows, dtype=_F32, device=x.device)
    return ((kind, rows, width, vocab, x.data_ptr(), ldx, w.data_ptr(), ldw, pt,
             64 if targets.dtype is torch.int64 else 32), REDUCTIONS[reduction], loss, torch.empty_like(loss),
            torch.empty((), dtype=_F32, device=x.device))


def vocab_loss(x, w, targets, ignore_index=-100, reduction="mean", stream=None):
    """(total, loss, lse): softmax cross entropy of the logits x @ w.T, which are never stored.

    x: rows x width, w: vocab x width, of one type; targets: int64 or int32,
    one per row.  loss and lse are float32 per row (loss 0 where the target
    is ignore_index), total their sum, or mean over the rows that count.  A
    target outside the vocabulary counts as ignored and is reported by
    gemm_f32_status()."""
    matrix = _matrix("x", x)
    if stream is not None or _current_device() != matrix[1]:
        with elsewhere(matrix[1], stream):
            return vocab_loss(x, w, targets, ignore_index, reduction)
    args, code, loss, lse, total = _loss_args(x, w, targets, reduction, matrix)
    _call("gemm_f32_vocab_loss", *args, ignore_index, code, loss.data_ptr(), lse.data_ptr(), total.data_ptr(),
          _raw_stream(matrix[1]))
    return total, loss, lse


def vocab_loss_grad(x, w, targets, ignore_index=-100, reduction="mean", grad_scale=1.0, need_dx=True, need_dw=True,
                    piece_bytes=0, stream=None):
    """(total, loss, lse, dx, dw): vocab_loss and the gradients of grad_scale * total.

    dx and dw hold x's type; need_dx / need_dw False leaves one out (None).
    piece_bytes bounds the scratch that holds a piece of the rows (0: the
    library's default)."""
    matrix = _matrix("x", x)
    if stream is not None or _current_device() != matrix[1]:
        with elsewhere(matrix[1], stream):
            return vocab_loss_grad(x, w, targets, ignore_index, reduction, grad_scale, need_dx, need_dw, piece_bytes)
    args, code, loss, lse, total = _loss_args(x, w, targets, reduction, matrix)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
    dw = torch.empty_like(w, memory_format=torch.contiguous_format) if need_dw else None
    _call("gemm_f32_vocab_loss_grad", *args, ignore_index, code, grad_scale, loss.data_ptr(), lse.data_ptr(),
          total.data_ptr(), dx.data_ptr() if need_dx else 0, args[2], dw.data_ptr() if need_dw else 0, args[2],
          piece_bytes, _raw_stream(matrix[1]))
    return total, loss, lse, dx, dw
