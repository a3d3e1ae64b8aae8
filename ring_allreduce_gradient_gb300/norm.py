"""The root-mean-square norm in front of a layer's products: residual addition,
norm and the operand's quantised form in one pass, and its backward pass.

    n = rms_norm(x, weight, residual=h, format="mxfp8")
    y = mx8.matmul(n.q, wq)                          # the layer, on n.q
    ...                                              # n.h: the next residual
    # backward: dy, the gradient of the norm's output, and dh, that of n.h past it
    dx, dweight = rms_norm_backward(dy, n.h, weight, n.rstd, dh=dh)

The calls record no gradient: an autograd function calls the first in its forward
and the second in its backward.  No arithmetic happens here: it allocates with
PyTorch and calls the binding.
"""
from __future__ import annotations

from functools import lru_cache
from typing import NamedTuple

import torch

from . import binding as B
from .collectives import _code
from .mx4 import Mx4Tensor, _check_scale, _on, _rows
from .mx8 import Mx8Tensor

FORMATS = {"mxfp4": B.DP_NORM_MXFP4, "nvfp4": B.DP_NORM_NVFP4, "mxfp8": B.DP_NORM_MXFP8}


class Normed(NamedTuple):
    """``y``: the output, or None; ``h``: x + residual (x itself without one);
    ``rstd``: 1 / root-mean-square of each row, fp32; ``q``: y quantised, or None."""
    y: torch.Tensor | None
    h: torch.Tensor
    rstd: torch.Tensor
    q: Mx4Tensor | Mx8Tensor | None


_workspace_size = lru_cache(256)(B.dp_rms_norm_backward_workspace_size)   # of (M, D) alone


def _weight(weight, cols, device):
    if weight.dim() != 1 or weight.numel() != cols or weight.device != device or \
            not weight.is_contiguous():
        raise ValueError(f"weight: {cols} contiguous values on {device}")
    return _code(weight)


def _like(name, t, x):
    """A matrix of x's shape, dtype and device as the library takes it."""
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name}: {tuple(t.shape)} of {t.dtype} on {t.device}, "
                         f"x is {tuple(x.shape)} of {x.dtype} on {x.device}")
    return _rows(t)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6,
             format: str | None = None, tensor_scale=None, keep: bool = False,
             stream=None) -> Normed:
    """y = h / rms(h) * weight with h = x + residual, for the rows of x [M, D]
    (fp32 or bf16; ``residual``: like x; ``weight``: D values, fp32 or bf16).

    ``format``: "mxfp4", "nvfp4" (``tensor_scale``: its fp32 device value,
    calibrated beforehand) or "mxfp8": y is quantised as it is formed, into ``q``,
    and is itself kept only with ``keep`` (a weight gradient needs it).  Rows of no
    elements have rstd NaN."""
    if format is not None and format not in FORMATS:
        raise ValueError(f"format: None, 'mxfp4', 'nvfp4' or 'mxfp8', not {format!r}")
    if stream is not None:
        with _on(stream, x.device):
            return rms_norm(x, weight, residual, eps, format, tensor_scale, keep)
    xs, ld = _rows(x)
    M, D = x.shape
    dev, code = x.device, _code(x)
    wcode = _weight(weight, D, dev)
    rs, ldr = (None, 0) if residual is None else _like("residual", residual, x)
    if tensor_scale is not None:
        if format != "nvfp4":
            raise ValueError("tensor_scale belongs to nvfp4")
        _check_scale(tensor_scale, dev)
    here = B._stream_on(dev, "rms_norm")
    h = x if residual is None else torch.empty((M, D), dtype=x.dtype, device=dev)
    rstd = torch.empty(M, dtype=torch.float32, device=dev)
    if D == 0:
        rstd.fill_(float("nan"))     # a mean of nothing; the library writes nothing then
    y = torch.empty((M, D), dtype=x.dtype, device=dev) if keep or format is None else None
    q = c = None
    if format is not None:
        q = Mx8Tensor._empty(M, D, dev) if format == "mxfp8" else \
            Mx4Tensor._empty(M, D, format, tensor_scale, dev)
        c = q._c
    st = (B._lib or B.load()).dp_rms_norm(
        xs.data_ptr(), ld, None if rs is None else rs.data_ptr(), ldr, M, D, code,
        weight.data_ptr(), wcode, eps, None if rs is None else h.data_ptr(),
        None if y is None else y.data_ptr(), rstd.data_ptr(),
        B.DP_NORM_PLAIN if q is None else FORMATS[format], None if c is None else c.tensor_scale,
        None if c is None else c.codes, None if c is None else c.scales, here)
    if st:
        raise B.DpError(st, "dp_rms_norm")
    return Normed(y, h, rstd, q)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                      rstd: torch.Tensor, dh=None, stream=None):
    """(dx, dweight) from the gradient ``dy`` of the norm's output and ``dh``, the
    gradient that reaches h past the norm (or None); ``h`` and ``rstd`` are the
    forward's.  dx, of h's dtype, is the gradient of x and of the residual alike;
    dweight is fp32.  A quantised output's gradient passes straight through."""
    if stream is not None:
        with _on(stream, h.device):
            return rms_norm_backward(dy, h, weight, rstd, dh)
    hs, ldh = _rows(h)
    M, D = h.shape
    dev, code = h.device, _code(h)
    wcode = _weight(weight, D, dev)
    ys, ldy = _like("dy", dy, h)
    ds, ldd = (None, 0) if dh is None else _like("dh", dh, h)
    if rstd.dtype != torch.float32 or rstd.numel() != M or rstd.device != dev or \
            not rstd.is_contiguous():
        raise ValueError(f"rstd: {M} contiguous fp32 values on {dev}")
    here = B._stream_on(dev, "rms_norm_backward")
    dx = torch.empty((M, D), dtype=h.dtype, device=dev)
    dw = torch.empty(D, dtype=torch.float32, device=dev)
    # scratch of this call alone: the allocator hands it on in stream order
    n = _workspace_size(M, D)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    st = (B._lib or B.load()).dp_rms_norm_backward(
        ys.data_ptr(), ldy, hs.data_ptr(), ldh, None if ds is None else ds.data_ptr(), ldd, M, D,
        code, weight.data_ptr(), wcode, rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(),
        ws.data_ptr(), n, here)
    if st:
        raise B.DpError(st, "dp_rms_norm_backward")
    return dx, dw
