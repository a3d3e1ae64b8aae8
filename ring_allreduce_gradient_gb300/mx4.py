"""Microscaled 4-bit matrices: quantisation of parameter shards, activations
and gradients, and the all-gather product of two such operands.

    wq = [quantize(w, "nvfp4", tensor_scale=tensor_scale(w)) for w in shards]
    y = linear(x, wq, x_scale=x_scale)            # y = x . w^T, both in 4 bits
    # backward, in 4 bits too: blocks along the contracted dimension
    wt = quantize(shards, "nvfp4", tensor_scale=s, transpose=True)   # [D, F], gathered
    dx = linear(dy, [wt])                                            # dy . w
    dw = matmul(quantize(dy, transpose=True), [quantize(x, transpose=True)])  # dy^T . x

No arithmetic happens here: it allocates with PyTorch and calls the binding.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B
from .collectives import _DT, _code

FORMATS = {"mxfp4": B.DP_MXFP4, "nvfp4": B.DP_NVFP4}


def _format(name) -> int:
    if name not in FORMATS:
        raise ValueError(f"format: 'mxfp4' or 'nvfp4', not {name!r}")
    return FORMATS[name]


@dataclass
class Mx4Tensor:
    """A [rows, cols] matrix in 4 bits (layout: ``include/dp.h``).

    ``codes``: uint8, rows x cols/2 bytes; ``scales``: uint8 tiles;
    ``tensor_scale``: one fp32 device value or None (nvfp4 only).
    """

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    format: str
    tensor_scale: Optional[torch.Tensor] = None

    def __post_init__(self):
        need = B.dp_mx4_scales_size(self.rows, self.cols, _format(self.format))
        for name, t, n in (("codes", self.codes, self.rows * (self.cols // 2)),
                           ("scales", self.scales, need)):
            if t.dtype != torch.uint8 or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name}: {n} contiguous bytes for a {self.format} matrix of "
                                 f"{self.rows} x {self.cols}")
        _check_scale(self.tensor_scale, self.codes.device)

    def _triple(self):
        return (self.codes, self.scales, self.tensor_scale)


def _check_scale(scale, device):
    if scale is not None and (scale.dtype != torch.float32 or scale.numel() != 1 or
                              scale.device != device):
        raise ValueError(f"tensor_scale: one fp32 value on {device}")


def tensor_scale(x, out=None, stream=None) -> torch.Tensor:
    """The nvfp4 scale of a tensor (or of a list of them, say all of a
    matrix's shards): its largest magnitude / 2688, one fp32 device value."""
    xs = [x] if isinstance(x, torch.Tensor) else list(x)
    if not xs or any(t.dtype != xs[0].dtype or t.device != xs[0].device or
                     not t.is_contiguous() for t in xs):
        raise ValueError("need contiguous tensors of one dtype and device")
    dev = xs[0].device
    out = torch.empty(1, dtype=torch.float32, device=dev) if out is None else out
    _check_scale(out, dev)
    with torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else _same():
        ws = torch.zeros(B.dp_grad_norm_workspace_size(len(xs)), dtype=torch.uint8, device=dev)
    B.dp_mx4_tensor_scale(xs, [t.numel() for t in xs], len(xs), _code(xs[0]), out, ws,
                          stream=stream)
    return out


class _same:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


def quantize(x, format: str = "mxfp4", tensor_scale=None, transpose: bool = False,
             stream=None) -> Mx4Tensor:
    """4-bit form of a matrix (fp32 or bf16, unit stride along its rows), or of
    the row concatenation of a list of shards; with ``transpose``, of its
    transpose.  ``tensor_scale`` (nvfp4): one fp32 device value, as
    ``tensor_scale()`` gives it or calibrated beforehand."""
    fmt = _format(format)
    xs = [x] if isinstance(x, torch.Tensor) else list(x)
    if not xs:
        raise ValueError("need at least one shard")
    x0 = xs[0]
    for t in xs:
        if t.dim() != 2 or t.shape != x0.shape or t.dtype != x0.dtype or t.device != x0.device \
                or t.stride() != x0.stride() or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError("need matrices of one shape, dtype, device and row stride, with unit "
                             "stride along the rows")
    rows, cols = x0.shape
    ld = x0.stride(0) if rows > 1 else cols
    _check_scale(tensor_scale, x0.device)
    K = len(xs)
    R, L = (cols, K * rows) if transpose else (K * rows, cols)
    codes = torch.empty(R, L // 2, dtype=torch.uint8, device=x0.device)
    scales = torch.empty(B.dp_mx4_scales_size(R, L, fmt), dtype=torch.uint8, device=x0.device)
    B.dp_mx4_quantize(xs, K, rows, cols, max(ld, cols), _code(x0), fmt, transpose, tensor_scale,
                      codes, scales, stream)
    return Mx4Tensor(codes, scales, R, L, format, tensor_scale)


def dequantize(q: Mx4Tensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values a 4-bit matrix stands for."""
    out = torch.empty(q.rows, q.cols, dtype=dtype, device=q.codes.device)
    B.dp_mx4_dequantize(q.codes, q.scales, q.rows, q.cols, _format(q.format), q.tensor_scale, out,
                        _code(out), stream)
    return out


def matmul(x: Mx4Tensor, w_shards, y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x . w^T with w the row concatenation of the 4-bit shards."""
    w0 = w_shards[0]
    for w in w_shards:
        if (w.rows, w.cols, w.format) != (w0.rows, w0.cols, w0.format) or \
                w.codes.device != x.codes.device:
            raise ValueError("need shards of one shape, format and device")
    if w0.cols != x.cols or w0.format != x.format:
        raise ValueError(f"x is {x.format} with {x.cols} columns, the shards {w0.format} "
                         f"with {w0.cols}")
    if y_dtype not in _DT:
        raise TypeError(f"unsupported dtype {y_dtype}")
    y = torch.empty(x.rows, len(w_shards) * w0.rows, dtype=y_dtype, device=x.codes.device)
    B.dp_allgather_matmul_mx4(x._triple(), x.rows, x.cols, [w._triple() for w in w_shards],
                              len(w_shards), w0.rows, _format(x.format), y, _DT[y_dtype], stream)
    return y


def linear(x: torch.Tensor, w_shards, x_scale=None, y_dtype=torch.bfloat16,
           stream=None) -> torch.Tensor:
    """y = x . w^T with x [M, D] quantised to the shards' format on the way."""
    return matmul(quantize(x, w_shards[0].format, x_scale, stream=stream), w_shards, y_dtype,
                  stream)
