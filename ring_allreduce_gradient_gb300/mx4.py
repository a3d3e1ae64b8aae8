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

import torch

from . import binding as B
from .collectives import _DT, _code

FORMATS = {"mxfp4": B.DP_MXFP4, "nvfp4": B.DP_NVFP4}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}


def _format(name) -> int:
    if name not in FORMATS:
        raise ValueError(f"format: 'mxfp4' or 'nvfp4', not {name!r}")
    return FORMATS[name]


def _scale_bytes(rows: int, cols: int, format: str) -> int:
    """dp_mx4_scales_size."""
    return -(-rows // 128) * -(-cols // (4 * _BLOCK[format])) * 512


class Mx4Tensor:
    """A [rows, cols] matrix in 4 bits (layout: ``include/dp.h``), read-only
    once made: it keeps its buffers and their addresses for the calls.

    ``codes``: uint8, rows x cols/2 bytes; ``scales``: uint8 tiles;
    ``tensor_scale``: one fp32 device value or None (nvfp4 only).
    """

    __slots__ = ("_codes", "_scales", "_store", "_tensor_scale", "_kind", "_c")

    def __init__(self, codes, scales, rows: int, cols: int, format: str, tensor_scale=None):
        _format(format)
        for name, t, n in (("codes", codes, rows * (cols // 2)),
                           ("scales", scales, _scale_bytes(rows, cols, format))):
            if t.dtype != torch.uint8 or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name}: {n} contiguous bytes for a {format} matrix of "
                                 f"{rows} x {cols}")
        if scales.device != codes.device:
            raise ValueError("codes and scales on one device")
        _check_scale(tensor_scale, codes.device)
        self._codes, self._scales, self._store = codes, scales, None
        self._tensor_scale = tensor_scale
        self._kind = (rows, cols, format, codes.device)
        self._c = B.Mx4(codes.data_ptr(), scales.data_ptr(),
                        None if tensor_scale is None else tensor_scale.data_ptr())

    @classmethod
    def _empty(cls, rows, cols, format, tensor_scale, device):
        """A matrix to be written, codes and scales in one allocation."""
        q = cls.__new__(cls)
        n = -(-rows * (cols // 2) // 256) * 256
        q._store = torch.empty(n + _scale_bytes(rows, cols, format), dtype=torch.uint8,
                               device=device)
        q._codes = q._scales = None      # views, made when they are asked for
        q._tensor_scale = tensor_scale
        q._kind = (rows, cols, format, device)
        at = q._store.data_ptr()
        q._c = B.Mx4(at, at + n, None if tensor_scale is None else tensor_scale.data_ptr())
        return q

    @property
    def codes(self):
        if self._codes is None:
            rows, cols = self.rows, self.cols
            self._codes = self._store[:rows * (cols // 2)].view(rows, cols // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            n = _scale_bytes(self.rows, self.cols, self.format)
            self._scales = self._store[self._store.numel() - n:]
        return self._scales

    rows = property(lambda self: self._kind[0])
    cols = property(lambda self: self._kind[1])
    format = property(lambda self: self._kind[2])
    device = property(lambda self: self._kind[3])
    tensor_scale = property(lambda self: self._tensor_scale)

    def __repr__(self):
        return f"Mx4Tensor({self.rows} x {self.cols}, {self.format}, {self.device})"


def _check_scale(scale, device):
    if scale is not None and (scale.dtype != torch.float32 or scale.numel() != 1 or
                              scale.device != device):
        raise ValueError(f"tensor_scale: one fp32 value on {device}")


def _on(stream, device):
    """A context in which allocations, fills and calls belong to ``stream``."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def tensor_scale(x, out=None, stream=None) -> torch.Tensor:
    """The nvfp4 scale of a tensor (or of a list of them, say all of a
    matrix's shards): its largest magnitude / 2688, one fp32 device value."""
    xs = [x] if isinstance(x, torch.Tensor) else list(x)
    if not xs or any(t.dtype != xs[0].dtype or t.device != xs[0].device or
                     not t.is_contiguous() for t in xs):
        raise ValueError("need contiguous tensors of one dtype and device")
    dev = xs[0].device
    if stream is not None:
        with _on(stream, dev):
            return tensor_scale(xs, out)
    out = torch.empty(1, dtype=torch.float32, device=dev) if out is None else out
    _check_scale(out, dev)
    ws = torch.zeros(B.dp_grad_norm_workspace_size(len(xs)), dtype=torch.uint8, device=dev)
    B.dp_mx4_tensor_scale(xs, [t.numel() for t in xs], len(xs), _code(xs[0]), out, ws,
                          stream=B._stream_on(dev, "tensor_scale"))
    return out


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
    if stream is not None:
        with _on(stream, xs[0].device):
            return quantize(xs, format, tensor_scale, transpose)
    x0 = xs[0]
    first, ld = _rows(x0)
    rows, cols = x0.shape
    for t in xs[1:]:
        if t.shape != x0.shape or t.dtype != x0.dtype or t.device != x0.device or \
                t.stride() != x0.stride():
            raise ValueError("need shards of one shape, dtype, device and row stride")
    if first is not x0:
        xs = [first] + [_rows(t)[0] for t in xs[1:]]
    dev = x0.device
    if tensor_scale is not None:
        _check_scale(tensor_scale, dev)
    K = len(xs)
    R, L = (cols, K * rows) if transpose else (K * rows, cols)
    q = Mx4Tensor._empty(R, L, format, tensor_scale, dev)
    c = q._c
    st = (B._lib or B.load()).dp_mx4_quantize(
        B._parray(xs), K, rows, cols, ld, _code(x0), fmt, 1 if transpose else 0,
        c.tensor_scale, c.codes, c.scales, B._stream_on(dev, "quantize"))
    if st:
        raise B.DpError(st, "dp_mx4_quantize")
    return q


def _rows(x):
    """A matrix as the library takes it, and the elements between its rows, which
    are at least a row's length.  Rows that overlap (one row expanded to many, a
    window moved over a vector) are copied out."""
    if x.dim() != 2:
        raise ValueError(f"need a matrix, got {tuple(x.shape)}: flatten the other dimensions first")
    rows, cols = x.shape
    ld, unit = x.stride()
    if unit != 1 and cols > 1:
        raise ValueError("need a matrix with unit stride along its rows")
    if rows <= 1:
        return x, cols
    if ld < cols:
        return x.contiguous(), cols
    return x, ld


def dequantize(q: Mx4Tensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values a 4-bit matrix stands for."""
    rows, cols, format, dev = q._kind
    if stream is not None:
        with _on(stream, dev):
            return dequantize(q, dtype)
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    out = torch.empty((rows, cols), dtype=dtype, device=dev)
    c = q._c
    st = (B._lib or B.load()).dp_mx4_dequantize(c.codes, c.scales, rows, cols, FORMATS[format],
                                                c.tensor_scale, out.data_ptr(), _DT[dtype],
                                                B._stream_on(dev, "dequantize"))
    if st:
        raise B.DpError(st, "dp_mx4_dequantize")
    return out


def _shards(w_shards, cols, format, device):
    """The shards' structures, after checking that they make one matrix for this operand."""
    if not w_shards:
        raise ValueError("need at least one shard")
    w0 = w_shards[0]
    kind = (w0._kind[0], cols, format, device)
    if w0._kind != kind:
        raise ValueError(f"x is {format} with {cols} columns on {device}, the shards {w0!r}")
    for w in w_shards:
        if w._kind != kind:
            raise ValueError("need shards of one shape, format and device")
    return (B.Mx4 * len(w_shards))(*[w._c for w in w_shards])


def matmul(x: Mx4Tensor, w_shards, y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x . w^T with w the row concatenation of the 4-bit shards."""
    M, D, format, dev = x._kind
    if stream is not None:
        with _on(stream, dev):
            return matmul(x, w_shards, y_dtype)
    if y_dtype not in _DT:
        raise TypeError(f"unsupported dtype {y_dtype}")
    K = len(w_shards)
    arr = _shards(w_shards, D, format, dev)
    y = torch.empty((M, K * w_shards[0].rows), dtype=y_dtype, device=dev)
    B.dp_allgather_matmul_mx4(x._c, M, D, arr, K, w_shards[0].rows, FORMATS[format], y,
                              _DT[y_dtype], stream=B._stream_on(dev, "matmul"))
    return y


def linear(x: torch.Tensor, w_shards, x_scale=None, y_dtype=torch.bfloat16,
           stream=None) -> torch.Tensor:
    """y = x . w^T with x [M, D] quantised to the shards' format on the way
    (``x_scale``: its nvfp4 tensor scale), in one call.  Like every call here it
    records no gradient: an autograd function calls it in its forward, and its
    backward products (above) in its backward."""
    if stream is not None:
        with _on(stream, x.device):
            return linear(x, w_shards, x_scale, y_dtype)
    # One token's product takes the GPU less time than this function: it makes
    # the call itself, without the binding's marshalling.
    x, ld = _rows(x)
    M, D = x.shape
    if y_dtype not in _DT:
        raise TypeError(f"unsupported dtype {y_dtype}")
    if not w_shards:
        raise ValueError("need at least one shard")
    dev, K = x.device, len(w_shards)
    F, _, format, _ = w_shards[0]._kind
    arr = _shards(w_shards, D, format, dev)
    if x_scale is not None:
        _check_scale(x_scale, dev)
    # scratch of this call alone: the allocator hands it on in stream order
    nbytes = -(-M * (D // 2) // 256) * 256 + _scale_bytes(M, D, format)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    y = torch.empty((M, K * F), dtype=y_dtype, device=dev)
    st = (B._lib or B.load()).dp_allgather_linear_mx4(
        x.data_ptr(), M, D, ld, _code(x),
        None if x_scale is None else x_scale.data_ptr(), arr, K, F, FORMATS[format],
        y.data_ptr(), _DT[y_dtype], ws.data_ptr(), nbytes, B._stream_on(dev, "linear"))
    if st:
        raise B.DpError(st, "dp_allgather_linear_mx4")
    return y
