"""Activations in the 8-bit microscaled form (mxfp8: e4m3 values, a power of two
for each 32 of a row): quantisation, decoding, and their all-gather product with
4-bit weight shards, for layers whose activations need more bits than their
weights.

    wq = [mx4.quantize(w, "mxfp4") for w in shards]
    y = mx8.linear(x, wq)                  # x . w^T, x in 8 bits, w in 4
    y = mx8.matmul(n.q, wq)                # n = norm.rms_norm(x, weight, format="mxfp8")

No arithmetic happens here: it allocates with PyTorch and calls the binding.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B
from .collectives import _DT, _code
from .mx4 import _on, _rows, _scale_bytes, _shard_bytes


class Mx8Tensor:
    """A [rows, cols] matrix in 8 bits (layout: ``include/dp.h``), read-only
    once made.  ``codes``: uint8 [rows, cols]; ``scales``: uint8 tiles."""

    __slots__ = ("_store", "_codes", "_scales", "_kind", "_c")

    def __init__(self, codes, scales, rows: int, cols: int):
        for name, t, n in (("codes", codes, rows * cols),
                           ("scales", scales, _scale_bytes(rows, cols, "mxfp4"))):
            if t.dtype != torch.uint8 or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name}: {n} contiguous bytes for an mxfp8 matrix of "
                                 f"{rows} x {cols}")
        if scales.device != codes.device:
            raise ValueError("codes and scales on one device")
        self._store, self._codes, self._scales = None, codes, scales
        self._kind = (rows, cols, "mxfp8", codes.device)
        self._c = B.Mx4(codes.data_ptr(), scales.data_ptr(), None)

    @classmethod
    def _empty(cls, rows, cols, device):
        """A matrix to be written, codes and scales in one allocation."""
        q = cls.__new__(cls)
        n = -(-rows * cols // 256) * 256
        q._store = torch.empty(n + _scale_bytes(rows, cols, "mxfp4"), dtype=torch.uint8,
                               device=device)
        q._codes = q._scales = None      # views, made when they are asked for
        q._kind = (rows, cols, "mxfp8", device)
        at = q._store.data_ptr()
        q._c = B.Mx4(at, at + n, None)
        return q

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._store[:self.rows * self.cols].view(self.rows, self.cols)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            n = _scale_bytes(self.rows, self.cols, "mxfp4")
            self._scales = self._store[self._store.numel() - n:]
        return self._scales

    rows = property(lambda self: self._kind[0])
    cols = property(lambda self: self._kind[1])
    format = property(lambda self: self._kind[2])
    device = property(lambda self: self._kind[3])

    def __repr__(self):
        return f"Mx8Tensor({self.rows} x {self.cols}, {self.device})"


def quantize(x: torch.Tensor, stream=None) -> Mx8Tensor:
    """8-bit form of a matrix (fp32 or bf16, unit stride along its rows)."""
    if stream is not None:
        with _on(stream, x.device):
            return quantize(x)
    x, ld = _rows(x)
    rows, cols = x.shape
    code = _code(x)
    q = Mx8Tensor._empty(rows, cols, x.device)
    c = q._c
    st = (B._lib or B.load()).dp_mx8_quantize(x.data_ptr(), rows, cols, ld, code, c.codes,
                                              c.scales, B._stream_on(x.device, "quantize"))
    if st:
        raise B.DpError(st, "dp_mx8_quantize")
    return q


def dequantize(q: Mx8Tensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values an 8-bit matrix stands for."""
    rows, cols, format, dev = q._kind
    if format != "mxfp8":
        raise ValueError(f"need an mxfp8 matrix, not {q!r}")
    if stream is not None:
        with _on(stream, dev):
            return dequantize(q, dtype)
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    out = torch.empty((rows, cols), dtype=dtype, device=dev)
    c = q._c
    st = (B._lib or B.load()).dp_mx8_dequantize(c.codes, c.scales, rows, cols, out.data_ptr(),
                                                _DT[dtype], B._stream_on(dev, "dequantize"))
    if st:
        raise B.DpError(st, "dp_mx8_dequantize")
    return out


def matmul(x: Mx8Tensor, w_shards, y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x . w^T with w the row concatenation of the mxfp4 shards."""
    M, D, format, dev = x._kind
    if format != "mxfp8":
        raise ValueError(f"need an mxfp8 matrix, not {x!r}")
    if stream is not None:
        with _on(stream, dev):
            return matmul(x, w_shards, y_dtype)
    if y_dtype not in _DT:
        raise TypeError(f"unsupported dtype {y_dtype}")
    arr = _shard_bytes(w_shards, D, "mxfp4", dev)
    K, F = len(w_shards), w_shards[0].rows
    y = torch.empty((M, K * F), dtype=y_dtype, device=dev)
    st = (B._lib or B.load()).dp_allgather_matmul_mx8(
        ctypes.byref(x._c), M, D, arr, K, F, y.data_ptr(), _DT[y_dtype],
        B._stream_on(dev, "matmul"))
    if st:
        raise B.DpError(st, "dp_allgather_matmul_mx8")
    return y


def linear(x: torch.Tensor, w_shards, y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x . w^T with x [M, D] quantised to 8 bits on the way and w the row
    concatenation of the mxfp4 shards, in one call.  Records no gradient."""
    if stream is not None:
        with _on(stream, x.device):
            return linear(x, w_shards, y_dtype)
    x, ld = _rows(x)
    M, D = x.shape
    if y_dtype not in _DT:
        raise TypeError(f"unsupported dtype {y_dtype}")
    dev, code = x.device, _code(x)
    arr = _shard_bytes(w_shards, D, "mxfp4", dev)
    K, F = len(w_shards), w_shards[0].rows
    here = B._stream_on(dev, "linear")
    # scratch of this call alone: the allocator hands it on in stream order
    nbytes = -(-M * D // 256) * 256 + _scale_bytes(M, D, "mxfp4")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    y = torch.empty((M, K * F), dtype=y_dtype, device=dev)
    st = (B._lib or B.load()).dp_allgather_linear_mx8(
        x.data_ptr(), M, D, ld, code, arr, K, F, y.data_ptr(), _DT[y_dtype], ws.data_ptr(), nbytes,
        here)
    if st:
        raise B.DpError(st, "dp_allgather_linear_mx8")
    return y
