"""Refusals of the norm and of the 8-bit form, all made on the host before any
device call; and the backward formula against differences, in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import build as cuda_build
from ring_allreduce_gradient_gb300 import mx4, mx8, norm

BASE = 0x7F0000000000
OK, INVALID, UNSUPPORTED, ALIAS = (B.DP_OK, B.DP_ERR_INVALID_ARG, B.DP_ERR_UNSUPPORTED,
                                   B.DP_ERR_ALIAS)
PLAIN, MX4, NV4, MX8 = B.DP_NORM_PLAIN, B.DP_NORM_MXFP4, B.DP_NORM_NVFP4, B.DP_NORM_MXFP8


def fake(i, off=0):
    return BASE + (i << 26) + off


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return B.load()


def fwd(x=fake(0), ldx=64, r=None, ldr=0, M=64, D=64, dt=B.DP_BF16, w=fake(1), wdt=B.DP_BF16,
        eps=1e-6, h=None, y=fake(2), rstd=fake(3), fmt=PLAIN, ts=None, codes=None, scales=None):
    return B.dp_rms_norm(x, ldx, r, ldr, M, D, dt, w, wdt, eps, h, y, rstd, fmt, ts, codes, scales,
                         stream=0, check=False)


def test_norm_checks():
    q = dict(fmt=MX8, codes=fake(5), scales=fake(6))
    assert fwd(M=-1) == INVALID and fwd(D=-1) == INVALID and fwd(ldx=63) == INVALID
    assert fwd(x=None) == INVALID and fwd(w=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(eps=float("inf")) == INVALID
    assert fwd(dt=3) == UNSUPPORTED and fwd(wdt=9) == UNSUPPORTED
    assert fwd(fmt=4) == UNSUPPORTED and fwd(fmt=-1) == UNSUPPORTED
    assert fwd(D=32769, ldx=32769) == UNSUPPORTED
    assert fwd(M=0x7fff0001) == UNSUPPORTED
    assert fwd(x=fake(0, 1)) == UNSUPPORTED and fwd(w=fake(1, 1)) == UNSUPPORTED
    assert fwd(rstd=fake(3, 2)) == UNSUPPORTED
    assert fwd(r=fake(4), ldr=64) == INVALID                       # a residual without h
    assert fwd(h=fake(4)) == INVALID                               # h without a residual
    assert fwd(r=fake(4), ldr=63, h=fake(7)) == INVALID
    assert fwd(codes=fake(5)) == INVALID                           # codes without a format
    assert fwd(fmt=MX8, codes=fake(5)) == INVALID and fwd(fmt=MX8, scales=fake(6)) == INVALID
    assert fwd(D=48, ldx=48, **q) == UNSUPPORTED                   # no whole blocks
    assert fwd(**{**q, "codes": fake(5, 8)}) == UNSUPPORTED
    assert fwd(**{**q, "scales": fake(6, 4)}) == UNSUPPORTED
    assert fwd(ts=fake(8), **q) == INVALID and fwd(ts=fake(8)) == INVALID
    assert fwd(fmt=NV4, codes=fake(5), scales=fake(6), ts=fake(8, 2)) == UNSUPPORTED
    assert fwd(y=fake(0)) == ALIAS and fwd(y=fake(0, 64 * 64 * 2 - 2)) == ALIAS
    assert fwd(y=fake(1, 2)) == ALIAS and fwd(rstd=fake(2, 64)) == ALIAS
    assert fwd(r=fake(4), ldr=64, h=fake(4)) == ALIAS              # not in place
    assert fwd(r=fake(4), ldr=64, h=fake(2)) == ALIAS
    assert fwd(**{**q, "codes": fake(2, 16)}) == ALIAS
    assert fwd(**{**q, "scales": fake(5, 64 * 64 - 16)}) == ALIAS  # 8 bits: 64 x 64 bytes of codes
    assert fwd(fmt=NV4, codes=fake(5), scales=fake(6), ts=fake(6, 4)) == ALIAS
    assert fwd(M=0, y=None, x=None) == OK and fwd(D=0, ldx=0, y=None) == OK


def test_backward_checks(lib):
    need = B.dp_rms_norm_backward_workspace_size(64, 64)
    assert need == 8 * 64 * 4                      # sets of eight rows
    assert B.dp_rms_norm_backward_workspace_size(100000, 4096) == 304 * 4096 * 4
    assert B.dp_rms_norm_backward_workspace_size(100000, 8192) == 152 * 8192 * 4
    assert B.dp_rms_norm_backward_workspace_size(0, 64) == 0

    def bwd(dy=fake(0), ldy=64, h=fake(1), ldh=64, dh=None, ldd=0, M=64, D=64, dt=B.DP_BF16,
            w=fake(2), wdt=B.DP_FP32, rstd=fake(3), dx=fake(4), dw=fake(5), ws=fake(6), wb=need):
        return B.dp_rms_norm_backward(dy, ldy, h, ldh, dh, ldd, M, D, dt, w, wdt, rstd, dx, dw, ws,
                                      wb, stream=0, check=False)

    assert bwd(M=-1) == INVALID and bwd(ldy=63) == INVALID and bwd(ldh=1) == INVALID
    assert bwd(dh=fake(7), ldd=63) == INVALID
    for name in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert bwd(**{name: None}) == INVALID
    assert bwd(wb=need - 1) == INVALID
    assert bwd(dt=7) == UNSUPPORTED and bwd(wdt=2) == UNSUPPORTED
    assert bwd(D=32800, ldy=32800, ldh=32800) == UNSUPPORTED
    assert bwd(dy=fake(0, 1)) == UNSUPPORTED and bwd(ws=fake(6, 16)) == UNSUPPORTED
    assert bwd(dw=fake(5, 2)) == UNSUPPORTED
    assert bwd(dx=fake(0)) == ALIAS and bwd(dx=fake(1, 64)) == ALIAS
    assert bwd(dw=fake(4, 64)) == ALIAS and bwd(ws=fake(4, 64)) == ALIAS
    assert bwd(dh=fake(4), ldd=64) == ALIAS and bwd(ws=fake(3)) == ALIAS
    assert bwd(D=0, ldy=0, ldh=0) == OK
    n = ctypes.c_size_t(3)
    assert lib.dp_rms_norm_backward_workspace_size(1, 1, None) == INVALID
    assert lib.dp_rms_norm_backward_workspace_size(-1, 1, ctypes.byref(n)) == INVALID
    assert n.value == 0
    assert lib.dp_rms_norm_backward_workspace_size(1, 32769, ctypes.byref(n)) == UNSUPPORTED


def test_eight_bit_checks():
    def q(x=fake(0), rows=64, cols=64, ld=64, dt=B.DP_BF16, codes=fake(4), scales=fake(5)):
        return B.dp_mx8_quantize(x, rows, cols, ld, dt, codes, scales, stream=0, check=False)

    assert q(rows=-1) == INVALID and q(ld=63) == INVALID and q(x=None) == INVALID
    assert q(codes=None) == INVALID and q(scales=None) == INVALID
    assert q(dt=4) == UNSUPPORTED and q(cols=48) == UNSUPPORTED
    assert q(cols=0x7fff0020, ld=0x7fff0020, rows=1) == UNSUPPORTED
    assert q(x=fake(0, 1)) == UNSUPPORTED and q(codes=fake(4, 8)) == UNSUPPORTED
    assert q(codes=fake(0, 64 * 64)) == ALIAS and q(scales=fake(4, 64 * 64 - 16)) == ALIAS
    assert q(rows=0, codes=None, scales=None) == OK

    def d(codes=fake(0), scales=fake(1), rows=64, cols=64, out=fake(2), dt=B.DP_BF16):
        return B.dp_mx8_dequantize(codes, scales, rows, cols, out, dt, stream=0, check=False)

    assert d(rows=-1) == INVALID and d(codes=None) == INVALID and d(out=None) == INVALID
    assert d(dt=9) == UNSUPPORTED and d(cols=40) == UNSUPPORTED
    assert d(out=fake(2, 8)) == UNSUPPORTED
    assert d(out=fake(0, 16)) == ALIAS and d(out=fake(1, 16)) == ALIAS
    assert d(cols=0, codes=None) == OK


def test_the_helpers_check():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    r = torch.zeros(4)
    for args, kw, err, word in [
            ((x, w), dict(format="int8"), ValueError, "format"),
            ((x, w[:63]), {}, ValueError, "weight: 64"),
            ((x, torch.ones(128)[::2]), {}, ValueError, "weight"),
            ((x, w.half()), {}, TypeError, "dtype"),
            ((x.half(), w), {}, TypeError, "dtype"),
            ((x, w), dict(residual=x[:3]), ValueError, "residual"),
            ((x, w), dict(residual=x.float()), ValueError, "residual"),
            ((x, w), dict(tensor_scale=torch.ones(1)), ValueError, "nvfp4"),
            ((x, w), dict(tensor_scale=torch.ones(2), format="nvfp4"), ValueError, "tensor_scale"),
            ((x[0], w), {}, ValueError, "need a matrix"),
            ((x.t(), torch.ones(4)), {}, ValueError, "unit stride"),
            ((x, w), {}, B.DpError, "not the current CUDA device")]:
        with pytest.raises(err, match=word):
            norm.rms_norm(*args, **kw)
    for args, kw, err, word in [
            ((x[:3], x, w, r), {}, ValueError, "dy"),
            ((x, x, w, r[:3]), {}, ValueError, "rstd"),
            ((x, x, w, r.double()), {}, ValueError, "rstd"),
            ((x, x, w, r), dict(dh=x.float()), ValueError, "dh"),
            ((x, x, w, r), {}, B.DpError, "not the current CUDA device")]:
        with pytest.raises(err, match=word):
            norm.rms_norm_backward(*args, **kw)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    q = mx8.Mx8Tensor(u8(2 * 32), u8(512), 2, 32)
    assert q.format == "mxfp8" and q.rows == 2 and q.cols == 32
    with pytest.raises(AttributeError):
        q.codes = u8(64)
    with pytest.raises(ValueError, match="codes"):
        mx8.Mx8Tensor(u8(63), u8(512), 2, 32)
    with pytest.raises(ValueError, match="scales"):
        mx8.Mx8Tensor(u8(64), u8(511), 2, 32)
    with pytest.raises(TypeError, match="dtype"):
        mx8.dequantize(q, torch.float16)
    with pytest.raises(TypeError, match="dtype"):
        mx8.quantize(x.half())
    with pytest.raises(ValueError, match="unit stride"):
        mx8.quantize(x.t())
    for call in (lambda: mx8.quantize(x), lambda: mx8.dequantize(q)):
        with pytest.raises(B.DpError, match="not the current CUDA device"):
            call()
    assert mx4._scale_bytes(2, 32, "mxfp4") == 512


def test_the_backward_formula_is_the_derivative():
    """The formula that the GPU tests hold the kernel to, against central differences:
    their error is step^2 / 6 times a third derivative of order 1, and 1e-16 / step."""
    rng = np.random.default_rng(0)
    M, D, eps = 3, 10, 1e-3
    h, dy, dh = rng.standard_normal((3, M, D))
    w = rng.standard_normal(D)

    def loss(h, w):
        r = 1 / np.sqrt((h * h).mean(1) + eps)
        return (dy * h * r[:, None] * w).sum() + (dh * h).sum()

    r = 1 / np.sqrt((h * h).mean(1) + eps)[:, None]
    g, xh = dy * w, h * r
    dx = r * (g - xh * (g * xh).mean(1, keepdims=True)) + dh
    dw = (dy * xh).sum(0)
    step = 1e-5
    for i in range(M):
        for j in range(D):
            a, b = h.copy(), h.copy()
            a[i, j] += step
            b[i, j] -= step
            assert abs((loss(a, w) - loss(b, w)) / (2 * step) - dx[i, j]) < 1e-7
    for j in range(D):
        a, b = w.copy(), w.copy()
        a[j] += step
        b[j] -= step
        assert abs((loss(h, a) - loss(h, b)) / (2 * step) - dw[j]) < 1e-7
