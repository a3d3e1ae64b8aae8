"""Refusals of the 4-bit calls: every one is made on the host before any device
call, so none of them needs a GPU."""
import ctypes

import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import build as cuda_build
from ring_allreduce_gradient_gb300 import mx4

BASE = 0x7F0000000000
OK, INVALID, UNSUPPORTED, ALIAS = (B.DP_OK, B.DP_ERR_INVALID_ARG, B.DP_ERR_UNSUPPORTED,
                                   B.DP_ERR_ALIAS)
MX, NV = B.DP_MXFP4, B.DP_NVFP4


def fake(i, off=0):
    return BASE + (i << 26) + off


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return B.load()


def test_scales_size(lib):
    assert B.dp_mx4_scales_size(0, 64, MX) == 0
    assert B.dp_mx4_scales_size(1, 32, MX) == 512          # one tile
    assert B.dp_mx4_scales_size(128, 128, MX) == 512
    assert B.dp_mx4_scales_size(129, 160, MX) == 4 * 512
    assert B.dp_mx4_scales_size(128, 128, NV) == 2 * 512
    for r in (0, 1, 127, 300):
        for c in (0, 32, 96, 4096):
            for name, f in mx4.FORMATS.items():
                assert B.dp_mx4_scales_size(r, c, f) == mx4._scale_bytes(r, c, name)
    n = ctypes.c_size_t(3)
    assert lib.dp_mx4_scales_size(1, 32, MX, None) == INVALID
    assert lib.dp_mx4_scales_size(-1, 32, MX, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.dp_mx4_scales_size(1, 32, 5, ctypes.byref(n)) == UNSUPPORTED


def test_quantize_checks():
    def q(x=(fake(0),), K=1, rows=64, cols=64, ld=64, dt=B.DP_BF16, fmt=MX, tr=0, ts=None,
          codes=fake(4), scales=fake(5)):
        return B.dp_mx4_quantize(list(x), K, rows, cols, ld, dt, fmt, tr, ts, codes, scales,
                                 stream=0, check=False)

    assert q(K=0) == INVALID and q(K=17) == INVALID
    assert q(rows=-1) == INVALID and q(cols=-32) == INVALID
    assert q(ld=63) == INVALID
    assert q(x=(None,)) == INVALID
    assert q(codes=None) == INVALID and q(scales=None) == INVALID
    assert q(dt=4) == UNSUPPORTED and q(fmt=2) == UNSUPPORTED
    assert q(ts=fake(6)) == INVALID                        # mxfp4 has no tensor scale
    assert q(fmt=NV, ts=fake(6, 2)) == UNSUPPORTED
    assert q(cols=48) == UNSUPPORTED                       # not whole blocks for the tensor core
    assert q(rows=48, tr=1) == UNSUPPORTED
    assert q(rows=16, K=3, x=(fake(0), fake(1), fake(2)), tr=1) == UNSUPPORTED
    assert q(x=(fake(0, 1),)) == UNSUPPORTED
    assert q(codes=fake(4, 8)) == UNSUPPORTED and q(scales=fake(5, 4)) == UNSUPPORTED
    assert q(codes=fake(0, 64 * 64)) == ALIAS              # inside x
    assert q(codes=fake(0, 64 * 64 * 2 - 16)) == ALIAS
    assert q(scales=fake(4, 64 * 32 - 16)) == ALIAS        # inside the codes
    assert q(fmt=NV, ts=fake(4, 4)) == ALIAS
    assert q(rows=0, codes=None, scales=None) == OK        # nothing to do
    assert q(cols=0, ld=0, codes=None, scales=None) == OK


def test_dequantize_checks():
    def d(codes=fake(0), scales=fake(1), rows=64, cols=64, fmt=MX, ts=None, out=fake(2),
          dt=B.DP_BF16):
        return B.dp_mx4_dequantize(codes, scales, rows, cols, fmt, ts, out, dt, stream=0,
                                   check=False)

    assert d(rows=-1) == INVALID and d(codes=None) == INVALID and d(out=None) == INVALID
    assert d(fmt=3) == UNSUPPORTED and d(dt=9) == UNSUPPORTED
    assert d(ts=fake(3)) == INVALID
    assert d(cols=40) == UNSUPPORTED
    assert d(out=fake(2, 8)) == UNSUPPORTED
    assert d(out=fake(0, 1024)) == ALIAS and d(out=fake(1)) == ALIAS
    assert d(rows=0, codes=None, out=None) == OK


def test_tensor_scale_checks():
    need = B.dp_grad_norm_workspace_size(1)

    def t(x=(fake(0),), n=(100,), dt=B.DP_FP32, out=fake(1), ws=fake(2), wb=need):
        return B.dp_mx4_tensor_scale(list(x), list(n), len(x), dt, out, ws, wb, stream=0,
                                     check=False)

    assert t(out=None) == INVALID and t(ws=None) == INVALID and t(wb=need - 1) == INVALID
    assert t(x=(None,)) == INVALID
    assert t(dt=3) == UNSUPPORTED and t(x=(fake(0, 2),)) == UNSUPPORTED
    assert t(out=fake(0, 4)) == ALIAS


def test_product_checks():
    ws = [(fake(2 * k + 2), fake(2 * k + 3), None) for k in range(2)]

    def m(x=(fake(0), fake(1), None), M=64, D=64, w=ws, K=2, Fs=32, fmt=MX, y=fake(20),
          dt=B.DP_BF16):
        return B.dp_allgather_matmul_mx4(x, M, D, w, K, Fs, fmt, y, dt, stream=0, check=False)

    assert m(K=0) == INVALID and m(K=17) == INVALID
    assert m(M=-1) == INVALID and m(D=-32) == INVALID and m(Fs=-16) == INVALID
    assert m(x=(None, fake(1), None)) == INVALID and m(x=(fake(0), None, None)) == INVALID
    assert m(w=[ws[0], (fake(4), None, None)]) == INVALID
    assert m(y=None) == INVALID
    assert m(x=(fake(0), fake(1), fake(9))) == INVALID     # a tensor scale with mxfp4
    assert m(fmt=7) == UNSUPPORTED and m(dt=5) == UNSUPPORTED
    assert m(D=48) == UNSUPPORTED and m(Fs=24) == UNSUPPORTED
    assert m(x=(fake(0, 8), fake(1), None)) == UNSUPPORTED
    assert m(y=fake(20, 4)) == UNSUPPORTED
    assert m(fmt=NV, x=(fake(0), fake(1), fake(9, 2))) == UNSUPPORTED
    assert m(y=fake(0)) == ALIAS and m(y=fake(3)) == ALIAS
    assert m(y=fake(4, 512)) == ALIAS
    assert m(fmt=NV, x=(fake(0), fake(1), fake(20, 64))) == ALIAS
    assert m(M=0, y=None) == OK and m(Fs=0, y=None) == OK


def test_linear_checks(lib):
    ws = [(fake(2 * k + 2), fake(2 * k + 3), None) for k in range(2)]
    need = B.dp_allgather_linear_mx4_workspace_size(64, 64, MX)
    assert need == 64 * 32 + 512

    def m(x=fake(0), M=64, D=64, ld=64, xdt=B.DP_BF16, xs=None, w=ws, Fs=32, fmt=MX, y=fake(20),
          dt=B.DP_BF16, work=fake(30), wb=need):
        return B.dp_allgather_linear_mx4(x, M, D, ld, xdt, xs, w, 2, Fs, fmt, y, dt, work, wb,
                                         stream=0, check=False)

    assert m(work=None) == INVALID and m(wb=need - 1) == INVALID
    assert m(work=fake(30, 8)) == UNSUPPORTED
    assert m(M=-1) == INVALID
    assert m(fmt=4) == UNSUPPORTED
    assert m(D=48, ld=48) == UNSUPPORTED
    assert m(xs=fake(31)) == INVALID
    assert m(work=fake(20)) == ALIAS                       # the scratch and y
    assert m(work=fake(2)) == ALIAS                        # the scratch and a weight shard
    assert m(work=fake(3)) == ALIAS
    assert m(y=fake(0, 64)) == ALIAS                       # y and x
    n = ctypes.c_size_t(3)
    assert lib.dp_allgather_linear_mx4_workspace_size(1, 32, MX, None) == INVALID
    assert lib.dp_allgather_linear_mx4_workspace_size(-1, 32, MX, ctypes.byref(n)) == INVALID


def test_the_tensor_helpers_check():
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    q = mx4.Mx4Tensor(u8(2 * 16), u8(512), 2, 32, "mxfp4")
    with pytest.raises(AttributeError):
        q.codes = u8(32)                                   # read-only: its address is kept
    with pytest.raises(ValueError, match="format"):
        mx4.Mx4Tensor(u8(32), u8(512), 2, 32, "fp4")
    with pytest.raises(ValueError, match="codes"):
        mx4.Mx4Tensor(u8(31), u8(512), 2, 32, "mxfp4")
    with pytest.raises(ValueError, match="scales"):
        mx4.Mx4Tensor(u8(2 * 64), u8(512), 2, 128, "nvfp4")
    with pytest.raises(ValueError, match="tensor_scale"):
        mx4.Mx4Tensor(u8(32), u8(512), 2, 32, "nvfp4", torch.zeros(2))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="format"):
        mx4.quantize(x, "int4")
    with pytest.raises(ValueError, match="unit stride"):
        mx4.quantize(x.t())
    with pytest.raises(ValueError, match="shards"):
        mx4.quantize([x, x[:2]])
    with pytest.raises(ValueError, match="at least one"):
        mx4.quantize([])
    with pytest.raises(TypeError, match="dtype"):
        mx4.quantize(x.half())
    with pytest.raises(B.DpError, match="UNSUPPORTED"):
        mx4.quantize(x[:, :48])
    with pytest.raises(ValueError, match="tensor_scale"):
        mx4.quantize(x, "nvfp4", tensor_scale=torch.zeros(3))
    with pytest.raises(TypeError, match="dtype"):
        mx4.dequantize(q, torch.float16)
    other = mx4.Mx4Tensor(u8(2 * 32), u8(512), 2, 64, "mxfp4")
    with pytest.raises(ValueError, match="columns"):
        mx4.matmul(q, [other])
    with pytest.raises(ValueError, match="one shape"):
        mx4.matmul(other, [other, mx4.Mx4Tensor(u8(32), u8(512), 1, 64, "mxfp4")])
    with pytest.raises(TypeError, match="dtype"):
        mx4.matmul(q, [q], torch.float16)
    with pytest.raises(ValueError, match="columns"):
        mx4.linear(x, [q])
    with pytest.raises(ValueError, match="contiguous tensors"):
        mx4.tensor_scale([])


def test_a_product_needs_a_shard():
    with pytest.raises(ValueError, match="at least one shard"):
        mx4.linear(torch.zeros(4, 64), [])


@pytest.mark.parametrize("cols", [0x7fff0020, 0x7fffff00])
def test_rows_too_long_to_index(cols):
    def q(tr, rows, n):
        return B.dp_mx4_quantize([fake(0)], 1, rows, n, n, B.DP_BF16, MX, tr, None, fake(4),
                                 fake(5), stream=0, check=False)

    assert q(0, 1, cols) == UNSUPPORTED and q(1, 32, cols) == UNSUPPORTED
    assert q(0, cols, 32) == UNSUPPORTED
    assert B.dp_mx4_dequantize(fake(0), fake(1), 1, cols, MX, None, fake(2), B.DP_BF16, stream=0,
                               check=False) == UNSUPPORTED


def views():
    """Matrices whose rows overlap, are expanded from one, or lie apart, and single rows."""
    base = torch.arange(4096, dtype=torch.float32)
    return [base[:64].expand(128, 64), base[64:128].view(1, 64).expand(3, 64),
            base[100:].as_strided((4, 64), (16, 1), 100), base.unfold(0, 96, 32),
            base[:1].expand(32, 1), base.view(64, 64)[:, :32], base.view(32, 128)[3:9, 5:37],
            base[:64].view(1, 64), base.view(64, 64)[:1, :32], base.view(128, 32)[:, :1],
            base.view(64, 64)[:0]]


@pytest.mark.parametrize("i", range(len(views())))
def test_rows_that_the_library_gets_are_the_views(i):
    """Row r at r * ld of the buffer that is handed on, inside its storage, ld a row or more."""
    x = views()[i]
    t, ld = mx4._rows(x)
    rows, cols = x.shape
    assert ld >= cols
    if rows:
        assert (rows - 1) * ld + cols <= t.untyped_storage().nbytes() // 4 - t.storage_offset()
        assert torch.equal(t.as_strided((rows, cols), (ld, 1)), x)


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """Host memory, or another GPU's: the library is not called at all."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = mx4.Mx4Tensor(torch.zeros(4 * 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                      4, 64, "mxfp4")
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or (b"" if name.endswith("_string") else 0)

    monkeypatch.setattr(B, "_lib", Library())
    for with_gpu in (False, True):
        if with_gpu:      # as on a machine whose current device is cuda:0
            monkeypatch.setattr(B, "_raw_stream", lambda d: 0)
            monkeypatch.setattr(B, "_current_device", lambda: 0)
        for call in (lambda: mx4.quantize(x), lambda: mx4.quantize([x, x]),
                     lambda: mx4.dequantize(q), lambda: mx4.matmul(q, [q]),
                     lambda: mx4.linear(x, [q]), lambda: mx4.tensor_scale(x)):
            with pytest.raises(B.DpError, match="tensors on cpu, which is not the current"):
                call()
    assert B._stream_on(torch.device("cuda", 0), "here") == 0
    with pytest.raises(B.DpError, match="cuda:1"):
        B._stream_on(torch.device("cuda", 1), "here")
    assert [c for c in calls if not c.endswith(("_size", "_string"))] == []


@pytest.mark.parametrize("shape", [(64,), (2, 4, 64), (1, 1, 2, 64)])
def test_what_is_no_matrix_is_named(shape):
    x = torch.zeros(shape, dtype=torch.bfloat16)
    q = mx4.Mx4Tensor(torch.zeros(4 * 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                      4, 64, "mxfp4")
    for call in (lambda: mx4.linear(x, [q]), lambda: mx4.quantize(x), lambda: mx4.quantize([x])):
        with pytest.raises(ValueError, match=r"need a matrix, got \(.*\): flatten"):
            call()
