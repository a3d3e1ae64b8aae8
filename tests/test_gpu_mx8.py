"""Products of 8-bit x with 4-bit shards against the decoded operands in 64 bits, and
the layer's operators one after another.

The products of e4m3 and e2m1 values are exact; y differs from their sum by fp32
additions: at most D + 8, each within 2^-24 of the sum of magnitudes and twice that
where the tensor core truncates, and one rounding of y.  With small integers all of
it is exact.
"""
import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import mx4, mx8, norm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def no_expired_wait():
    yield
    assert B.dp_get_device_error() == B.DP_OK


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g) * scale


def check(y, x, shards):
    """y against the 64-bit product of the values x and the shards stand for (on the GPU)."""
    w = torch.cat([mx4.dequantize(q, torch.float32) for q in shards]).double()
    v = mx8.dequantize(x, torch.float32).double()
    want, size = v @ w.t(), v.abs() @ w.abs().t()
    tol = 2 * (x.cols + 8) * U * size
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert y.shape == want.shape
    assert bool(((y.double() - want).abs() <= tol + 2.0 ** -140).all())


SHAPES = [  # M, D, K, F_shard
    (1, 32, 1, 16), (1, 64, 1, 48), (3, 96, 2, 16), (16, 128, 1, 128), (17, 160, 1, 144),
    (31, 544, 4, 64), (33, 256, 1, 256), (64, 288, 2, 272), (65, 1024, 1, 128), (100, 672, 8, 64),
    (128, 512, 8, 64), (129, 416, 3, 80), (200, 1120, 2, 208), (257, 1056, 4, 208), (1, 4096, 8, 512),
    (300, 8192, 1, 64), (1000, 736, 2, 1040), (2049, 512, 2, 640), (4100, 320, 1, 4096)]


@pytest.mark.parametrize("M,D,K,Fs", SHAPES)
def test_product(M, D, K, Fs):
    w = normal((K * Fs, D), M + D, 0.02)
    x = (normal((M, D), M * D) * torch.exp(2 * normal((M, 1), 3))).bfloat16()
    s = [mx4.quantize(c.contiguous(), "mxfp4") for c in w.chunk(K)]
    q = mx8.quantize(x)
    a, b = mx8.matmul(q, s, torch.float32), mx8.matmul(q, s)
    check(a, q, s)
    check(b, q, s)
    assert torch.equal(mx8.linear(x, s, torch.float32), a) and torch.equal(mx8.linear(x, s), b)
    assert torch.equal(mx8.linear(x.float(), s), b)


@pytest.mark.parametrize("M,D,K,Fs", [(5, 64, 1, 16), (130, 416, 2, 144), (300, 1024, 2, 640),
                                      (70, 2048, 1, 32)])
def test_integers_are_exact(M, D, K, Fs):
    rng = np.random.default_rng(D)
    vals = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    w = rng.choice(vals, (K * Fs, D)) * rng.choice([-1, 1], (K * Fs, D))
    x = rng.integers(-15, 16, (M, D))
    scale = 2.0 ** rng.integers(-3, 4, (1, D // 32)).repeat(32, 1)      # blocks of different scales
    to = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    s = [mx4.quantize(c.contiguous(), "mxfp4") for c in to(w / scale).chunk(K)]
    y = mx8.linear(to(x * scale), s, torch.float32)
    w4 = np.concatenate([mx4.dequantize(q, torch.float32).double().cpu().numpy() for q in s])
    assert np.array_equal(y.double().cpu().numpy(), (x * scale) @ w4.T)


def test_each_block_of_d_counts_once():
    """One nonzero value of x, one of w: y is their product wherever they lie."""
    D, F = 416, 48
    w = torch.zeros(F, D, device=DEV)
    at = torch.arange(D, device=DEV)
    w[at % F, at] = 2.0 ** (at % 7 - 3).float()
    x = torch.zeros(D, D, device=DEV)
    x[at, at] = 1.0 + (at % 8).float() / 8
    y = mx8.linear(x, [mx4.quantize(w, "mxfp4")], torch.float32)
    assert torch.equal(y, x @ mx4.dequantize(mx4.quantize(w, "mxfp4"), torch.float32).t())


def test_not_finite():
    w = normal((96, 320), 1)
    x = normal((140, 320), 2)
    s = [mx4.quantize(w, "mxfp4")]
    clean = mx8.linear(x, s)
    x[7, 100] = float("nan")
    x[133, 319] = float("inf")
    y = mx8.linear(x, s)
    assert y[7].isnan().all() and y[133].isnan().all()
    keep = [i for i in range(140) if i not in (7, 133)]
    assert torch.equal(y[keep], clean[keep])
    w[5, 0] = float("nan")
    y = mx8.linear(normal((140, 320), 2), [mx4.quantize(w, "mxfp4")])
    assert y[:, 5].isnan().all() and y[:, 6:].isfinite().all() and y[:, :5].isfinite().all()


def test_empty():
    s = [mx4.quantize(normal((32, 64), 1), "mxfp4")]
    assert mx8.linear(torch.zeros(0, 64, device=DEV), s).shape == (0, 32)
    z = [mx4.quantize(torch.zeros(16, 0, device=DEV), "mxfp4")]
    y = mx8.linear(torch.zeros(3, 0, device=DEV), z)
    assert y.shape == (3, 16) and (y == 0).all()


def test_same_bits_under_any_cta_limit():
    saved = B.dp_get_cta_limits()
    for M, D, F in ((700, 512, 640), (16, 4096, 128)):
        s = [mx4.quantize(normal((F, D), 1), "mxfp4")]
        x = normal((M, D), 2)
        want = mx8.linear(x, s)
        try:
            for limit in (1, 5, 40):
                B.dp_set_cta_limits(limit, limit)
                assert torch.equal(mx8.linear(x, s), want)
        finally:
            B.dp_set_cta_limits(*saved)


def test_nothing_else_is_written_and_streams_and_graphs():
    M, D, F = 137, 544, 208
    s = [mx4.quantize(c.contiguous(), "mxfp4") for c in normal((2 * F, D), 1).chunk(2)]
    x = normal((M, D), 2).bfloat16()
    want = mx8.linear(x, s)
    torch.cuda.synchronize()
    need = B.dp_allgather_linear_mx8_workspace_size(M, D)
    y = torch.full((M * 2 * F * 2 + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    B.dp_allgather_linear_mx8(x, M, D, D, B.DP_BF16, [q._c for q in s], 2, F, y.data_ptr() + 256,
                              B.DP_BF16, ws.data_ptr() + 256, need)
    for b in (y, ws):
        assert (b[:256] == 0xA5).all() and (b[-256:] == 0xA5).all()
    assert torch.equal(y[256:-256].view(torch.bfloat16).view(M, 2 * F), want)
    side = torch.cuda.Stream()
    got, other = mx8.linear(x, s, stream=side), mx8.linear(x, s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx8.linear(x, s)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mx8.linear(x, s))


@pytest.mark.parametrize("M,D,H", [(1, 64, 128), (130, 192, 512), (300, 1024, 256)])
def test_a_layer_with_its_gradient(M, D, H):
    """residual + norm -> 8-bit product -> few-token product of the same weights; then back:
    4-bit transposed product, norm's backward.  Each against 64 bits on what the one before
    left, with and without waits between the calls."""
    def run(wait):
        x, res = normal((M, D), 1).bfloat16(), normal((M, D), 2).bfloat16()
        nw = (1 + 0.1 * normal(D, 3)).bfloat16()
        shards = [c.contiguous() for c in normal((H, D), 4, D ** -0.5).bfloat16().chunk(4)]
        w4 = [mx4.quantize(c, "mxfp4") for c in shards]
        w4_t = mx4.quantize(shards, "mxfp4", transpose=True)
        wait()
        n = norm.rms_norm(x, nw, residual=res, format="mxfp8", keep=True)
        wait()
        y = mx8.matmul(n.q, w4)
        wait()
        few = mx4.linear_w4(n.y, w4)
        wait()
        dn = mx8.linear(y, [w4_t])
        wait()
        dx, dw = norm.rms_norm_backward(dn, n.h, nw, n.rstd, dh=x)
        wait()
        return x, n, w4, w4_t, y, few, dn, dx, dw, nw

    a, b = run(torch.cuda.synchronize), run(lambda: None)
    torch.cuda.synchronize()
    for i in (4, 5, 6, 7, 8):
        assert torch.equal(a[i], b[i])
    x, n, w4, w4_t, y, few, dn, dx, dw, nw = b
    check(y, n.q, w4)
    w64 = torch.cat([mx4.dequantize(q, torch.float32) for q in w4]).double()
    y64 = n.y.double()
    want, size = y64 @ w64.t(), y64.abs() @ w64.abs().t()
    assert bool(((few.double() - want).abs() <= 2.02 * (D + 8) * U * size +
                 2.0 ** -8 * want.abs()).all())
    check(dn, mx8.quantize(y), [w4_t])
    xh = n.h.double() * n.rstd.double()[:, None]
    g = dn.double() * nw.double()
    c = (g * xh).mean(1, keepdim=True)
    want = n.rstd.double()[:, None] * (g - xh * c) + x.double()
    big = n.rstd.double()[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= 40 * U * (big + x.double().abs()) +
                 2.0 ** -8 * 1.01 * want.abs()).all())
    size = (dn.double() * xh).abs().sum(0)
    assert bool(((dw.double() - (dn.double() * xh).sum(0)).abs() <= (M + 24) * U * size).all())
