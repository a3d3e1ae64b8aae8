"""Microscaled 4-bit matrices against a plain implementation in 64 bits.

Quantisation is a rounding: every decoded value is the nearest one that its
block's scale offers, up to a tie that the fp32 quotient x / (s t) or the fp32
scale a / 6 / t may round to either side: values and scales within 4u (u =
2^-24) of such a tie may go either way, all others are equal.  mxfp4 divides by
powers of two, so it is equal everywhere.

Products: with small integers every product and sum is exact in fp32, so y
equals the integer result (rounded once to bf16).  With general values the
fp32 sums of D exact products are within D u of the sum of magnitudes, and one
rounding of y follows.
"""
import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import mx4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24
BLOCK = {"mxfp4": 32, "nvfp4": 16}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def nearest(x, grid):
    """Nearest of an ascending grid, ties to the even index, saturating; and how near to a tie."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")
    tie = (i < mid.size) & (np.take(mid, np.minimum(i, mid.size - 1)) == x)
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    near = np.abs(x[..., None] - mid).min(-1) / np.maximum(x, 1e-300) if x.size else x
    return i, near


def oracle(x, fmt, t=1.0):
    """(scale bytes, block steps, values, doubtful) of fp64 x [R, L]."""
    R, L = x.shape
    b = x.reshape(R, L // BLOCK[fmt], BLOCK[fmt])
    top = np.abs(b).max(2)
    if fmt == "mxfp4":
        e = np.where(top > 0, np.frexp(top)[1] - 3, -127).clip(-127, 127)
        byte, step, near = e + 127, np.exp2(e.astype(float)), np.ones_like(top)
    else:
        byte, near = nearest(top / 6 / t, E4M3)
        step = E4M3[byte] * t
    q = np.abs(b) / np.where(step > 0, step, 1)[..., None]
    i, near_q = nearest(q, GRID)
    vals = np.where(step[..., None] > 0, np.sign(b) * GRID[i] * step[..., None], 0)
    doubt = (near < 4 * U)[..., None] | (near_q < 4 * U) if fmt == "nvfp4" else np.zeros(b.shape, bool)
    return byte, step, vals.reshape(R, L), np.broadcast_to(doubt, b.shape).reshape(R, L)


def linear_scales(q):
    """Scale bytes [rows, blocks] out of their tiles, and whether the rest is zero."""
    nb = q.cols // BLOCK[q.format]
    Rt, Ct = -(-q.rows // 128), -(-nb // 4)
    full = q.scales.cpu().numpy().reshape(Rt, Ct, 32, 4, 4).transpose(0, 3, 2, 1, 4) \
        .reshape(Rt * 128, Ct * 4)
    rest = full.copy()
    rest[:q.rows, :nb] = 0
    return full[:q.rows, :nb], not rest.any()


def unpack(q):
    c = q.codes.cpu().numpy()
    c = np.stack([c & 15, c >> 4], 2).reshape(q.rows, q.cols)
    return GRID[c & 7] * np.where(c & 8, -1, 1)


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def check(q, x64, fmt, t=1.0):
    byte, step, vals, doubt = oracle(x64, fmt, t)
    got_bytes, padded = linear_scales(q)
    assert padded
    block_doubt = doubt.reshape(*byte.shape, -1).all(2)
    assert np.array_equal(got_bytes[~block_doubt], byte[~block_doubt])
    got = mx4.dequantize(q, torch.float32).double().cpu().numpy()
    sure = ~doubt
    assert np.all(np.abs(got - vals)[sure] <= 2 * U * np.abs(vals)[sure])
    assert doubt.mean() < 0.25
    # what decoding gives is the codes times their scales
    if fmt == "mxfp4":
        st = np.exp2(got_bytes.astype(float) - 127)
    else:
        st = E4M3[np.minimum(got_bytes, 126)] * t
    mine = unpack(q) * np.repeat(st, BLOCK[fmt], 1)
    assert np.all(np.abs(mine - got) <= 2 * U * np.abs(mine))


SHAPES = [(1, 32), (3, 64), (127, 96), (128, 256), (130, 512 + 32), (257, 1056), (2050, 1120),
          (2049, 2080)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(rows, cols, dtype, fmt, transpose):
    rng = np.random.default_rng(rows * 7 + cols)
    a = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-6, 3, (rows, 1)))
    a[rng.random((rows, cols)) < 0.05] = 0
    x = dev(a.T if transpose else a, dtype)
    t = mx4.tensor_scale(x) if fmt == "nvfp4" else None
    x64 = x.double().cpu().numpy()
    x64 = x64.T if transpose else x64
    if t is not None:
        want = np.abs(x64).max() / 2688
        assert abs(float(t) - want) <= 2 * U * want
    q = mx4.quantize(x, fmt, tensor_scale=t, transpose=transpose)
    assert (q.rows, q.cols) == (rows, cols)
    check(q, x64, fmt, float(t) if t is not None else 1.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 3), (2, 5)])
def test_quantize_views_and_shards(fmt, transpose, off, pad):
    """Rows that are not packed, at odd offsets, and a matrix in several shards."""
    rng = np.random.default_rng(3)
    K, rows, cols = 3, 32, 160
    buf = [dev(rng.standard_normal((rows, cols + pad + off)), torch.bfloat16) for _ in range(K)]
    xs = [b[:, off:off + cols] for b in buf]
    q = mx4.quantize(xs, fmt, transpose=transpose)
    whole = torch.cat(xs).contiguous()
    ref = mx4.quantize(whole.t().contiguous() if transpose else whole, fmt)
    assert (q.rows, q.cols) == (ref.rows, ref.cols)
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_every_code_and_tie(fmt):
    """Values on the grid and halfway between, at every sign: ties go to the even code."""
    ties = (GRID[1:] + GRID[:-1]) / 2
    row = np.concatenate([[6.0], GRID, ties, np.nextafter(ties, 9), np.nextafter(ties, 0)])
    row = row.astype(np.float32)
    row = np.concatenate([row, -row])
    B_ = BLOCK[fmt]
    n = -(-row.size // (B_ - 1))
    blocks = np.zeros((n, B_), np.float32)
    blocks[:, 0] = 6.0                        # fixes the scale at 1
    flat = np.zeros(n * (B_ - 1), np.float32)
    flat[:row.size] = row
    blocks[:, 1:] = flat.reshape(n, B_ - 1)
    x = np.zeros((n, 32), np.float32)
    x[:, :B_] = blocks
    q = mx4.quantize(dev(x), fmt)
    i, _ = nearest(np.abs(x.astype(np.float64)), GRID)
    assert np.array_equal(unpack(q), GRID[i] * np.where(np.signbit(x), -1, 1))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("transpose", [False, True])
def test_zeros_extremes_and_non_finite_blocks(fmt, transpose):
    x = np.zeros((8, 64), np.float32)
    x[1, 5] = np.nan
    x[2, 40] = np.inf
    x[3, :] = 1.0
    x[3, 3] = -np.inf
    x[4, 0] = 3.4e38
    x[5, 0] = 1e-40
    x[6, :] = 2.0 ** -126
    q = mx4.quantize(dev(x.T if transpose else x), fmt, transpose=transpose)
    got = mx4.dequantize(q, torch.float32).cpu().numpy()
    b = BLOCK[fmt]
    for r, c in ((1, 5), (2, 40), (3, 3)):
        lo = c // b * b
        assert np.isnan(got[r, lo:lo + b]).all()
        rest = np.delete(got[r], np.s_[lo:lo + b])
        assert np.isfinite(rest).all()
    assert (got[0] == 0).all() and (got[7] == 0).all()
    if fmt == "mxfp4":
        assert got[4, 0] == 1.5 * 2.0 ** 127 and got[6, 0] == 2.0 ** -126
        assert abs(got[5, 0] - 1e-40) <= 2.0 ** -128     # half of 2^-127's smallest step
    else:   # one e4m3 scale alone: above 6 * 448 all saturates, far below all is zero
        assert got[4, 0] == 2688 and got[5, 0] == 0 and got[6, 0] == 0
    t = torch.zeros(1, device=DEV)
    if fmt == "nvfp4":                                    # an all-zero tensor's scale is 0
        z = mx4.quantize(torch.zeros(3, 32, device=DEV), fmt, tensor_scale=t)
        assert not mx4.dequantize(z).any()
        assert torch.isnan(mx4.tensor_scale(dev(x)[1:2])).all()
        assert torch.isinf(mx4.tensor_scale(dev(x)[2:4])).all()


# --- products ------------------------------------------------------------------------

def integers(rng, rows, cols):
    """Values that both formats hold exactly: e2m1 integers with a 6 in each block of 16, which
    makes every block's scale 1."""
    a = rng.choice([-4, -3, -2, -1, 0, 1, 2, 3, 4], (rows, cols)).astype(np.float32)
    a[:, ::16] = 6
    return a


PRODUCTS = [  # M, D, K, F_shard
    (1, 32, 1, 16), (1, 256, 1, 128), (5, 96, 2, 48), (16, 512, 8, 64), (17, 1056, 3, 144),
    (128, 512, 8, 64), (129, 320, 2, 256), (255, 2048, 4, 80), (300, 4096, 1, 128),
    (1, 4096, 8, 512), (700, 288, 8, 512), (2100, 512, 4, 400), (5000, 160, 5, 336),
    (40, 96, 16, 2048), (100, 704, 2, 272), (200, 2048, 1, 512), (64, 1024, 8, 16),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,D,K,Fs", PRODUCTS)
def test_product_of_integers_is_exact(M, D, K, Fs, fmt):
    rng = np.random.default_rng(M + D)
    x, w = integers(rng, M, D), integers(rng, K * Fs, D)
    xq = mx4.quantize(dev(x), fmt)
    assert np.array_equal(mx4.dequantize(xq, torch.float32).cpu().numpy(), x)
    wq = [mx4.quantize(s, fmt) for s in dev(w).chunk(K)]
    want = x.astype(np.float64) @ w.astype(np.float64).T
    y = mx4.matmul(xq, wq, torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), want)
    yb = mx4.matmul(xq, wq)
    assert torch.equal(yb, dev(want.astype(np.float32)).to(torch.bfloat16))
    assert B.dp_get_device_error() == B.DP_OK


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,D,K,Fs", PRODUCTS)
def test_product_of_general_values(M, D, K, Fs, fmt):
    rng = np.random.default_rng(M * 3 + D)
    x = dev(rng.standard_normal((M, D)), torch.bfloat16)
    ws = [dev(rng.standard_normal((Fs, D)) * 0.02 * (k + 1)) for k in range(K)]
    nv = fmt == "nvfp4"
    xq = mx4.quantize(x, fmt, mx4.tensor_scale(x) if nv else None)
    wq = [mx4.quantize(w, fmt, mx4.tensor_scale(w) if nv else None) for w in ws]  # a scale per shard
    x64 = mx4.dequantize(xq, torch.float32).double()
    w64 = torch.cat([mx4.dequantize(w, torch.float32) for w in wq]).double()
    want, size = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    y = mx4.matmul(xq, wq, torch.float32).double()
    assert bool(((y - want).abs() <= (D + 8) * U * size).all())
    yb = mx4.matmul(xq, wq).double()
    assert bool(((yb - want).abs() <= (D + 8) * U * size * 1.01 + 2.0 ** -8 * want.abs()).all())
    assert torch.equal(mx4.linear(x, wq, xq.tensor_scale).double(), yb)
    assert B.dp_get_device_error() == B.DP_OK


def test_scales_of_every_row_and_block_reach_their_own_products():
    """One block nonzero at a time: a misplaced scale or block changes the result."""
    rng = np.random.default_rng(11)
    M, D, Fs = 160, 640, 160
    for fmt in ("mxfp4", "nvfp4"):
        b = BLOCK[fmt]
        x = np.zeros((M, D), np.float32)
        w = np.zeros((Fs, D), np.float32)
        for i in range(M):
            j = (i * 7) % (D // b)
            x[i, j * b:(j + 1) * b] = 6 * 2.0 ** rng.integers(-3, 4)
        for i in range(Fs):
            w[i] = np.repeat(6 * 2.0 ** rng.integers(-3, 4, D // b), b)
        y = mx4.matmul(mx4.quantize(dev(x), fmt), [mx4.quantize(dev(w), fmt)], torch.float32)
        assert np.array_equal(y.double().cpu().numpy(), x.astype(np.float64) @ w.T)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_non_finite_row_stays_in_its_row(fmt):
    rng = np.random.default_rng(2)
    x, w = integers(rng, 40, 256), integers(rng, 64, 256)
    want = x.astype(np.float64) @ w.T
    x[7, 33] = np.nan
    x[9, 200] = np.inf
    y = mx4.matmul(mx4.quantize(dev(x), fmt), [mx4.quantize(dev(w), fmt)], torch.float32)
    y = y.double().cpu().numpy()
    assert np.isnan(y[[7, 9]]).all()
    keep = np.delete(np.arange(40), [7, 9])
    assert np.array_equal(y[keep], want[keep])


def test_cta_limits_streams_and_graphs_give_the_same_bits():
    rng = np.random.default_rng(5)
    for M, D, K, Fs in [(3, 2048, 8, 64), (600, 512, 4, 256)]:
        x = dev(rng.standard_normal((M, D)), torch.bfloat16)
        wq = [mx4.quantize(dev(rng.standard_normal((Fs, D))), "nvfp4") for _ in range(K)]
        y = mx4.linear(x, wq, y_dtype=torch.float32)
        saved = B.dp_get_cta_limits()
        try:
            for lim in (1, 7, 20):
                B.dp_set_cta_limits(lim, lim)
                assert torch.equal(mx4.linear(x, wq, y_dtype=torch.float32), y)
        finally:
            B.dp_set_cta_limits(*saved)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(mx4.linear(x, wq, y_dtype=torch.float32), y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = mx4.linear(x, wq, y_dtype=torch.float32)
            x2 = dev(rng.standard_normal((M, D)), torch.bfloat16)
            x.copy_(x2)
            graph.replay()
            assert torch.equal(out, mx4.linear(x2, wq, y_dtype=torch.float32))
        torch.cuda.current_stream().wait_stream(side)


def test_empty_products():
    w = [mx4.quantize(torch.ones(16, 32, device=DEV))]
    x0 = mx4.quantize(torch.ones(0, 32, device=DEV))
    assert mx4.matmul(x0, w).shape == (0, 16)
    xe = mx4.quantize(torch.ones(3, 0, device=DEV))
    we = [mx4.quantize(torch.ones(16, 0, device=DEV))]
    assert torch.equal(mx4.matmul(xe, we), torch.zeros(3, 16, dtype=torch.bfloat16, device=DEV))
    we = [mx4.quantize(torch.ones(0, 32, device=DEV))]
    assert mx4.matmul(mx4.quantize(torch.ones(3, 32, device=DEV)), we).shape == (3, 0)


def test_backward_products_are_the_gradients_of_the_decoded_forward():
    """dx = dy . w and dw = dy^T . x through transposed operands, gathered from the shards:
    against the formula in 64 bits and against differences of the loss sum(dy * y)."""
    rng = np.random.default_rng(8)
    M, D, K, Fs = 96, 160, 4, 32
    x, dy = integers(rng, M, D), integers(rng, M, K * Fs)
    w = integers(rng, K * Fs, D)
    for a in (x, dy, w):   # a 6 in every block in the other direction too: all values exact
        a[::16] = 6
    wt = mx4.quantize(list(dev(w).chunk(K)), "nvfp4", transpose=True)
    dx = mx4.matmul(mx4.quantize(dev(dy), "nvfp4"), [wt], torch.float32)
    dw = mx4.matmul(mx4.quantize(dev(dy), "nvfp4", transpose=True),
                    [mx4.quantize(dev(x), "nvfp4", transpose=True)], torch.float32)
    assert np.array_equal(dx.double().cpu().numpy(), dy.astype(np.float64) @ w)
    assert np.array_equal(dw.double().cpu().numpy(), dy.astype(np.float64).T @ x)
    loss = lambda x_, w_: float((dy.astype(np.float64) * (x_.astype(np.float64) @ w_.T)).sum())  # noqa: E731
    for _ in range(4):   # the loss is linear in each: a difference of any size is the gradient
        i, j, f = rng.integers(M), rng.integers(D), rng.integers(K * Fs)
        e = np.zeros_like(x)
        e[i, j] = 1
        assert loss(x + e, w) - loss(x, w) == float(dx[i, j])
        e = np.zeros_like(w)
        e[f, j] = 1
        assert loss(x, w + e) - loss(x, w) == float(dw[f, j])


def test_counts_past_32_bits():
    """More than 2^31 elements of x and of y: the last rows are those of a call on them alone."""
    rows, cols = (1 << 20) + 128 * 9, 2048
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = dev(np.random.default_rng(1).standard_normal((256, cols)), torch.bfloat16)
    x[-256:] = tail
    q, ref = mx4.quantize(x, "nvfp4"), mx4.quantize(tail, "nvfp4")
    assert x.numel() > 2 ** 31
    assert torch.equal(q.codes[-256:], ref.codes) and not q.codes[:-256].any()
    assert torch.equal(q.scales[-ref.scales.numel():], ref.scales)
    back = mx4.dequantize(q)
    assert torch.equal(back[-256:], mx4.dequantize(ref))
    del back, q
    t = mx4.quantize(x, "mxfp4", transpose=True)
    ref = mx4.quantize(tail, "mxfp4", transpose=True)
    assert torch.equal(t.codes[:, -128:], ref.codes)
    del t
    w = [mx4.quantize(dev(np.random.default_rng(2).standard_normal((2048, 32))), "mxfp4")]
    a = x[:, :32]                        # rows 2048 elements apart
    y = mx4.linear(a, w)
    assert y.numel() > 2 ** 31
    assert torch.equal(y[-256:], mx4.linear(tail[:, :32], w)) and not y[:-256].any()


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_stream_given_by_hand(as_handle):
    """Every call on the stream it is given, its results allocated there."""
    side = torch.cuda.Stream()
    st = side.cuda_stream if as_handle else side
    rng = np.random.default_rng(6)
    x = dev(rng.standard_normal((48, 256)), torch.bfloat16)
    w = dev(rng.standard_normal((64, 256)))
    s = mx4.tensor_scale(x)
    want = mx4.linear(x, [mx4.quantize(w, "nvfp4", s)], s)
    side.wait_stream(torch.cuda.current_stream())
    s2 = mx4.tensor_scale(x, stream=st)
    wq = mx4.quantize(w, "nvfp4", s2, stream=st)
    y = mx4.linear(x, [wq], s2, stream=st)
    xq = mx4.quantize(x, "nvfp4", s2, stream=st)
    y2 = mx4.matmul(xq, [wq], stream=st)
    d = mx4.dequantize(xq, stream=st)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s, s2) and torch.equal(y, want) and torch.equal(y2, want)
    assert torch.equal(d, mx4.dequantize(mx4.quantize(x, "nvfp4", s)))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_overlap(fmt, dtype):
    """One row expanded to many and a window moved over a vector: the bits of their copies."""
    rng = np.random.default_rng(12)
    row, line = dev(rng.standard_normal((1, 256)), dtype), dev(rng.standard_normal(4096), dtype)
    w = [mx4.quantize(dev(rng.standard_normal((64, 256))), fmt) for _ in range(2)]
    for x in (row.expand(96, 256), line.as_strided((160, 256), (16, 1)), line.unfold(0, 256, 64)[:32]):
        c = x.contiguous()
        for tr in (False, True):
            for a, b in ((x, c), ([x, x], [c, c])):
                q, ref = mx4.quantize(a, fmt, transpose=tr), mx4.quantize(b, fmt, transpose=tr)
                assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
        assert torch.equal(mx4.linear(x, w), mx4.linear(c, w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("transpose", [False, True])
def test_values_far_above_the_tensor_scale_saturate(dtype, transpose):
    """Spikes up to the type's largest value under a small calibrated scale: the block's scale is
    e4m3's largest and the spike is 6 of it with its own sign, the values beside it as ever."""
    rng = np.random.default_rng(14)
    for t in np.exp(rng.uniform(np.log(1e-32), np.log(1e-6), 40)).astype(np.float32):
        a = rng.standard_normal((32, 64)) * 900.0 * float(t)
        spike = np.zeros(a.shape, bool)
        spike[rng.integers(0, 32, 24), rng.integers(0, 64, 24)] = True
        a[spike] = rng.uniform(1e36, 3.38e38, spike.sum()) * rng.choice([-1, 1], spike.sum())
        x = dev(a.T if transpose else a, dtype)
        q = mx4.quantize(x, "nvfp4", torch.tensor([t], device=DEV), transpose=transpose)
        x64 = x.double().cpu().numpy()
        x64 = x64.T if transpose else x64
        bytes_, _ = linear_scales(q)
        assert (bytes_[spike.reshape(32, 4, 16).any(2)] == 0x7e).all()
        assert np.array_equal(unpack(q)[spike], 6 * np.sign(x64[spike]))
        check(q, x64, "nvfp4", float(t))
