"""The norm with its quantised outputs, its backward pass and the 8-bit form,
against plain implementations in 64 bits.

Tolerances, with u = 2^-24:
  * h is one fp32 addition rounded to the dtype: equal bits.
  * rstd: a sum of squares is 8 products to an accumulator, 2 additions to join
    four, 5 among lanes and 5 among warps, each within u: 20 u of a sum of
    positive terms; mean, eps, root and quotient add 4 roundings, the root halves
    what came before: within 16 u.  (The correction of the quotient only lowers it.)
  * y: two products more, 18 u, and the rounding to the dtype, eps / 2.
  * quantised y: the oracle's value, unless y lies within 32 u of a tie or its
    block's largest within 32 u of where the scale changes.
  * dx: g and xh are within u and 2 u; their products' sum within 22 u of the sum
    S of magnitudes, c within 24 u S / D of itself; the difference is one rounding
    of g - xh c, the product with rstd and the addition of dh one each.
  * dw: a chain of `rows of a set` products, the 8 or fewer rows that a CTA takes at
    once, then at most 15 + 5 additions, and the factor's 2 u, of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import mx4, mx8, norm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24
EPS = 1e-5
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
BLOCK = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def nearest(x, grid):
    """Index of the nearest of an ascending grid, ties to even, saturating; distance to a tie."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")
    tie = (i < mid.size) & (np.take(mid, np.minimum(i, mid.size - 1)) == x)
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    near = np.minimum(np.abs(x - np.take(mid, np.minimum(i, mid.size - 1))),
                      np.abs(x - np.take(mid, np.maximum(i - 1, 0)))) / np.maximum(x, 1e-300)
    return i, near


def oracle(y, fmt, t=1.0, margin=0.0):
    """(scale bytes, block doubtful, values, value doubtful) of fp64 y [R, L]."""
    R, L = y.shape
    b = y.reshape(R, -1, BLOCK[fmt])
    top = np.abs(b).max(2)
    if fmt == "nvfp4":
        byte, near = nearest(top / 6 / t, E4M3)
        step = E4M3[byte] * t
    else:
        frac, e = np.frexp(top)                       # top = frac 2^e, frac in [0.5, 1)
        if fmt == "mxfp4":
            e, near = e - 3, np.minimum(frac - 0.5, 1 - frac)
        else:
            e, near = e - 9 + (frac > 0.875), np.abs(frac - 0.875)
        byte = np.where(top > 0, np.clip(e, -127, 127) + 127, 0)
        step = np.exp2(byte - 127.0)
        near = np.where(top > 0, near, 1.0)
    z = np.where(step[..., None] > 0, np.abs(b) / np.where(step > 0, step, 1)[..., None], 0)
    grid = E4M3 if fmt == "mxfp8" else E2M1
    i, nq = nearest(z, grid)
    vals = np.sign(b) * grid[i] * step[..., None]
    block = near <= margin
    doubt = block[..., None] | (nq <= margin)
    return byte, block, vals.reshape(R, L), doubt.reshape(R, L)


def scale_bytes(q):
    nb = q.cols // BLOCK[q.format]
    Rt, Ct = -(-q.rows // 128), -(-nb // 4)
    full = q.scales.cpu().numpy().reshape(Rt, Ct, 32, 4, 4).transpose(0, 3, 2, 1, 4) \
        .reshape(Rt * 128, Ct * 4)
    rest = full.copy()
    rest[:q.rows, :nb] = 0
    return full[:q.rows, :nb], not rest.any()


def decoded(q, dtype=torch.float32):
    return (mx8 if q.format == "mxfp8" else mx4).dequantize(q, dtype)


def check_quantised(q, y64, t=1.0, margin=32 * U):
    byte, block, vals, doubt = oracle(y64, q.format, t, margin)
    got_bytes, padded = scale_bytes(q)
    assert padded
    assert np.array_equal(got_bytes[~block], byte[~block])
    got = decoded(q).double().cpu().numpy()
    assert np.all(np.abs(got - vals)[~doubt] <= 2 * U * np.abs(vals)[~doubt])
    assert doubt.mean() < 0.05
    # a doubtful value is one of the two around it: within a step of the coarser scale
    step = np.repeat(np.where(E4M3[np.minimum(byte, 126)] > 0, E4M3[np.minimum(byte, 126)] * t, t)
                     if q.format == "nvfp4" else np.exp2(byte - 127.0), BLOCK[q.format], 1)
    assert np.all(np.abs(got - y64) <= (64 if q.format == "mxfp8" else 4) * step)


@pytest.fixture(autouse=True)
def no_expired_wait():
    yield
    assert B.dp_get_device_error() == B.DP_OK


def f64(t):
    return t.double().cpu().numpy()


def matrix(rng, M, D, dtype, ld=None, offset=0, spread=True):
    """A random matrix whose rows lie ld apart, `offset` elements into its buffer."""
    ld = ld or D
    a = rng.standard_normal((M, D))
    if spread and M:
        a = a * np.exp(rng.uniform(-3, 3, (M, 1)))
    buf = torch.full((offset + M * ld + 64,), float("nan"), dtype=dtype, device=DEV)
    x = buf[offset:offset + M * ld].view(M, ld)[:, :D]
    x.copy_(torch.from_numpy(a))
    return x


def forward(x, w, res, fmt, t, keep=False, eps=EPS):
    """The formula in 64 bits on what is stored, and the checks of a call against it."""
    n = norm.rms_norm(x, w, residual=res, eps=eps, format=fmt, tensor_scale=t, keep=keep)
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(n.h, h)
    if res is None:
        assert n.h is x
    h64 = f64(h)
    r64 = 1 / np.sqrt((h64 * h64).mean(1) + eps)
    y64 = h64 * r64[:, None] * f64(w)
    assert n.rstd.dtype == torch.float32 and n.rstd.shape == (x.shape[0],)
    assert np.all(np.abs(f64(n.rstd) - r64) <= 16 * U * r64)
    if fmt is None or keep:
        assert n.y.dtype == x.dtype
        assert np.all(np.abs(f64(n.y) - y64) <= (18 * U + HALF[x.dtype] * (1 + 18 * U)) * np.abs(y64))
    else:
        assert n.y is None
    if fmt is not None:
        check_quantised(n.q, y64, 1.0 if t is None else float(t))
    else:
        assert n.q is None
    return n


# --- the 8-bit form -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (127, 96), (130, 544), (257, 1056),
                                       (2050, 1120), (2049, 2080), (0, 64), (5, 0)])
def test_eight_bits(rows, cols, dtype):
    """A division by a power of two is exact: the oracle's values everywhere."""
    rng = np.random.default_rng(rows + cols)
    a = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-9, 9, (rows, 1)))
    a[rng.random((rows, cols)) < 0.05] = 0
    x = torch.from_numpy(a).to(DEV).to(dtype)
    q = mx8.quantize(x)
    if rows == 0 or cols == 0:
        assert mx8.dequantize(q).shape == (rows, cols)
        return
    byte, _, vals, _ = oracle(f64(x), "mxfp8")
    got_bytes, padded = scale_bytes(q)
    assert padded and np.array_equal(got_bytes, byte)
    assert np.array_equal(f64(mx8.dequantize(q, torch.float32)), vals)
    assert np.array_equal(f64(mx8.dequantize(q)), vals)          # e4m3 times 2^e is a bf16 value
    codes = q.codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    assert np.array_equal(codes * np.repeat(np.exp2(byte - 127.0), 32, 1), vals)


def test_eight_bit_edges():
    """The largest value at, just below and just above 448 times a power of two, zeros, the
    smallest and largest scales, subnormals, NaN and infinities."""
    top = np.float32(448.0)
    rows = [[448.0], [np.nextafter(top, np.float32(500))], [np.nextafter(top, np.float32(0))],
            [449.0, 447.9], [256.0], [511.0], [0.0], [-0.0, 2.0 ** -149], [2.0 ** -118 * 1.75],
            [2.0 ** -120], [3.3e38], [-3.4e38, 1.0], [np.nan], [np.inf, 3.0], [1.0, -np.inf],
            [2.0 ** -6, 448.0], [2.0 ** -10, 448.0], [1.5 * 2.0 ** -10, 448.0]]
    x = np.zeros((len(rows), 64), np.float32)
    for i, r in enumerate(rows):
        x[i, :len(r)] = r
        x[i, 32] = 1.0                                  # the block beside it is its own
    q = mx8.quantize(torch.from_numpy(x).to(DEV))
    bad = ~np.isfinite(x[:, :32]).all(1)
    byte, _, vals, _ = oracle(np.where(np.isfinite(x), x, 0).astype(np.float64), "mxfp8")
    got_bytes, padded = scale_bytes(q)
    assert padded
    assert np.array_equal(got_bytes[~bad], byte[~bad]) and np.all(got_bytes[bad, 0] == 255)
    assert np.array_equal(got_bytes[bad, 1], byte[bad, 1])
    got = f64(mx8.dequantize(q, torch.float32))
    # 3.3e38 is 1.94 * 2^127: its code is 256 and its scale 2^120, and their product, 2^128,
    # rounds to infinity in fp32
    with np.errstate(over="ignore"):
        vals = vals.astype(np.float32).astype(np.float64)
    assert np.isinf(vals[10, 0]) and np.isinf(vals[11, 0]) and np.isinf(vals).sum() == 2
    assert np.array_equal(got[~bad], vals[~bad])
    assert np.isnan(got[bad, :32]).all() and np.array_equal(got[bad, 32:], vals[bad, 32:])
    assert not q.codes.cpu().numpy()[bad, :32].any()


def test_eight_bit_strided_and_unaligned():
    rng = np.random.default_rng(5)
    for ld, off in ((96, 0), (65, 0), (64, 1), (80, 3)):
        x = matrix(rng, 33, 64, torch.bfloat16, ld=ld, offset=off)
        assert torch.equal(mx8.dequantize(mx8.quantize(x)),
                           mx8.dequantize(mx8.quantize(x.contiguous())))


# --- forward --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(1, 1), (3, 17), (5, 33), (300, 48), (4, 511), (7, 768), (2, 1601),
                                 (6, 2049), (3, 4096), (2, 8191), (2, 16384), (2, 32767),
                                 (1, 32768)])
def test_plain(M, D, dtype):
    rng = np.random.default_rng(M * 31 + D)
    x, res = matrix(rng, M, D, dtype), matrix(rng, M, D, dtype)
    w32 = torch.from_numpy(rng.standard_normal(D)).float().to(DEV)
    forward(x, w32, None, None, None)
    forward(x, w32.bfloat16(), res, None, None)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(1, 32), (3, 64), (127, 96), (130, 512), (257, 768), (5, 1120),
                                 (2, 2080), (129, 4096), (3, 6432), (2, 16384), (2, 32768)])
def test_quantised(M, D, dtype, fmt):
    rng = np.random.default_rng(M * 31 + D)
    x, res = matrix(rng, M, D, dtype), matrix(rng, M, D, dtype)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float().to(DEV)
    t = torch.tensor([0.004], device=DEV) if fmt == "nvfp4" else None
    forward(x, w, res, fmt, t)
    forward(x, w.bfloat16(), None, fmt, None, keep=True)


@pytest.mark.parametrize("fmt", [None, "mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("M,D,dtype", [(2600, 4096, torch.bfloat16), (2433, 2080, torch.float32),
                                       (19500, 64, torch.bfloat16), (40001, 32, torch.float32),
                                       (2440, 8192, torch.bfloat16), (2440, 9216, torch.float32),
                                       (2500, 16384, torch.bfloat16), (7300, 1120, torch.bfloat16)])
def test_many_rows(M, D, dtype, fmt):
    """Enough rows that they come by bulk copies, several to a CTA, with and without a residual."""
    rng = np.random.default_rng(M)
    x, res = matrix(rng, M, D, dtype, ld=D + 16), matrix(rng, M, D, dtype)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float().to(DEV)
    t = torch.tensor([0.004], device=DEV) if fmt == "nvfp4" else None
    a = norm.rms_norm(x, w, residual=res, eps=EPS, format=fmt, tensor_scale=t, keep=True)
    b = norm.rms_norm(res, w, eps=EPS, format=fmt, tensor_scale=t)
    some = torch.from_numpy(np.unique(np.concatenate(
        [rng.integers(0, M, 40), np.arange(8), np.arange(M - 20, M)]))).to(DEV)
    # rows do not depend on one another: a few of them, checked as a small call's are
    one = forward(x[some], w, res[some], fmt, t, keep=True)
    two = forward(res[some], w, None, fmt, t)
    for big, small in ((a, one), (b, two)):
        assert torch.equal(big.rstd[some], small.rstd) and torch.equal(big.h[some], small.h)
        if small.y is not None:
            assert torch.equal(big.y[some], small.y)
        if fmt:
            assert torch.equal(decoded(big.q)[some], decoded(small.q))
    # and all of them against the formula, in fp32 on the GPU (its own error: 64 u)
    h = (x.float() + res.float()).to(dtype)
    assert torch.equal(a.h, h)
    want = torch.rsqrt(h.float().square().mean(1) + EPS)
    assert bool(((a.rstd - want).abs() <= 64 * U * want).all())
    want = h.float() * want[:, None] * w
    assert bool(((a.y.float() - want).abs() <= (96 * U + 1.01 * HALF[dtype]) * want.abs()).all())
    if fmt:
        assert scale_bytes(a.q)[1] and scale_bytes(b.q)[1]


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of a small call."""
    M, D = 66000, 32768
    x = torch.empty(M, D, dtype=torch.bfloat16, device=DEV)
    x[:-300] = 1
    g = torch.Generator(device=DEV).manual_seed(1)
    x[-300:] = torch.randn(300, D, device=DEV, generator=g).bfloat16()
    w = torch.ones(D, device=DEV)
    n = norm.rms_norm(x, w, format="mxfp8", keep=True)
    small = norm.rms_norm(x[-300:].clone(), w, format="mxfp8", keep=True)
    assert torch.equal(n.y[-300:], small.y) and torch.equal(n.rstd[-300:], small.rstd)
    assert torch.equal(n.q.codes[-300:], small.q.codes)
    assert bool((n.y[:-300] == 1).all())
    del n
    dx, dw = norm.rms_norm_backward(x, x, w, torch.ones(M, device=DEV))
    d1, _ = norm.rms_norm_backward(x[-300:].clone(), x[-300:].clone(), w, torch.ones(300, device=DEV))
    assert torch.equal(dx[-300:], d1)


@pytest.mark.parametrize("ld,off", [(64, 0), (96, 0), (65, 0), (64, 1), (100, 7)])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "nvfp4"])
def test_strides_and_alignment(ld, off, fmt):
    rng = np.random.default_rng(ld + off)
    x = matrix(rng, 37, 64, torch.bfloat16, ld=ld, offset=off)
    res = matrix(rng, 37, 64, torch.bfloat16, ld=96, offset=0)
    w = matrix(rng, 1, 64, torch.float32, offset=off, spread=False).reshape(64)
    a = forward(x, w, res, fmt, None, keep=True)
    b = norm.rms_norm(x.contiguous(), w.clone(), residual=res.contiguous(), eps=EPS, format=fmt,
                      keep=True)
    # unaligned rows are summed in another order: within the tolerances of both
    assert np.all(np.abs(f64(a.rstd) - f64(b.rstd)) <= 32 * U * f64(b.rstd))


def test_overlapping_and_expanded_rows():
    rng = np.random.default_rng(2)
    base = matrix(rng, 1, 64, torch.float32)
    x = base.expand(9, 64)
    w = torch.ones(64, device=DEV)
    n = norm.rms_norm(x, w, eps=EPS)
    one = norm.rms_norm(base, w, eps=EPS)
    assert torch.equal(n.y, one.y.expand(9, 64))
    dx, dw = norm.rms_norm_backward(x, x, w, n.rstd)
    d1, _ = norm.rms_norm_backward(base, base, w, one.rstd)
    assert torch.equal(dx, d1.expand(9, 64))


def test_empty():
    w = torch.ones(64, device=DEV)
    n = norm.rms_norm(torch.zeros(0, 64, device=DEV), w, format="mxfp8", keep=True)
    assert n.y.shape == (0, 64) and n.q.rows == 0 and n.rstd.shape == (0,)
    dx, dw = norm.rms_norm_backward(torch.zeros(0, 64, device=DEV), torch.zeros(0, 64, device=DEV),
                                    w, n.rstd)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device=DEV))
    n = norm.rms_norm(torch.zeros(3, 0, device=DEV), torch.ones(0, device=DEV))
    assert n.y.shape == (3, 0)


def test_rows_that_are_not_finite():
    rng = np.random.default_rng(8)
    x = matrix(rng, 6, 96, torch.float32, spread=False)
    clean = norm.rms_norm(x, torch.ones(96, device=DEV), format="mxfp8", keep=True)
    x[1, 5] = float("nan")
    x[3, 95] = float("inf")
    x[4] = 0
    n = norm.rms_norm(x, torch.ones(96, device=DEV), format="mxfp8", keep=True)
    assert n.y[1].isnan().all() and decoded(n.q)[1].isnan().all()
    assert n.y[3].isnan().sum() == 1 and n.y[3, :95].abs().max() == 0     # 1 / rms is 0
    assert (n.y[4] == 0).all() and (decoded(n.q)[4] == 0).all()           # eps alone
    for i in (0, 2, 5):
        assert torch.equal(n.y[i], clean.y[i])
        assert torch.equal(decoded(n.q)[i], decoded(clean.q)[i])


# --- backward --------------------------------------------------------------------------

def backward(dy, h, w, rstd, dh):
    dx, dw = norm.rms_norm_backward(dy, h, w, rstd, dh=dh)
    M, D = h.shape
    y, hh, ww, r = f64(dy), f64(h), f64(w), f64(rstd)[:, None]
    d = 0 if dh is None else f64(dh)
    xh, g = hh * r, y * ww
    c = (g * xh).mean(1, keepdims=True)
    S = np.abs(g * xh).mean(1, keepdims=True)
    want = r * (g - xh * c) + d
    tol = 1.01 * (r * (np.abs(g) * 4 * U + np.abs(xh) * (6 * U * np.abs(c) + 24 * U * S)) +
                  2 * U * (np.abs(want) + np.abs(d)) + HALF[h.dtype] * np.abs(want))
    tol += 2.0 ** -149
    assert dx.dtype == h.dtype and np.all(np.abs(f64(dx) - want) <= tol)
    per = 8 // -(-D // 512) if D <= 4096 else 1          # rows of a CTA at once
    sets = min(-(-M // per), 304 if D <= 4096 else 152)
    chain = -(-M // (sets * per)) + per + 15 + 5 + 2
    size = np.abs(y * xh).sum(0)
    assert dw.dtype == torch.float32
    assert np.all(np.abs(f64(dw) - (y * xh).sum(0)) <= 1.01 * chain * U * size + 2.0 ** -149)
    return dx, dw


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(1, 1), (1, 64), (3, 17), (128, 512), (457, 513), (1031, 1024),
                                 (500, 1601), (459, 2048), (1000, 4096), (13, 8192), (11, 16384),
                                 (5, 32767), (3, 32768), (5000, 96), (700, 2048), (400, 8192),
                                 (400, 16384), (200, 32768)])
def test_backward(M, D, dtype):
    rng = np.random.default_rng(M + D)
    h, dy, dh = (matrix(rng, M, D, dtype) for _ in range(3))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float().to(DEV)
    n = norm.rms_norm(h, w, eps=EPS)
    backward(dy, h, w, n.rstd, dh)
    backward(dy, h, w.bfloat16(), n.rstd, None)


@pytest.mark.parametrize("ld,off", [(64, 0), (96, 0), (65, 0), (64, 1)])
def test_backward_strides(ld, off):
    rng = np.random.default_rng(ld + off)
    h = matrix(rng, 37, 64, torch.bfloat16, ld=ld, offset=off)
    dy = matrix(rng, 37, 64, torch.bfloat16, ld=128)
    dh = matrix(rng, 37, 64, torch.bfloat16, offset=off)
    w = torch.ones(64, device=DEV)
    backward(dy, h, w, norm.rms_norm(h, w, eps=EPS).rstd, dh)


def test_gradient_against_differences():
    """Central differences of the 64-bit forward, at the fp32 inputs."""
    rng = np.random.default_rng(1)
    M, D, eps, step = 4, 24, 1e-3, 1e-5
    h, dy, dh = (matrix(rng, M, D, torch.float32, spread=False) for _ in range(3))
    w = torch.from_numpy(rng.standard_normal(D)).float().to(DEV)
    n = norm.rms_norm(h, w, eps=eps)
    dx, dw = norm.rms_norm_backward(dy, h, w, n.rstd, dh=dh)
    h64, y64, d64, w64 = f64(h), f64(dy), f64(dh), f64(w)

    def loss(h, w):
        return (y64 * h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w).sum() + (d64 * h).sum()

    for i in range(M):
        for j in range(D):
            a, b = h64.copy(), h64.copy()
            a[i, j] += step
            b[i, j] -= step
            assert abs((loss(a, w64) - loss(b, w64)) / (2 * step) - float(dx[i, j])) < 2e-5
    for j in range(D):
        a, b = w64.copy(), w64.copy()
        a[j] += step
        b[j] -= step
        assert abs((loss(h64, a) - loss(h64, b)) / (2 * step) - float(dw[j])) < 2e-5


# --- how the calls are made ---------------------------------------------------------------

def test_same_bits_under_any_cta_limit():
    rng = np.random.default_rng(4)
    saved = B.dp_get_cta_limits()
    for M, D in ((700, 512), (700, 4096), (3, 9000), (2600, 4096), (20000, 96)):
        x, dy = matrix(rng, M, D, torch.bfloat16), matrix(rng, M, D, torch.bfloat16)
        w = torch.ones(D, device=DEV)
        fmt = "mxfp8" if D % 32 == 0 else None

        def run():
            n = norm.rms_norm(x, w, residual=dy, format=fmt, keep=True)
            out = [n.y, n.h, n.rstd, *norm.rms_norm_backward(dy, n.h, w, n.rstd, dh=x)]
            return out + ([n.q.codes, n.q.scales] if fmt else [])
        want = run()
        try:
            for limit in (1, 7):
                B.dp_set_cta_limits(0, limit)
                assert all(torch.equal(a, b) for a, b in zip(run(), want))
        finally:
            B.dp_set_cta_limits(*saved)


def test_nothing_outside_is_written():
    """Bytes around every output of the C call stay as they were."""
    rng = np.random.default_rng(6)
    M, D = 130, 96
    x, res = matrix(rng, M, D, torch.bfloat16), matrix(rng, M, D, torch.bfloat16)
    w = torch.ones(D, device=DEV)
    sb = B.dp_mx4_scales_size(M, D, B.DP_MXFP4)
    need = B.dp_rms_norm_backward_workspace_size(M, D)
    sizes = {"h": M * D * 2, "y": M * D * 2, "rstd": M * 4, "codes": M * D, "scales": sb,
             "dx": M * D * 2, "dw": D * 4, "ws": need}
    buf = {k: torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV) for k, n in sizes.items()}
    at = {k: b.data_ptr() + 256 for k, b in buf.items()}
    B.dp_rms_norm(x, D, res, D, M, D, B.DP_BF16, w, B.DP_FP32, EPS, at["h"], at["y"], at["rstd"],
                  B.DP_NORM_MXFP8, None, at["codes"], at["scales"])
    B.dp_rms_norm_backward(x, D, at["h"], D, res, D, M, D, B.DP_BF16, w, B.DP_FP32, at["rstd"],
                           at["dx"], at["dw"], at["ws"], need)
    torch.cuda.synchronize()
    for k, n in sizes.items():
        assert (buf[k][:256] == 0xA5).all() and (buf[k][256 + n:] == 0xA5).all(), k
    want = norm.rms_norm(x, w, residual=res, eps=EPS, format="mxfp8", keep=True)
    assert torch.equal(buf["codes"][256:256 + M * D], want.q.codes.reshape(-1))
    assert torch.equal(buf["h"][256:256 + M * D * 2].view(torch.bfloat16), want.h.reshape(-1))


def test_streams_and_graphs():
    rng = np.random.default_rng(7)
    M, D = 300, 1024
    x, res, dy = (matrix(rng, M, D, torch.bfloat16) for _ in range(3))
    w = torch.ones(D, device=DEV)

    def step(stream=None):
        n = norm.rms_norm(x, w, residual=res, format="mxfp8", stream=stream)
        return n.q, n.h, *norm.rms_norm_backward(dy, n.h, w, n.rstd, dh=dy, stream=stream)

    def flat(out):
        return [out[0].codes, out[0].scales, *out[1:]]

    want = [t.clone() for t in flat(step())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = flat(step(side))
    got2 = flat(step(side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(got2, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.mul_(2)                      # the replay reads what is there then
    res.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1], flat(step())[2])
    assert all(torch.equal(a, b) for a, b in zip(flat(out), flat(step())))


def test_two_calls_at_once():
    rng = np.random.default_rng(9)
    xs = [matrix(rng, 3000, 2048, torch.bfloat16) for _ in range(2)]
    w = torch.ones(2048, device=DEV)
    want = [norm.rms_norm_backward(x, x, w, norm.rms_norm(x, w).rstd) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(norm.rms_norm_backward(x, x, w, norm.rms_norm(x, w).rstd))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --- magnitudes far from 1 --------------------------------------------------------------------

def check_range(n, h, w, eps, q=False):
    """The tolerances of any row: times a power of two a sum is as exact.  Two roundings more
    for the smallest rows: h w below 2^-126 is 2^-150 off, which an rstd up to 2^62 takes to
    2^-88; a thread's squares times that power are 2^-150 off at most, of 2^-124 or more (32
    of them from 5e-19 on, over 1024), within the 16 u whose own terms come to 14."""
    h64 = f64(h)
    r64 = 1 / np.sqrt((h64 * h64).mean(1) + eps)
    y64 = h64 * r64[:, None] * f64(w)
    assert np.all(np.abs(f64(n.rstd) - r64) <= 16 * U * r64)
    if n.y is not None:
        tol = (18 * U + HALF[h.dtype] * (1 + 18 * U)) * np.abs(y64) + 2.0 ** -88
        assert np.all(np.abs(f64(n.y) - y64) <= tol)
    if q:
        check_quantised(n.q, y64)


def sized(M, D, sizes, dtype, seed):
    """Rows of the magnitudes `sizes` (0.5 to 2 times that), others of 1."""
    rng = np.random.default_rng(seed)
    a = np.sign(rng.standard_normal((M, D))) * rng.uniform(0.5, 2, (M, D))
    a[:len(sizes)] *= np.array(sizes)[:, None]
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).float().to(DEV)
    return torch.from_numpy(a).to(DEV).to(dtype), w


@pytest.mark.parametrize("fmt", [None, "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(9, 96), (9, 513), (9, 4096), (2700, 4096), (9, 6432), (9, 16384),
                                 (9, 32768)])
def test_large_rows(M, D, dtype, fmt):
    """4096 values of 1e18 have a sum of squares past fp32 and a mean of them well inside it."""
    fmt = fmt if D % 32 == 0 else None
    sizes = [1e12, 1e16, 1e17, 3e17, 1e18, 1.6e18]
    x, w = sized(M, D, sizes, dtype, D)
    n = norm.rms_norm(x, w, eps=EPS, format=fmt, keep=True)
    few = torch.arange(9, device=DEV)
    small = norm.rms_norm(x[few].clone(), w, eps=EPS, format=fmt, keep=True)
    check_range(small, x[few], w, EPS, fmt is not None)
    assert torch.equal(n.y[few], small.y) and torch.equal(n.rstd[few], small.rstd)
    check_range(n, x, w, EPS)
    m = norm.rms_norm(torch.zeros_like(x), w, residual=x, eps=EPS, format=fmt, keep=True)
    assert torch.equal(m.h, x) and torch.equal(m.y, n.y) and torch.equal(m.rstd, n.rstd)
    check_range(norm.rms_norm(x, w, eps=1e36), x, w, float(np.float32(1e36)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(9, 96), (9, 513), (2700, 4096), (9, 16384), (9, 32768)])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-27])
def test_small_rows(M, D, dtype, eps):
    x, w = sized(M, D, [1e-12, 1e-14, 1e-16, 1e-17, 3e-18, 1e-18], dtype, D)
    check_range(norm.rms_norm(x, w, eps=eps), x, w, float(np.float32(eps)))


def test_rows_past_the_range():
    """What the header says of them: an infinite mean makes y 0; squares that vanish leave eps."""
    x, w = sized(4, 4096, [1e25, 1e38], torch.float32, 1)
    n = norm.rms_norm(x, w)
    fits = (x.double() * w.double()).abs() <= torch.finfo(torch.float32).max
    assert (n.rstd[:2] == 0).all() and (n.y[:2][fits[:2]] == 0).all()
    assert fits[0].all() and n.y[~fits].isnan().all()      # h w comes first: infinity times 0
    x, w = sized(4, 4096, [1e-24, 0.0], torch.float32, 1)
    n = norm.rms_norm(x, w, eps=0.0)
    assert n.rstd[:2].isinf().all() and n.y[0].isinf().all() and n.y[1].isnan().all()
    n = norm.rms_norm(x, w, eps=1e-12)
    assert bool(((n.rstd[:2] - 1e6).abs() <= 16 * U * 1e6).all()) and (n.y[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_of_large_and_small_rows(dtype):
    h, w = sized(9, 4096, [1e18, 1.6e18, 3e17, 1e12, 1e-12, 1e-16, 1e-17], dtype, 3)
    rng = np.random.default_rng(3)
    dy, dh = matrix(rng, 9, 4096, dtype), matrix(rng, 9, 4096, dtype)
    n = norm.rms_norm(h, w, eps=0.0)
    check_range(n, h, w, 0.0)
    backward(dy, h, w, n.rstd, dh)
    backward(dy, h, w, n.rstd, None)


def test_a_row_of_nothing_has_no_mean():
    """Rows of no elements: the mean of their squares, and so rstd, is NaN."""
    held = torch.full((3,), 7.0, device=DEV)     # what the allocator hands out next
    del held
    n = norm.rms_norm(torch.zeros(3, 0, device=DEV), torch.ones(0, device=DEV))
    assert n.rstd.shape == (3,) and n.rstd.dtype == torch.float32 and n.rstd.isnan().all()
    n = norm.rms_norm(torch.zeros(2, 0, device=DEV), torch.ones(0, device=DEV),
                      residual=torch.zeros(2, 0, device=DEV), format="mxfp8")
    assert n.rstd.isnan().all() and n.q.rows == 2 and n.q.cols == 0


def test_which_calls_have_the_same_bits():
    """A row's bits are one in all calls with a format, and in calls without one whose buffers are
    all on 32-byte boundaries; otherwise sums have another order, within both tolerances."""
    rng = np.random.default_rng(11)
    M, D = 40, 1120
    x, res = matrix(rng, M, D, torch.bfloat16), matrix(rng, M, D, torch.bfloat16)
    odd = matrix(rng, M, D, torch.bfloat16, ld=D + 3, offset=1)
    odd.copy_(x)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D + 1)).float().to(DEV)
    w_odd, w = w[1:], w[1:].clone()
    want = norm.rms_norm(x, w, residual=res)
    for a, b, fmt in ((x, w, "mxfp8"), (odd, w, "mxfp8"), (x, w_odd, "mxfp4"), (odd, w_odd, "nvfp4")):
        n = norm.rms_norm(a, b, residual=res, format=fmt, keep=True)
        assert torch.equal(n.rstd, want.rstd) and torch.equal(n.y, want.y)
    for a, b in ((odd, w), (x, w_odd), (odd, w_odd)):
        n = norm.rms_norm(a, b, residual=res)
        assert bool(((n.rstd - want.rstd).abs() <= 32 * U * want.rstd).all())
