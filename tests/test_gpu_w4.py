"""A few tokens times 4-bit shards, against the decoded weights in 64 bits.

Every product of an f16 weight and an f16 x is exact, so y differs from the sum by
the fp32 additions: at most D + 8 of them (the tensor core's within an instruction,
an instruction a step, the shares'), 2^-24 of the sum of magnitudes each and twice
that where the tensor core truncates; plus what x and mxfp4's scales lose below
2^-27 of the largest, 2^-35 of it, and one rounding of y.  With small integers all
of it is exact.
"""
import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import mx4

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def no_expired_wait():
    yield
    assert B.dp_get_device_error() == B.DP_OK


def f64(t):
    return t.double().cpu().numpy()


def shards_of(w, K, fmt, t=None):
    return [mx4.quantize(s.contiguous(), fmt, t) for s in w.chunk(K)]


def check(x, shards, y_dtype=torch.float32):
    """The call against 64 bits on what is stored; returns y."""
    y = mx4.linear_w4(x, shards, y_dtype)
    w = np.concatenate([f64(mx4.dequantize(q, torch.float32)) for q in shards])
    x64 = f64(x)
    want, size = x64 @ w.T, np.abs(x64) @ np.abs(w).T
    D = x.shape[1]
    lost = D * 2.0 ** -35 * 2 * np.abs(x64).max(1, initial=0)[:, None] * \
        np.abs(w).max(1, initial=0)[None, :]
    tol = 2 * (D + 8) * U * size + lost
    if y_dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert y.dtype == y_dtype and y.shape == want.shape
    assert np.all(np.abs(f64(y) - want) <= tol + 2.0 ** -140)
    return y


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g) * scale


SHAPES = [  # M, D, K, F_shard
    (1, 32, 1, 16), (1, 64, 2, 48), (1, 96, 1, 128), (2, 128, 1, 144), (3, 160, 4, 16),
    (8, 512, 8, 64), (9, 544, 2, 208), (16, 1056, 1, 336), (17, 1024, 3, 80), (32, 4096, 1, 64),
    (33, 288, 2, 32), (70, 96, 1, 256), (1, 4096, 8, 512), (5, 1120, 2, 4112), (12, 640, 1, 20000),
    (24, 224, 4, 5008), (7, 16384, 1, 32)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,D,K,Fs", SHAPES)
def test_values(M, D, K, Fs, fmt):
    w = normal((K * Fs, D), M + D, 0.02)
    x = normal((M, D), M * D) * torch.exp(2 * normal((M, 1), 3))
    t = mx4.tensor_scale(w) if fmt == "nvfp4" else None
    s = shards_of(w, K, fmt, t)
    a = check(x.bfloat16(), s)
    b = check(x.bfloat16(), s, torch.bfloat16)
    assert torch.equal(a.bfloat16(), b)
    assert torch.equal(a, mx4.linear_w4(x.bfloat16(), s, torch.float32))   # the same bits again


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,D,K,Fs", [(1, 64, 1, 16), (5, 416, 2, 144), (20, 256, 1, 20000),
                                      (11, 1024, 2, 96)])
def test_integers_are_exact(M, D, K, Fs, fmt):
    """Weights that their form holds exactly, x of small integers: every sum is exact."""
    rng = np.random.default_rng(D)
    vals = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    w = rng.choice(vals, (K * Fs, D)) * rng.choice([-1, 1], (K * Fs, D))
    w[:, ::16] = 6                      # every block's scale is 1 in both forms
    x = rng.integers(-8, 9, (M, D))
    s = shards_of(torch.from_numpy(w).float().to(DEV), K, fmt)
    y = mx4.linear_w4(torch.from_numpy(x).to(DEV).bfloat16(), s, torch.float32)
    assert np.array_equal(f64(y), x @ w.T)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [1, 10, 30])
def test_growing_and_shrinking_magnitudes(M, fmt):
    """x and the weights' scales rise and fall along d, past what f16 spans."""
    D, F = 2048, 160
    ramp = torch.linspace(-40, 40, D, device=DEV)
    w = normal((F, D), 1)
    for dx, dw in ((ramp, 0 * ramp), (-ramp, 0 * ramp), (0 * ramp, ramp), (0 * ramp, -ramp),
                   (ramp, -ramp), (-ramp, ramp), (ramp.abs(), ramp)):
        if fmt == "nvfp4":
            dw = dw.clamp(-5, 5)        # its block scales span 2^17
        s = shards_of(w * torch.exp2(dw), 1, fmt, torch.tensor([1.0], device=DEV) if fmt == "nvfp4"
                      else None)
        check((normal((M, D), 2) * torch.exp2(dx)).bfloat16(), s)


def test_extreme_magnitudes():
    """Tokens and weights at the ends of bf16 and of the scales."""
    D, F = 256, 48
    w, x = normal((F, D), 1), normal((4, D), 2)
    for sw in (2.0 ** -100, 1.0, 2.0 ** 100):
        s = shards_of(w * sw, 1, "mxfp4")
        for sx in (2.0 ** -120, 2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** 110):
            if 2.0 ** -90 < sw * sx < 2.0 ** 110:      # where fp32 holds the sums
                check((x * sx).bfloat16(), s)
    rows = x.bfloat16()
    rows[0] = 0
    rows[1, 1:] = 0
    y = check(rows, shards_of(w, 1, "mxfp4"))
    assert (y[0] == 0).all()
    z = shards_of(torch.zeros(F, D, device=DEV), 1, "nvfp4")
    assert (check(rows, z) == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_not_finite(fmt):
    D, F = 512, 96
    w = normal((F, D), 1)
    x = normal((5, D), 2).bfloat16()
    clean = mx4.linear_w4(x, shards_of(w, 1, fmt), torch.float32)
    x[1, 300] = float("nan")
    x[3, 7] = float("inf")
    y = mx4.linear_w4(x, shards_of(w, 1, fmt), torch.float32)
    assert y[1].isnan().all() and not y[3].isfinite().any()
    for i in (0, 2, 4):
        assert torch.equal(y[i], clean[i])
    x = normal((5, D), 2).bfloat16()
    w[17, 200] = float("nan")           # a NaN block: that feature, and no other
    y = mx4.linear_w4(x, shards_of(w, 1, fmt), torch.float32)
    assert y[:, 17].isnan().all()
    keep = [f for f in range(F) if f != 17]
    assert torch.equal(y[:, keep], clean[:, keep])


def test_strides_and_alignment():
    D, F = 320, 112
    s = shards_of(normal((F, D), 1), 1, "nvfp4")
    x = normal((6, D), 2).bfloat16()
    want = mx4.linear_w4(x, s)
    for ld, off in ((D + 8, 0), (D + 1, 0), (D, 1), (2 * D, 3), (D + 4, 4)):
        buf = torch.full((off + 6 * ld + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
        v = buf[off:off + 6 * ld].view(6, ld)[:, :D]
        v.copy_(x)
        assert torch.equal(mx4.linear_w4(v, s), want)
    many = normal((19, D), 3).bfloat16()          # prepared beforehand
    want = mx4.linear_w4(many, s)
    for ld, off in ((D + 8, 0), (D + 1, 0), (D, 1), (D + 4, 4)):
        buf = torch.full((off + 19 * ld + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
        v = buf[off:off + 19 * ld].view(19, ld)[:, :D]
        v.copy_(many)
        assert torch.equal(mx4.linear_w4(v, s), want)
    one = mx4.linear_w4(many[:1].expand(9, D), s)
    assert torch.equal(one, one[:1].expand(9, F))


def test_offsets_past_32_bits():
    """A shard of more than 4 GB: its last rows are those of a shard of these rows alone."""
    D, F, last = 16384, 524288 + 256, 256
    g = torch.Generator(device=DEV).manual_seed(4)
    codes = torch.randint(0, 256, (F, D // 2), dtype=torch.uint8, device=DEV, generator=g)
    tiles = D // 128 * 512
    scales = torch.randint(118, 131, (F // 128 * tiles,), dtype=torch.uint8, device=DEV, generator=g)
    big = mx4.Mx4Tensor(codes, scales, F, D, "mxfp4")
    end = mx4.Mx4Tensor(codes[-last:].clone(), scales[-last // 128 * tiles:].clone(), last, D, "mxfp4")
    for M in (1, 10):
        x = normal((M, D), M).bfloat16()
        y = mx4.linear_w4(x, [big], torch.float32)[:, -last:]
        want = check(x, [end])
        # d is split otherwise there, so the sums come in another order: each is within
        # 2 (D + 8) 2^-24 of the sum of magnitudes of the exact one (see above), and the
        # two within twice that of one another
        size = x.double().abs() @ mx4.dequantize(end, torch.float32).double().abs().t()
        assert bool(((y - want).double().abs() <= 4 * (D + 8) * U * size).all())
        # rows of another place would be off by the size of y itself
        assert bool(((y - want).abs() <= 1e-2 * want.abs().amax()).all())


def test_two_calls_at_once():
    D, F = 1024, 4096
    s = shards_of(normal((F, D), 1), 4, "nvfp4")
    xs = [normal((M, D), M).bfloat16() for M in (3, 12, 30)]
    want = [mx4.linear_w4(x, s) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [mx4.linear_w4(x, s, stream=st) for x, st in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty():
    s = shards_of(normal((32, 64), 1), 1, "mxfp4")
    assert mx4.linear_w4(torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV), s).shape == (0, 32)
    z = mx4.quantize(torch.zeros(16, 0, device=DEV), "mxfp4")
    y = mx4.linear_w4(torch.zeros(3, 0, dtype=torch.bfloat16, device=DEV), [z])
    assert y.shape == (3, 16) and (y == 0).all()


def test_nothing_else_is_written_and_streams_and_graphs():
    from ring_allreduce_gradient_gb300 import binding as B
    D, F, M = 544, 224, 9
    s = shards_of(normal((F, D), 1), 2, "nvfp4")
    x = normal((M, D), 2).bfloat16()
    want = mx4.linear_w4(x, s)
    torch.cuda.synchronize()
    buf = torch.full((M * F * 2 + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    need = B.dp_allgather_linear_w4_workspace_size(M, D)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    B.dp_allgather_linear_w4(x, M, D, D, [q._c for q in s], 2, F // 2, B.DP_NVFP4,
                             buf.data_ptr() + 256, B.DP_BF16, ws.data_ptr() + 256, need)
    assert (ws[:256] == 0xA5).all() and (ws[-256:] == 0xA5).all()
    assert (buf[:256] == 0xA5).all() and (buf[-256:] == 0xA5).all()
    assert torch.equal(buf[256:-256].view(torch.bfloat16).view(M, F), want)
    side = torch.cuda.Stream()
    got = mx4.linear_w4(x, s, stream=side)
    other = mx4.linear_w4(x, s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mx4.linear_w4(x, s)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, mx4.linear_w4(x, s)) and torch.equal(y.float(), want.float() * 2)


def test_tokens_do_not_meet():
    """Each token is scaled by itself: tokens of one call, in another order and among others of
    other magnitudes, keep their bits."""
    D, F = 1024, 96
    s = shards_of(normal((F, D), 1), 1, "mxfp4")
    for M in (8, 30):
        x = (normal((M, D), 2) * torch.exp2(10 * normal((M, 1), 3))).bfloat16()
        y = mx4.linear_w4(x, s, torch.float32)
        order = torch.randperm(M, device=DEV)
        assert torch.equal(mx4.linear_w4(x[order].contiguous(), s, torch.float32), y[order])
        x2 = (normal((M, D), 5) * 1e4).bfloat16()
        x2[3] = x[5]
        assert torch.equal(mx4.linear_w4(x2, s, torch.float32)[3], y[5])


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def made(codes, byte):
    """An mxfp4 matrix of e2m1 codes [F, D] and scale bytes [F, D / 32], and its values."""
    F, D = codes.shape
    Rt, Ct = -(-F // 128), -(-D // 128)
    full = np.zeros((Rt * 128, Ct * 4), np.uint8)
    full[:F, :D // 32] = byte
    tiles = full.reshape(Rt, 4, 32, Ct, 4).transpose(0, 3, 2, 1, 4)
    packed = (codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)
    q = mx4.Mx4Tensor(torch.from_numpy(packed).to(DEV),
                      torch.from_numpy(tiles.reshape(-1).copy()).to(DEV), F, D, "mxfp4")
    scale = np.where(byte == 255, np.nan, np.exp2(byte - 127.0)).repeat(32, 1)
    return q, E2M1[codes & 7] * np.where(codes & 8, -1, 1) * scale


@pytest.mark.parametrize("M", [1, 10, 20])
@pytest.mark.parametrize("top", [200, 245, 246, 250, 254])
def test_a_nan_block_after_one_of_the_largest_scales(top, M):
    """Byte 255 is NaN whatever scales its row has had; D is long enough that a warp comes to
    it after them."""
    rng = np.random.default_rng(top)
    F, D = 48, 8192
    byte = np.full((F, D // 32), 120)
    byte[3] = byte[40] = byte[41] = top
    codes = rng.integers(0, 16, (F, D))
    x = torch.from_numpy(rng.integers(-8, 9, (M, D)) * 2.0 ** -40).to(DEV).bfloat16()
    q, v = made(codes, byte)
    want, size = f64(x) @ v.T, np.abs(f64(x)) @ np.abs(v).T
    y = f64(mx4.linear_w4(x, [q], torch.float32))
    assert np.all(np.abs(y - want) <= 2 * (D + 8) * U * size)
    byte[3, 5] = byte[40, 250] = 255                 # the second step of a warp; a later one
    q, v = made(codes, byte)
    y = f64(mx4.linear_w4(x, [q], torch.float32))
    assert np.isnan(y[:, [3, 40]]).all()
    keep = [f for f in range(F) if f not in (3, 40)]
    assert np.all(np.abs(y - want)[:, keep] <= 2 * (D + 8) * U * size[:, keep])


@pytest.mark.parametrize("M", [1, 10, 20])
@pytest.mark.parametrize("top", [9, 10, 18, 19, 27])
def test_blocks_of_the_smallest_scale_count(top, M):
    """Scale byte 0 is 2^-127, not nothing: with one of 2^27 times it in the row before."""
    F, D = 16, 8192
    codes, byte = np.zeros((F, D), int), np.zeros((F, D // 32), int)
    codes[:, :32] = 1
    byte[:, 0] = top
    codes[:, 4 * 32:5 * 32] = 7
    q, v = made(codes, byte)
    x = torch.zeros(M, D, device=DEV, dtype=torch.bfloat16)
    x[:, 4 * 32:5 * 32] = 2.0 ** 60
    want = f64(x) @ v.T
    assert want[0, 0] == 192 * 2.0 ** -67
    assert np.array_equal(f64(mx4.linear_w4(x, [q], torch.float32)), want)


@pytest.mark.parametrize("M", [1, 10, 20])
@pytest.mark.parametrize("top", [30, 60, 130])
def test_blocks_far_below_their_rows_largest(top, M):
    """Blocks down to 2^-27 of the largest scale of their row are exact; below, a weight is off
    by at most 2^-25 of that scale.  x is nothing where the large ones are, and a power of two
    elsewhere, so that sums of one block's weights are exact."""
    rng = np.random.default_rng(top)
    F, D = 64, 8192
    codes = rng.integers(0, 8, (F, D))
    for below in (20, 26, 27, 28, 29, 30, 40):
        low = top - below
        if low < 0:
            continue
        byte = np.full((F, D // 32), low)
        byte[:, ::4] = top                            # a block of each step
        q, v = made(codes, byte)
        x = torch.zeros(M, D, device=DEV, dtype=torch.bfloat16)
        at = rng.choice([b for b in range(D // 32) if b % 4], M)
        for m in range(M):
            x[m, 32 * at[m]:32 * at[m] + 32] = 1.0
        y, want = f64(mx4.linear_w4(x, [q], torch.float32)), f64(x) @ v.T
        if below <= 27:
            assert np.array_equal(y, want)
        else:
            assert np.all(np.abs(y - want) <= 32 * 2.0 ** (top - 127 - 25))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_one_token_and_the_same_one_in_a_batch(fmt):
    """A call's own sizes order its sums, M among them.  Alone and in a batch a token's y are
    each within 2 (D + 8) 2^-24 of the sum of magnitudes of the exact one, and so within twice
    that of one another; where d is one step there is one order."""
    for D, F in ((128, 96), (1024, 96), (2080, 400), (8192, 64)):
        s = shards_of(normal((F, D), 1), 1, fmt)
        w = mx4.dequantize(s[0], torch.float32).double()
        x = normal((40, D), 2).bfloat16()
        size = x.double().abs() @ w.abs().t()
        alone = torch.cat([mx4.linear_w4(x[i:i + 1], s, torch.float32) for i in range(40)])
        for M in (2, 5, 8, 9, 16, 17, 33, 40):
            y = mx4.linear_w4(x[:M], s, torch.float32)
            if D == 128:
                assert torch.equal(y, alone[:M])
            assert bool(((y - alone[:M]).double().abs() <= 4 * (D + 8) * U * size[:M]).all())


def test_weights_rewritten_by_another_thread_on_the_same_stream():
    """A product of prepared tokens is of the weights before or after the other thread's
    quantisation, never of some of both: the call's two kernels stay together."""
    import threading
    D, F, M, runs = 1024, 8192, 12, 300
    w = [normal((F, D), i, 0.02).bfloat16() for i in range(2)]
    q = mx4.quantize(w[0], "nvfp4")
    x = normal((M, D), 3).bfloat16()
    want = []
    for i in range(2):
        B.dp_mx4_quantize([w[i]], 1, F, D, D, B.DP_BF16, B.DP_NVFP4, False, None, q.codes, q.scales)
        want.append(mx4.linear_w4(x, [q]))
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    stream = torch.cuda.Stream()
    got, errors = [], []
    go = threading.Barrier(2)

    def quantise():
        try:
            go.wait()
            for i in range(2 * runs):
                B.dp_mx4_quantize([w[i % 2]], 1, F, D, D, B.DP_BF16, B.DP_NVFP4, False, None,
                                  q.codes, q.scales, stream=stream.cuda_stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    other = threading.Thread(target=quantise)
    other.start()
    with torch.cuda.stream(stream):
        go.wait()
        for _ in range(runs):
            got.append(mx4.linear_w4(x, [q]))
    other.join()
    torch.cuda.synchronize()
    assert not errors
    same = [[torch.equal(y, z) for z in want] for y in got]
    assert all(any(s) for s in same)
