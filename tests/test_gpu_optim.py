"""AdamW over lists of tensors (32- and 8-bit states) and the global gradient
norm, against the formulas in 64 bits.

Bounds, with u = 2^-24: m' and v' are two products, a sum and rounded
constants, at most 6u of the sum of their terms' magnitudes; the parameter adds
its own two roundings (3u |p|) and a quotient whose operands carry those errors
(24u of the step).  A bf16 result lies between the rounded ends of that
interval.  An 8-bit value is within half a step of e4m3 of the value it stands for, with 16u
for the scale.  The norm sums 32 squares in fp32: at most 17u of the norm, and
its own rounding.
"""
import numpy as np
import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import optim

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24
LR, BETAS, EPS = 3e-3, (0.9, 0.98), 1e-8
BLOCK = B.DP_STATE_BLOCK


def flat_views(sizes, dtype, shift, fill):
    """Tensors back to back in one buffer, `shift` elements in; fill(n) -> fp64 values."""
    buf = torch.zeros(sum(sizes) + shift + 8, dtype=dtype, device=DEV)
    out, at = [], shift
    for n in sizes:
        v = buf[at:at + n]
        v.copy_(torch.from_numpy(fill(n)).to(DEV))
        out.append(v)
        at += n
    return out


def host(t):
    return t.double().cpu().numpy()


def decode(codes, scale):
    x = codes.float().double().cpu().numpy()
    return x * np.repeat(host(scale), BLOCK)[:x.size]


def formula(p, g, m, v, t, decay, c=1.0, lr=LR):
    """One step in 64 bits: (p', m', v', the step's magnitude)."""
    g = g * c
    m1 = BETAS[0] * m + (1 - BETAS[0]) * g
    v1 = BETAS[1] * v + (1 - BETAS[1]) * g * g
    step = lr / (1 - BETAS[0] ** t) * m1 / (np.sqrt(v1 / (1 - BETAS[1] ** t)) + EPS)
    return p * (1 - lr * decay) - step, m1, v1, np.abs(step)


def check_step(p1, old, new, decay, t, c, pdtype, m1=None, v1=None):
    p, g, m, v = old
    want, wm, wv, step = formula(p, g, m, v, t, decay, c)
    # the quotient's numerator may cancel: its error is 6u of its terms, over the same denominator
    terms = BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g * c)
    denom = np.sqrt(wv / (1 - BETAS[1] ** t)) + EPS
    bound = 3 * U * np.abs(p) + 24 * U * (step + LR / (1 - BETAS[0] ** t) * terms / denom)
    got, bound = host(p1), bound + 1e-38
    if pdtype == torch.bfloat16:   # rounding is monotone: the interval's ends, rounded, enclose the result
        ends = [torch.from_numpy(e).to(torch.bfloat16).double().numpy()
                for e in (want - bound, want + bound)]
        assert np.all((ends[0] <= got) & (got <= ends[1]))
    else:
        assert np.all(np.abs(got - want) <= bound)
    if m1 is not None:
        assert np.all(np.abs(host(m1) - wm) <= 6 * U * terms + 1e-38)
        assert np.all(np.abs(host(v1) - wv) <= 8 * U * wv + 1e-38)
    return want, wm, wv


SIZES = [[1], [3, 0, 255, 256, 257, 1, 700], [5000, 8, 1024, 16384 + 5]]
DTYPES = [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
          (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]


def make(sizes, pd, gd, shift, seed=0, states="f32", copies=False, step=7, decay=None):
    rng = np.random.default_rng(seed)
    params = flat_views(sizes, pd, shift, lambda n: rng.standard_normal(n) * 0.05)
    grads = flat_views(sizes, gd, shift, lambda n: rng.standard_normal(n) * 1e-2)
    kw = {}
    if copies:
        kw["copies"] = flat_views(sizes, torch.bfloat16, shift, lambda n: np.zeros(n))
    if states == "f32":
        kw["exp_avg"] = flat_views(sizes, torch.float32, shift,
                                   lambda n: rng.standard_normal(n) * 3e-3)
        kw["exp_avg_sq"] = flat_views(sizes, torch.float32, shift,
                                      lambda n: rng.uniform(0, 1e-4, n))
    decay = [0.1 * (i % 2) for i in range(len(sizes))] if decay is None else decay
    opt = optim.AdamW(params, grads, lr=LR, betas=BETAS, eps=EPS, weight_decay=decay,
                      states=states, step=step, **kw)
    return opt, decay


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("pd,gd", DTYPES)
@pytest.mark.parametrize("sizes", SIZES)
def test_adamw_f32_states(sizes, pd, gd, shift):
    opt, decay = make(sizes, pd, gd, shift, copies=pd == torch.float32)
    old = [[host(x) for x in four] for four in
           zip(opt.params, opt.grads, opt.exp_avg, opt.exp_avg_sq)]
    coef = torch.tensor([0.625], device=DEV)
    opt.step(grad_scale=coef)
    assert opt.steps == 8
    for i in range(len(sizes)):
        check_step(opt.params[i], old[i], None, decay[i], 8, 0.625, pd, opt.exp_avg[i],
                   opt.exp_avg_sq[i])
        if opt.copies:
            assert torch.equal(opt.copies[i], opt.params[i].to(torch.bfloat16))
        assert np.array_equal(host(opt.grads[i]), old[i][1])


def half_step(x, scale):
    """Half of e4m3's step around x (both scaled), the largest that rounding may move."""
    a = np.abs(x) / np.where(scale > 0, scale, 1.0)
    return np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -9))) - 3, -9)) * scale / 2


def check_codes(codes, scale, want, positive=False):
    n = want.size
    nb = -(-n // BLOCK)
    tops = np.array([np.abs(want[b * BLOCK:(b + 1) * BLOCK]).max() for b in range(nb)])
    sc = host(scale)
    assert np.all(np.abs(sc - tops / 448) <= 16 * U * tops / 448 + 1e-38)
    full = np.repeat(tops / 448, BLOCK)[:n]
    got = decode(codes, scale)
    slack = half_step(want, full) * (1 + 1e-3) + 64 * U * np.abs(want) + 1e-38
    if positive:   # a root above zero keeps the smallest code at least
        low = (want > 0) & (want < full * 2.0 ** -9)
        assert np.all(np.abs(got[low] - (full * 2.0 ** -9)[low]) <= full[low] * 2.0 ** -20)
        got, want, slack = got[~low], want[~low], slack[~low]
    assert np.all(np.abs(got - want) <= slack)


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("pd,gd", DTYPES)
@pytest.mark.parametrize("sizes", SIZES)
def test_adamw_8bit_states(sizes, pd, gd, shift):
    opt, decay = make(sizes, pd, gd, shift, states="8bit", copies=pd == torch.float32, step=0)
    for t in range(1, 4):   # from zero states, each step from the stored states
        old = [[host(p), host(g), decode(m, ms), decode(r, rs) ** 2] for p, g, m, ms, r, rs in
               zip(opt.params, opt.grads, opt.exp_avg, opt.exp_avg_scale, opt.exp_avg_sq,
                   opt.exp_avg_sq_scale)]
        opt.step()
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            _, wm, wv = check_step(opt.params[i], old[i], None, decay[i], t, 1.0, pd)
            check_codes(opt.exp_avg[i], opt.exp_avg_scale[i], wm)
            check_codes(opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], np.sqrt(wv), positive=True)
            if opt.copies:
                assert torch.equal(opt.copies[i], opt.params[i].to(torch.bfloat16))


def test_adamw_8bit_blocks_of_zeros_spikes_and_tiny_values():
    n = 4 * BLOCK + 9
    g = np.zeros(n)
    g[BLOCK:2 * BLOCK] = 1e-7
    g[BLOCK] = 100.0                       # a spike: the rest of its block falls far below
    g[2 * BLOCK:3 * BLOCK] = 1e-19         # squares near the smallest normal number
    g[3 * BLOCK:] = np.linspace(-1, 1, n - 3 * BLOCK)
    params = [torch.zeros(n, device=DEV)]
    grads = [torch.from_numpy(g).float().to(DEV)]
    opt = optim.AdamW(params, grads, lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, states="8bit")
    for _ in range(20):
        opt.step()
    p = host(params[0])
    assert np.all(np.isfinite(p)) and np.all(p[:BLOCK] == 0)
    # Adam's steps are at most lr in size for a constant gradient; a root that fell to zero would
    # have made the spike's neighbours move by lr * m / eps
    assert np.abs(p).max() <= 20 * LR * 1.1
    r = opt.exp_avg_sq[0].float()[BLOCK:2 * BLOCK]
    assert float(r.min()) >= 2.0 ** -9


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_a_nan_coefficient_changes_nothing(states):
    opt, _ = make([257, 4096], torch.float32, torch.bfloat16, 0, states=states, copies=True)
    opt.step()
    bufs = opt.params + opt.copies + opt.exp_avg + opt.exp_avg_sq + \
        (opt.exp_avg_scale + opt.exp_avg_sq_scale if states == "8bit" else [])
    before = [b.clone().view(torch.uint8) for b in bufs]
    opt.grads[1][17] = float("inf")
    norm, coef = optim.GradNorm(opt.grads, 1.0)()
    assert torch.isinf(norm).all() and torch.isnan(coef).all()
    opt.step(grad_scale=coef)
    for a, b in zip(bufs, before):
        assert torch.equal(a.view(torch.uint8), b)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_bits_do_not_depend_on_list_limits_or_stream(states):
    """A list of two launches, under a CTA limit and on another stream, gives the same bits."""
    sizes = [300 + 7 * (i % 11) for i in range(500)]
    opt, _ = make(sizes, torch.float32, torch.float32, 0, states=states, decay=0.01, copies=True)
    other, _ = make(sizes, torch.float32, torch.float32, 0, states=states, decay=0.01, copies=True)
    start = opt.params[499].clone()
    opt.step()
    saved = B.dp_get_cta_limits()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    try:
        B.dp_set_cta_limits(0, 3)
        with torch.cuda.stream(side):
            other.step()
    finally:
        B.dp_set_cta_limits(*saved)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(opt.params + opt.exp_avg + opt.exp_avg_sq + opt.copies,
                    other.params + other.exp_avg + other.exp_avg_sq + other.copies):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert bool((opt.params[499] != start).all())   # the last tensor of the second launch moved


def test_schedule_in_a_captured_step():
    """A captured step replayed with the schedule's new values is the eager steps, bit for bit."""
    sizes = [1000, 33]
    opt, _ = make(sizes, torch.float32, torch.float32, 0, step=0)
    ref, _ = make(sizes, torch.float32, torch.float32, 0, step=0)
    sched = torch.tensor([LR, 1 - BETAS[0], 1 - BETAS[1]], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            opt.step(schedule=sched)
    for t in range(1, 5):
        lr = LR / t
        sched.copy_(torch.tensor([lr, 1 - BETAS[0] ** t, 1 - BETAS[1] ** t], dtype=torch.float64))
        graph.replay()
        torch.cuda.synchronize()
        old = [[host(x) for x in four] for four in
               zip(ref.params, ref.grads, ref.exp_avg, ref.exp_avg_sq)]
        ref.step(lr=lr)
        for i in range(len(sizes)):
            assert torch.equal(opt.exp_avg[i], ref.exp_avg[i])
            assert torch.equal(opt.exp_avg_sq[i], ref.exp_avg_sq[i])
            # lr and the corrections are rounded to fp32 in the schedule: 4u of the step more, each step
            step = formula(*old[i], t, 0.0, lr=lr)[3]
            assert np.all(np.abs(host(opt.params[i]) - host(ref.params[i])) <=
                          t * (8 * U * np.abs(old[i][0]) + 16 * U * step.max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("sizes", [[1], [0, 5], [1023, 1024, 1025, 31], [700000, 3, 100001],
                                   [17 + i % 5 for i in range(1700)]])
def test_grad_norm(sizes, dtype, shift):
    rng = np.random.default_rng(4)
    grads = flat_views(sizes, dtype, shift, lambda n: rng.standard_normal(n) * 3)
    want = np.sqrt(sum((host(g) ** 2).sum() for g in grads))
    gn = optim.GradNorm(grads, max_norm=0.5)
    norm, coef = (float(x) for x in gn())
    assert abs(norm - want) <= 19 * U * want
    c = min(1.0, 0.5 / (want + 1e-6))
    assert abs(coef - c) <= 24 * U * c
    first = gn.norm.clone()
    saved = B.dp_get_cta_limits()
    try:      # the same bits again, and under a CTA limit
        B.dp_set_cta_limits(0, 5)
        for _ in range(3):
            gn()
            assert torch.equal(gn.norm, first)
    finally:
        B.dp_set_cta_limits(*saved)


def test_grad_norm_of_zeros_infinities_and_nan():
    g = [torch.zeros(3000, device=DEV), torch.zeros(5, device=DEV)]
    gn = optim.GradNorm(g, max_norm=1.0)
    norm, coef = gn()
    assert float(norm) == 0 and float(coef) == 1
    for bad in (float("inf"), float("-inf"), float("nan")):
        g[1][4] = bad
        norm, coef = gn()
        assert not torch.isfinite(norm).any() and torch.isnan(coef).all()
    g[1][4] = 1e-30       # its square is below the smallest number
    assert float(gn()[0]) == 0
    assert float(optim.GradNorm([torch.full((4,), 2.0, device=DEV)])()[1]) == 1   # no limit


def test_counts_past_32_bits():
    """A tensor of more than 2^31 elements: the last ones are stepped, and the norm counts all."""
    n = (1 << 31) + 301
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    norm, _ = optim.GradNorm([g], 1.0)()
    want = 0.5 * np.sqrt(float(n))
    assert abs(float(norm) - want) <= 19 * U * want
    opt = optim.AdamW([p], [g], lr=0.5, betas=BETAS, eps=EPS, weight_decay=0.0, states="8bit")
    opt.step()
    q = torch.zeros(301, dtype=torch.bfloat16, device=DEV)
    ref = optim.AdamW([q], [g[-301:].clone()], lr=0.5, betas=BETAS, eps=EPS, weight_decay=0.0,
                      states="8bit")
    ref.step()
    assert float(q[0]) != 0
    assert torch.equal(p[-301:], q) and torch.equal(p[:301], q)
    assert bool((p == q[0]).all())
    assert torch.equal(opt.exp_avg[0].view(torch.uint8)[-301:], ref.exp_avg[0].view(torch.uint8))


def test_clipped_steps_follow_the_formula_over_a_run():
    """Norm, clip and step together, ten times, against 64 bits."""
    rng = np.random.default_rng(9)
    sizes = [513, 40]
    opt, decay = make(sizes, torch.float32, torch.float32, 0, step=0)
    clip = optim.GradNorm(opt.grads, max_norm=0.1)
    ref = [[host(x) for x in four] for four in
           zip(opt.params, opt.grads, opt.exp_avg, opt.exp_avg_sq)]
    travel = [np.zeros(n) for n in sizes]
    for t in range(1, 11):
        for i, n in enumerate(sizes):
            g = (rng.standard_normal(n) * 1e-2).astype(np.float32)
            opt.grads[i].copy_(torch.from_numpy(g))
            ref[i][1] = g.astype(np.float64)
        c = min(1.0, 0.1 / (np.sqrt(sum((r[1] ** 2).sum() for r in ref)) + 1e-6))
        assert c < 1
        opt.step(grad_scale=clip()[1])
        for i in range(len(sizes)):
            p, m, v, step = formula(*ref[i], t, decay[i], c)
            ref[i] = [p, ref[i][1], m, v]
            terms = LR / (1 - BETAS[0] ** t) / (np.sqrt(v / (1 - BETAS[1] ** t)) + EPS)
            travel[i] += 3 * U * np.abs(p) + 200 * U * (step + terms * 3e-3)
    for i in range(len(sizes)):
        assert np.all(np.abs(host(opt.params[i]) - ref[i][0]) <= travel[i])


def test_a_stream_given_by_hand():
    opt, _ = make([1000, 33], torch.float32, torch.float32, 0, step=0)
    ref, _ = make([1000, 33], torch.float32, torch.float32, 0, step=0)
    clip = optim.GradNorm(opt.grads, max_norm=0.01)
    ref.step(grad_scale=optim.GradNorm(ref.grads, max_norm=0.01)()[1])
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        coef = clip(stream=st)[1]
        if st is side:
            opt.step(grad_scale=coef, stream=st)
        torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(opt.params + opt.exp_avg, ref.params + ref.exp_avg):
        assert torch.equal(a, b)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_second_moments_below_the_normal_range(states):
    """Squares of gradients from 1e-22 to 1e-18 under an eps far below their root: v is the fp32
    one, its root is not dropped, and no step is longer than the formula's."""
    eps = 1e-25
    mags = np.float32(10.0) ** np.linspace(-21, -18, 7, dtype=np.float32)
    g = np.repeat(mags, BLOCK).astype(np.float32)
    params, grads = [torch.zeros(g.size, device=DEV)], [torch.from_numpy(g).to(DEV)]
    opt = optim.AdamW(params, grads, lr=LR, betas=BETAS, eps=eps, weight_decay=0.0, states=states)
    opt.step()
    # fp32 as written in the header: products below 2^-126 are multiples of 2^-149
    v = (g * g) * np.float32(1 - BETAS[1])
    assert (v > 0).all() and (v < 2.0 ** -126).any()
    if states == "f32":
        assert np.array_equal(host(opt.exp_avg_sq[0]), v.astype(np.float64))
    m = g.astype(np.float64) * (1 - BETAS[0])
    step = LR / (1 - BETAS[0]) * m / (np.sqrt(v.astype(np.float64) / (1 - BETAS[1])) + eps)
    assert np.all(np.abs(host(params[0]) + step) <= 24 * U * step)


@pytest.mark.parametrize("gd", [torch.float32, torch.bfloat16])
def test_the_step_of_fp32_parameters_and_states_is_the_rounded_operations(gd):
    """Every operation of the step rounded once to fp32: the bits of the same steps in numpy."""
    f = np.float32
    n, t = 5000, 8
    opt, _ = make([n], torch.float32, gd, 0, step=t - 1, decay=0.1)
    for x in (opt.grads[0], opt.exp_avg[0], opt.exp_avg_sq[0]):
        x[:9] = 0
    p, g, m, v = [host(x).astype(f) for x in (opt.params[0], opt.grads[0], opt.exp_avg[0],
                                               opt.exp_avg_sq[0])]
    opt.step(grad_scale=torch.tensor([0.625], device=DEV))
    g = g * f(0.625)
    m = m * f(BETAS[0]) + g * f(1 - BETAS[0])
    v = v * f(BETAS[1]) + (g * g) * f(1 - BETAS[1])
    denom = np.sqrt(v) * f(1 / np.sqrt(1 - BETAS[1] ** t)) + f(EPS)
    want = p * f(1 - LR * 0.1) - f(LR / (1 - BETAS[0] ** t)) * (m / denom)
    assert np.array_equal(host(opt.params[0]), want.astype(np.float64))
    assert np.array_equal(host(opt.exp_avg[0]), m.astype(np.float64))
    assert np.array_equal(host(opt.exp_avg_sq[0]), v.astype(np.float64))


@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("count", [1, 500])
def test_a_left_out_step_does_not_count(states, count):
    """Steps with a NaN coefficient before and between others, on one launch and on two: each step
    that is taken is the formula's for the number of steps taken.  With steps left out the factors
    of t are formed in fp32: 8u in lr / (1 - beta1^t) and 5u in the root's, so 16u of the step
    beside the other errors."""
    sizes = [257 + i % 3 for i in range(count)]
    opt, decay = make(sizes, torch.float32, torch.float32, 0, states=states, step=0,
                      decay=[0.0] * count)
    for x in opt.exp_avg + opt.exp_avg_sq:
        x.view(torch.uint8).zero_()
    nan, one = (torch.tensor([c], device=DEV) for c in (float("nan"), 1.0))
    taken = 0
    for skip in (True, False, False, True, True, False, False):
        old = [[host(x[0]), host(x[1])] + ([host(x[2]), host(x[3])] if states == "f32" else
               [decode(x[2], x[4]), decode(x[3], x[5]) ** 2])
               for x in zip(opt.params, opt.grads, opt.exp_avg, opt.exp_avg_sq,
                            *([opt.exp_avg_scale, opt.exp_avg_sq_scale] if states == "8bit" else []))]
        opt.step(grad_scale=nan if skip else one)
        taken += not skip
        for i in {0, count - 1}:
            if skip:
                assert np.array_equal(host(opt.params[i]), old[i][0])
                continue
            p, g, m, v = old[i]
            want, _, _, step = formula(p, g, m, v, taken, 0.0)
            terms = BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g)
            v1 = BETAS[1] * v + (1 - BETAS[1]) * g * g
            size = LR / (1 - BETAS[0] ** taken) * terms / (np.sqrt(v1 / (1 - BETAS[1] ** taken)) + EPS)
            assert np.all(np.abs(host(opt.params[i]) - want) <=
                          3 * U * np.abs(p) + 24 * U * (step + size) + 16 * U * step + 1e-38)
    assert opt.steps == 7 and int(opt.skipped) == 3
    # a run resumed with the steps taken goes on as one that has left none out
    other = optim.AdamW([p.clone() for p in opt.params], opt.grads, lr=LR, betas=BETAS, eps=EPS,
                        weight_decay=0.0, states=states, step=opt.steps - int(opt.skipped),
                        **{k: [x.clone() for x in getattr(opt, k)] for k in
                           (("exp_avg", "exp_avg_sq") if states == "f32" else
                            ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"))})
    before = [host(p) for p in opt.params]
    opt.step(grad_scale=one)
    other.step(grad_scale=one)
    for a, b, c in zip(opt.params, other.params, before):
        moved = np.abs(host(b) - c)
        assert np.all(np.abs(host(a) - host(b)) <= 16 * U * moved + 3 * U * np.abs(c))


def test_left_out_steps_of_a_replayed_graph():
    """Replays with a NaN coefficient add to the count; the schedule's corrections stay the caller's."""
    opt, _ = make([300], torch.float32, torch.float32, 0, step=4)
    ref, _ = make([300], torch.float32, torch.float32, 0, step=4)
    coef = torch.ones(1, device=DEV)
    sched = torch.tensor([LR, 1 - BETAS[0] ** 5, 1 - BETAS[1] ** 5], dtype=torch.float64).float().to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            opt.step(grad_scale=coef, schedule=sched)
    for c in (float("nan"), float("nan"), 1.0):
        coef.fill_(c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
    ref.step(grad_scale=torch.ones(1, device=DEV), schedule=sched)
    assert int(opt.skipped) == 2 and int(ref.skipped) == 0
    assert torch.equal(opt.params[0], ref.params[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [5000, 4096])
def test_the_range_of_the_norm(n, dtype):
    """What fp32 squares hold, as the header says: every element up to 2.3e18 in magnitude, a single
    one up to 1.8e19, none above; tiny ones lose bits, and 0 is left below half of 2^-149."""
    norm = lambda x: [float(v) for v in optim.GradNorm([x], 1.0)()]  # noqa: E731
    x = torch.full((n,), 2.25e18, dtype=dtype, device=DEV)
    want = np.sqrt((host(x) ** 2).sum())
    got, coef = norm(x)
    assert abs(got - want) <= 19 * U * want and abs(coef - 1 / want) <= 24 * U / want
    got, coef = norm(torch.full((n,), 4e18, dtype=dtype, device=DEV))
    assert np.isinf(got) and np.isnan(coef)
    x.zero_()
    x[77] = 1.8e19
    assert abs(norm(x)[0] - float(x[77])) <= 19 * U * 1.8e19
    x[77] = 1.9e19
    assert np.isinf(norm(x)[0])
    x.fill_(2e-19)
    want = np.sqrt((host(x) ** 2).sum())
    assert abs(norm(x)[0] - want) <= 19 * U * want
    assert norm(x.fill_(2.5e-23))[0] == 0
    assert norm(x.fill_(2.8e-23))[0] > 0


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_adamw_8bit_states_over_a_long_run(beta2):
    """After 1200 steps, half of each block's gradients a tenth from step 600 on: the next step is
    still the formula's from the stored states, and its states the nearest codes.  At beta2 = 0.95
    the stored roots follow v: a code is held until it is off by half a code's step (6 %) and v
    itself wanders between steps, so three quarters of the 1.25 in the header bound the median."""
    n = 64 * BLOCK
    gen = torch.Generator(device=DEV).manual_seed(5)
    params, grads = [torch.zeros(n, device=DEV)], [torch.zeros(n, device=DEV)]
    opt = optim.AdamW(params, grads, lr=LR, betas=(BETAS[0], beta2), eps=EPS, weight_decay=0.0,
                      states="8bit")
    low = torch.arange(n, device=DEV) % BLOCK < BLOCK // 2
    v = torch.zeros(n, dtype=torch.float64, device=DEV)
    for t in range(1, 1202):
        g = torch.randn(n, device=DEV, generator=gen) * 1e-3
        grads[0].copy_(torch.where(low, g * 0.1, g) if t > 600 else g)
        v.mul_(beta2).addcmul_(grads[0].double(), grads[0].double(), value=1 - beta2)
        if t == 1201:
            old = [host(params[0]), host(grads[0]), decode(opt.exp_avg[0], opt.exp_avg_scale[0]),
                   decode(opt.exp_avg_sq[0], opt.exp_avg_sq_scale[0]) ** 2]
        opt.step()
    p, g, m, v0 = old
    m1, v1 = BETAS[0] * m + (1 - BETAS[0]) * g, beta2 * v0 + (1 - beta2) * g * g
    size = LR / (1 - BETAS[0] ** 1201) / (np.sqrt(v1 / (1 - beta2 ** 1201)) + EPS)
    terms = BETAS[0] * np.abs(m) + (1 - BETAS[0]) * np.abs(g)
    assert np.all(np.abs(host(params[0]) - (p - size * m1)) <=
                  3 * U * np.abs(p) + 24 * U * size * (np.abs(m1) + terms) + 1e-38)
    check_codes(opt.exp_avg[0], opt.exp_avg_scale[0], m1)
    check_codes(opt.exp_avg_sq[0], opt.exp_avg_sq_scale[0], np.sqrt(v1), positive=True)
    if beta2 == 0.95:
        ratio = decode(opt.exp_avg_sq[0], opt.exp_avg_sq_scale[0]) / np.sqrt(host(v))
        for half in (low.cpu().numpy(), ~low.cpu().numpy()):
            a, b, c = np.quantile(ratio[half], [0.05, 0.5, 0.95])
            assert 0.85 < a and 0.9 < b < 1.19 and c < 1.35


def test_the_coefficient_is_the_rounded_quotient():
    """max_norm / (norm + 1e-6) rounded once from the fp32 norm, at ordinary and at extreme limits."""
    rng = np.random.default_rng(21)
    for size, limit in [(rng.uniform(0.5, 2), rng.uniform(0.1, 0.5)) for _ in range(40)] + \
            [(1.7e19, 3e-20), (1.7e19, 1e18), (1e-18, 1e-9)]:
        norm, coef = optim.GradNorm([torch.full((1,), float(size), device=DEV)], float(limit))()
        want = np.float32(limit) / (np.float32(norm.item()) + np.float32(1e-6))
        assert np.float32(coef.item()) == min(want, np.float32(1))
