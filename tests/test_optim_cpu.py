"""Refusals of the optimizer calls: every one is made on the host before any
device call, so none of them needs a GPU."""
import ctypes

import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import build as cuda_build
from ring_allreduce_gradient_gb300 import optim

BASE = 0x7F0000000000
INVALID, UNSUPPORTED, ALIAS = B.DP_ERR_INVALID_ARG, B.DP_ERR_UNSUPPORTED, B.DP_ERR_ALIAS


def fake(i, off=0):
    return BASE + (i << 26) + off


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return B.load()


def row(i=0, n=1000, **kw):
    r = dict(param=fake(8 * i), grad=fake(8 * i + 1), copy=None, exp_avg=fake(8 * i + 2),
             exp_avg_sq=fake(8 * i + 3), exp_avg_scale=fake(8 * i + 4),
             exp_avg_sq_scale=fake(8 * i + 5), numel=n, weight_decay=0.1)
    r.update(kw)
    return r


def create(rows, pd=B.DP_FP32, gd=B.DP_FP32, state=B.DP_STATE_FP32):
    st, h = B.dp_adamw_create(rows, len(rows), pd, gd, state, check=False)
    if h:
        B.dp_adamw_destroy(h)
    assert (st == B.DP_OK) == bool(h)
    return st


def test_adamw_create_checks_its_list(lib):
    assert create([row()]) == B.DP_OK
    assert create([row(copy=fake(6))], state=B.DP_STATE_8BIT) == B.DP_OK
    assert create([row(i) for i in range(900)]) == B.DP_OK     # several launches
    assert create([]) == B.DP_OK
    for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert create([row(**{name: None})]) == INVALID
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        assert create([row(**{name: None})]) == B.DP_OK        # 32-bit states have none
        assert create([row(**{name: None})], state=B.DP_STATE_8BIT) == INVALID
    none = dict.fromkeys(("param", "grad", "exp_avg", "exp_avg_sq"))
    assert create([row(n=0, **none)]) == B.DP_OK               # an empty tensor has no pointers
    assert create([row(weight_decay=-0.1)]) == INVALID
    assert create([row(weight_decay=float("nan"))]) == INVALID
    assert create([row()], pd=7) == UNSUPPORTED
    assert create([row()], gd=7) == UNSUPPORTED
    assert create([row()], state=2) == UNSUPPORTED
    assert create([row(param=fake(0, 2))]) == UNSUPPORTED      # not on an element's boundary
    assert create([row(grad=fake(1, 1))], gd=B.DP_BF16) == UNSUPPORTED
    assert lib.dp_adamw_create(None, 1, 0, 0, 0, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.dp_adamw_create(None, 0, 0, 0, 0, None) == INVALID


def test_adamw_create_finds_overlaps():
    assert create([row(grad=fake(0, 400))]) == ALIAS           # gradient inside the parameter
    assert create([row(), row(1, param=fake(0, 3996))]) == ALIAS
    assert create([row(), row(1, param=fake(0, 4000))]) == B.DP_OK
    assert create([row(), row(1, exp_avg=fake(3, 16))]) == ALIAS
    assert create([row(), row(1, grad=fake(1))]) == B.DP_OK    # gradients are only read
    assert create([row(copy=fake(2, 64))]) == ALIAS
    assert create([row(exp_avg_scale=fake(5, 12))], state=B.DP_STATE_8BIT) == ALIAS
    assert create([row(exp_avg_scale=fake(5, 16))], state=B.DP_STATE_8BIT) == B.DP_OK


def test_adamw_step_checks_its_numbers():
    _, h = B.dp_adamw_create([], 0, B.DP_FP32, B.DP_FP32, B.DP_STATE_FP32)
    ok = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1)
    step = lambda **kw: B.dp_adamw_step(h, stream=0, check=False, **{**ok, **kw})  # noqa: E731
    assert step() == B.DP_OK
    for bad in (dict(step=0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0),
                dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
                dict(eps=-1e-8), dict(eps=1e-60), dict(eps=float("nan"))):
        assert step(**bad) == INVALID, bad
    assert step(grad_scale=fake(0, 2)) == UNSUPPORTED
    assert step(schedule=fake(0, 2)) == UNSUPPORTED
    assert B.dp_adamw_step(0, 1e-3, 0.9, 0.99, 1e-8, 1, stream=0, check=False) == INVALID
    B.dp_adamw_destroy(h)
    B.dp_adamw_destroy(0)


def test_grad_norm_checks(lib):
    need = B.dp_grad_norm_workspace_size(2)
    assert need > B.dp_grad_norm_workspace_size(0) - 1 > 0
    assert B.dp_grad_norm_workspace_size(2000) > need

    def norm(grads=(fake(0), fake(1)), numels=(100, 50), dt=B.DP_FP32, max_norm=1.0, out=fake(2),
             coef=fake(3), ws=fake(4), wb=need):
        return B.dp_grad_norm(list(grads), list(numels), len(grads), dt, max_norm, out, coef, ws,
                              wb, stream=0, check=False)

    assert norm(out=None, coef=None) == INVALID
    assert norm(ws=None) == INVALID
    assert norm(wb=need - 1) == INVALID
    assert norm(grads=(fake(0), None)) == INVALID
    for bad in (0.0, -1.0, float("nan")):
        assert norm(max_norm=bad) == INVALID
    assert norm(dt=5) == UNSUPPORTED
    assert norm(grads=(fake(0, 2), fake(1))) == UNSUPPORTED
    assert norm(ws=fake(4, 8)) == UNSUPPORTED
    assert norm(out=fake(0, 396)) == ALIAS
    assert norm(coef=fake(2)) == ALIAS
    assert norm(ws=fake(1, 16)) == ALIAS
    assert lib.dp_grad_norm_workspace_size(1, None) == INVALID
    assert lib.dp_grad_norm_workspace_size(-1, ctypes.byref(ctypes.c_size_t())) == INVALID


def test_the_tensor_objects_check_their_lists():
    p = [torch.zeros(10), torch.zeros(4)]
    g = [torch.zeros(10), torch.zeros(4)]
    with pytest.raises(ValueError, match="at least one"):
        optim.AdamW([], [])
    with pytest.raises(ValueError, match="states"):
        optim.AdamW(p, g, states="4bit")
    with pytest.raises(ValueError, match="grads: 1 tensors for 2"):
        optim.AdamW(p, g[:1])
    with pytest.raises(ValueError, match=r"grads\[1\]: 5 elements"):
        optim.AdamW(p, [g[0], torch.zeros(5)])
    with pytest.raises(ValueError, match="contiguous"):
        optim.AdamW(p, [torch.zeros(20)[::2], g[1]])
    with pytest.raises(ValueError, match="contiguous"):
        optim.AdamW([p[0], p[1].bfloat16()], g)
    with pytest.raises(ValueError, match="copies"):
        optim.AdamW(p, g, copies=[torch.zeros(10), torch.zeros(4)])
    with pytest.raises(ValueError, match="weight_decay"):
        optim.AdamW(p, g, weight_decay=[0.1])
    with pytest.raises(ValueError, match="exp_avg"):
        optim.AdamW(p, g, states="8bit", exp_avg=[torch.zeros(10), torch.zeros(4)])
    with pytest.raises(ValueError, match="scales"):
        optim.AdamW(p, g, exp_avg_scale=[torch.zeros(1), torch.zeros(1)])
    with pytest.raises(TypeError, match="dtype"):
        optim.AdamW([x.half() for x in p], g)
    with pytest.raises(B.DpError):
        optim.AdamW(p, p)                      # a parameter that is its own gradient
    opt = optim.AdamW(p, g)
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.zeros(2))
    with pytest.raises(ValueError, match="schedule"):
        opt.step(schedule=torch.zeros(2))
    with pytest.raises(B.DpError):
        opt.step(lr=float("nan"))
    assert opt.steps == 0


def test_the_count_of_left_out_steps_checks_its_word():
    rows = [row(), row(1)]
    _, h = B.dp_adamw_create(rows, 2, B.DP_FP32, B.DP_FP32, B.DP_STATE_FP32)
    count = lambda p, h=h: B.dp_adamw_count_skips(h, p, check=False)  # noqa: E731
    assert count(fake(20)) == B.DP_OK and count(None) == B.DP_OK
    assert count(fake(20, 2)) == UNSUPPORTED
    assert count(fake(0, 3996)) == ALIAS and count(fake(0, 4000)) == B.DP_OK
    assert count(fake(9)) == ALIAS                             # a gradient, which is read
    assert count(fake(20), h=0) == INVALID
    B.dp_adamw_destroy(h)
    opt = optim.AdamW([torch.zeros(4)], [torch.zeros(4)])
    assert opt.skipped.tolist() == [0]


def test_steps_on_host_tensors_are_refused():
    g = [torch.zeros(10), torch.zeros(4)]
    opt, norm = optim.AdamW([torch.zeros(10), torch.zeros(4)], g), optim.GradNorm(g)
    for call in (opt.step, norm, lambda: opt.step(stream=0), lambda: norm(stream=0)):
        with pytest.raises(B.DpError, match="tensors on cpu, which is not the current"):
            call()
    assert opt.steps == 0


def test_the_memory_of_a_list_outlives_a_tensor_that_leaves_it():
    """A step writes through the addresses it was made with: their storage is not freed before it."""
    p, g = [torch.zeros(1000), torch.zeros(70)], [torch.ones(1000), torch.ones(70)]
    c, m = [x.bfloat16() for x in p], [torch.zeros_like(x) for x in p]
    was = [t.data_ptr() for ts in (p, g, c, m) for t in ts]
    opt, norm = optim.AdamW(p, g, copies=c, exp_avg=m), optim.GradNorm(g)
    for ts in (p, g, c, m):
        for t in ts:
            t.data = torch.zeros_like(t)
    assert set(was) <= {s.data_ptr() for s in opt._held}
    assert {x for x in was[2:4]} == {s.data_ptr() for s in norm._held}
