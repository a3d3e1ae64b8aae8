"""The optimizer step on the reduced gradients: the global gradient norm with
its clip coefficient, and AdamW with 32- or 8-bit states over a list of
tensors.  The tensors are those of a training step: parameter shards with the
gradients that a reduce-scatter or the Reducer leaves in place each step, so
each object takes them once and a step passes no lists.  It works on the memory
that they have when it is made, and keeps that memory: a tensor that is given
other storage later (``p.data = ...``, ``module.to(...)``) is not followed.

    clip = GradNorm(grads, max_norm=1.0)
    opt = AdamW(params, grads, lr=3e-4, states="8bit", copies=bf16_shards)
    ...
    norm, coef = clip()
    opt.step(grad_scale=coef)

No arithmetic happens here: it allocates with PyTorch and calls the binding.
"""
from __future__ import annotations


import torch

from . import binding as B
from .collectives import _code

_STATES = {"f32": B.DP_STATE_FP32, "8bit": B.DP_STATE_8BIT}


def _check_list(name, ts, numels=None, dtype=None, device=None):
    """One dtype and device, contiguous, and the sizes of the parameters."""
    ts = list(ts)
    if not ts:
        raise ValueError(f"{name}: need at least one tensor")
    dtype, device = dtype or ts[0].dtype, device or ts[0].device
    if numels is not None and len(ts) != len(numels):
        raise ValueError(f"{name}: {len(ts)} tensors for {len(numels)} parameters")
    for i, t in enumerate(ts):
        if t.dtype != dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name}[{i}]: need contiguous {dtype} tensors on {device}")
        if numels is not None and t.numel() != numels[i]:
            raise ValueError(f"{name}[{i}]: {t.numel()} elements, the parameter needs {numels[i]}")
    return ts


def _storages(*lists):
    """What the addresses of some tensors point into, kept from being freed when a
    tensor is given other storage (``p.data = ...``, ``module.to(...)``)."""
    return [t.untyped_storage() for ts in lists if ts is not None for t in ts]


class GradNorm:
    """The global norm of a list of gradients and its clip coefficient.

    Calling it enqueues one pass over the gradients and returns two device
    tensors of one float: the norm, and min(1, max_norm / (norm + 1e-6)) -- NaN
    when the norm is not finite, which makes ``AdamW.step`` leave everything as
    it is.  Every call writes the same two tensors; calls that overlap on the
    GPU need an object each.
    """

    def __init__(self, grads, max_norm: float = float("inf")):
        self.grads = _check_list("grads", grads)
        self.max_norm = float(max_norm)
        dev = self._device = self.grads[0].device
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.coef = torch.ones(1, dtype=torch.float32, device=dev)
        self._n = len(self.grads)
        self._ws = torch.zeros(B.dp_grad_norm_workspace_size(self._n), dtype=torch.uint8,
                               device=dev)
        self._dtype = _code(self.grads[0])
        self._ptrs = B._parray(self.grads)
        self._held = _storages(self.grads)
        self._numels = B._sizes(g.numel() for g in self.grads)

    def __call__(self, stream=None):
        here = B._stream_on(self._device, "GradNorm")
        B.dp_grad_norm(self._ptrs, self._numels, self._n, self._dtype, self.max_norm, self.norm,
                       self.coef, self._ws, stream=here if stream is None else stream)
        return self.norm, self.coef


class AdamW:
    """AdamW over a list of parameters in one launch (per 384 tensors).

    ``params``: fp32 or bf16, updated in place; ``grads``: fp32 or bf16, read by
    every step.  ``weight_decay``: a number, or one for each parameter.
    ``copies``: bf16 tensors that receive the new parameters rounded (the
    compute copy of fp32 masters).

    States, allocated here as zeros or taken over (a resumed run, with
    ``step`` the number of steps already taken):

    * ``states="f32"``: ``exp_avg`` and ``exp_avg_sq``, fp32;
    * ``states="8bit"``: ``exp_avg`` and ``exp_avg_sq`` are float8_e4m3fn codes
      of m and of sqrt(v), with ``exp_avg_scale`` / ``exp_avg_sq_scale``, one
      fp32 scale for each 256 elements of a tensor.  Made for beta2 of 0.95 or
      less: nearer to 1 (the default among them) a step's change of v is below
      the codes' rounding, and stored roots stay several times too large where
      gradients shrink (figures: ``include/dp.h``).

    ``steps`` counts the calls of ``step``; ``skipped``, one int32 on the device,
    those that a NaN coefficient left out, which the bias corrections do not
    count.  A run is resumed with ``step = opt.steps - int(opt.skipped)``.
    """

    def __init__(self, params, grads, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, states: str = "f32", copies=None, exp_avg=None,
                 exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None, step: int = 0):
        self.handle = 0
        if states not in _STATES:
            raise ValueError(f"states: 'f32' or '8bit', not {states!r}")
        self.params = _check_list("params", params)
        numels = [p.numel() for p in self.params]
        dev = self._device = self.params[0].device
        self.grads = _check_list("grads", grads, numels, device=dev)
        self.copies = None if copies is None else \
            _check_list("copies", copies, numels, torch.bfloat16, dev)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else \
            [float(weight_decay)] * len(numels)
        if len(decay) != len(numels):
            raise ValueError(f"weight_decay: {len(decay)} values for {len(numels)} parameters")
        eight = states == "8bit"
        sdt = torch.float8_e4m3fn if eight else torch.float32
        blocks = [-(-n // B.DP_STATE_BLOCK) for n in numels]

        def kept(name, given, sizes, dt):
            if given is None:
                return [torch.zeros(n, dtype=torch.uint8 if dt == torch.float8_e4m3fn else dt,
                                    device=dev).view(dt) for n in sizes]
            return _check_list(name, given, sizes, dt, dev)

        self.exp_avg = kept("exp_avg", exp_avg, numels, sdt)
        self.exp_avg_sq = kept("exp_avg_sq", exp_avg_sq, numels, sdt)
        if not eight and (exp_avg_scale is not None or exp_avg_sq_scale is not None):
            raise ValueError("scales belong to 8-bit states")
        self.exp_avg_scale = kept("exp_avg_scale", exp_avg_scale, blocks, torch.float32) \
            if eight else None
        self.exp_avg_sq_scale = kept("exp_avg_sq_scale", exp_avg_sq_scale, blocks,
                                     torch.float32) if eight else None
        self.lr, self.betas, self.eps, self.steps = lr, tuple(betas), eps, int(step)
        self._held = _storages(self.params, self.grads, self.copies, self.exp_avg,
                               self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)
        none = [None] * len(numels)
        rows = list(zip(self.params, self.grads, self.copies or none, self.exp_avg,
                        self.exp_avg_sq, self.exp_avg_scale or none,
                        self.exp_avg_sq_scale or none, numels, decay))
        _, self.handle = B.dp_adamw_create(rows, len(rows), _code(self.params[0]),
                                           _code(self.grads[0]), _STATES[states])
        self.skipped = torch.zeros(1, dtype=torch.int32, device=dev)
        B.dp_adamw_count_skips(self.handle, self.skipped)

    def step(self, lr=None, grad_scale=None, schedule=None, stream=None) -> None:
        """One step.  ``lr`` replaces the constructor's for this step;
        ``grad_scale``: a device float that multiplies the gradients
        (``GradNorm``'s coefficient); ``schedule``: three device floats (lr,
        1 - beta1^t, 1 - beta2^t) read when the kernel runs, for a step that is
        captured in a graph and replayed."""
        for name, t, n in (("grad_scale", grad_scale, 1), ("schedule", schedule, 3)):
            if t is not None and (t.dtype != torch.float32 or t.numel() != n or
                                  t.device != self._device or not t.is_contiguous()):
                raise ValueError(f"{name}: {n} fp32 value(s) on {self._device}")
        here = B._stream_on(self._device, "AdamW.step")
        B.dp_adamw_step(self.handle, self.lr if lr is None else lr, self.betas[0], self.betas[1],
                        self.eps, self.steps + 1, grad_scale, schedule,
                        here if stream is None else stream)
        self.steps += 1

    def __del__(self):
        h = getattr(self, "handle", 0)
        if h:
            self.handle = 0
            B.dp_adamw_destroy(h)
