"""A sharded training step with 4-bit products and 8-bit optimizer states.

Two linear layers with a ReLU between them, trained over K virtual
data-parallel ranks on a fixed synthetic regression.  Each layer's weight lives
as K shards: an fp32 master, its bf16 copy, 8-bit AdamW states, and the 4-bit
form that the products gather.  One step:

    forward    y_r = relu(x_r . w1^T) . w2^T        4-bit all-gather products
    backward   dh_r = dy_r . w2                     4-bit, w2's shards gathered transposed
               dw = mean over ranks of dy_r^T x_r   bf16 GEMM fused with its reduce-scatter
    step       global norm -> clip -> AdamW on every rank's shards, in one launch each
    publish    bf16 copies -> 4-bit shards

    python examples/sharded_step.py [--steps 60] [--format nvfp4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from ring_allreduce_gradient_gb300 import binding, mx4, optim  # noqa: E402
from ring_allreduce_gradient_gb300 import collectives as col  # noqa: E402


class ShardedLinear:
    """y = x . w^T, w [F, D] as K row shards."""

    def __init__(self, K, F, D, format, gen, device):
        w = torch.randn(F, D, device=device, generator=gen) * D ** -0.5
        self.format = format
        self.master = [s.clone() for s in w.chunk(K)]
        self.copy = [s.to(torch.bfloat16) for s in self.master]
        self.grad = [torch.zeros_like(s) for s in self.master]
        self.publish()

    def scale(self, x):
        """An nvfp4 tensor scale; mxfp4 has none."""
        return mx4.tensor_scale(x) if self.format == "nvfp4" else None

    def publish(self):
        """The 4-bit shards of the current weights, as they are and transposed."""
        s = self.scale(self.copy)
        self.w4 = [mx4.quantize(w, self.format, s) for w in self.copy]
        self.w4_t = mx4.quantize(self.copy, self.format, s, transpose=True)

    def forward(self, x):
        return mx4.linear(x, self.w4, self.scale(x))

    def backward_input(self, dy):
        """dx = dy . w through the transposed shards, for dy of every rank."""
        return mx4.linear(dy, [self.w4_t], self.scale(dy))

    def backward_weight(self, dys, xs):
        for g, s in zip(self.grad, col.wgrad_reduce_scatter(dys, xs, dw_dtype=torch.float32)):
            g.copy_(s)


def run(steps=60, format="nvfp4", K=8, tokens=256, D=256, H=512, F=256, seed=0, report=None):
    """Trains for `steps` steps; returns the mean loss of each."""
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(seed)
    xs = [torch.randn(tokens, D, device=dev, generator=gen).bfloat16() for _ in range(K)]
    true = torch.randn(F, D, device=dev, generator=gen) * D ** -0.5
    target = [torch.relu(x.float() @ true.t()) for x in xs]
    layers = [ShardedLinear(K, H, D, format, gen, dev), ShardedLinear(K, F, H, format, gen, dev)]
    one, two = layers
    grads = [g for m in layers for g in m.grad]
    clip = optim.GradNorm(grads, max_norm=1.0)
    opt = optim.AdamW([w for m in layers for w in m.master], grads, lr=3e-3, betas=(0.9, 0.95),
                      weight_decay=0.01, states="8bit", copies=[c for m in layers for c in m.copy])
    losses = []
    for step in range(steps):
        hs, dys, dhs, loss = [], [], [], 0.0
        for x, t in zip(xs, target):
            h = torch.relu(one.forward(x))
            err = two.forward(h).float() - t
            loss = loss + err.square().mean() / K
            dy = (err * (2.0 / err.numel())).bfloat16()
            hs.append(h)
            dys.append(dy)
            dhs.append(two.backward_input(dy) * (h > 0))
        two.backward_weight(dys, hs)
        one.backward_weight(dhs, xs)
        norm, coef = clip()
        opt.step(grad_scale=coef)
        for m in layers:
            m.publish()
        losses.append(float(loss))
        if report:
            report(f"step {step:3d}  loss {losses[-1]:.5f}  gradient norm {float(norm):.4f}")
    status = binding.dp_get_device_error()
    if status != binding.DP_OK:
        raise binding.DpError(status, "sharded step")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--format", choices=sorted(mx4.FORMATS), default="nvfp4")
    a = ap.parse_args()
    run(a.steps, a.format, report=print)
