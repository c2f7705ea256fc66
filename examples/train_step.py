"""A sharded data-parallel training step with every operator of this package where a user would call it.

W ranks are played on one GPU, each with its own shard, gradients and microbatch, as the collectives' rank buffers are
separate allocations.  The model is a stack of residual blocks x + relu(layer_norm(x) @ A) @ B in bf16 that learns a
fixed random map; its matrix products are torch's.  One step:

  1. gather      allgather_param_contig_shards: W parameter shards -> every parameter whole
  2. forward     layer_norm_forward, which also adds the previous block's output to the residual stream
  3. backward    layer_norm_backward, with the residual stream's own gradient and the weights' gradients
  4. reduce      allreduce_sum over the ranks' gradient buffers (fp32 accumulation in rank order)
  5. clip        grad_norm: the mean gradient's norm and clip factor, left on the device
  6. update      adamw_step on each rank's pieces of every parameter: moments in 8 or 32 bits, fp32 master copies

Run: python examples/train_step.py [--bits 8] [--steps 100]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import all_gather_amd as mr

EPS = 1e-5


class Sharded:
    """Parameters as W flat bf16 shards, gathered into one buffer in which every parameter is whole."""

    def __init__(self, shapes, W, gen):
        self.W, self.shapes = W, shapes
        dev = gen.device
        self.splits = [s.numel() // W for s in shapes]           # elements of a parameter on one rank
        assert all(n * W == s.numel() for n, s in zip(self.splits, shapes))
        self.full = torch.empty(W * sum(self.splits), dtype=torch.bfloat16, device=dev)
        self.params = [p.view(s) for p, s in zip(self.full.split([n * W for n in self.splits]), shapes)]
        self.shards = [torch.empty(sum(self.splits), dtype=torch.bfloat16, device=dev) for _ in range(W)]
        for i, (p, s) in enumerate(zip(self.params, shapes)):    # gamma, beta, A, B of every block
            p.fill_(1.0 if i % 4 == 0 else 0.0) if len(s) == 1 else p.normal_(0, s[0] ** -0.5, generator=gen)
        for r in range(W):
            for mine, piece in zip(self.shards[r].split(self.splits), self.pieces(self.full, r)):
                mine.copy_(piece)

    def pieces(self, full, r):
        """Rank r's piece of every parameter in a buffer laid out like ``full``."""
        return [p[r * n:(r + 1) * n] for p, n in zip(full.split([n * self.W for n in self.splits]), self.splits)]

    def gather(self):
        mr.allgather_param_contig_shards(self.shards, self.W, self.splits, self.full)


def forward_backward(params, x, target, grads, blocks):
    """Loss of one microbatch; its gradients go to ``grads`` (views shaped like ``params``)."""
    rows, d = x.shape
    dev, kept = x.device, []
    stream, add = x, None                                        # the residual stream and what is still to be added to it
    for i in range(blocks):
        gamma, beta, A, B = params[4 * i:4 * i + 4]
        y, xo = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        terms = [stream] if add is None else [add]
        mr.layer_norm_forward(terms, gamma, beta, y, eps=EPS, residual=None if add is None else stream, x_out=xo, mean=mean,
                              rstd=rstd)
        h = y @ A
        a = torch.relu(h)
        add = a @ B
        kept.append((y, xo, mean, rstd, h, a))
        stream = xo
    diff = (stream + add).float() - target
    loss = (diff * diff).mean()
    g = (diff * (2.0 / diff.numel())).to(torch.bfloat16)          # gradient of the stream and of the last block's output
    for i in reversed(range(blocks)):
        gamma, beta, A, B = params[4 * i:4 * i + 4]
        y, xo, mean, rstd, h, a = kept[i]
        grads[4 * i + 3].copy_(a.t() @ g)
        gh = (g @ B.t()) * (h > 0)
        grads[4 * i + 2].copy_(y.t() @ gh)
        gx = torch.empty_like(g)
        mr.layer_norm_backward(gh @ A.t(), xo, gamma, mean, rstd, gx, dgamma=grads[4 * i], dbeta=grads[4 * i + 1], dres=g)
        g = gx
    return loss


def train(steps=100, bits=8, W=4, rows=512, width=256, blocks=3, lr=2e-3, seed=0, device="cuda"):
    """The losses (mean over ranks) of ``steps`` steps."""
    gen = torch.Generator(device=device).manual_seed(seed)
    S = torch.Size
    shapes = [S((width,)), S((width,)), S((width, 2 * width)), S((2 * width, width))] * blocks
    model = Sharded(shapes, W, gen)
    teacher = torch.randn(width, width, generator=gen, device=device) * width ** -0.5
    data = [torch.randn(rows, width, generator=gen, device=device) for _ in range(W)]
    targets = [x + torch.tanh(x @ teacher) for x in data]
    inputs = [x.to(torch.bfloat16) for x in data]
    rank_grads = [torch.empty_like(model.full) for _ in range(W)]
    rank_views = [[p.view(s) for p, s in zip(g.split([n * W for n in model.splits]), shapes)] for g in rank_grads]
    total, record = torch.empty_like(model.full), torch.empty(3, device=device)
    mine = [list(sh.split(model.splits)) for sh in model.shards]
    states = [mr.adamw_init(p, bits=bits, master=True) for p in mine]
    # parameters, gradients and state stay in place from step to step: marshalled once
    clip = mr.prepare_grad_norm([total], record, max_norm=1.0, scale=1.0 / W)
    update = [mr.prepare_adamw(mine[r], model.pieces(total, r), states[r], weight_decay=0.01, clip=record, seed=seed + r)
              for r in range(W)]
    losses = []
    for step in range(1, steps + 1):
        model.gather()
        loss = [forward_backward(model.params, inputs[r], targets[r], rank_views[r], blocks) for r in range(W)]
        mr.allreduce_sum(rank_grads, total)
        clip()
        for u in update:
            u(lr=lr, step=step)
        losses.append(torch.stack(loss).mean())
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    for i, x in enumerate(train(a.steps, a.bits), 1):
        if i == 1 or i % 10 == 0:
            print(f"step {i:4d}  loss {x:.5f}", flush=True)
