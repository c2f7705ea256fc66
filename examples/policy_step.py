"""A data-parallel post-training step, from logits to updated weights, with the operators of this package where a user would call them.

W ranks are played on one GPU, each with its own tokens and gradients.  The model reads a token through an embedding, a stack of
residual blocks x + relu(layer_norm(x) @ A) @ B and a head, all in bf16; its matrix products are torch's.  One step:

  1. forward     layer_norm_forward in every block and before the head
  2. loss        policy_loss on the logits (in place: they become their gradient), or, for pairs of sequences,
                 token_logprob_forward, preference_loss and token_logprob_backward
  3. backward    layer_norm_backward
  4. reduce      allreduce_sum over the ranks' gradient buffers
  5. clip        grad_norm: the norm and clip factor, left on the device
  6. update      muon_step on the blocks' matrices, each rank those that it owns; adamw_step on everything else

Run: python examples/policy_step.py [--loss preference] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import all_gather_amd as mr

EPS, IGNORED = 1e-5, -100


class Model:
    """Embedding, gamma and beta of every norm, A and B of every block, head: views of one flat bf16 buffer."""

    def __init__(self, vocab, width, blocks, gen):
        self.blocks = blocks
        S = torch.Size
        block = [S((width,)), S((width,)), S((width, 2 * width)), S((2 * width, width))]
        self.shapes = [S((vocab, width))] + block * blocks + [S((width,)), S((width,)), S((width, vocab))]
        self.flat = torch.empty(sum(s.numel() for s in self.shapes), dtype=torch.bfloat16, device=gen.device)
        self.params = self.views(self.flat)
        for p in self.params:
            p.normal_(0, p.shape[0] ** -0.5, generator=gen) if p.dim() == 2 else p.zero_()
        self.params[0].normal_(0, 1, generator=gen)
        for i in range(1, len(self.params) - 1, 4):
            self.params[i].fill_(1.0)                              # gamma
        self.matrices = [k for i in range(blocks) for k in (4 * i + 3, 4 * i + 4)]
        self.others = [k for k in range(len(self.params)) if k not in self.matrices]

    def views(self, flat):
        return [p.view(s) for p, s in zip(flat.split([s.numel() for s in self.shapes]), self.shapes)]


def _norm(x, add, gamma, beta):
    """The norm of x + add, with what its backward pass takes."""
    y, xo = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(x.shape[0], device=x.device) for _ in range(2))
    mr.layer_norm_forward([x if add is None else add], gamma, beta, y, eps=EPS, residual=None if add is None else x, x_out=xo,
                          mean=mean, rstd=rstd)
    return y, (xo, mean, rstd)


def forward(m, tokens):
    """Logits of every token, and what the backward pass takes."""
    p, kept = m.params, []
    x, add = p[0][tokens], None
    for i in range(m.blocks):
        gamma, beta, A, B = p[4 * i + 1:4 * i + 5]
        y, stats = _norm(x, add, gamma, beta)
        h = y @ A
        a = torch.relu(h)
        x, add = stats[0], a @ B
        kept.append((y, stats, h, a))
    y, stats = _norm(x, add, p[-3], p[-2])
    kept.append((y, stats))
    return y @ p[-1], kept


def backward(m, tokens, kept, dlogits, grads):
    """Gradients of every parameter, into ``grads``."""
    p = m.params
    y, (xo, mean, rstd) = kept[-1]
    grads[-1].copy_(y.t() @ dlogits)
    g = torch.empty_like(y)
    mr.layer_norm_backward(dlogits @ p[-1].t(), xo, p[-3], mean, rstd, g, dgamma=grads[-3], dbeta=grads[-2])
    for i in reversed(range(m.blocks)):
        gamma, _, A, B = p[4 * i + 1:4 * i + 5]
        y, (xo, mean, rstd), h, a = kept[i]
        grads[4 * i + 4].copy_(a.t() @ g)
        gh = (g @ B.t()) * (h > 0)
        grads[4 * i + 3].copy_(y.t() @ gh)
        gx = torch.empty_like(g)
        mr.layer_norm_backward(gh @ A.t(), xo, gamma, mean, rstd, gx, dgamma=grads[4 * i + 1], dbeta=grads[4 * i + 2], dres=g)
        g = gx
    grads[0].copy_(torch.zeros(p[0].shape, device=g.device).index_add_(0, tokens, g.float()))


def policy(m, batch, grads):
    """[loss, KL, clipped share, weight] of one rank's packed sequences, and their gradients."""
    logits, kept = forward(m, batch["tokens"])
    record = torch.empty(4, device=logits.device)
    mr.policy_loss(logits, batch["targets"], batch["advantages"], record, old_logp=batch["old"], ref_logp=batch["ref"],
                   weights=batch["weights"], dlogits=logits, clip=(0.2, 0.28), kl=0.02)
    backward(m, batch["tokens"], kept, logits, grads)
    return record


def preference(m, batch, grads):
    """[loss, share of pairs ranked right, mean margin] of one rank's pairs, and their gradients."""
    logits, kept = forward(m, batch["tokens"])
    rows = logits.shape[0]
    logp, stats, record = torch.empty(rows, device=logits.device), torch.empty(rows, 2, device=logits.device), torch.empty(3, device=logits.device)
    mr.token_logprob_forward(logits, batch["targets"], logp, stats=stats)
    mr.preference_loss(logp, batch["offsets"], record, ref_logp=batch["ref"], dlogp=logp, beta=0.5)
    mr.token_logprob_backward(logits, batch["targets"], stats, logp, logits)
    backward(m, batch["tokens"], kept, logits, grads)
    return record


def make_batch(m, gen, pairs=4, longest=60):
    """Packed prompts and answers: the targets of prompts carry no loss, and the log-probabilities are the first model's."""
    dev, vocab = gen.device, m.shapes[0][0]
    lens = torch.randint(8, longest, (2 * pairs,), generator=gen, device=dev)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), lens.cumsum(0)])
    n = int(offsets[-1])
    tokens, targets = (torch.randint(0, vocab, (n,), generator=gen, device=dev) for _ in range(2))
    at = torch.arange(n, device=dev)
    seq = torch.searchsorted(offsets, at, right=True) - 1
    targets[at - offsets[seq] < 5] = IGNORED                       # the prompts
    live = targets >= 0
    logp = torch.empty(n, device=dev)
    mr.token_logprob_forward(forward(m, tokens)[0], targets, logp)
    advantages = torch.randn(2 * pairs, generator=gen, device=dev)[seq]
    return dict(tokens=tokens, targets=targets, offsets=offsets, old=logp, ref=logp.clone(), advantages=advantages,
                weights=live.float() / live.sum())


def train(loss="policy", steps=20, W=2, vocab=1000, width=128, blocks=2, seed=0, device="cuda"):
    """The records (mean over ranks) of ``steps`` steps."""
    gen = torch.Generator(device=device).manual_seed(seed)
    m = Model(vocab, width, blocks, gen)
    one = {"policy": policy, "preference": preference}[loss]
    batches = [make_batch(m, gen) for _ in range(W)]
    rank_grads = [torch.empty_like(m.flat) for _ in range(W)]
    total, clip = torch.empty_like(m.flat), torch.empty(3, device=device)
    tv = m.views(total)
    pick = lambda t, ks: [t[k] for k in ks]  # noqa: E731
    # each rank updates the matrices that it owns; parameters, gradients and states stay in place: marshalled once
    norm = mr.prepare_grad_norm([total], clip, max_norm=1.0, scale=1.0 / W)
    muon = [mr.prepare_muon(pick(m.params, own), pick(tv, own), mr.muon_init(pick(m.params, own), master=True), weight_decay=0.01,
                            adjust="rms", clip=clip) for own in (m.matrices[r::W] for r in range(W))]
    others = pick(m.params, m.others)
    adam = mr.prepare_adamw(others, pick(tv, m.others), mr.adamw_init(others, bits=8, master=True), weight_decay=0.0, clip=clip)
    records = []
    for step in range(1, steps + 1):
        records.append(torch.stack([one(m, b, m.views(g)) for b, g in zip(batches, rank_grads)]).mean(dim=0))
        mr.allreduce_sum(rank_grads, total)
        norm()
        for update in muon:
            update(lr=3e-3)
        adam(lr=1e-3, step=step)
    return torch.stack(records).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--loss", default="policy", choices=("policy", "preference"))
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    for i, x in enumerate(train(a.loss, a.steps), 1):
        print(f"step {i:4d}  " + "  ".join(f"{v:.5f}" for v in x), flush=True)
