"""The operators of a post-training step together, as the example runs them: norms, losses on logits, reduction, clipping, Muon and
AdamW; and the example's gradients against torch's own derivative of the same model in 64 bits."""
import importlib.util
import math
import os

import pytest
import torch

import all_gather_amd as mr
from gpu_util import device

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("policy_step_example", os.path.join(ROOT, "examples", "policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def exact(ex, m, batch, loss):
    """The model, its loss and the gradients by torch in 64 bits."""
    p = [x.double().requires_grad_(True) for x in m.params]
    norm = lambda x, k: torch.nn.functional.layer_norm(x, x.shape[1:], p[k], p[k + 1], ex.EPS)  # noqa: E731
    x = p[0][batch["tokens"]]
    for i in range(m.blocks):
        x = x + torch.relu(norm(x, 4 * i + 1) @ p[4 * i + 3]) @ p[4 * i + 4]
    z = norm(x, len(p) - 3) @ p[-1]
    t = batch["targets"]
    live = t >= 0
    lp = torch.where(live, torch.log_softmax(z, dim=1).gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0)
    ref = batch["ref"].double()
    if loss == "policy":
        adv, w = batch["advantages"].double(), batch["weights"].double()
        r, d = torch.exp(lp - batch["old"].double()), ref - lp
        value = (w * (torch.maximum(-adv * r, -adv * r.clamp(0.8, 1.28)) + 0.02 * (torch.exp(d) - d - 1))).sum()
    else:
        off = batch["offsets"].tolist()
        s = torch.stack([(lp - ref)[a:b].sum() for a, b in zip(off, off[1:])])
        value = -torch.nn.functional.logsigmoid(0.5 * (s[0::2] - s[1::2])).mean()
    return float(value.detach()), torch.autograd.grad(value, p)


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_gradients(ex, loss):
    gen = torch.Generator(device=device()).manual_seed(3)
    m = ex.Model(501, 64, 2, gen)
    batch = ex.make_batch(m, gen)
    batch["old"] = batch["old"] + 0.1 * torch.randn(batch["old"].shape, generator=gen, device=device())
    batch["ref"] = torch.where(batch["targets"] >= 0, batch["ref"] + 0.2 * torch.randn(batch["ref"].shape, generator=gen, device=device()), 0.0)
    r = torch.exp(batch["ref"] - batch["old"])
    grads = m.views(torch.empty_like(m.flat))
    record = getattr(ex, loss)(m, batch, grads)
    value, want = exact(ex, m, batch, loss)
    # bf16 activations and gradients: about a dozen roundings of 2^-9 in a row between a logit and a weight's gradient, each
    # raised at most a few times by the layers behind it; and a token whose ratio is near a border may fall on its other side
    assert abs(float(record[0]) - value) <= 2.0 ** -4 * (abs(value) + 1) and torch.isfinite(r).all()
    for i, (g, w) in enumerate(zip(grads, want)):
        assert float((g.double() - w).norm()) <= 2.0 ** -3 * float(w.norm()), (i, float((g.double() - w).norm() / w.norm()))


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_runs_and_repeats(ex, loss):
    a, b = ex.train(loss, steps=4), ex.train(loss, steps=4)
    assert all(math.isfinite(v) for r in a for v in r)
    if loss == "policy":
        assert all(abs(r[3] - 1) < 1e-5 for r in a)                # the weights of a rank add up to one
    # index_add_ and torch's products may sum in another order: the first step's forward pass does not
    assert abs(a[0][0] - b[0][0]) <= 2.0 ** -7 * (abs(a[0][0]) + 2.0 ** -10)


def test_steps_beside_each_other_and_captured(ex):
    """One captured step (loss, reduction, norm, Muon), replayed, beside the same step run eagerly on another stream: the same bits
    every time."""
    gen = torch.Generator(device=device()).manual_seed(9)
    rows, cols, W = 300, 2003, 3
    logits = [torch.randn(rows, cols, generator=gen, device=device()).bfloat16() for _ in range(W)]
    targets = torch.randint(0, cols, (rows,), generator=gen, device=device())
    adv = torch.randn(rows, generator=gen, device=device())

    def make():
        d = dict(dz=[torch.empty_like(z) for z in logits], rec=torch.empty(4, device=device()), total=torch.empty_like(logits[0]),
                 clip=torch.empty(3, device=device()), p=[torch.zeros(rows, cols, dtype=torch.bfloat16, device=device())])
        d["st"] = mr.muon_init(d["p"])
        return d

    def step(d):
        for z, dz in zip(logits, d["dz"]):
            mr.policy_loss(z, targets, adv, d["rec"], dlogits=dz)
        mr.allreduce_sum(d["dz"], d["total"])
        mr.grad_norm([d["total"]], d["clip"], max_norm=1.0)
        mr.muon_step(d["p"], [d["total"]], d["st"], 0.02, clip=d["clip"])

    a, b = make(), make()
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(a)
    a["p"][0].zero_()
    a["st"].m.zero_()
    for i in range(4):
        for z in logits:
            z.copy_(torch.randn(rows, cols, generator=gen, device=device()))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["rec"], b["rec"]) and torch.equal(a["total"], b["total"]) and torch.equal(a["clip"], b["clip"]), i
        assert torch.equal(a["p"][0], b["p"][0]) and torch.equal(a["st"].m, b["st"].m), i
