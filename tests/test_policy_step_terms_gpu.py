"""The example's gradients with one term of its loss at a time, against torch's own derivative in 64 bits: a term that was lost, or that had
another sign or size, is most of the gradient here."""
import pytest
import torch

from gpu_util import device
from test_policy_step_gpu import ex, exact  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("term", ["kl", "ratio", "clipped", "preference"])
def test_one_term(ex, term):  # noqa: F811
    gen = torch.Generator(device=device()).manual_seed(5)
    m = ex.Model(501, 64, 2, gen)
    batch = ex.make_batch(m, gen)
    live = batch["targets"] >= 0
    n = live.numel()
    if term == "kl":                                 # no advantages: the KL term's gradient alone, of either sign
        batch["advantages"] = torch.zeros(n, device=device())
        batch["ref"] = torch.where(live, batch["ref"] + torch.where(torch.arange(n, device=device()) % 3 == 0, 2.0, -2.0), 0.0)
    elif term == "clipped":                          # ratios far past both borders, so that no rounding decides: half of them are held
        batch["old"] = torch.where(live, batch["old"] + torch.where(torch.arange(n, device=device()) % 2 == 0, 1.0, -1.0), 0.0)
    elif term == "preference":                       # margins apart from 0: each pair's weight differs
        batch["ref"] = torch.where(live, batch["ref"] + 0.2 * torch.randn(n, generator=gen, device=device()), 0.0)
    loss = "preference" if term == "preference" else "policy"
    grads = m.views(torch.empty_like(m.flat))
    record = getattr(ex, loss)(m, batch, grads)
    value, want = exact(ex, m, batch, loss)
    # bf16 activations and gradients: about a dozen roundings of 2^-9 in a row between a logit and a weight's gradient, each raised
    # at most a few times by the layers behind it
    assert abs(float(record[0]) - value) <= 2.0 ** -4 * (abs(value) + 0.02)
    if term == "clipped":
        assert 0.2 < float(record[2]) < 0.8
    for i, (g, w) in enumerate(zip(grads, want)):
        assert float(w.norm()) > 0 and float((g.double() - w).norm()) <= 2.0 ** -3 * float(w.norm()), (i, float((g.double() - w).norm() / w.norm()))
