"""The policy loss's terms where an exponential passes fp32's range, against the formulas in 64 bits, on every path.

Tolerances.  A log-probability is off by at most 2^-16 (test_loss_gpu.py), and exp of a difference of x by as much of itself, by 2^-24 |x|
for the argument's rounding to fp32 (|x| <= 100: 6e-6) and by 2^-20 for expf's error in the eighth power: 2.3e-5 < 2^-15 together."""
import pytest
import torch

import all_gather_amd as mr
from gpu_util import device
from test_loss_gpu import S_TOL, case, check_gradient, exact_gradient, exact_logp, exact_policy

pytestmark = pytest.mark.gpu

# one workgroup a row in registers; rows over several workgroups and a second launch for the gradient; rows that are too long
PATHS = [(300, 100), (40, 4099), (8, 131072), (300, 140000)]
REL = 2.0 ** -15


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", PATHS)
@pytest.mark.parametrize("kl", [0.0, 1e-6])
def test_differences_past_fp32_range(rows, cols, dtype, kl):
    print(f"[case] {rows}x{cols} {dtype} kl={kl}", flush=True)
    z, t, rand = case(rows, cols, dtype, seed=21, dead=0.1)
    lp, _, live = exact_logp(z, t, 1.0)
    i = torch.arange(rows, device=device())
    adv = rand(rows)
    old, ref = (lp + 0.05 * rand(rows).clamp(-2, 2)).float(), (lp + 0.3 * rand(rows)).float()
    far = i % 4 == 0
    ref = torch.where(far, lp + 100.0, lp + (ref.double() - lp)).float()      # exp(100) = 2.7e43
    none = i % 4 == 1
    old = torch.where(none, lp - 100.0, old.double()).float()                 # a ratio of 2.7e43 ...
    adv = torch.where(none, 0.0, adv)                                         # ... of a token without an advantage
    cut = i % 4 == 2
    old = torch.where(cut, lp - 95.0, old.double()).float()                   # clipped
    adv = torch.where(cut, adv.abs() + 0.1, adv)
    w = torch.where(far, 1e-20, 1.0) if kl else None                          # the KL term's gradient is an fp32 number
    want, p, on, g, size, sums, sizes = exact_policy(z, t, adv, old, ref, w, (0.2, 0.3), kl, 1.0)
    assert torch.isfinite(g).all() and float(g.abs().max()) < 1e20
    # a clipped ratio leaves the clipped term alone, with no error of its own
    r, a, ww = torch.exp(lp - old.double()), adv.double(), 1.0 if w is None else w.double()
    term = torch.maximum(-a * r, -a * r.clamp(0.8, 1.3)).abs() + kl * (torch.expm1(ref.double() - lp).abs() + 1)
    sizes[0] = torch.where(on, ww * term, 0.0).sum()
    for grad in (True, False):
        out = torch.empty_like(z)
        logp, record = torch.empty(rows, device=device()), torch.empty(4, device=device())
        mr.policy_loss(z, t, adv, record, old_logp=old, ref_logp=ref, weights=w, clip=(0.2, 0.3), kl=kl, logp=logp, dlogits=out if grad else None)
        assert ((logp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        big = torch.finfo(torch.float32).max
        for k in (0, 1, 2, 3):                                                # the divergence's sum may pass fp32: infinite then
            if float(sums[k]) > big:
                assert float(record[k]) == float("inf"), k
            else:
                assert abs(float(record[k]) - float(sums[k])) <= REL * float(sizes[k]) + 2.0 ** -23 * abs(float(sums[k])), (k, record, sums)
        if grad:
            # where the ratio is clipped nothing of it passes: only what passes carries its error.  Where the two terms cancel
            # the KL term's size counts, below 8 kl w in rows of small differences (exp(d) < 7)
            kept = g.abs() + 8 * kl * (0.0 if w is None else w.double())
            check_gradient(out, exact_gradient(p, t, on, g, 1.0), p, t, on, kept, 1.0, dtype, more=REL)


@pytest.mark.parametrize("rows,cols", PATHS)
def test_small_differences_keep_their_bits(rows, cols):
    """A divergence that is reported and one that is not asked for: the same loss and the same gradient."""
    z, t, rand = case(rows, cols, "bf16", seed=22)
    lp = exact_logp(z, t, 1.0)[0]
    old, ref, adv = (lp + 0.2 * rand(rows)).float(), (lp + 0.4 * rand(rows)).float(), rand(rows)
    a, b = torch.empty(4, device=device()), torch.empty(4, device=device())
    da, db = torch.empty_like(z), torch.empty_like(z)
    mr.policy_loss(z, t, adv, a, old_logp=old, ref_logp=ref, kl=0.0, dlogits=da)
    mr.policy_loss(z, t, adv, b, old_logp=old, kl=0.0, dlogits=db)
    assert torch.equal(da, db) and torch.equal(a[[0, 2, 3]], b[[0, 2, 3]]) and float(a[1]) > 0 and float(b[1]) == 0


@pytest.mark.parametrize("rows,cols", PATHS)
def test_a_ruled_out_target_under_its_own_policy(rows, cols):
    """Without old_logp the ratio is 1 in every row, also where the target's logit is -inf: a loss of -A, and the gradient that r = 1 gives."""
    z, t, rand = case(rows, cols, "fp32", seed=23, dead=0.0)
    z[2, 5], t[2] = -float("inf"), 5
    z[3], t[3] = -float("inf"), 5                    # nothing left in the row: NaN
    adv = rand(rows)
    for grad in (True, False):
        w = torch.ones(rows, device=device())
        w[3] = 0.0
        record, logp, out = torch.empty(4, device=device()), torch.empty(rows, device=device()), torch.empty_like(z)
        mr.policy_loss(z, t, adv, record, weights=w, logp=logp, dlogits=out if grad else None)
        assert float(logp[2]) == -float("inf")
        want = -adv.double()[w != 0].sum()
        assert abs(float(record[0]) - float(want)) <= 2.0 ** -23 * float(adv.double().abs().sum()) and float(record[2]) == 0
        if grad:
            lp, p, live = exact_logp(z, t, 1.0)
            live = live & (w != 0)
            g, p = torch.where(live, -adv.double(), 0.0), torch.where(live[:, None], p, 0.0)  # (a row of nothing has no probabilities)
            check_gradient(out, exact_gradient(p, t, live, g, 1.0), p, t, live, g, 1.0, "fp32")
        w[3] = 1.0
        mr.policy_loss(z, t, adv, record, weights=w)
        assert record[0].isnan() and float(record[3]) == rows
