"""The losses' row loops in their steady state, against the formulas in 64 bits: many rows a workgroup, live and ignored ones mixed, for
every number of packs a lane that holds a row, and the statistics' loops over several rows.  Tolerances are test_loss_gpu.py's."""
import pytest
import torch

import all_gather_amd as mr
from gpu_util import device
from test_logit_rows import held_row
from test_loss_gpu import P_TOL, S_TOL, case, check_gradient, exact_gradient, exact_logp, exact_policy

pytestmark = pytest.mark.gpu

CLIP, KL = (0.2, 0.3), 0.05
# dtype, columns on the 16-byte grid and off it, rows: a compute unit holds 16 or 24 waves, so one-wave rows need 3 x 4096 and more
HELD = [("bf16", 504, 501, 13000, 1), ("fp16", 1000, 1001, 12500, 2), ("bf16", 2000, 2001, 13001, 4), ("fp16", 2800, 2801, 13000, 6),
        ("bf16", 4000, 4001, 12400, 8), ("fp16", 5000, 5003, 12400, 10), ("bf16", 6000, 6007, 12400, 12), ("fp16", 7000, 7001, 12400, 14),
        ("bf16", 8000, 8009, 12400, 16), ("bf16", 50000, 50001, 2000, 14), ("fp16", 131072, 131063, 900, 16), ("bf16", 98304, 98299, 900, 16),
        ("fp32", 252, 250, 13000, 1), ("fp32", 500, 501, 12500, 2), ("fp32", 1000, 1001, 13001, 4), ("fp32", 1400, 1401, 13000, 6),
        ("fp32", 2000, 2001, 12400, 8), ("fp32", 2500, 2503, 12400, 10), ("fp32", 3000, 3001, 12400, 12), ("fp32", 3500, 3503, 12400, 14),
        ("fp32", 4000, 4005, 12400, 16), ("fp32", 25000, 25003, 2000, 14), ("fp32", 65536, 65533, 900, 16), ("fp32", 49152, 49149, 900, 16)]


def vectors(z, t, rand, temp):
    rows = z.shape[0]
    lp = exact_logp(z, t, temp)[0]
    old, ref = (lp + 0.4 * rand(rows)).float(), (lp + 0.5 * rand(rows)).float()
    r = torch.exp(lp - old.double())
    near = ((r - 0.8).abs() < 1e-4) | ((r - 1.3).abs() < 1e-4)      # no ratio within its own error of a border
    old = torch.where(near, old + 0.01, old)
    w = (rand(rows).abs() + 0.1) * (torch.arange(rows, device=device()) % 5 != 3)
    return rand(rows), old, ref, w


@pytest.mark.parametrize("dtype,on,off,rows,packs", HELD)
def test_policy_rows_one_after_another(dtype, on, off, rows, packs):
    V = 4 if dtype == "fp32" else 8
    for cols, pad, shift, temp in ((on, 0, 0, 1.0), (off, 3, 1, 0.8)):
        print(f"[case] policy {rows}x{cols} (+{pad}) {dtype}", flush=True)
        waves, K = held_row(rows, cols, V, pad == 0)
        per_cu = min(16, (24 if K <= 4 else 16) // waves)
        assert K == packs and rows > 3 * 256 * per_cu               # the shape under test, and what makes a workgroup walk rows
        z, t, rand = case(rows, cols, dtype, pad, shift, seed=31, dead=0.25)
        adv, old, ref, w = vectors(z, t, rand, temp)
        want, p, live, g, size, sums, sizes = exact_policy(z, t, adv, old, ref, w, CLIP, KL, temp)
        args = dict(old_logp=old, ref_logp=ref, weights=w, clip=CLIP, kl=KL, temperature=temp, grad_scale=8.0)
        flat = torch.full((shift + rows * (cols + pad),), 5.0, dtype=z.dtype, device=device())
        out = flat[shift:].view(rows, cols + pad)[:, :cols]
        logp, record = torch.full((rows,), 9.0, device=device()), torch.full((4,), 9.0, device=device())
        mr.policy_loss(z, t, adv, record, logp=logp, dlogits=out, **args)
        assert ((logp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        assert ((record.double() - sums).abs() <= 2.0 ** -15 * sizes + 2.0 ** -23 * sums.abs()).all(), (record, sums)
        gs = g * 8.0
        check_gradient(out, exact_gradient(p, t, live, gs, temp), p, t, live, size * 8.0, temp, dtype, more=2.0 ** -15)
        if pad:
            assert (flat[shift:].view(rows, cols + pad)[:, cols:] == 5.0).all() and (flat[:shift] == 5.0).all()
        del p
        again = torch.empty_like(record)
        mr.policy_loss(z, t, adv, again, dlogits=z, **args)          # in place
        assert torch.equal(z, out) and torch.equal(again, record)


# one wave a row, many rows; several waves (256 and 512 lanes) of more rows than workgroups; rows shorter than a pack
STATS = [("bf16", 2048, 20000), ("fp16", 2001, 20001), ("fp32", 1001, 20000), ("bf16", 511, 30000), ("bf16", 2200, 13000), ("fp16", 4099, 13000),
         ("fp32", 2050, 13000), ("bf16", 5, 13000), ("fp32", 3, 13000), ("bf16", 65600, 8300)]


@pytest.mark.parametrize("dtype,cols,rows", STATS)
def test_statistics_of_many_rows(dtype, cols, rows):
    for pad, shift, temp in ((0, 0, 1.0), (3, 1, 0.6)):
        print(f"[case] statistics {rows}x{cols} (+{pad}) {dtype}", flush=True)
        z, t, rand = case(rows, cols, dtype, pad, shift, seed=33, dead=0.25)
        want, p, live = exact_logp(z, t, temp)
        logp, stats = torch.full((rows,), 9.0, device=device()), torch.full((rows, 2), 9.0, device=device())
        mr.token_logprob_forward(z, t, logp, stats=stats, temperature=temp)
        assert ((logp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        assert (logp[~live] == 0).all() and (stats[~live] == 0).all()
        top = z.amax(dim=1)
        assert torch.equal(stats[live, 0], top[live].float())
        total = 1 / p.amax(dim=1)                                    # exp((max - max) / T) over the sum
        assert ((stats[live, 1].double() - total[live]).abs() <= S_TOL * total[live]).all()
        adv, old, ref, w = vectors(z, t, rand, temp)
        want, _, _, _, _, sums, sizes = exact_policy(z, t, adv, old, ref, w, CLIP, KL, temp)
        record, lp = torch.empty(4, device=device()), torch.empty(rows, device=device())
        mr.policy_loss(z, t, adv, record, logp=lp, old_logp=old, ref_logp=ref, weights=w, clip=CLIP, kl=KL, temperature=temp)
        assert ((lp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        assert ((record.double() - sums).abs() <= 2.0 ** -15 * sizes + 2.0 ** -23 * sums.abs()).all()
        if cols < 8:                                                 # the gradient by way of the same statistics
            out = torch.empty_like(z)
            want, p, live, g, size, sums, sizes = exact_policy(z, t, adv, old, ref, w, CLIP, KL, temp)
            mr.policy_loss(z, t, adv, record, old_logp=old, ref_logp=ref, weights=w, clip=CLIP, kl=KL, temperature=temp, dlogits=out)
            check_gradient(out, exact_gradient(p, t, live, g, temp), p, t, live, size, temp, dtype, more=2.0 ** -15)
            assert P_TOL == 2.0 ** -15
