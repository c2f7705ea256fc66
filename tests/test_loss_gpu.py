"""Losses on logits against their formulas in 64 bits: token log-probabilities, their backward pass, the clipped policy loss
with its gradient, and the preference loss.

Tolerances.  A row's sum S adds exponentials that are each off by at most 2^-23 (exp2) and 2^-23 |arg| ln 2 (the exponent's two
roundings and the rounded 1/T, with |arg| 2^-|arg| <= 0.54), in chains of at most 128 additions a lane and 32 to join lanes and
parts, each off by 2^-24 of the partial sum: 2^-23 (1 + 1 + 80) < 2^-16 of S.  So a log-probability is off by at most 2^-16, and by
2^-24 of itself where it is stored; a probability by 2^-15 of itself; a gradient by that and a storage rounding of eps / 2."""
import math

import pytest
import torch

import all_gather_amd as mr
from gpu_util import TORCH_DT, device

pytestmark = pytest.mark.gpu

S_TOL, P_TOL = 2.0 ** -16, 2.0 ** -15
SHAPES = [(1, 1), (3, 2), (5, 7), (130, 8), (300, 9), (4, 63), (257, 100), (131, 513), (1, 4097), (140, 4096), (200, 8193), (2, 32771),
          (129, 32771), (3, 131072), (128, 131072), (129, 65537), (130, 131073), (6, 262144), (62, 50000), (300, 70001)]


def case(rows, cols, dtype, pad=0, shift=0, seed=0, dead=0.3):
    """Logits inside a larger buffer (``shift`` elements in, ``pad`` after each row), targets (some ignored), per-row vectors."""
    g = torch.Generator(device=device()).manual_seed(seed * 1000003 + rows * 1009 + cols)
    rand = lambda *s: torch.randn(*s, generator=g, device=device())  # noqa: E731
    flat = torch.full((shift + rows * (cols + pad),), 7.0, dtype=TORCH_DT[dtype], device=device())
    z = flat[shift:].view(rows, cols + pad)[:, :cols]
    z.copy_(3 * rand(rows, cols))
    t = torch.randint(0, cols, (rows,), generator=g, device=device())
    t[0] = cols - 1
    if rows > 2:
        t[1] = 0
        drop = torch.rand(rows, generator=g, device=device()) < dead
        drop[:2] = False
        t = torch.where(drop, torch.tensor([-100, cols, -1, 1 << 40], device=device())[torch.arange(rows, device=device()) % 4], t)
    return z, t, rand


def exact_logp(z, t, temp):
    live = (t >= 0) & (t < z.shape[1])
    x = torch.log_softmax(z.double() / temp, dim=1)
    return torch.where(live, x.gather(1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0], 0.0), x.exp(), live


def exact_gradient(p, t, live, g, temp):
    d = -p * g[:, None] / temp
    i = live.nonzero()[:, 0]
    d[i, t[i]] += g[i] / temp
    return torch.where(live[:, None], d, 0.0)


def check_gradient(got, want, p, t, live, g, temp, dtype, more=0.0):
    """``more``: relative error of g itself."""
    eps = torch.finfo(got.dtype).eps / 2
    scale = p.clone()
    i = live.nonzero()[:, 0]
    scale[i, t[i]] += more + 2.0 ** -22          # g ([j = t] - p): g's own error there, and fp32's of the difference
    tol = scale * (g.abs() / temp)[:, None] * (P_TOL + more) + want.abs() * (eps + more)
    tol = tol + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps  # what subnormal storage loses
    i = live.nonzero()[:, 0]
    tol[i, t[i]] += (g.abs() / temp)[i] * (more + 2.0 ** -22)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_logprob_forward_and_backward(rows, cols, dtype):
    print(f"[case] logprob {rows}x{cols} {dtype}", flush=True)
    for pad, shift, temp in ((0, 0, 1.0), (3, 1, 0.6)):
        z, t, rand = case(rows, cols, dtype, pad, shift)
        logp, stats = torch.full((rows,), 9.0, device=device()), torch.full((rows, 2), 9.0, device=device())
        mr.token_logprob_forward(z, t, logp, stats=stats, temperature=temp)
        want, p, live = exact_logp(z, t, temp)
        assert ((logp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        assert (logp[~live] == 0).all() and (stats[~live] == 0).all()
        top = z.double().amax(dim=1)
        assert (stats[live, 0].double() == top[live]).all()
        total = torch.exp((z.double() - top[:, None]) / temp).sum(dim=1)
        assert ((stats[live, 1].double() - total[live]).abs() <= S_TOL * total[live]).all()
        only = torch.empty_like(logp)
        mr.token_logprob_forward(z, t, only, temperature=temp)
        assert torch.equal(only, logp)
        g = rand(rows)
        flat = torch.full((shift + rows * (cols + pad),), 5.0, dtype=z.dtype, device=device())
        out = flat[shift:].view(rows, cols + pad)[:, :cols]
        mr.token_logprob_backward(z, t, stats, g, out, temperature=temp)
        check_gradient(out, exact_gradient(p, t, live, g.double(), temp), p, t, live, g.double(), temp, dtype)
        if pad:
            assert (flat[shift:].view(rows, cols + pad)[:, cols:] == 5.0).all() and (flat[:shift] == 5.0).all()
        mr.token_logprob_backward(z, t, stats, g, z, temperature=temp)  # in place
        assert torch.equal(z, out)


def exact_policy(z, t, adv, old, ref, w, clip, kl, temp):
    lp, p, live = exact_logp(z, t, temp)
    w = torch.where(live, w.double() if w is not None else torch.ones_like(lp), 0.0)
    live = live & (w != 0)
    lp = torch.where(live, lp, 0.0)
    r = torch.exp(lp - old.double()) if old is not None else torch.ones_like(lp)
    a = adv.double()
    free, held = -a * r, -a * r.clamp(1 - clip[0], 1 + clip[1])
    k, more = torch.zeros_like(lp), torch.zeros_like(lp)
    if ref is not None:
        d = ref.double() - lp
        k, more = torch.expm1(d) - d, -torch.expm1(d)
    g = torch.where(live, w * (torch.where(free >= held, free, 0.0) + kl * more), 0.0)
    size = torch.where(live, w.abs() * (free.abs() + abs(kl) * (1 + more.abs())), 0.0)
    z0 = torch.zeros_like(lp)
    terms = torch.stack([torch.where(live, x, z0) for x in (w * (torch.maximum(free, held) + kl * k), w * k, w * (held > free), w)])
    sizes = torch.stack([torch.where(live, x, z0) for x in (w.abs() * (free.abs() + held.abs() + abs(kl) * (k.abs() + 1)),
                                                            w.abs() * (k.abs() + 1), z0, w.abs())])
    return lp, p, live, g, size, terms.sum(dim=1), sizes.sum(dim=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_policy_loss(rows, cols, dtype):
    print(f"[case] policy {rows}x{cols} {dtype}", flush=True)
    for pad, shift, temp, kl, has_old, has_w in ((0, 0, 1.0, 0.05, True, True), (5, 1, 0.8, 0.0, True, False), (0, 0, 1.3, 0.2, False, True)):
        z, t, rand = case(rows, cols, dtype, pad, shift, seed=1)
        lp = exact_logp(z, t, temp)[0]
        old = (lp + 0.4 * rand(rows)).float() if has_old else None
        ref = (lp + 0.5 * rand(rows)).float() if kl else None
        adv = rand(rows)
        w = (rand(rows).abs() + 0.1) * (torch.arange(rows, device=device()) % 5 != 3) if has_w else None
        clip = (0.2, 0.3)
        if has_old:  # no ratio within its own error of a border, where a rounding may decide
            r = torch.exp(lp - old.double())
            near = ((r - 0.8).abs() < 1e-4) | ((r - 1.3).abs() < 1e-4)
            old = torch.where(near, old + 0.01, old)
        want, p, live, g, size, sums, sizes = exact_policy(z, t, adv, old, ref, w, clip, kl, temp)
        scale = 8.0
        flat = torch.full((shift + rows * (cols + pad),), 5.0, dtype=z.dtype, device=device())
        out = flat[shift:].view(rows, cols + pad)[:, :cols]
        logp, record = torch.full((rows,), 9.0, device=device()), torch.full((4,), 9.0, device=device())
        args = dict(old_logp=old, ref_logp=ref, weights=w, clip=clip, kl=kl, temperature=temp)
        mr.policy_loss(z, t, adv, record, logp=logp, dlogits=out, grad_scale=scale, **args)
        assert ((logp.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        # r and exp(d) are off by the log-probability's error and 2^-22 (expf, expm1f, their arguments' rounding): 2^-15
        # of `size`, which bounds both; the record's terms likewise, then one rounding to fp32
        gs = g * scale
        check_gradient(out, exact_gradient(p, t, live, gs, temp), p, t, live, size * scale, temp, dtype, more=2.0 ** -15)
        assert ((record.double() - sums).abs() <= 2.0 ** -15 * sizes + 2.0 ** -23 * sums.abs()).all(), (record, sums)
        if pad:
            assert (flat[shift:].view(rows, cols + pad)[:, cols:] == 5.0).all() and (flat[:shift] == 5.0).all()
        # the value alone, on whichever path: no gradient wanted
        again, lp2 = torch.empty_like(record), torch.empty_like(logp)
        mr.policy_loss(z, t, adv, again, logp=lp2, **args)
        assert ((again.double() - sums).abs() <= 2.0 ** -15 * sizes + 2.0 ** -23 * sums.abs()).all()
        assert ((lp2.double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all()
        mr.policy_loss(z, t, adv, again, dlogits=z, grad_scale=scale, **args)  # in place, no logp
        assert torch.equal(z, out) and torch.equal(again, record)


@pytest.mark.parametrize("rows,cols", [(6, 40), (6, 70000), (160, 40), (160, 70000), (160, 140000)])
def test_policy_gradient_against_differences(rows, cols):
    """The gradient of the loss along a direction, against a difference of losses (fp32 logits, kl and clipping on)."""
    z, t, rand = case(rows, cols, "fp32", seed=2)
    lp = exact_logp(z, t, 1.0)[0]
    old, ref = (lp + 0.05 * rand(rows)).float(), (lp + 0.3 * rand(rows)).float()
    adv, record = rand(rows), torch.empty(4, device=device())
    out = torch.empty_like(z)
    mr.policy_loss(z, t, adv, record, old_logp=old, ref_logp=ref, kl=0.1, clip=(0.5, 0.5), dlogits=out)
    step = torch.zeros_like(z)
    step[torch.arange(rows, device=device()), t.clamp(0, cols - 1)] = rand(rows) * 0.02
    ends = []
    for s in (1.0, -1.0):
        mr.policy_loss(z + s * step, t, adv, record, old_logp=old, ref_logp=ref, kl=0.1, clip=(0.5, 0.5))
        ends.append(float(record[0]))
    slope = float((out.double() * step.double()).sum()) * 2
    # third derivatives of exp-like terms are at most a few times |A| + kl: 0.02^3 each; and the losses' own 2^-15
    tol = rows * (2 * 4 * 0.02 ** 3) + rows * 4 * 2.0 ** -15
    assert abs((ends[0] - ends[1]) - slope) <= tol, (ends, slope, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [8, 200])
@pytest.mark.parametrize("cols", [65, 40000, 150000])
def test_masked_and_extreme_logits(rows, cols, dtype):
    z, t, rand = case(rows, cols, dtype, seed=3, dead=0.0)
    low = torch.finfo(z.dtype).min
    z[0], t[0] = low, 3                              # every element the type's lowest value: uniform
    z[1, 1:], t[1] = -math.inf, 0                    # one token left: probability 1
    z[2, ::2], t[2] = low, 1                         # masked by the lowest value
    z[3], t[3] = -math.inf, 2                        # nothing left: NaN
    z[4, 5], t[4] = math.nan, 6
    z[5, 5], t[5] = math.inf, 6
    z[6, 7:], t[6] = -math.inf, 9                    # the target itself is ruled out: -inf
    z[7], t[7] = -math.inf, -100                     # a row that is not read
    logp, stats = torch.empty(rows, device=device()), torch.empty(rows, 2, device=device())
    mr.token_logprob_forward(z, t, logp, stats=stats)
    lp = logp.double()
    assert abs(float(lp[0]) + math.log(cols)) <= S_TOL + 2.0 ** -20 and float(lp[1]) == 0.0
    n = (cols + 1) // 2
    want, p, live = exact_logp(z[2:3, 1::2].contiguous(), torch.zeros(1, dtype=torch.int64, device=device()), 1.0)
    assert abs(float(lp[2] - want[0])) <= S_TOL + 2.0 ** -20 and n
    assert lp[3].isnan() and lp[4].isnan() and lp[5].isnan() and float(lp[6]) == -math.inf and float(lp[7]) == 0.0
    assert torch.isfinite(lp[8:]).all()
    out = torch.empty_like(z)
    mr.token_logprob_backward(z, t, stats, torch.ones(rows, device=device()), out)
    assert ((out[0, :3].double() + 1 / cols).abs() <= (P_TOL + torch.finfo(z.dtype).eps) / cols + 2.0 ** -24).all()
    assert (out[1] == 0).all() and (out[2, ::2] == 0).all() and (out[7] == 0).all()
    assert out[3].isnan().all() and out[4].isnan().all()
    assert torch.isfinite(out[8:].float()).all()
    # the policy loss: the same rows, others untouched by them
    adv = torch.ones(rows, device=device())
    w = torch.ones(rows, device=device())
    w[3:7] = 0.0                                     # rows without a probability carry no loss here
    record, d = torch.empty(4, device=device()), torch.empty_like(z)
    mr.policy_loss(z, t, adv, record, weights=w, dlogits=d)
    assert (d[3:8] == 0).all() and torch.isfinite(record).all() and torch.isfinite(d.float()).all()
    assert float(record[3]) == rows - 5 and float(record[0]) == -(rows - 5)
    w[3] = 1.0
    mr.policy_loss(z, t, adv, record, weights=w, dlogits=d)
    assert record[0].isnan() and d[3].isnan().all() and torch.isfinite(d[4:].float()).all() and torch.isfinite(d[:3].float()).all()


def test_all_rows_ignored():
    for rows, cols in ((3, 100), (300, 100), (300, 40000)):
        z, t, _ = case(rows, cols, "bf16")
        t.fill_(-100)
        z.fill_(math.nan)
        logp, record, d = torch.ones(rows, device=device()), torch.ones(4, device=device()), torch.ones_like(z)
        mr.policy_loss(z, t, torch.ones(rows, device=device()), record, logp=logp, dlogits=d)
        assert (record == 0).all() and (logp == 0).all() and (d == 0).all()


def test_empty_calls():
    z = torch.empty(0, 10, device=device())
    t = torch.empty(0, dtype=torch.int64, device=device())
    f = torch.empty(0, device=device())
    mr.token_logprob_forward(z, t, f, stats=torch.empty(0, 2, device=device()))
    mr.token_logprob_backward(z, t, torch.empty(0, 2, device=device()), f, z)
    record = torch.ones(4, device=device())
    mr.policy_loss(z, t, f, record, dlogits=z)
    assert (record == 0).all()
    # no columns: every row is ignored
    z = torch.empty(5, 0, device=device())
    t, logp = torch.zeros(5, dtype=torch.int64, device=device()), torch.ones(5, device=device())
    mr.token_logprob_forward(z, t, logp)
    assert (logp == 0).all()
    record.fill_(1)
    mr.policy_loss(z, t, torch.ones(5, device=device()), record, dlogits=z)
    assert (record == 0).all()


def exact_preference(lp, ref, off, beta, ls, scale):
    x = lp.double() - (ref.double() if ref is not None else 0.0)
    s = torch.stack([x[a:b].sum() for a, b in zip(off, off[1:])]) if len(off) > 1 else x.new_zeros(0)
    h = beta * (s[0::2] - s[1::2])
    f = torch.nn.functional.logsigmoid
    loss = -scale * ((1 - ls) * f(h) + (ls * f(-h) if ls else 0.0))
    gh = scale * beta * (ls - torch.sigmoid(-h))
    d = torch.zeros_like(x)
    for i, (a, b) in enumerate(zip(off, off[1:])):
        d[a:b] = gh[i // 2] if i % 2 == 0 else -gh[i // 2]
    return loss.sum(), h, d


@pytest.mark.parametrize("offsets", [
    (0, 5, 9), (0, 0, 0), (0, 0, 7), (0, 7, 7), (3, 10, 12, 12, 40, 41, 41), tuple(range(0, 9000, 500)) + (9000,), (2, 6000, 6001),
    (0, 40000, 100001), tuple(i * i // 3 for i in range(0, 2401))])
@pytest.mark.parametrize("with_ref", [True, False])
def test_preference_loss(offsets, with_ref):
    rows = offsets[-1] + 13
    g = torch.Generator(device=device()).manual_seed(rows)
    lp = -torch.randn(rows, generator=g, device=device()).abs()
    ref = lp + 0.1 * torch.randn(rows, generator=g, device=device()) if with_ref else None
    off = torch.tensor(offsets, device=device())
    pairs = (len(offsets) - 1) // 2
    for beta, ls, scale, gs in ((0.1, 0.0, None, 1.0), (0.5, 0.1, 2.0, 4.0)):
        record, margins, d = torch.empty(3, device=device()), torch.empty(pairs, device=device()), torch.full((rows,), 9.0, device=device())
        mr.preference_loss(lp, off, record, ref_logp=ref, margins=margins, dlogp=d, beta=beta, smoothing=ls, loss_scale=scale, grad_scale=gs)
        sc = 1 / pairs if scale is None else scale
        loss, h, want = exact_preference(lp, ref, list(offsets), beta, ls, sc)
        # sums and functions in 64 bits (their errors far below), one rounding to fp32 each
        r = 2.0 ** -24 * 1.001
        assert ((margins.double() - h).abs() <= r * h.abs() + 1e-9).all()
        assert abs(float(record[0]) - float(loss)) <= r * abs(float(loss)) + 1e-9 * pairs
        assert abs(float(record[1]) - float((h > 0).double().mean())) <= r and abs(float(record[2]) - float(h.mean())) <= r * abs(float(h.mean())) + 1e-9
        assert ((d.double() - gs * want).abs() <= r * (gs * want).abs() + 1e-12).all()
        first = record.clone()
        mr.preference_loss(lp, off, record, ref_logp=ref, margins=None, dlogp=None, beta=beta, smoothing=ls, loss_scale=scale)
        assert torch.equal(record, first)
        place = lp.clone()
        mr.preference_loss(place, off, record, ref_logp=ref, dlogp=place, beta=beta, smoothing=ls, loss_scale=scale, grad_scale=gs)
        assert torch.equal(place, d) and torch.equal(record, first)


def test_preference_extremes():
    off = torch.tensor([0, 2, 4, 6, 8, 10, 12], device=device())
    lp = torch.zeros(12, device=device())
    lp[0], lp[6], lp[8] = 1e6, 1e6, math.nan         # h huge, minus huge, NaN
    record, margins, d = torch.empty(3, device=device()), torch.empty(3, device=device()), torch.empty(12, device=device())
    mr.preference_loss(lp, off, record, margins=margins, dlogp=d, beta=1.0, loss_scale=1.0)
    assert record[0].isnan() and float(margins[0]) == 1e6 and float(margins[1]) == -1e6 and margins[2].isnan()
    assert (d[:4] == 0).all() and (d[4:6] == -1).all() and (d[6:8] == 1).all() and d[8:].isnan().all()
    mr.preference_loss(lp[:8].contiguous(), off[:5], record, beta=1.0, loss_scale=1.0)
    assert abs(float(record[0]) - 1e6) <= 1 and float(record[1]) == 0.5
    # no pairs; offsets past the rows are held to them
    mr.preference_loss(lp, off[:1], record, dlogp=d)
    assert (record == 0).all() and (d == 0).all()
    far = torch.tensor([-5, 3, 1 << 50], device=device())
    one = torch.ones(6, device=device())
    mr.preference_loss(one, far, record, dlogp=torch.empty(6, device=device()), beta=1.0)
    assert float(record[2]) == 0.0


def test_two_streams_and_replays():
    """Calls of every kind captured into one graph: each replay, on new inputs, gives the eager results, bit for bit, with eager
    calls on another stream between them."""
    rows, cols, few = 300, 4099, 5
    z, t, rand = case(rows, cols, "bf16", seed=4)
    zf, tf, _ = case(few, 90001, "fp16", seed=5)
    adv = rand(rows)
    off = torch.tensor([0, 50, 100, 180, 300], device=device())

    def bufs():
        e = lambda *s: torch.empty(*s, device=device())  # noqa: E731
        return dict(rec=e(4), d=torch.empty_like(z), lp=e(rows), lpf=e(few), stf=e(few, 2), df=torch.empty_like(zf), recf=e(4), pref=e(3), dl=e(rows))

    def step(b):
        mr.policy_loss(z, t, adv, b["rec"], logp=b["lp"], dlogits=b["d"])
        mr.token_logprob_forward(zf, tf, b["lpf"], stats=b["stf"])
        mr.token_logprob_backward(zf, tf, b["stf"], b["lpf"], b["df"])
        mr.policy_loss(zf, tf, adv[:few].contiguous(), b["recf"], dlogits=b["df"], weights=None)
        mr.preference_loss(b["lp"], off, b["pref"], dlogp=b["dl"])

    graphed, eager, other = bufs(), bufs(), bufs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(graphed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(graphed)
    for i in range(3):
        z.copy_(3 * rand(rows, cols))
        zf.copy_(3 * rand(few, 90001))
        torch.cuda.synchronize()
        for v in graphed.values():
            v.fill_(float("nan"))
        graph.replay()
        with torch.cuda.stream(s):
            step(other)                              # beside the replay: another workspace
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(graphed[k], eager[k]) and torch.equal(other[k], eager[k]), (i, k)


def test_row_offsets_past_32_bits():
    """The last rows of logits of more than 2^32 elements."""
    rows, cols = 70000, 65536
    z = torch.empty(rows, cols, dtype=torch.bfloat16, device=device())
    z[-3:] = 3 * torch.randn(3, cols, device=device())
    t = torch.full((rows,), -100, device=device())
    t[-3:] = torch.tensor([5, cols - 1, 0], device=device())
    logp, record = torch.empty(rows, device=device()), torch.empty(4, device=device())
    want, p, live = exact_logp(z[-3:], t[-3:], 1.0)
    mr.policy_loss(z, t, torch.ones(rows, device=device()), record, logp=logp, dlogits=z)
    assert ((logp[-3:].double() - want).abs() <= S_TOL + 2.0 ** -24 * want.abs()).all() and float(record[3]) == 3.0
    g = torch.full((3,), -1.0, dtype=torch.float64, device=device())
    check_gradient(z[-3:], exact_gradient(p, t[-3:], live, g, 1.0), p, t[-3:], live, g, 1.0, "bf16", more=2.0 ** -15)
    assert (z[:7] == 0).all() and (z[-10:-3] == 0).all()
