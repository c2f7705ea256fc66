"""The two ends of a training step as measured cases: losses on logits with their gradients, and Muon's update.

Five operators: the log-probabilities of target tokens from logits, their backward pass, a clipped policy
loss with a KL term (value and gradient of the logits in one call), a preference loss over pairs of
sequences, and one Muon step over a list of matrices (momentum, Newton-Schulz orthogonalisation, update).
``run`` computes each in its plain form (elementary torch operations in 32 bits, a row's few scalars and
long sums in 64) or, where ``own`` is set, through this package's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
CLIP, KL = (0.2, 0.28), 0.04                     # policy loss
BETA, SMOOTH = 0.1, 0.05                         # preference loss
MOMENTUM, DECAY, LR, NS_EPS = 0.95, 0.1, 0.02, 1e-7
COEF, STEPS = (3.4445, -4.775, 2.0315), 5
BLOCK = 32                                       # a matrix's part of the flat state starts on such a multiple
IGNORED = -100                                   # target of a token that carries no loss
MOST = {"logits": 4.4e9, "preference": 4.2e7, "muon": 1.6e13}   # the largest listed cases' work, which no drawn one exceeds


def listed():
    return [
        # the last few tokens of a batch that is scored while it is generated: latency
        dict(name="logprob few", op="logprob", rows=3, cols=131072, pad=0, dtype="bf16", active=1.0, temp=1.0),
        # scoring packed sequences under a reference model, odd vocabulary in fp16
        dict(name="logprob large", op="logprob", rows=16384, cols=50001, pad=0, dtype="fp16", active=0.9, temp=1.0),
        # the gradient of a small evaluation batch, odd vocabulary inside a padded buffer
        dict(name="logprob bwd ragged", op="logprob_bwd", rows=1001, cols=32003, pad=61, dtype="bf16", active=0.6, temp=0.7),
        # a preference batch whose logits are kept in fp32
        dict(name="logprob bwd fp32", op="logprob_bwd", rows=4096, cols=65536, pad=0, dtype="fp32", active=0.8, temp=1.0),
        # one short answer's tokens
        dict(name="policy short", op="policy", rows=24, cols=32768, pad=0, dtype="bf16", active=0.7, temp=1.0),
        # an ordinary microbatch of prompts and answers, sampled at a temperature, odd vocabulary
        dict(name="policy step", op="policy", rows=4096, cols=50001, pad=0, dtype="bf16", active=0.75, temp=0.9),
        # a long packed microbatch under a large vocabulary
        dict(name="policy large", op="policy", rows=8192, cols=131072, pad=0, dtype="bf16", active=1.0, temp=1.0),
        # one rank's few pairs
        dict(name="preference small", op="preference", pairs=4, lo=20, hi=200, shape_seed=1),
        # a large batch of long pairs
        dict(name="preference large", op="preference", pairs=1024, lo=200, hi=8192, shape_seed=2),
        # the small matrices of an adapter or of a small model, all odd: latency
        dict(name="muon small", op="muon", width=0, matrices=16, lo=16, hi=512, mult=1, shape_seed=3, dtype="bf16", gdtype="bf16",
             master=False, products=16),
        # one block of a model of width 4096 trained in bf16: four square matrices and two of 1 : 4
        dict(name="muon block", op="muon", width=4096, matrices=6, lo=0, hi=0, mult=1, shape_seed=0, dtype="bf16", gdtype="bf16",
             master=False, products=16),
        # odd sizes in mixed precision: fp32 master copies, products as exact as fp32
        dict(name="muon master ragged", op="muon", width=0, matrices=8, lo=700, hi=2500, mult=1, shape_seed=5, dtype="bf16",
             gdtype="fp32", master=True, products=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        op = rng.choice(("logprob", "logprob_bwd", "policy", "policy", "preference", "muon", "muon"))
        if op == "preference":
            lo = _log(rng, 1, 400)
            c = dict(op=op, pairs=_log(rng, 1, 4096), lo=lo, hi=max(lo, _log(rng, 16, 16384)), shape_seed=rng.randrange(1 << 20))
        elif op == "muon":
            lo = _log(rng, 1, 2048)
            c = dict(op=op, width=0, matrices=_log(rng, 1, 96), lo=lo, hi=max(lo, _log(rng, 64, 9000)), mult=rng.choice((1, 1, 64)),
                     shape_seed=rng.randrange(1 << 20), gdtype=rng.choice(("bf16", "fp16", "fp32")))
            c["dtype"] = rng.choice(("fp32", "bf16")) if c["gdtype"] == "fp32" else c["gdtype"]
            c["master"] = c["dtype"] != "fp32" and rng.random() < 0.4
            c["products"] = 32 if c["dtype"] == "fp32" or c["master"] else 16
        else:
            c = dict(op=op, rows=_log(rng, 1, 65536), cols=_log(rng, 2, 262144), pad=rng.choice((0, 0, rng.randrange(1, 200))),
                     dtype=rng.choice(("bf16", "fp16", "fp32")), active=rng.choice((1.0, round(rng.uniform(0.05, 1.0), 2))),
                     temp=rng.choice((1.0, round(rng.uniform(0.3, 1.5), 2))))
        w = work(c)
        if (w["flops"] if op == "muon" else w["bytes"]) <= MOST["logits" if "cols" in c else op]:
            return c


def _active(case):
    return max(1, int(case["active"] * case["rows"]))


def _lengths(case):
    """Tokens of each chosen and each rejected sequence, log-uniform in [lo, hi]."""
    r = random.Random(case["shape_seed"])
    return [_log(r, case["lo"], case["hi"]) for _ in range(2 * case["pairs"])]


def _shapes(case):
    """(rows, columns) of the case's matrices."""
    d = case["width"]
    if d:
        return [(d, d)] * 4 + [(4 * d, d), (d, 4 * d)]
    r, mult = random.Random(case["shape_seed"]), case["mult"]
    return [tuple(max(mult, _log(r, case["lo"], case["hi"]) // mult * mult) for _ in range(2)) for _ in range(case["matrices"])]


def work(case):
    op = case["op"]
    if op == "preference":
        n = sum(_lengths(case))
        return {"bytes": 12 * n + 8 * (2 * case["pairs"] + 1) + 4 * case["pairs"], "flops": 3 * n}
    if op == "muon":
        shapes, s = _shapes(case), SIZE[case["dtype"]]
        n = sum(a * b for a, b in shapes)
        # X X^T and A^2 are symmetric: half of each; P X whole
        flops = STEPS * sum(3 * min(a, b) ** 2 * max(a, b) + min(a, b) ** 3 for a, b in shapes)
        return {"bytes": n * (8 + SIZE[case["gdtype"]] + (8 + s if case["master"] else 2 * s)), "flops": flops}
    rows, cols, s, live = case["rows"], case["cols"], SIZE[case["dtype"]], _active(case)
    if op == "logprob":
        return {"bytes": live * cols * s + 20 * rows, "flops": 5 * live * cols}
    return {"bytes": (live + rows) * cols * s + (20 if op == "logprob_bwd" else 28) * rows,
            "flops": (5 if op == "logprob_bwd" else 9) * live * cols}


# ------------------------------------------------------------------------------------------ inputs

def _padded(counts):
    return [-(-n // BLOCK) * BLOCK for n in counts]


def _logprob64(z, t, temp):
    """Log-probabilities of the targets, in 64 bits, a few rows at a time."""
    rows = max(1, (1 << 26) // z.shape[1])
    return torch.cat([torch.log_softmax(z[i:i + rows].double() / temp, dim=1).gather(1, t[i:i + rows].clamp_min(0)[:, None])
                      for i in range(0, z.shape[0], rows)])[:, 0]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] == "preference":
        lens = torch.tensor(_lengths(case), dtype=torch.int64)
        n = int(lens.sum())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(dev)
        s["logp"] = -normal(n).square()                              # of targets; the prompts' tokens carry none
        s["logp"][torch.rand(n, generator=g, device=dev) < 0.3] = 0.0
        s["ref"] = torch.where(s["logp"] == 0, s["logp"], s["logp"] + 0.1 * normal(n))
        s["margins"], s["dlogp"], s["record"] = torch.empty(case["pairs"], device=dev), torch.empty(n, device=dev), torch.empty(3, device=dev)
        return s
    if case["op"] == "muon":
        shapes = _shapes(case)
        s["shapes"], counts = shapes, [a * b for a, b in shapes]
        total, padded = sum(counts), _padded(counts)
        # gradients of a layer: a few strong directions over noise; their momentum has seen the same directions
        weak, strong = 1e-4 * normal(total), []
        s["m"] = torch.zeros(sum(padded), device=dev)
        for (a, b), w, m in zip(shapes, weak.split(counts), s["m"].split(padded)):
            k = min(8, a, b)
            low = (normal(a, k) * torch.logspace(0, -2, k, device=dev)) @ normal(k, b) * 1e-4
            strong.append((w.view(a, b) + low).to(DT[case["gdtype"]]))
            m[:a * b] = (0.3 * normal(a, b) * 1e-4 + low).view(-1)
        s["grads"] = strong
        p = 0.02 * normal(total)
        flat = p.to(DT[case["dtype"]])
        s["params"] = [x.view(q) for x, q in zip(flat.split(counts), shapes)]
        s["out_flat"] = torch.empty_like(flat)
        s["params_out"] = [x.view(q) for x, q in zip(s["out_flat"].split(counts), shapes)]
        s["m_out"] = torch.empty_like(s["m"])
        s["master"] = s["master_out"] = None
        if case["master"]:
            s["master"], s["master_out"] = torch.zeros_like(s["m"]), torch.empty_like(s["m"])
            for x, m, n in zip(p.split(counts), s["master"].split(padded), counts):
                m[:n] = x
        s["record"] = torch.tensor([1.25, 0.8, 1.0], device=dev)     # norm, clip factor, all finite
        return s
    rows, cols, dt, temp, live = case["rows"], case["cols"], DT[case["dtype"]], case["temp"], _active(case)
    buf = torch.empty(rows, cols + case["pad"], device=dev, dtype=dt)
    z = s["logits"] = buf[:, :cols]
    step = max(1, (1 << 28) // cols)
    for i in range(0, rows, step):
        z[i:i + step] = 2.5 * normal(min(step, rows - i), cols)
    half = -(-cols // 2)
    z[::16, half:] = -math.inf                                       # rows whose later tokens are ruled out
    # a target is the likeliest of some tokens, as sampling would find it
    some = torch.randint(0, half, (rows, 64), generator=g, device=dev)
    t = some.gather(1, z.gather(1, some).float().argmax(dim=1, keepdim=True))[:, 0]
    off = torch.randperm(rows, generator=g, device=dev)[live:]
    t[off] = IGNORED
    s["targets"] = t
    s["out"] = torch.zeros(rows, cols + case["pad"], device=dev, dtype=dt)[:, :cols] if case["op"] != "logprob" else None
    # the loss is a mean over the tokens; fp16 gradients carry a loss scale
    s["grad_scale"] = 16.0 * live if case["dtype"] == "fp16" else 1.0
    if case["op"] == "logprob_bwd":
        m = z.float().amax(dim=1)
        rows_at = max(1, (1 << 26) // cols)
        total = torch.cat([torch.exp((z[i:i + rows_at].double() - m[i:i + rows_at, None].double()) / temp).sum(dim=1)
                           for i in range(0, rows, rows_at)])
        s["stats"] = torch.where((t >= 0)[:, None], torch.stack([m, total.float()], dim=1), torch.zeros(1, device=dev))
        s["dlogp"] = normal(rows) / live * s["grad_scale"]
        return s
    s["logp"], s["stats"] = torch.empty(rows, device=dev), torch.empty(rows, 2, device=dev)
    if case["op"] == "policy":
        lp = _logprob64(z, t, temp)
        s["old"], s["ref"] = (lp + 0.15 * normal(rows)).float(), (lp + 0.3 * normal(rows)).float()
        s["adv"] = normal(rows)
        s["weights"] = torch.full((rows,), 1.0 / live, device=dev)
        s["weights"][off] = 0.0
        s["record"] = torch.empty(4, device=dev)
    return s


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"logprob": _logprob, "logprob_bwd": _logprob_bwd, "policy": _policy, "preference": _preference, "muon": _muon}[s["case"]["op"]](s)


def _run_own(s):
    import all_gather_amd as mr

    c = s["case"]
    if c["op"] == "logprob":
        mr.token_logprob_forward(s["logits"], s["targets"], s["logp"], stats=s["stats"], temperature=c["temp"])
        return {"logp": s["logp"], "stats": s["stats"]}
    if c["op"] == "logprob_bwd":
        mr.token_logprob_backward(s["logits"], s["targets"], s["stats"], s["dlogp"], s["out"], temperature=c["temp"])
        return {"dlogits": s["out"]}
    if c["op"] == "policy":
        mr.policy_loss(s["logits"], s["targets"], s["adv"], s["record"], old_logp=s["old"], ref_logp=s["ref"], weights=s["weights"],
                       logp=s["logp"], dlogits=s["out"], clip=CLIP, kl=KL, temperature=c["temp"], grad_scale=s["grad_scale"])
        return {"dlogits": s["out"], "logp": s["logp"], "record": s["record"]}
    if c["op"] == "preference":
        mr.preference_loss(s["logp"], s["offsets"], s["record"], ref_logp=s["ref"], margins=s["margins"], dlogp=s["dlogp"], beta=BETA,
                           smoothing=SMOOTH)
        return {"record": s["record"], "margins": s["margins"], "dlogp": s["dlogp"]}
    mr.muon_step(s["params"], s["grads"], mr.MuonState(s["m"], s["master"]), LR, params_out=s["params_out"],
                 state_out=mr.MuonState(s["m_out"], s["master_out"]), momentum=MOMENTUM, nesterov=True, weight_decay=DECAY, eps=NS_EPS,
                 coefficients=COEF, steps=STEPS, adjust="ratio", products=c["products"], clip=s["record"])
    return {"params": s["out_flat"], "m": s["m_out"], "master": s["master_out"]}


def _softmax(s):
    """(exp of the logits less their maximum, its sums in rows, the maxima, the targets' log-probabilities in 64 bits)."""
    temp = s["case"]["temp"]
    z = s["logits"].float()
    m = z.amax(dim=1, keepdim=True)
    at = s["targets"].clamp_min(0)[:, None]
    x = ((z.gather(1, at) - m).double() / temp)[:, 0]
    e = z.sub_(m).div_(temp).exp_() if z.data_ptr() != s["logits"].data_ptr() else ((z - m) / temp).exp()
    total = e.sum(dim=1, keepdim=True)
    return e, total, m, x - total.double().log()[:, 0]


def _logprob(s):
    live = s["targets"] >= 0
    _, total, m, logp = _softmax(s)
    return {"logp": torch.where(live, logp, 0.0).float(), "stats": torch.where(live[:, None], torch.cat([m, total], dim=1), 0.0)}


def _scatter_gradient(s, p, g):
    """g ([j = target] - p) / temp, with zeros where the target is ignored; p is used up."""
    live, at = (s["targets"] >= 0)[:, None], s["targets"].clamp_min(0)[:, None]
    g = torch.where(live, g[:, None] / s["case"]["temp"], 0.0)
    d = p.scatter_(1, at, p.gather(1, at) - 1).mul_(-g)
    return d.masked_fill_(~live, 0.0).to(s["out"].dtype)


def _logprob_bwd(s):
    z = s["logits"].float()
    m, total = s["stats"][:, :1], s["stats"][:, 1:]
    return {"dlogits": _scatter_gradient(s, torch.exp((z - m) / s["case"]["temp"]).div_(total), s["dlogp"])}


def _policy(s):
    live, w, adv = s["targets"] >= 0, s["weights"].double(), s["adv"].double()
    e, total, _, logp = _softmax(s)
    r = torch.exp(logp - s["old"].double())
    d = s["ref"].double() - logp
    k = torch.exp(d)
    free, held = -adv * r, -adv * r.clamp(1 - CLIP[0], 1 + CLIP[1])
    kl = k - d - 1
    g = w * (torch.where(free >= held, free, 0.0) + KL * (1 - k))
    # rows that carry no loss add nothing
    sums = torch.where(live, torch.stack([w * (torch.maximum(free, held) + KL * kl), w * kl, w * (held > free), w]), 0.0).sum(dim=1)
    return {"dlogits": _scatter_gradient(s, e.div_(total), (g * s["grad_scale"]).float()),
            "logp": torch.where(live, logp, 0.0).float(), "record": sums.float()}


def _preference(s):
    pairs = s["case"]["pairs"]
    at = torch.cat([torch.zeros(1, device=s["logp"].device, dtype=torch.float64), (s["logp"] - s["ref"]).double().cumsum(0)])
    sums = at[s["offsets"][1:]] - at[s["offsets"][:-1]]
    h = BETA * (sums[0::2] - sums[1::2])
    up, down = torch.log1p(torch.exp(-h.abs())) + (-h).clamp_min(0), torch.log1p(torch.exp(-h.abs())) + h.clamp_min(0)
    loss = ((1 - SMOOTH) * up + SMOOTH * down).sum() / pairs
    gh = (SMOOTH - 1 / (1 + torch.exp(h))) * BETA / pairs
    lens = s["offsets"][1:] - s["offsets"][:-1]
    dlogp = torch.repeat_interleave(torch.stack([gh, -gh], dim=1).view(-1), lens, output_size=s["logp"].numel())
    return {"record": torch.stack([loss, (h > 0).double().mean(), h.mean()]).float(), "margins": h.float(), "dlogp": dlogp.float()}


def _newton_schulz(u):
    if u.shape[0] > u.shape[1]:
        return _newton_schulz(u.t().contiguous()).t()
    x = u / torch.linalg.vector_norm(u, dtype=torch.float64).clamp_min(NS_EPS).float()
    a, b, c = COEF
    for _ in range(STEPS):
        q = x @ x.t()
        x = a * x + (b * q + c * (q @ q)) @ x
    return x


def _muon(s):
    c, shapes = s["case"], s["shapes"]
    counts = [a * b for a, b in shapes]
    padded = _padded(counts)
    zero = torch.zeros(BLOCK, device=s["m"].device)
    g = torch.cat([t for x, n, q in zip(s["grads"], counts, padded) for t in (x.float().reshape(-1), zero[:q - n])]) * s["record"][1]
    m = s["m"] * MOMENTUM + g * (1 - MOMENTUM)
    u = m * MOMENTUM + g * (1 - MOMENTUM)
    o = [_newton_schulz(x[:n].view(q)) * math.sqrt(max(1.0, q[0] / q[1])) for x, n, q in zip(u.split(padded), counts, shapes)]
    old = [x[:n].view(q) for x, n, q in zip(s["master"].split(padded), counts, shapes)] if c["master"] else s["params"]
    p = [x.float() * (1 - LR * DECAY) - LR * y for x, y in zip(old, o)]
    master = torch.cat([t for x, n, q in zip(p, counts, padded) for t in (x.reshape(-1), zero[:q - n])]) if c["master"] else None
    return {"params": torch.cat([x.reshape(-1) for x in p]).to(DT[c["dtype"]]), "m": m, "master": master}


# ------------------------------------------------------------------------------------------ in 64 bits

def _exact_rows(s):
    """The logits' operators by torch's own log_softmax and its derivative in 64 bits, a few rows at a time."""
    c = s["case"]
    rows, cols = s["logits"].shape
    out = {"dlogits": [], "logp": [], "stats": [], "sums": torch.zeros(4, dtype=torch.float64, device=s["logits"].device)}
    step = max(1, (1 << 27) // cols)
    for i in range(0, rows, step):
        at = slice(i, min(rows, i + step))
        t = s["targets"][at]
        live = t >= 0
        z = s["logits"][at].double().requires_grad_(c["op"] != "logprob")
        lp = -torch.nn.functional.nll_loss(torch.log_softmax(z / c["temp"], dim=1), t, ignore_index=IGNORED, reduction="none")
        if c["op"] == "logprob":
            top = z.amax(dim=1)
            total = torch.exp(torch.logsumexp(z / c["temp"], dim=1) - top / c["temp"])
            out["stats"].append(torch.where(live[:, None], torch.stack([top, total], dim=1), 0.0))
            out["logp"].append(lp)
            continue
        if c["op"] == "logprob_bwd":
            value = (lp * s["dlogp"][at].double()).sum()
        else:
            w = torch.where(live, s["weights"][at].double(), 0.0)
            r = torch.exp(lp - s["old"][at].double())
            adv, d = s["adv"][at].double(), s["ref"][at].double() - lp
            held = r.clamp(1 - CLIP[0], 1 + CLIP[1])
            gain = torch.minimum(adv * r, adv * held)
            kl = torch.expm1(d) - d
            loss = (w * (KL * kl - gain)).sum()
            out["sums"] += torch.stack([loss, (w * kl).sum(), (w * (gain < adv * r)).sum(), w.sum()]).detach()
            out["logp"].append(lp.detach())
            value = loss * s["grad_scale"]
        out["dlogits"].append(torch.autograd.grad(value, z)[0])
    if c["op"] == "logprob":
        return {"logp": torch.cat(out["logp"]), "stats": torch.cat(out["stats"])}
    if c["op"] == "logprob_bwd":
        return {"dlogits": torch.cat(out["dlogits"])}
    return {"dlogits": torch.cat(out["dlogits"]), "logp": torch.cat(out["logp"]), "record": out["sums"]}


def _exact_polar(u):
    """The same odd polynomial of u's singular values, iterated on the smaller Gram matrix: X_k = Q_k X_0 with
    Q_{k+1} = p(A_k) Q_k and A_{k+1} = p(A_k) A_k p(A_k)."""
    wide = u.shape[0] <= u.shape[1]
    x = (u if wide else u.t().contiguous()) / max(float(torch.linalg.vector_norm(u)), NS_EPS)
    gram = torch.mm(x, x.t().contiguous())
    total = None
    for _ in range(STEPS):
        p = torch.mm(gram, gram).mul_(COEF[2]).add_(gram, alpha=COEF[1])
        p.diagonal().add_(COEF[0])
        total = p if total is None else torch.mm(p, total)
        gram = torch.mm(torch.mm(p, gram), p)
    x = torch.mm(total, x)
    return x if wide else x.t()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "preference":
        off = s["offsets"].cpu().tolist()
        ratio = (s["logp"].double() - s["ref"].double()).cpu()
        sums = torch.stack([x.sum() for x in ratio.split([b - a for a, b in zip(off, off[1:])])])
        h = (BETA * (sums[0::2] - sums[1::2])).requires_grad_(True)
        ls = torch.nn.functional.logsigmoid
        loss = -((1 - SMOOTH) * ls(h) + SMOOTH * ls(-h)).mean()
        gh = torch.autograd.grad(loss, h)[0] * BETA
        h = h.detach()
        return {"record": torch.stack([loss.detach(), (h > 0).double().mean(), h.mean()]), "margins": h,
                "dlogp": torch.cat([x.expand(b - a) for x, a, b in zip(torch.stack([gh, -gh], dim=1).view(-1), off, off[1:])])}
    if case["op"] != "muon":
        return _exact_rows(s)
    params, ms, masters = [], torch.zeros_like(s["m"], dtype=torch.float64), None
    if case["master"]:
        masters = torch.zeros_like(ms)
    at = 0
    for i, (a, b) in enumerate(s["shapes"]):
        here = slice(at, at + a * b)
        g = s["grads"][i].double() * s["record"][1].double()
        m = torch.lerp(g, s["m"][here].double().view(a, b), MOMENTUM)
        ms[here] = m.view(-1)
        o = _exact_polar(torch.lerp(g, m, MOMENTUM)) * math.sqrt(max(1.0, a / b))
        p = (s["master"][here].view(a, b) if case["master"] else s["params"][i]).double()
        p = p - LR * DECAY * p - LR * o
        if case["master"]:
            masters[here] = p.reshape(-1)
        params.append(p.reshape(-1))
        at += _padded([a * b])[0]
    return {"params": torch.cat(params), "m": ms, "master": masters}
