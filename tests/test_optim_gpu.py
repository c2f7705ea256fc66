"""Gradient norm and AdamW on the GPU against their formulas in 64 bits.

Tolerances (u = 2^-24), from the roundings of the formulas' fp32 operations and constants, set before the first run:
  m'   6 u (|b1 m| + |c1 g|)          v'   8 u v'
  p'   uo |p'| + 6 u (|p| + |step|) + 24 u lr_t (|b1 m| + |c1 g|) / (r / sqrt(bc2) + eps)
  norm 4 u relative (fp64 sums, one rounding), the factor the same
Stored 8-bit values: each must be the neighbour that the hash picks; where the exact position is within 2^-15 of a spacing of the
point at which the pick changes, either neighbour passes (fp32 places a value to 2^-20 of a spacing)."""
import math

import pytest
import torch

import all_gather_amd as mr
from gpu_util import TORCH_DT, device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UO = {"fp32": U, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
HY = dict(betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def tensors(gen, counts, dtype, scale, gap=0):
    """Views of one flat buffer, `gap` elements between them (so they start at any phase)."""
    total = sum(counts) + gap * (len(counts) + 1)
    flat = (scale * torch.randn(max(total, 1), generator=gen)).to(TORCH_DT[dtype]).to(device())
    out, at = [], gap
    for n in counts:
        out.append(flat[at:at + n])
        at += n + gap
    return out


def random_state(gen, params, bits, master, scale=1e-2):
    st = mr.adamw_init(params, bits, master)
    at, n = mr.adamw_offsets([p.numel() for p in params])
    live = torch.zeros(n, dtype=torch.bool)
    for a, p in zip(at, params):
        live[a:a + p.numel()] = True
    if bits == 32:
        st.m.copy_(torch.where(live, scale * torch.randn(n, generator=gen), 0.0))
        st.v.copy_(torch.where(live, (scale * torch.randn(n, generator=gen)) ** 2, 0.0))
    else:
        st.m.view(torch.uint8).copy_(torch.where(live, torch.randint(0, 256, (n,), generator=gen), 0).to(torch.uint8))
        codes = st.m.view(torch.uint8)
        codes[(codes & 127) == 127] = 0x38   # no NaN codes
        st.v.view(torch.uint8).copy_(torch.where(live, torch.randint(0, 127, (n,), generator=gen), 0).to(torch.uint8))
        for s in (st.m_scale, st.v_scale):
            s.view(torch.uint8).copy_(torch.randint(105, 120, (n // 32,), generator=gen).to(torch.uint8))
    return st


def clone(st):
    return mr.AdamWState(*(None if t is None else t.clone() for t in (st.m, st.v, st.m_scale, st.v_scale, st.master)))


def flat64(parts, at, n):
    out = torch.zeros(n, dtype=torch.float64)
    for a, p in zip(at, parts):
        out[a:a + p.numel()] = p.detach().double().cpu()
    return out


def key(seed, step):
    mask = (1 << 64) - 1
    z = (seed + 0x9E3779B97F4A7C15 * step) & mask
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
    return (z ^ (z >> 31)) & 0xFFFFFFFF


def hash_bits(n, seed, step):
    x = (torch.arange(n) * 0x9E3779B1 + key(seed, step)) & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    return x ^ (x >> 15)


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {int(bad.nonzero()[0])}: " \
        f"got {got[bad][0]!r} want {want[bad][0]!r} tol {tol[bad][0]!r}"


def check_codes(codes, scale, x, r16, floor, what):
    """Stored codes and scales against the exact values x (64 bits): the scale is the smallest that brings the block's
    largest to 448 or less, every code the neighbour that r16 picks."""
    x = x.view(-1, 32)
    byte = scale.view(torch.uint8).cpu().int()
    top = x.abs().amax(1)
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-127).nan_to_num(neginf=-127).int() + 127
    edge = (top / 448 / torch.exp2(e.double() - 127 - 1) - 1).abs() < 16 * U  # within rounding of a power of two
    edge |= (top / 448 / torch.exp2(e.double() - 127) - 1).abs() < 16 * U
    assert bool(((byte == e) | edge).all()), f"{what}: scales"
    y = x.abs() / torch.exp2(byte.double() - 127)[:, None]
    q = codes.view(torch.uint8).cpu()
    got = q.view(torch.float8_e4m3fn).double().view(-1, 32)
    assert bool(((got == 0) | (torch.sign(got) == torch.sign(x))).all()), f"{what}: signs"
    spacing = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    pos = y / spacing + r16.view(-1, 32).double() / 65536
    want = torch.floor(pos) * spacing
    near = (pos - torch.round(pos)).abs() < 2.0 ** -15
    other = (torch.round(pos) + torch.where(torch.floor(pos) == torch.round(pos), -1, 0)) * spacing
    if floor:
        want = torch.where((y > 0) & (want == 0), 2.0 ** -9, want)
        other = torch.where((y > 0) & (other == 0), 2.0 ** -9, other)
    bad = (got.abs() != want) & ~(near & (got.abs() == other))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} codes, y {y[bad][:3]} got {got[bad][:3]} want {want[bad][:3]}"


def check_adamw(counts, dtype, gdtype="same", bits=32, master=False, clip=None, in_place=True, gap=0, step=3, lr=1e-3, seed=11, gen=0):
    print(f"[case] adamw {len(counts)} tensors {sum(counts)} elements {dtype}/{gdtype} bits={bits} master={master} clip={clip} "
          f"in_place={in_place} gap={gap}", flush=True)
    gen = torch.Generator().manual_seed(gen)
    gname = dtype if gdtype == "same" else gdtype
    params, grads = tensors(gen, counts, dtype, 0.5, gap), tensors(gen, counts, gname, 1e-2, gap)
    st = random_state(gen, params, bits, master)
    if master:
        st.master.add_(1e-4 * (st.master != 0))
    at, n = mr.adamw_offsets(counts)
    f = 1.0 if clip is None else clip[1]
    g = flat64(grads, at, n) * float(torch.tensor(f))
    p = st.master.double().cpu() if master else flat64(params, at, n)
    m0, v0 = (t.double().cpu() for t in st.moments())
    if bits == 8:  # v0 as the exact square
        r0 = (st.v.double().cpu().view(-1, 32) * st.v_scale.double().cpu().view(-1, 1)).view(-1)
        v0 = r0 * r0
    (b1, b2), eps, wd = HY["betas"], HY["eps"], HY["weight_decay"]
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    den = torch.sqrt(v) / math.sqrt(1 - b2 ** step) + eps
    lr_t = lr / (1 - b1 ** step)
    new = p * (1 - lr * wd) - lr_t * m / den
    mag = (b1 * m0).abs() + ((1 - b1) * g).abs()
    c = None if clip is None else torch.tensor(clip, device=device())
    po, so = params, st
    if not in_place:
        po = [torch.full_like(t, float("nan")) for t in params]
        so = clone(st)
        for t in (so.m, so.v, so.m_scale, so.v_scale, so.master):
            if t is not None:
                t.view(torch.uint8).fill_(0x55)
    before = [t.clone() for t in params]
    mr.adamw_step(params, grads, st, lr, step, params_out=None if in_place else po, state_out=None if in_place else so, clip=c,
                  seed=seed, **HY)
    torch.cuda.synchronize()
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(before, params))
    tol = 6 * U * (p.abs() + (p - new).abs()) + 24 * U * lr_t * mag / den
    live = torch.zeros(n, dtype=torch.bool)
    for a, k in zip(at, counts):
        live[a:a + k] = True
    got = flat64(po, at, n)
    lowest = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}[dtype]
    close(got[live], new[live], (UO[dtype] * new.abs() + tol + lowest)[live], "params")
    if master:
        close(so.master.cpu()[live], new[live], (U * new.abs() + tol)[live], "master")
        assert torch.equal(torch.cat([t.cpu() for t in po]), so.master.cpu()[live].to(TORCH_DT[dtype]))
        assert not bool(so.master.cpu()[~live].any())
    m, v = torch.where(live, m, 0.0), torch.where(live, v, 0.0)
    if bits == 32:
        close(so.m, m, 6 * U * mag, "m")
        close(so.v, v, 8 * U * v + 2.0 ** -149, "v")
    else:
        bits32 = hash_bits(n, seed, step)
        check_codes(so.m, so.m_scale, m, bits32 & 0xFFFF, False, "m")
        check_codes(so.v, so.v_scale, torch.sqrt(v), bits32 >> 16, True, "v")


COUNTS = [[1], [31], [32], [33, 1, 0, 64], [7, 1024, 1025, 2047, 2048, 2049, 5], [100003], [0, 8, 4096, 0, 333, 0]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("dtype,gdtype,master", [("fp32", "same", False), ("bf16", "same", False), ("bf16", "fp32", False),
                                                 ("bf16", "fp32", True), ("bf16", "same", True), ("fp16", "same", False),
                                                 ("fp16", "fp32", False), ("fp16", "fp32", True), ("fp16", "same", True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(counts, dtype, gdtype, master, bits):
    k = len(counts) + sum(counts)
    check_adamw(counts, dtype, gdtype, bits, master, clip=(2.0, 0.375, 1.0) if k % 2 else None, in_place=k % 3 != 0, gap=k % 4)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors(bits):
    """More tensors than one launch takes, empty ones between."""
    gen = torch.Generator().manual_seed(1)
    counts = [int(c) for c in torch.randint(0, 3000, (203,), generator=gen)]
    counts[79] = counts[80] = counts[81] = 0
    check_adamw(counts, "bf16", "same", bits, gap=1)
    check_adamw(counts[:81], "fp32", "same", bits, in_place=False)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_step_left_out(bits, master):
    """clip says a gradient is not finite: every output is its input, in place and not."""
    gen = torch.Generator().manual_seed(2)
    counts = [33, 5000, 1]
    params, grads = tensors(gen, counts, "bf16", 0.5, 1), tensors(gen, counts, "bf16", float("inf"), 0)
    st = random_state(gen, params, bits, master)
    c = torch.tensor([float("inf"), 0.0, 0.0], device=device())
    keep, pk = clone(st), [p.clone() for p in params]
    out, po = clone(st), [torch.zeros_like(p) for p in params]
    for t in (out.m, out.v, out.m_scale, out.v_scale, out.master):
        if t is not None:
            t.view(torch.uint8).fill_(0x55)
    mr.adamw_step(params, grads, st, 1e-3, 1, params_out=po, state_out=out, clip=c)
    mr.adamw_step(params, grads, st, 1e-3, 1, clip=c)
    torch.cuda.synchronize()
    for a in (st, out):
        for x, y in zip((a.m, a.v, a.m_scale, a.v_scale, a.master), (keep.m, keep.v, keep.m_scale, keep.v_scale, keep.master)):
            assert (x is None) == (y is None) and (x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)))
    for a, b, c2 in zip(params, pk, po):
        assert torch.equal(a, b) and torch.equal(c2, b)


def test_not_finite_gradient_without_clip():
    """Only the element (32-bit moments) or its block (8-bit) is lost."""
    for bits in (32, 8):
        for bad in (float("nan"), float("inf")):
            p, g = torch.ones(200, device=device()), torch.full((200,), 1e-2, device=device())
            g[70] = bad
            st = mr.adamw_init([p], bits)
            mr.adamw_step([p], [g], st, 1e-3, 1)
            mr.adamw_step([p], [torch.full_like(g, 1e-2)], st, 1e-3, 2)
            ok = torch.ones(200, dtype=torch.bool)
            ok[70 if bits == 32 else slice(64, 96)] = False
            assert torch.isfinite(p.cpu()[ok]).all() and torch.isnan(p.cpu()[~ok]).all(), (bits, bad)


@pytest.mark.parametrize("bits,low", [(32, -55), (8, -70)])
def test_gradients_of_every_size(bits, low):
    """With eps = 0 the first step moves a parameter by lr whatever the gradient's size: no over- or underflow on the way to the
    quotient, from 2^low (where the fp32 v of the 32-bit form is still normal) to 2^46.  A tolerance of 24 u of the step, 2 u of p."""
    e = torch.arange(low, 47)
    g = torch.ldexp(torch.ones(len(e)), e).repeat_interleave(32).to(device())
    for sign in (1.0, -1.0):
        p, st = torch.ones_like(g), mr.adamw_init([g], bits)
        mr.adamw_step([p], [sign * g], st, 0.125, 1, weight_decay=0.0, eps=0.0)
        assert float((p.double() - (1 - sign * 0.125)).abs().max()) <= 24 * U * 0.125 + 2 * U
        m, v = st.moments()
        # the 8-bit form's roots as they are stored: their squares leave fp32's range
        r = v.sqrt() if bits == 32 else (st.v.float().view(-1, 32) * st.v_scale.float().view(-1, 1)).view(-1)
        assert float((m / (sign * 0.1 * g) - 1).abs().max()) <= (1 / 8 if bits == 8 else 8 * U)
        assert float((r / (0.001 ** 0.5 * g) - 1).abs().max()) <= (1 / 8 if bits == 8 else 16 * U)


def test_zero_state_and_zero_gradient():
    for bits in (32, 8):
        p, g = torch.ones(100, device=device()), torch.zeros(100, device=device())
        st = mr.adamw_init([p], bits)
        for t in range(1, 4):
            mr.adamw_step([p], [g], st, 1e-3, t, weight_decay=0.0)
        m, v = st.moments()
        assert torch.all(p == 1) and not m.any() and not v.any()


def test_eight_bit_moments_follow_the_gradients():
    """The stored second moment follows a fall of the gradients by 16, which rounding to nearest would never show: its mean square
    root over 65536 elements ends within 5% of the exact recurrence's (the mean's sampling error is below 1%), the first moment's
    mean too."""
    n = 65536
    p = torch.zeros(n, device=device())
    st = mr.adamw_init([p], 8)
    m64 = v64 = 0.0
    b1, b2 = 0.9, 0.995
    steps = 3000
    high, low = torch.full((n,), 1.0, device=device()), torch.full((n,), 1.0 / 16, device=device())
    for t in range(1, steps + 1):
        x, g = (1.0, high) if t < steps // 2 else (1.0 / 16, low)
        mr.adamw_step([p], [g], st, 0.0, t, betas=(b1, b2), seed=5)
        m64, v64 = b1 * m64 + (1 - b1) * x, b2 * v64 + (1 - b2) * x * x
    m, v = st.moments()
    assert abs(float(v.sqrt().double().mean()) / math.sqrt(v64) - 1) < 0.05
    assert abs(float(m.double().mean()) / m64 - 1) < 0.05


def test_stochastic_rounding_keeps_the_mean():
    """One value stored under 512 seeds: the mean of what is stored is the value to 6 standard errors (a spacing of at
    most 1/8 of the value gives a deviation of at most half of it)."""
    n = 32 * 64
    g = torch.linspace(0.5, 1.0, n, device=device())
    total = torch.zeros(n, dtype=torch.float64, device=device())
    for seed in range(512):
        p, st = torch.zeros(n, device=device()), mr.adamw_init([torch.empty(n, device=device())], 8)
        mr.adamw_step([p], [g], st, 0.0, 1, betas=(0.0, 0.0), seed=seed)
        total += st.moments()[0].double()
    err = (total / 512 - g.double()).abs() / g.double()
    assert float(err.max()) < 6 * (1 / 16) / math.sqrt(512)


def test_seed_and_step_change_the_rounding_and_nothing_else_does():
    gen = torch.Generator().manual_seed(4)
    p, g = tensors(gen, [5000], "bf16", 1.0), tensors(gen, [5000], "bf16", 1e-2)
    st0 = random_state(gen, p, 8, False)

    def codes(seed, step):
        st, q = clone(st0), [t.clone() for t in p]
        mr.adamw_step(q, g, st, 1e-3, step, seed=seed)
        return st.m.view(torch.uint8)

    a = codes(1, 2)
    assert torch.equal(a, codes(1, 2)) and not torch.equal(a, codes(2, 2)) and not torch.equal(a, codes(1, 3))


def check_norm(counts, dtype, max_norm=1.0, scale=1.0, gap=0, spread=1.0):
    print(f"[case] grad norm {len(counts)} tensors {sum(counts)} elements {dtype} max_norm={max_norm} scale={scale} gap={gap}", flush=True)
    grads = tensors(torch.Generator().manual_seed(len(counts)), counts, dtype, spread, gap)
    out = torch.full((3,), 7.0, device=device())
    mr.grad_norm(grads, out, max_norm=max_norm, scale=scale)
    norm = scale * math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in grads))
    f = scale * (min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0)
    got = out.double().cpu().tolist()
    assert got[2] == 1.0 and abs(got[0] - norm) <= 4 * U * norm and abs(got[1] - f) <= 4 * U * f, (got, norm, f)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts", [[1], [5, 0, 3], [4095, 4096, 4097, 1], [1 << 20, 77, 123457], [3] * 129, [40000] * 257], ids=len)
def test_grad_norm(counts, dtype):
    check_norm(counts, dtype)
    check_norm(counts, dtype, max_norm=0.0, scale=0.25, gap=1)
    check_norm(counts, dtype, max_norm=1e6, gap=3)


def test_grad_norm_of_nothing():
    out = torch.full((3,), 7.0, device=device())
    mr.grad_norm([], out, max_norm=1.0, scale=0.5)
    assert out.tolist() == [0.0, 0.5, 1.0]
    mr.grad_norm([torch.empty(0, device=device())], out)
    assert out.tolist() == [0.0, 1.0, 1.0]


def test_grad_norm_range_and_not_finite():
    """Squares far outside fp32's range are summed; an infinity or NaN anywhere clears the flag."""
    out = torch.empty(3, device=device())
    for x in (1e30, 1e-30):
        mr.grad_norm([torch.full((10000,), x, device=device())], out, max_norm=1.0)
        assert abs(float(out[0]) / (float(torch.tensor(x)) * 100) - 1) < 4 * U and float(out[2]) == 1.0
    for bad in (float("inf"), float("-inf"), float("nan")):
        for dt in (torch.bfloat16, torch.float16, torch.float32):
            gs = [torch.ones(5000, dtype=dt, device=device()) for _ in range(3)]
            gs[1][4999] = bad
            mr.grad_norm(gs, out, max_norm=1.0)
            assert float(out[1]) == 0.0 and float(out[2]) == 0.0 and not math.isfinite(float(out[0]))
    mr.grad_norm([torch.ones(4, device=device())], out)
    assert out.tolist() == [2.0, 1.0, 1.0]  # the workspace is as it was


def test_norm_feeds_the_step_in_a_graph():
    """Norm and step captured together, replayed with new gradients and eager work between: every replay equals the eager
    pair's bits."""
    gen = torch.Generator().manual_seed(12)
    counts = [100, 70001, 3]
    params = tensors(gen, counts, "bf16", 1.0)
    grads = [t.clone() for t in tensors(gen, counts, "bf16", 1e-1)]
    st = mr.adamw_init(params, 8)
    st0, p0 = clone(st), [p.clone() for p in params]
    rec, rec2 = torch.empty(3, device=device()), torch.empty(3, device=device())
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        mr.grad_norm(grads, rec, max_norm=1.0)
        mr.adamw_step(params, grads, st, 1e-2, 1, clip=rec)
    for k in range(4):
        for g in grads:
            g.mul_(1.5).add_(1e-3)
        mr.grad_norm(grads, rec2, max_norm=1.0)
        mr.adamw_step(p0, grads, st0, 1e-2, 1, clip=rec2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rec, rec2) and all(torch.equal(a, b) for a, b in zip(params, p0)), k
        assert torch.equal(st.m.view(torch.uint8), st0.m.view(torch.uint8))
        assert torch.equal(st.v.view(torch.uint8), st0.v.view(torch.uint8))
    del graph


def test_offsets_past_32_bits():
    n = (1 << 32) + 4001
    p = torch.ones(n, dtype=torch.bfloat16, device=device())
    g = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device=device())
    g[-1] = 2.0 ** -4
    st = mr.adamw_init([p], 8)
    out = torch.empty(3, device=device())
    mr.grad_norm([g], out)
    assert abs(float(out[0]) / math.sqrt((n - 1) * 2.0 ** -20 + 2.0 ** -8) - 1) <= 4 * U
    mr.adamw_step([p], [g], st, 2.0 ** -3, 1, weight_decay=0.0, eps=0.0)
    # the first step moves every element by lr
    assert float(p[:4096].float().max()) == float(p[-4096:].float().min()) == 0.875
    assert float(p[(1 << 32) - 8:(1 << 32) + 8].float().max()) == 0.875
    m = st.m[-64:].float() * torch.repeat_interleave(st.m_scale[-2:].float(), 32)
    tail = n % 32
    assert abs(float(m[32 + tail - 1]) / (0.1 * 2.0 ** -4) - 1) <= 1 / 8 and not bool(m[32 + tail:].any())


@pytest.mark.parametrize("low,high", [(-133, -80), (-90, -60), (-149, -120)])
def test_eight_bit_second_moments_of_the_smallest_sizes(low, high):
    """Second moments far below fp32's squares: the root of a gradient of 2^low and more is kept, a zero gradient leaves it decayed, and
    none becomes zero.  fp32 gradients below 2^-126 have fewer bits, which the tolerance of one E4M3 spacing covers."""
    e = torch.arange(low, high)
    g = torch.ldexp(torch.ones(len(e), dtype=torch.float64), e).float().repeat_interleave(32).to(device())
    st = mr.adamw_init([g], 8)
    p = torch.ones_like(g)
    mr.adamw_step([p], [g], st, 0.125, 1, weight_decay=0.0, eps=1e-8, betas=(0.5, 0.75))

    def root():
        return st.v.cpu().double() * torch.exp2(st.v_scale.view(torch.uint8).cpu().double() - 127).repeat_interleave(32)

    want = 0.5 * g.double().cpu()
    # the smallest number of the format is 2^-9 * 2^-127: below it a root is raised to it
    tol = torch.maximum(want / 8, torch.tensor(2.0 ** -136, dtype=torch.float64))
    assert bool((root() > 0).all()) and bool(((root() - want).abs() <= tol).all())
    before = root()
    mr.adamw_step([p], [torch.zeros_like(g)], st, 0.125, 2, weight_decay=0.0, eps=1e-8, betas=(0.5, 0.75))
    want = before * 0.75 ** 0.5
    tol = torch.maximum(want / 8, torch.tensor(2.0 ** -136, dtype=torch.float64))
    assert bool((root() > 0).all()) and bool(((root() - want).abs() <= tol).all())


def test_eight_bit_step_without_eps_at_the_smallest_sizes():
    """With eps = 0 the first step moves a parameter by lr at every gradient down to 2^-120: neither the second moment nor the
    quotient leaves fp32's range on the way.  The tolerance is test_gradients_of_every_size's."""
    e = torch.arange(-120, -60)
    g = torch.ldexp(torch.ones(len(e), dtype=torch.float64), e).float().repeat_interleave(32).to(device())
    p, st = torch.ones_like(g), mr.adamw_init([g], 8)
    mr.adamw_step([p], [g], st, 0.125, 1, weight_decay=0.0, eps=0.0)
    assert float((p.double() - 0.875).abs().max()) <= 24 * U * 0.125 + 2 * U
