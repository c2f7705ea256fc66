"""Muon's step against its formulas in 64 bits.

Tolerances.  The orthogonalised update X is compared in the Frobenius norm with the iteration in 64 bits.  How far roundings move
it depends on the spectrum (a small singular value and the noise beside it are both raised up to 485-fold), so the bound is
measured with the documented arithmetic itself: the same iteration in 64 bits with X, A and P rounded to fp16 times 2^12 (products =
16) or in fp32 throughout (32).  The kernel's roundings are those, of other sums in another order: it may be off by 1.5 times as
much (16) or 4 times (32, whose two pieces resolve 2^-22 against fp32's 2^-24), and by 2^-20 for the fp32 arithmetic around it.
Everything elementwise (momentum, update, masters) is fp32 with a few roundings: 2^-21 of the terms."""
import math

import pytest
import torch

import all_gather_amd as mr
from gpu_util import TORCH_DT, device

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.775, 2.0315)


def half(x):
    return (x * 4096).half().double() / 4096


def same(x):
    return x


def iterate(u, rnd=same, steps=5, coef=COEF, eps=1e-7, dtype=torch.float64):
    if u.shape[0] > u.shape[1]:
        return iterate(u.t().contiguous(), rnd, steps, coef, eps, dtype).t()
    x = rnd((u.double() / max(float(u.double().norm()), eps)).to(dtype))
    flat = list(coef) * steps if not isinstance(coef[0], tuple) else [c for k in coef for c in k]
    eye = torch.eye(u.shape[0], device=u.device, dtype=dtype)
    for i in range(steps):
        a, b, c = flat[3 * i:3 * i + 3]
        q = rnd(x @ x.t())
        x = rnd(a * eye + b * q + c * (q @ q)) @ x
        if i + 1 < steps:
            x = rnd(x)
    return x.double()


def bound(u, products, **kw):
    want = iterate(u, **kw)
    if products == 16:
        return want, 1.5 * float((iterate(u, half, **kw) - want).norm()) + 2.0 ** -20 * float(want.norm())
    return want, 4 * float((iterate(u, dtype=torch.float32, **kw) - want).norm()) + 2.0 ** -20 * float(want.norm())


def matrix(r, c, kind, gen):
    n = lambda *s: torch.randn(*s, generator=gen, device=device())  # noqa: E731
    if kind == "low":
        k = min(4, r, c)
        return n(r, k) @ n(k, c) + 0.05 * n(r, c)
    return n(r, c)


def factor(r, c, adjust):
    return math.sqrt(max(1.0, r / c)) if adjust == "ratio" else 0.2 * math.sqrt(max(r, c))


def update_alone(u, products, **kw):
    """X, by a step of lr 1 without momentum on zero fp32 parameters."""
    p, g = [torch.zeros_like(x, dtype=torch.float32) for x in u], list(u)
    st = mr.muon_init(p)
    mr.muon_step(p, g, st, 1.0, momentum=0.0, nesterov=False, weight_decay=0.0, products=products, **kw)
    return [-x.double() / factor(*x.shape, kw.get("adjust", "ratio")) for x in p]


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (31, 33), (64, 64), (65, 63), (100, 300), (128, 127), (257, 129), (511, 700), (512, 512),
          (513, 512), (700, 1300), (1025, 640), (130, 5000), (2047, 300), (2048, 2048), (2049, 2500), (2600, 2050), (2304, 6001)]


@pytest.mark.parametrize("products", [16, 32])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalised(shape, products):
    print(f"[case] {shape} products={products}", flush=True)
    gen = torch.Generator(device=device()).manual_seed(shape[0] * 7919 + shape[1])
    for kind in ("full", "low"):
        u = matrix(*shape, kind, gen)
        got, = update_alone([u], products)
        want, tol = bound(u, products)
        off = float((got - want).norm())
        assert off <= tol, (kind, off, tol, float(want.norm()))


def test_singular_values_become_one():
    gen = torch.Generator(device=device()).manual_seed(5)
    x, = update_alone([matrix(256, 700, "full", gen)], 16)
    s = torch.linalg.svdvals(x.cpu())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("products", [16, 32])
def test_lists_of_every_size(products):
    """70 matrices of all tile sizes in one call, empty ones among them: each as if alone."""
    gen = torch.Generator(device=device()).manual_seed(11)
    shapes = [SHAPES[i % 16] if i % 9 else (0, 5) for i in range(70)]
    u = [matrix(*s, "full", gen) if s[0] else torch.zeros(s, device=device()) for s in shapes]
    got = update_alone(u, products)
    for i, s in enumerate(shapes):
        if s[0]:
            alone, = update_alone([u[i]], products)
            assert torch.equal(got[i], alone), (i, s)


@pytest.mark.parametrize("products", [16, 32])
def test_many_large_matrices(products):
    """Enough of them for the wide tiles: each against the iteration in 64 bits, both ways round.  Alone, on square tiles, a matrix gives
    the same bits: its sums run over the same columns in the same order.  Not so in two pieces, where an element of A or P is the sum
    hi lo + lo hi + hi hi of its row and column or, mirrored, of its column and row, by the tile that it falls in."""
    gen = torch.Generator(device=device()).manual_seed(14)
    shapes = [(2049, 2500)] * 4 + [(2500, 2047), (1025, 6001), (2304, 3001), (1500, 1100), (600, 700)]
    u = [matrix(*s, "low" if i % 2 else "full", gen) for i, s in enumerate(shapes)]
    got = update_alone(u, products)
    for i in (0, 3, 4, 5, 6, 7, 8):
        want, tol = bound(u[i], products)
        off = float((got[i] - want).norm())
        assert off <= tol, (shapes[i], off, tol)
        alone, = update_alone([u[i]], products)
        assert torch.equal(got[i], alone) if products == 16 else float((got[i] - alone).norm()) <= 2 * tol, shapes[i]


def test_group_larger_than_the_workspace_limit():
    """Matrices whose workspace passes 2 GiB together are worked off in parts."""
    gen = torch.Generator(device=device()).manual_seed(12)
    shapes = [(2048, 49152), (2048, 49152), (49152, 2048), (100, 100)]
    u = [matrix(*s, "full", gen) for s in shapes]
    got = update_alone(u, 16)
    for i in (0, 2, 3):
        alone, = update_alone([u[i]], 16)
        assert torch.equal(got[i], alone)


@pytest.mark.parametrize("coef,steps", [((2.0, -1.5, 0.5), 8), (((3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)), 3), ((1.5, -0.5, 0.0), 4),
                                        ((3.4445, -4.775, 2.0315), 1)])
def test_other_polynomials(coef, steps):
    gen = torch.Generator(device=device()).manual_seed(13)
    for products in (16, 32):
        u = matrix(150, 260, "full", gen)
        got, = update_alone([u], products, coefficients=coef, steps=steps)
        want, tol = bound(u, products, coef=coef, steps=steps)
        assert float((got - want).norm()) <= tol


@pytest.mark.parametrize("dtype,gdtype,master,products", [("bf16", "bf16", False, 16), ("fp16", "fp16", False, 16), ("fp32", "fp32", False, 32),
                                                          ("bf16", "fp32", True, 32), ("fp16", "fp32", True, 16), ("bf16", "bf16", True, 16)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(dtype, gdtype, master, products, nesterov):
    gen = torch.Generator(device=device()).manual_seed(21)
    n = lambda *s: torch.randn(*s, generator=gen, device=device())  # noqa: E731
    shapes = [(33, 70), (600, 515), (1, 1), (129, 128), (2100, 2060)]
    lr, wd, mu, f = 0.02, 0.1, 0.9, 0.7
    clip = torch.tensor([3.0, f, 1.0], device=device())
    flat = (0.02 * n(1 + sum(a * b for a, b in shapes))).to(TORCH_DT[dtype])      # one element off the 16-byte grid
    params = [x.view(s) for x, s in zip(flat[1:].split([a * b for a, b in shapes]), shapes)]
    gflat = (1e-3 * n(1 + flat.numel())).to(TORCH_DT[gdtype])
    grads = [x.view(s) for x, s in zip(gflat[1:-1].split([a * b for a, b in shapes]), shapes)]
    st = mr.muon_init(params, master=master)
    at, total = mr.adamw_offsets([a * b for a, b in shapes])
    for a, s in zip(at, shapes):
        st.m[a:a + s[0] * s[1]] = 1e-3 * n(s[0] * s[1])
        if master:
            st.master[a:a + s[0] * s[1]] += 1e-5 * n(s[0] * s[1])
    out = [torch.full_like(p, 9.0) for p in params]
    so = mr.MuonState(torch.full_like(st.m, 9.0), torch.full_like(st.m, 9.0) if master else None)
    kw = dict(momentum=mu, nesterov=nesterov, weight_decay=wd, adjust="rms", products=products, clip=clip)
    mr.muon_step(params, grads, st, lr, params_out=out, state_out=so, **kw)
    live = torch.zeros_like(st.m, dtype=torch.bool)
    for i, (a, s) in enumerate(zip(at, shapes)):
        k = s[0] * s[1]
        live[a:a + k] = True
        g, m = f * grads[i].double(), st.m[a:a + k].double().view(s)
        m2 = mu * m + (1 - mu) * g
        assert ((so.m[a:a + k].view(s).double() - m2).abs() <= 2.0 ** -21 * (m.abs() + g.abs())).all()
        u = mu * m2 + (1 - mu) * g if nesterov else m2
        x, tol = bound(u, products)
        scale = lr * factor(*s, "rms")
        old = (st.master[a:a + k].view(s) if master else params[i]).double()
        want = (1 - lr * wd) * old - scale * x
        tol = scale * (tol + 2.0 ** -20 * float(x.norm())) + 2.0 ** -22 * float(old.norm())
        if master:
            assert float((so.master[a:a + k].view(s).double() - want).norm()) <= tol
            assert torch.equal(out[i], so.master[a:a + k].view(s).to(out[i].dtype))
        eps = torch.finfo(out[i].dtype).eps / 2 if dtype != "fp32" else 0.0
        assert float((out[i].double() - want).norm()) <= tol + eps * float(want.norm()) + 2.0 ** -25 * math.sqrt(k)
    assert (so.m[~live] == 0).all() and (not master or (so.master[~live] == 0).all())
    # in place, the same bits; and again
    ip, ist = [p.clone() for p in params], mr.MuonState(st.m.clone(), st.master.clone() if master else None)
    mr.muon_step(ip, grads, ist, lr, **kw)
    assert all(torch.equal(a, b) for a, b in zip(ip, out)) and torch.equal(ist.m, so.m) and (not master or torch.equal(ist.master, so.master))
    # a step that is not taken leaves everything as it was
    clip[2] = 0.0
    clip[1] = 0.0
    gflat[5] = math.nan
    mr.muon_step(params, grads, st, lr, params_out=out, state_out=so, **kw)
    for i, (a, s) in enumerate(zip(at, shapes)):
        k = s[0] * s[1]
        assert torch.equal(so.m[a:a + k], st.m[a:a + k])
        if master:
            assert torch.equal(so.master[a:a + k], st.master[a:a + k]) and torch.equal(out[i].view(-1), st.master[a:a + k].to(out[i].dtype))
        else:
            assert torch.equal(out[i], params[i])


def test_zeros_infinities_and_tiny_gradients():
    gen = torch.Generator(device=device()).manual_seed(31)
    u = [matrix(70, 90, "full", gen) for _ in range(6)]
    alone = update_alone([u[5]], 16)[0]
    u[0].zero_()
    u[1][3, 4] = math.inf
    u[2][3, 4] = math.nan
    u[3] *= 1e30
    u[4] *= 1e-30
    got = update_alone(u, 16, eps=2.0 ** -114)
    assert (got[0] == 0).all() and got[1].isnan().any() and got[2].isnan().any()
    for i in (3, 4):
        want, tol = bound(u[i], 16, eps=2.0 ** -114)
        assert float((got[i] - want).norm()) <= tol, i
    assert torch.equal(got[5], alone)
    # a norm far below eps: the update is nearly zero
    small = update_alone([u[4]], 16)[0]
    assert float(small.abs().max()) < 1e-3


def test_workspace_of_the_caller():
    gen = torch.Generator(device=device()).manual_seed(41)
    shapes = [(300, 200), (64, 513), (700, 700)]
    u = [matrix(*s, "full", gen) for s in shapes]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        want = update_alone(u, 32)
        need = mr.muon_workspace_bytes(shapes, 32)
        buf = torch.empty(need, dtype=torch.uint8, device=device())
        mr.set_workspace(buf, s)
        got = update_alone(u, 32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        mr.set_workspace(buf[:need // 2 // 256 * 256], s)
        with pytest.raises(mr.MRError) as e:
            update_alone(u, 32)
        assert e.value.status == -4
        mr.set_workspace(None, s)
    torch.cuda.synchronize()


def test_replays_beside_eager_steps():
    gen = torch.Generator(device=device()).manual_seed(51)
    shapes = [(200, 300), (700, 513), (2048, 2100)]

    def make():
        p = [torch.zeros(s, device=device(), dtype=torch.bfloat16) for s in shapes]
        return p, mr.muon_init(p)

    grads = [matrix(*s, "full", gen).bfloat16() for s in shapes]
    pg, sg = make()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mr.muon_step(pg, grads, sg, 0.01)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mr.muon_step(pg, grads, sg, 0.01)
    for t in (*pg, sg.m):
        t.zero_()
    pe, se = make()
    po, so = make()
    for i in range(3):
        for g, sh in zip(grads, shapes):
            g.copy_(matrix(*sh, "full", gen))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(s):
            mr.muon_step(po, grads, so, 0.01)
        torch.cuda.synchronize()
        mr.muon_step(pe, grads, se, 0.01)
        torch.cuda.synchronize()
        for a, b, c in zip(pg, pe, po):
            assert torch.equal(a, b) and torch.equal(c, b), i
        assert torch.equal(sg.m, se.m) and torch.equal(so.m, se.m)
