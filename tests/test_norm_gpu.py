"""Layer norm on the GPU against the formula in 64 bits.

Tolerances, with u = 2^-24 (fp32) and uo the output type's unit roundoff, set from the kernels' longest chains of
fp32 operations (at most 128 for a row's sums, x included) before the first run:
  x       128 u sum|terms| + uo |x|
  mean    128 u A                      A = the row's largest sum|terms|
  rstd    rstd (256 u A rstd + 8 u)    (a relative error of the variance of 2 * 128 u A / sigma, halved, doubled to be safe)
  y       uo |y| + 128 u |gamma| (1 + |xh|) (1 + A rstd) + 8 u |beta|
  dx      uo |dx| + 128 u rstd (|gd| + avg|gd| + (|xh| + X) avg(|gd| (|xh| + X))) + u |dres|,  X = (|x| + |mean|) rstd
  dgamma  uo |dgamma| + (R + 64) u sum |dy| (|xh| + X),  dbeta the same with |dy|;  R = rows one lane adds up
Each also allows the output type's smallest subnormal."""
import numpy as np
import pytest
import torch

import all_gather_amd as mr
from gpu_util import TORCH_DT, device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UO = {"fp32": U, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}
EPS = 1e-5


def rand(gen, rows, cols, dtype, offset=0.0):
    x = torch.randn(rows, cols, generator=gen) * torch.exp(0.5 * torch.randn(cols, generator=gen)) + offset
    return x.to(TORCH_DT[dtype]).to(device())


def close(got, want, tol, dtype, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= tol + TINY[dtype])
    n = int(bad.sum())
    if n:
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {i}: got {got[i]!r} want {want[i]!r} tol {tol[i]!r}")


def fwd_ref(bufs, residual, gamma, beta, cols):
    terms = [b.double().cpu() for b in bufs] + ([residual.double().cpu()] if residual is not None else [])
    x = torch.stack(terms).sum(0)
    a = torch.stack(terms).abs().sum(0)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
    g = torch.ones(cols, dtype=torch.float64) if gamma is None else gamma.double().cpu()
    b = torch.zeros(cols, dtype=torch.float64) if beta is None else beta.double().cpu()
    xh = (x - mean) * rstd
    return x, a, mean, rstd, xh, g, b


def check_forward(rows, cols, dtype, wdtype="same", W=1, res=False, gamma=True, beta=True, offset=0.0, place=None, seed=0):
    print(f"[case] norm forward {rows}x{cols} {dtype}/{wdtype} W={W} res={res} place={place}", flush=True)
    gen = torch.Generator().manual_seed(seed)
    wdt = TORCH_DT[dtype if wdtype == "same" else wdtype]
    bufs = [rand(gen, rows, cols, dtype, offset) for _ in range(W)]
    residual = rand(gen, rows, cols, dtype) if res else None
    g = (1 + 0.2 * torch.randn(cols, generator=gen)).to(wdt).to(device()) if gamma else None
    b = (0.2 * torch.randn(cols, generator=gen)).to(wdt).to(device()) if beta else None
    x, a, mean, rstd, xh, g64, b64 = fwd_ref(bufs, residual, g, b, cols)
    y = torch.full((rows, cols), float("nan"), dtype=TORCH_DT[dtype], device=device())
    x_out = torch.full_like(y, float("nan"))
    if place:  # y and x_out in the place of inputs
        y = bufs[0]
        x_out = residual if res else bufs[-1] if W > 1 else None
    m, r = torch.empty(rows, device=device()), torch.empty(rows, device=device())
    mr.layer_norm_forward(bufs, g, b, y, eps=EPS, residual=residual, x_out=x_out, mean=m, rstd=r)
    torch.cuda.synchronize()
    uo, top = UO[dtype], a.max(1, keepdim=True).values
    close(m, mean[:, 0], 128 * U * top[:, 0], "fp32", "mean")
    close(r, rstd[:, 0], rstd[:, 0] * (256 * U * (top * rstd)[:, 0] + 8 * U), "fp32", "rstd")
    if x_out is not None:
        close(x_out, x, 128 * U * a + uo * x.abs(), dtype, "x")
    want = xh * g64 + b64
    close(y, want, uo * want.abs() + 128 * U * g64.abs() * (1 + xh.abs()) * (1 + top * rstd) + 8 * U * b64.abs(), dtype, "y")


# every variant: a wave per row (1 and 2 packs a lane), workgroups of each width, the longest held rows and beyond
SHAPES = [(1, 1), (3, 2), (5, 7), (4, 8), (7, 9), (1, 511), (66, 512), (9, 513), (3, 1024), (2, 1025), (5, 2048), (3, 2049), (6, 4096),
          (2, 4097), (3, 8192), (2, 8193), (2, 16384), (1, 16385), (2, 32768), (2, 32769), (1, 70001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_forward_shapes(rows, cols, dtype):
    check_forward(rows, cols, dtype)


@pytest.mark.parametrize("W,res", [(1, True), (2, False), (3, True), (8, True), (16, False)])
@pytest.mark.parametrize("rows,cols", [(5, 300), (300, 1000), (4, 4096), (3, 9001), (2, 33000)])
def test_forward_of_a_sum(W, res, rows, cols):
    check_forward(rows, cols, "bf16", "fp32", W=W, res=res)
    check_forward(rows, cols, "fp32", W=W, res=res)


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
def test_forward_without_weights(gamma, beta):
    check_forward(33, 777, "fp16", gamma=gamma, beta=beta)


@pytest.mark.parametrize("cols", [100, 3000, 40000])
def test_forward_in_place(cols):
    for W, res in ((1, False), (1, True), (3, True), (2, False)):
        check_forward(17, cols, "bf16", W=W, res=res, place=True)


def test_forward_far_mean():
    """Rows a hundred deviations away from zero: the second pass works on deviations, so nothing cancels."""
    check_forward(64, 2000, "fp32", offset=100.0)
    check_forward(8, 40000, "fp32", offset=100.0)


def test_constant_and_single_column_rows():
    for cols in (1, 500, 5000, 40000):
        x = torch.full((3, cols), 2.5, device=device())
        y, g, b = torch.empty_like(x), torch.full((cols,), 3.0, device=device()), torch.full((cols,), 0.25, device=device())
        r = torch.empty(3, device=device())
        mr.layer_norm_forward([x], g, b, y, eps=EPS, rstd=r)
        assert torch.all(y == 0.25) and torch.allclose(r, torch.full_like(r, EPS ** -0.5), rtol=4 * U * 2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cols", [60, 600, 3000, 40000])
def test_not_finite_stays_in_its_row(bad, cols):
    x = torch.randn(9, cols, device=device())
    dy = torch.randn(9, cols, device=device())
    clean, y = torch.empty_like(x), torch.empty_like(x)
    mr.layer_norm_forward([x], None, None, clean)
    x[4, cols // 2] = bad
    m, r = torch.empty(9, device=device()), torch.empty(9, device=device())
    mr.layer_norm_forward([x], None, None, y, mean=m, rstd=r)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[4]).all()
    dx = torch.empty_like(x)
    mr.layer_norm_backward(dy, x, None, m, r, dx)
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[4]).all()


def check_backward(rows, cols, dtype, wdtype="same", dres=False, gamma=True, want=("dx", "dgamma", "dbeta"), place=None, seed=1):
    print(f"[case] norm backward {rows}x{cols} {dtype}/{wdtype} dres={dres} want={want} place={place}", flush=True)
    gen = torch.Generator().manual_seed(seed)
    wname = dtype if wdtype == "same" else wdtype
    wdt = TORCH_DT[wname]
    x, dy = rand(gen, rows, cols, dtype, 0.5), rand(gen, rows, cols, dtype)
    dr = rand(gen, rows, cols, dtype) if dres else None
    g = (1 + 0.2 * torch.randn(cols, generator=gen)).to(wdt).to(device()) if gamma else None
    x64 = x.double().cpu()
    var, mean = torch.var_mean(x64, 1, correction=0)
    m, r = mean.float().to(device()), (1 / torch.sqrt(var + EPS)).float().to(device())
    mean, rstd = m.double().cpu()[:, None], r.double().cpu()[:, None]
    dy64, g64 = dy.double().cpu(), torch.ones(cols, dtype=torch.float64) if g is None else g.double().cpu()
    xh, gd = (x64 - mean) * rstd, dy64 * g64
    dx64 = rstd * (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True))
    dr64 = dr.double().cpu() if dres else torch.zeros_like(dx64)
    dx64 = dx64 + dr64
    big = xh.abs() + (x64.abs() + mean.abs()) * rstd
    nan = float("nan")
    out = {"dx": torch.full_like(dy, nan) if "dx" in want else None,
           "dgamma": torch.full((cols,), nan, dtype=wdt, device=device()) if "dgamma" in want else None,
           "dbeta": torch.full((cols,), nan, dtype=wdt, device=device()) if "dbeta" in want else None}
    if place:
        out["dx"] = {"dy": dy, "x": x, "dres": dr}[place]
    mr.layer_norm_backward(dy, x, g, m, r, out["dx"], dgamma=out["dgamma"], dbeta=out["dbeta"], dres=dr)
    torch.cuda.synchronize()
    if out["dx"] is not None:
        tol = UO[dtype] * dx64.abs() + U * dr64.abs() + 128 * U * rstd * (
            gd.abs() + gd.abs().mean(1, keepdim=True) + big * (gd.abs() * big).mean(1, keepdim=True))
        close(out["dx"], dx64, tol, dtype, "dx")
    depth = (min(rows, 2048) + 64) * U
    for name, w64, mag in (("dgamma", (dy64 * xh).sum(0), (dy64.abs() * big).sum(0)), ("dbeta", dy64.sum(0), dy64.abs().sum(0))):
        if out[name] is not None:
            close(out[name], w64, UO[wname] * w64.abs() + depth * mag, wname, name)


@pytest.mark.parametrize("rows,cols", [(1, 1), (4, 3), (2, 8), (9, 33), (300, 512), (70, 513), (5, 1024), (41, 1025), (3, 2048), (7, 2049),
                                       (600, 4096), (3, 4097), (5, 8192), (2, 8193), (3, 10001), (2, 12289), (4, 16384), (3, 16385), (70, 20001), (1, 66000),
                                       (5, 60), (130, 100), (40, 200), (300, 10000)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "fp32"), ("fp16", "same"), ("fp32", "same")])
def test_backward_shapes(rows, cols, dtype, wdtype):
    check_backward(rows, cols, dtype, wdtype, dres=(rows + cols) % 2 == 0)


def test_rows_shorter_than_a_pack():
    for cols in (1, 2, 3, 5, 7):
        for dtype, wdtype in (("bf16", "fp32"), ("fp16", "same"), ("fp32", "same")):
            check_forward(1000, cols, dtype, wdtype, W=2, res=True)
            if cols > 2:  # two elements' gradient is nothing but cancellation
                check_backward(70001, cols, dtype, wdtype, dres=True)
    check_backward(300, 3, "fp32", want=("dgamma", "dbeta"))
    check_backward(300, 3, "fp32", place="dy")


def test_backward_many_rows():
    check_backward(20011, 96, "fp32", dres=True)
    check_backward(5000, 1500, "bf16", "fp32")


@pytest.mark.parametrize("cols", [200, 3000, 20000])
def test_backward_parts(cols):
    for want in (("dx",), ("dgamma",), ("dbeta",), ("dgamma", "dbeta"), ("dx", "dgamma")):
        check_backward(37, cols, "fp32", want=want)
    check_backward(37, cols, "fp32", gamma=False)
    for place in ("dy", "x", "dres"):
        check_backward(37, cols, "bf16", dres=True, place=place)


def test_no_rows():
    x = torch.empty(0, 65, device=device())
    e = torch.empty(0, device=device())
    dg, db = torch.full((65,), float("nan"), device=device()), torch.full((65,), float("nan"), device=device())
    mr.layer_norm_forward([x], None, None, torch.empty_like(x), mean=e, rstd=e)
    mr.layer_norm_backward(x, x, None, e, e, torch.empty_like(x), dgamma=dg, dbeta=db)
    assert torch.all(dg == 0) and torch.all(db == 0)


@pytest.mark.parametrize("rows,cols", [(3, 5), (2, 700), (2, 2500)])
def test_gradient_against_differences(rows, cols):
    """d/dt of sum(c * y) along a direction, by central differences of the fp32 forward pass in steps of h = 2^-5,
    against the backward pass: truncation is below h^2 times the third derivative (of the order of the first), the forward's rounding
    below 2 * 64 u sum|c y| / (2 h)."""
    gen = torch.Generator().manual_seed(3)
    x, c, d = (torch.randn(rows, cols, generator=gen).to(device()) for _ in range(3))
    g, b, dg, db = (torch.randn(cols, generator=gen).to(device()) for _ in range(4))
    h = 2.0 ** -5

    def f(t):
        y = torch.empty_like(x)
        mr.layer_norm_forward([x + t * d], g + t * dg, b + t * db, y)
        return float((c.double() * y.double()).sum()), float((c.double() * y.double()).abs().sum())

    m, r, y = torch.empty(rows, device=device()), torch.empty(rows, device=device()), torch.empty_like(x)
    mr.layer_norm_forward([x], g, b, y, mean=m, rstd=r)
    dx, gg, gb = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    mr.layer_norm_backward(c, x, g, m, r, dx, dgamma=gg, dbeta=gb)
    parts = [(dx.double() * d.double()), (gg.double() * dg.double()), (gb.double() * db.double())]
    got = sum(float(p.sum()) for p in parts)
    size = sum(float(p.abs().sum()) for p in parts)
    (p, pa), (q, qa) = f(h), f(-h)
    assert abs((p - q) / (2 * h) - got) <= 8 * h * h * size + 64 * U * (pa + qa) / (2 * h)


def test_rows_off_the_16_byte_grid():
    """Every buffer one element past a 16-byte boundary, at its own phase."""
    rows, cols = 11, 1234
    gen = torch.Generator().manual_seed(5)

    def off(k, t):
        flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=device())
        v = flat[k:k + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    x, res, dy = (rand(gen, rows, cols, "bf16") for _ in range(3))
    g, b = (torch.randn(cols, generator=gen).to(torch.bfloat16).to(device()) for _ in range(2))
    m, r = torch.empty(rows, device=device()), torch.empty(rows, device=device())
    y, xo, dx, dg, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    mr.layer_norm_forward([x], g, b, y, residual=res, x_out=xo, mean=m, rstd=r)
    mr.layer_norm_backward(dy, xo, g, m, r, dx, dgamma=dg, dbeta=db)
    y2, xo2, dx2, dg2, db2 = off(3, y), off(5, xo), off(7, dx), off(1, dg), off(2, db)
    mr.layer_norm_forward([off(1, x)], off(2, g), off(3, b), y2, residual=off(4, res), x_out=xo2, mean=off(1, m), rstd=off(3, r))
    mr.layer_norm_backward(off(5, dy), xo2, off(1, g), off(3, m), off(1, r), dx2, dgamma=dg2, dbeta=db2)
    for p, q in ((y, y2), (xo, xo2), (dx, dx2), (dg, dg2), (db, db2)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("rows,cols", [(1000, 100), (5000, 300), (1111, 4096), (40, 20000)])
def test_same_bits_every_time(rows, cols):
    gen = torch.Generator().manual_seed(6)
    x, dy = rand(gen, rows, cols, "bf16"), rand(gen, rows, cols, "bf16")
    m, r = x.float().mean(1), 1 / x.float().std(1)
    first = None
    for _ in range(4):
        dx, dg, db = torch.empty_like(x), torch.empty(cols, device=device()), torch.empty(cols, device=device())
        mr.layer_norm_backward(dy, x, None, m, r, dx, dgamma=dg, dbeta=db)
        now = (dx, dg, db)
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("rows,cols", [(700, 1600), (300, 200)])  # a second launch adds the partial sums up; the last workgroup does
def test_side_stream_and_graph_replays(rows, cols):
    """The backward pass uses the stream's workspace: eager on two streams at once, then captured and replayed with eager
    work between the replays; all equal to the default stream's results."""
    gen = torch.Generator().manual_seed(8)
    sets = [(rand(gen, rows, cols, "bf16"), rand(gen, rows, cols, "bf16")) for _ in range(3)]
    g = torch.ones(cols, dtype=torch.bfloat16, device=device())

    def outputs():
        return [torch.empty(rows, cols, dtype=torch.bfloat16, device=device()), torch.empty(rows, device=device()),
                torch.empty(rows, device=device()), torch.empty(rows, cols, dtype=torch.bfloat16, device=device()),
                torch.empty_like(g), torch.empty_like(g)]

    def both(x, dy, o, stream=None):
        mr.layer_norm_forward([x], g, g, o[0], mean=o[1], rstd=o[2], stream=stream)
        mr.layer_norm_backward(dy, x, g, o[1], o[2], o[3], dgamma=o[4], dbeta=o[5], stream=stream)

    want = [outputs() for _ in sets]
    for (x, dy), o in zip(sets, want):
        both(x, dy, o)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [outputs() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (x, dy), o, s in zip(sets, got, streams):
            both(x, dy, o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, got) for a, b in zip(w, o))
    x, dy, o = sets[0][0].clone(), sets[0][1].clone(), outputs()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        both(x, dy, o)
    for k in (1, 2, 0, 1):
        x.copy_(sets[k][0])
        dy.copy_(sets[k][1])
        for t in o:
            t.fill_(7.0)
        both(*sets[2 - k], outputs())  # eager work on the default stream's own workspace
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[k], o)), k
    del graph


def test_offsets_past_32_bits():
    """More than 2^32 elements, more rows than one grid holds; checked rows at the start, across the grid's end and at the end."""
    rows, cols = (1 << 20) + 5, 4099
    assert rows * cols > 1 << 32
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=device())
    at = [0, 1, (1 << 20) - 1, 1 << 20, rows - 1]
    x.fill_(0.5)
    gen = torch.Generator().manual_seed(9)
    part = torch.randn(len(at), cols, generator=gen).to(torch.bfloat16).to(device())
    x[at] = part
    y = torch.empty_like(x)
    m, r = torch.empty(rows, device=device()), torch.empty(rows, device=device())
    mr.layer_norm_forward([x], None, None, y, mean=m, rstd=r)
    small = torch.empty_like(part)
    mr.layer_norm_forward([part], None, None, small)
    assert torch.equal(y[at], small)
    assert float(y[5].abs().max()) == 0.0 and float(y[rows - 2].abs().max()) == 0.0
    dg, db = torch.empty(cols, device=device()), torch.empty(cols, device=device())
    dy = x
    mr.layer_norm_backward(dy, x, None, m, r, y, dgamma=dg, dbeta=db)  # rows of 0.5 have xh = 0
    mr.layer_norm_backward(part, part, None, m[at], r[at], small)
    assert torch.equal(y[at], small)
    want = (part.double() * ((part.double() - m[at].double()[:, None]) * r[at].double()[:, None])).sum(0)
    mag = (part.double().abs() * (part.double().abs() + m[at].double()[:, None].abs()) * r[at].double()[:, None]).sum(0)
    assert bool(((dg.double() - want).abs() <= 128 * U * mag).all())
    assert np.isclose(float(db.double().mean()), 0.5 * (rows - len(at)) + float(part.double().sum(0).mean()), rtol=(4096 + 64) * U)


def test_prepared_calls_and_a_bound_workspace():
    """Prepared calls give the plain calls' bits; a caller's workspace is used, and refused when it is too small."""
    rows, cols = 900, 1600
    gen = torch.Generator().manual_seed(10)
    x, dy = rand(gen, rows, cols, "bf16"), rand(gen, rows, cols, "bf16")
    g, b = (torch.randn(cols, generator=gen).to(torch.bfloat16).to(device()) for _ in range(2))
    m, r = torch.empty(rows, device=device()), torch.empty(rows, device=device())
    want, got = ([torch.empty_like(x), torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)] for _ in range(2))
    mr.layer_norm_forward([x], g, b, want[0], mean=m, rstd=r)
    mr.layer_norm_backward(dy, x, g, m, r, want[1], dgamma=want[2], dbeta=want[3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    small, large = (torch.empty(n, dtype=torch.uint8, device=device()) for n in (1 << 18, 1 << 22))
    torch.cuda.synchronize()
    mr.prepare_layer_norm_forward([x], g, b, got[0], mean=m, rstd=r, stream=s)()
    backward = mr.prepare_layer_norm_backward(dy, x, g, m, r, got[1], dgamma=got[2], dbeta=got[3], stream=s)
    mr.set_workspace(small, stream=s)
    with pytest.raises(mr.MRError) as e:
        backward()
    assert e.value.status == -4
    mr.set_workspace(large, stream=s)
    backward()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    mr.set_workspace(None, stream=s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols", [(1 << 25) + 3, (1 << 26) + 37])
def test_backward_of_the_widest_rows(cols):
    """More columns than the launch that finishes the weight gradients has workgroups for: each takes several blocks of them.
    The tolerances are check_backward's, where a lane adds up cols / 1024 elements of a row."""
    print(f"[case] norm backward 2x{cols} bf16/fp32", flush=True)
    gen = torch.Generator(device=device()).manual_seed(12)
    x, dy = (torch.randn(2, cols, generator=gen, device=device()).to(torch.bfloat16) for _ in range(2))
    m, r = torch.tensor([0.25, -0.5], device=device()), torch.tensor([1.0, 0.75], device=device())
    dx, dg, db = torch.empty_like(x), torch.full((cols,), float("nan"), device=device()), torch.full((cols,), float("nan"), device=device())
    mr.layer_norm_backward(dy, x, None, m, r, dx, dgamma=dg, dbeta=db)
    dy64, xh = dy.double(), (x.double() - m.double()[:, None]) * r.double()[:, None]
    big = xh.abs() + (x.double().abs() + m.double().abs()[:, None]) * r.double()[:, None]
    assert bool(((dg.double() - (dy64 * xh).sum(0)).abs() <= 66 * U * (dy64.abs() * big).sum(0)).all())
    assert bool(((db.double() - dy64.sum(0)).abs() <= 66 * U * dy64.abs().sum(0)).all())
    chain = (cols // 1024 + 128) * U
    want = r.double()[:, None] * (dy64 - dy64.mean(1, keepdim=True) - xh * (dy64 * xh).mean(1, keepdim=True))
    tol = UO["bf16"] * want.abs() + chain * r.double()[:, None] * (
        dy64.abs() + dy64.abs().mean(1, keepdim=True) + big * (dy64.abs() * big).mean(1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= tol + TINY["bf16"]).all())


# rows past one round of the grid, with a ragged last set: lanes of 16, waves, two and four packs a lane (of which the last wave's
# second or fourth lies past the row's end), and rows past the registers
@pytest.mark.parametrize("rows,cols,dtype", [(20011, 96, "bf16"), (5001, 1500, "fp16"), (601, 8700, "bf16"), (601, 8700, "fp16"),
                                             (700, 14337, "bf16"), (601, 4100, "fp32"), (601, 12300, "fp32"), (601, 16383, "fp32"),
                                             (301, 20000, "bf16")])
def test_backward_in_place_over_many_rounds(rows, cols, dtype):
    gen = torch.Generator().manual_seed(13)
    x, dy, dr = (rand(gen, rows, cols, dtype) for _ in range(3))
    g = (1 + 0.2 * torch.randn(cols, generator=gen)).to(device())
    m, r = x.float().mean(1), torch.rsqrt(x.float().var(1) + EPS)
    for res, places in ((None, ("dy", "x")), (dr, ("dy", "x", "dres"))):
        want = torch.empty_like(x), torch.empty(cols, device=device()), torch.empty(cols, device=device())
        mr.layer_norm_backward(dy, x, g, m, r, want[0], dgamma=want[1], dbeta=want[2], dres=res)
        for place in places:
            print(f"[case] norm backward in place {rows}x{cols} {dtype} dres={res is not None} place={place}", flush=True)
            ins = {"dy": dy, "x": x, "dres": res}
            ins[place] = ins[place].clone()
            got = ins[place], torch.empty_like(want[1]), torch.empty_like(want[2])
            mr.layer_norm_backward(ins["dy"], ins["x"], g, m, r, got[0], dgamma=got[1], dbeta=got[2], dres=ins["dres"])
            assert all(torch.equal(a, b) for a, b in zip(want, got)), (res is not None, place)


@pytest.mark.parametrize("rows,cols,dtype", [(100003, 96, "bf16"), (5001, 1500, "fp16"), (9001, 1024, "bf16"), (3001, 8192, "bf16"),
                                             (3001, 8700, "bf16"), (3001, 8700, "fp16"), (2001, 17000, "fp16"), (3001, 4100, "fp32"),
                                             (2001, 12300, "fp32"), (601, 33000, "bf16")])
def test_forward_in_place_over_many_rounds(rows, cols, dtype):
    gen = torch.Generator().manual_seed(14)
    bufs = [rand(gen, rows, cols, dtype) for _ in range(3)]
    g, b = (torch.randn(cols, generator=gen).to(device()) for _ in range(2))
    for W in (1, 2):
        res = bufs[2] if W > 1 else None
        for x_out in (False, True):
            print(f"[case] norm forward in place {rows}x{cols} {dtype} W={W} x_out={x_out}", flush=True)
            want = [torch.empty_like(bufs[0]), torch.empty_like(bufs[0]) if x_out else None]
            mr.layer_norm_forward(bufs[:W], g, b, want[0], residual=res, x_out=want[1])
            ins, r = [t.clone() for t in bufs[:W]], None if res is None else res.clone()
            # y over the first buffer, x over the residual; with one buffer x over it and y apart
            got = [ins[0], r] if W > 1 else [torch.empty_like(ins[0]), ins[0]] if x_out else [ins[0], None]
            mr.layer_norm_forward(ins, g, b, got[0], residual=r, x_out=got[1] if x_out else None)
            assert all(torch.equal(p, q) for p, q in zip(want, got) if p is not None)
