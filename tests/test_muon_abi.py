"""Host-side checks of Muon's entry points: every refusal returns its code before any HIP call, so these run without a GPU."""
import ctypes

import pytest

import all_gather_amd as mr

OK, EINVAL, EDTYPE, EALIAS = 0, -1, -2, -3
BF16, FP16, FP32, INT32 = range(4)
A = [0x10000000 * (i + 1) for i in range(12)]  # far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return mr.lib()


def ptrs(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def u64(*c):
    return (ctypes.c_uint64 * max(len(c), 1))(*c)


def muon(L, params=(A[0], A[1]), grads=(A[2], A[3]), rows=(10, 7), cols=(10, 5), P=None, dt=BF16, gdt=BF16, m=A[4], master=None, pout=None,
         out=None, clip=None, hyper=True, coef=None, **h):
    c = None if coef is None else (ctypes.c_double * len(coef))(*coef)
    hy = mr._MuonHyperC(**{**dict(lr=1e-2, momentum=0.9, weight_decay=0.0, eps=1e-7, coefficients=c, steps=5, nesterov=1, products=16,
                                  adjust=0), **h})
    st = mr._MuonStateC(m, master)
    so = None if out is None else ctypes.byref(mr._MuonStateC(*out))
    return L.mr_muon_step(None if params is None else ptrs(*params), ptrs(*grads), u64(*rows), u64(*cols), len(rows) if P is None else P, dt,
                          gdt, ctypes.byref(st), None if pout is None else ptrs(*pout), so, ctypes.byref(hy) if hyper else None, clip, None)


def test_refusals(L):
    assert muon(L, dt=INT32, gdt=INT32) == EDTYPE and muon(L, dt=5) == EINVAL and muon(L, gdt=FP16) == EDTYPE and muon(L, dt=FP32) == EDTYPE
    assert muon(L, P=-1) == EINVAL and muon(L, hyper=False) == EINVAL
    for h in (dict(lr=NAN), dict(weight_decay=INF), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=NAN), dict(eps=0.0), dict(eps=INF),
              dict(eps=2.0 ** -115), dict(steps=0), dict(steps=17), dict(products=8), dict(adjust=2)):
        assert muon(L, **h) == EINVAL, h
    assert muon(L, rows=(65537, 7)) == EINVAL and muon(L, cols=(10, 65537)) == EINVAL
    assert muon(L, m=None) == EINVAL and muon(L, m=A[4] + 128) == EINVAL and muon(L, master=A[5] + 4) == EINVAL
    assert muon(L, dt=FP32, gdt=FP32, master=A[5]) == EDTYPE and muon(L, master=A[5], out=(A[6], None)) == EINVAL
    assert muon(L, params=None) == EINVAL and muon(L, params=(A[0], None)) == EINVAL and muon(L, grads=(None, A[3])) == EINVAL
    assert muon(L, grads=(A[2] + 1, A[3])) == EINVAL and muon(L, params=(A[0] + 1, A[1])) == EINVAL and muon(L, clip=A[6] + 2) == EINVAL
    assert muon(L, rows=(0, 7), cols=(5, 0), params=(None, None), grads=(None, None), m=None) == OK       # nothing to do
    assert muon(L, rows=(), cols=(), params=(), grads=()) == OK


def test_polynomials_that_leave_the_range_are_refused(L):
    for coef in ((4.0, -6.0, 2.5, 3.4445, -4.775, 2.0315, 2.0, -1.5, 0.5),   # 1.33, then 2.04: the third step's would pass 9
                 (20.0, 0.0, 0.0), (3.0, 0.0, 0.0, 3.0, 0.0, 0.0), (1.0, 0.0, NAN), (INF, 0.0, 0.0), (0.0, 20.0, 0.0), (0.0, 30.0, -29.0)):
        assert muon(L, coef=coef, steps=len(coef) // 3) == EINVAL, coef


def test_alias_rules(L):
    assert muon(L, params=(A[0], A[0] + 198)) == EALIAS and muon(L, grads=(A[0], A[3])) == EALIAS
    assert muon(L, pout=(A[0] + 2, A[7])) == EALIAS and muon(L, pout=(A[1], A[7])) == EALIAS
    assert muon(L, m=A[0] & ~255) == EALIAS and muon(L, master=A[4] + 256) == EALIAS     # 192 elements: 768 bytes of momentum
    assert muon(L, master=A[5], out=(A[5], A[4])) == EALIAS                              # exchanged
    assert muon(L, clip=A[4] + 4) == EALIAS


def test_workspace_sizes(L):
    def need(shapes, products=16):
        return mr.muon_workspace_bytes(shapes, products)

    one = need([(1000, 500)])
    assert one >= 2 * (512 * 1024 + 2 * 1000 * 512 + 2 * 500 * 512)
    assert need([(500, 1000)]) == one and need([(1000, 500)], 32) > 1.5 * one
    assert need([(1000, 500)] * 3) > 2 * one and need([(1000, 500)] * 64) == need([(1000, 500)] * 32)
    big = need([(16384, 16384)])
    assert need([(16384, 16384)] * 5) == big and need([]) > 0
    assert need([(65537, 1)]) == 0 and need([(10, 10)], 8) == 0


def test_binding_refuses_wrong_tensors():
    import torch

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mr.muon_step([x], [x], mr.MuonState(x), 1e-3)
    with pytest.raises(ValueError):
        mr.muon_step([torch.zeros(8)], [torch.zeros(8)], mr.MuonState(x), 1e-3)
