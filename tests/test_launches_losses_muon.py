"""What the host code of the losses and of Muon launches, without a GPU (the runtime of fake_hip.cpp): every launch fits the device,
calls of one stream stay together, documented workspaces are large enough, and sizes of nothing divide by nothing."""
import ctypes
import threading
import time

import pytest

import all_gather_amd as mr
from test_launches import BF16, FP16, FP32, counts, fake, launches, pytestmark, ptrs  # noqa: F401

A = [(i + 1) << 43 for i in range(12)]


def policy(L, rows, cols, dt=BF16, stride=None, dz=A[8], logp=A[7], stream=None, off=0):
    h = mr._PolicyHyperC(1.0, 0.2, 0.2, 0.0, 1.0)
    stride = cols if stride is None else stride
    return L.mr_policy_loss(A[0] + off, rows, cols, stride, dt, A[1], None, None, A[2], None, ctypes.byref(h), A[6], logp, dz, stride, stream)


def forward(L, rows, cols, dt=BF16, stream=None, off=0):
    return L.mr_token_logprob_forward(A[0] + off, rows, cols, cols, dt, A[1], 1.0, A[2], A[3], stream)


def backward(L, rows, cols, dt=BF16, stream=None):
    return L.mr_token_logprob_backward(A[0], rows, cols, cols, dt, A[1], 1.0, A[3], A[4], A[5], cols, stream)


def preference(L, rows, pairs, stream=None):
    h = mr._PreferenceHyperC(0.1, 0.0, 1.0, 1.0)
    return L.mr_preference_loss(A[0], A[1], rows, A[2], pairs, ctypes.byref(h), A[3], A[4], A[5], stream)


def muon(L, shapes, products=16, dt=BF16, stream=None, steps=5):
    hy = mr._MuonHyperC(1e-2, 0.9, 0.0, 1e-7, None, steps, 1, products, 0)
    st = mr._MuonStateC(A[4], None)
    n = len(shapes)
    return L.mr_muon_step(ptrs(*[A[0] + (i << 36) for i in range(n)]), ptrs(*[A[2] + (i << 36) for i in range(n)]),
                          counts(*[r for r, _ in shapes]), counts(*[c for _, c in shapes]), n, dt, dt, ctypes.byref(st), None, None,
                          ctypes.byref(hy), None, stream)


def fits(L, want=None):
    got = launches(L)
    assert got and not any(x["refused"] for x in got), got
    assert want is None or len(got) == want, [x["name"] for x in got]
    return got


SIZES = [(1, 1), (1, 2 ** 31 - 1), (3, 7), (7, 131072), (8, 131072), (8, 131073), (255, 9), (256, 16385), (257, 65537), (1023, 3),
         (1024, 200000), (100000, 5), (2 ** 20, 4096), (2 ** 24, 1), (2 ** 22, 2 ** 18), (5, 2 ** 31 - 1)]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_every_launch_over_logits_fits_the_device(fake, rows, cols, dt):
    for off in (0, 4):
        fake.fake_reset(0)
        assert policy(fake, rows, cols, dt, off=off) == 0
        assert len(fits(fake)) <= 3                  # a first call on a larger workspace clears its words
        fake.fake_reset(0)
        assert policy(fake, rows, cols, dt, dz=None, off=off) == 0
        fits(fake)
        fake.fake_reset(0)
        assert forward(fake, rows, cols, dt, off=off) == 0
        fits(fake)
    fake.fake_reset(0)
    assert backward(fake, rows, cols, dt) == 0
    fits(fake, 1)


def test_nothing_to_do(fake):
    for rows, cols in ((0, 0), (0, 100), (5, 0), (2000, 0)):
        fake.fake_reset(0)
        assert policy(fake, rows, cols) == 0
        fits(fake)                                   # the record becomes zeros
        assert forward(fake, rows, cols) == 0 and backward(fake, rows, cols) == 0
        assert not any(x["refused"] for x in launches(fake))
    for rows, pairs in ((0, 0), (0, 5), (100, 0), (1, 1), (2 ** 32, 2 ** 20), (2 ** 20, 1)):
        fake.fake_reset(0)
        assert preference(fake, rows, pairs) == 0
        fits(fake)
    fake.fake_reset(0)
    assert muon(fake, []) == 0 and muon(fake, [(0, 5), (5, 0)]) == 0 and fake.fake_launches() == 0


@pytest.mark.parametrize("products", [16, 32])
@pytest.mark.parametrize("shapes", [[(1, 1)], [(1, 65536)], [(65536, 1)], [(65536, 65536)], [(4096, 4096)] * 40, [(64, 64)] * 100,
                                    [(511, 512), (0, 3), (512, 511), (1024, 1023), (2048, 9000)] * 9])
def test_every_muon_launch_fits_the_device(fake, shapes, products):
    fake.fake_reset(0)
    assert muon(fake, shapes, products) == 0
    got = fits(fake)
    assert sum("momentum" in x["name"] for x in got) == sum("orient" in x["name"] for x in got) >= 1
    assert sum("ns_last" in x["name"] for x in got) >= 1


def test_small_matrices_of_one_size_take_17_launches(fake):
    assert muon(fake, [(64, 64)] * 32, stream=0x51) == 0
    fake.fake_reset(0)
    assert muon(fake, [(64, 64)] * 32, stream=0x51) == 0
    fits(fake, 17)


CALLS = {"muon": lambda L, st: muon(L, [(100, 200), (700, 700)], stream=st, steps=2), "policy": lambda L, st: policy(L, 3, 2 ** 20, stream=st),
         "preference": lambda L, st: preference(L, 1000, 10, stream=st), "forward": lambda L, st: forward(L, 5, 2 ** 20, stream=st)}


@pytest.mark.parametrize("first,second", [("muon", "policy"), ("policy", "muon"), ("policy", "forward"), ("muon", "preference"),
                                          ("policy", "policy"), ("muon", "muon")])
def test_a_call_s_launches_stay_together_on_a_stream(fake, first, second):
    n = {}
    for name in (first, second):
        assert CALLS[name](fake, 0x52) == 0          # the workspace is there
    for name in (first, second):
        fake.fake_reset(0)
        assert CALLS[name](fake, 0x52) == 0
        n[name] = fake.fake_launches()
    fake.fake_reset(20)
    status = []
    a = threading.Thread(target=lambda: status.append(CALLS[first](fake, 0x52)))
    b = threading.Thread(target=lambda: status.append(CALLS[second](fake, 0x52)))
    a.start()
    end = time.monotonic() + 10
    while not fake.fake_launches() and time.monotonic() < end:
        time.sleep(0.001)
    b.start()
    a.join()
    b.join()
    assert status == [0, 0]
    got = [x["thread"] for x in launches(fake)]
    assert len(got) == n[first] + n[second]
    assert len(set(got[:n[first]])) == 1 and len(set(got[n[first]:])) == 1, got
    fake.fake_reset(0)


@pytest.mark.parametrize("rows", [1, 7, 8, 100, 1023, 1024, 5000, 10 ** 6])
def test_a_caller_s_workspace_of_the_documented_size(fake, rows):
    """mr_workspace_bytes(1, 256 * rows + 65536, MR_FP32) is enough for the losses over any number of columns."""
    assert fake.mr_set_workspace(0x70, A[9], fake.mr_workspace_bytes(1, 256 * rows + 65536, FP32)) == 0
    before = fake.fake_allocated()
    for cols in (1, 9, 1000, 131072, 131073, 10 ** 6):
        for dt in (BF16, FP32):
            assert policy(fake, rows, cols, dt, stream=0x70) == 0 and policy(fake, rows, cols, dt, dz=None, stream=0x70) == 0, (cols, dt)
            assert forward(fake, rows, cols, dt, stream=0x70) == 0
    for pairs in (0, 1, 500, 10 ** 5):
        assert preference(fake, rows, pairs, stream=0x70) == 0
    assert fake.fake_allocated() == before
    assert fake.mr_set_workspace(0x70, None, 0) == 0


@pytest.mark.parametrize("products", [16, 32])
@pytest.mark.parametrize("shapes", [[(1, 1)], [(100, 7)] * 70, [(300, 200), (64, 513), (700, 700)], [(4096, 4096)] * 7 + [(5, 5)] * 40, [(8192, 30000)]])
def test_a_caller_s_workspace_for_muon(fake, shapes, products):
    need = mr.lib().mr_muon_workspace_bytes(counts(*[r for r, _ in shapes]), counts(*[c for _, c in shapes]), len(shapes), products)
    assert need > 0 and fake.mr_set_workspace(0x70, A[9], need) == 0
    before = fake.fake_allocated()
    assert muon(fake, shapes, products, stream=0x70) == 0
    assert fake.fake_allocated() == before
    if need > 1 << 21:
        assert fake.mr_set_workspace(0x70, A[9], need // 2 // 256 * 256) == 0
        fake.fake_reset(0)
        assert muon(fake, shapes, products, stream=0x70) == -4 and fake.fake_launches() == 0
    assert fake.mr_set_workspace(0x70, None, 0) == 0
