"""What the host code launches, without a GPU: the library's objects linked with a HIP runtime that only writes launches
down (fake_hip.cpp)."""
import ctypes
import os
import shutil
import subprocess
import threading
import time
from concurrent.futures import ThreadPoolExecutor

import pytest

import all_gather_amd as mr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_gather_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"
BF16, FP16, FP32 = 0, 1, 2
A = [(i + 1) << 40 for i in range(12)]  # far apart, never dereferenced
MOST_COLS = 2 ** 31 - 1

pytestmark = pytest.mark.skipif(not (os.path.exists(CLANG) and os.path.exists("/opt/rocm/bin/hipcc")),
                                reason="ROCm toolchain not present")


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from all_gather_amd import _build

    tmp = tmp_path_factory.mktemp("fake")
    headers = max(os.path.getmtime(os.path.join(CSRC, h)) for h in os.listdir(CSRC) if h.endswith(".h"))

    def compiled(src):
        path, built = os.path.join(CSRC, src), os.path.join(_build.OBJ, os.path.splitext(src)[0] + ".o")
        # a file whose interface headers are newer than its object is compiled here; the reduce and gather kernels' is not
        own = headers if src in ("api.hip", "train_api.hip", "norm_fwd.hip", "norm_bwd.hip", "optim_kernels.hip") else 0
        if os.path.exists(built) and os.path.getmtime(built) >= max(os.path.getmtime(path), own):
            return built
        obj = str(tmp / (src + ".o"))
        r = subprocess.run([_build.hipcc(), *_build.CFLAGS, "-c", path, "-o", obj], capture_output=True, text=True, timeout=900)
        assert r.returncode == 0, r.stderr[-2000:]
        return obj

    with ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(compiled, _build.SOURCES))
    lib = str(tmp / "libmr_fake.so")
    r = subprocess.run([CLANG, "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-Wl,-Bsymbolic", "-Wl,--no-undefined", os.path.join(ROOT, "tests", "fake_hip.cpp"), *objs, "-lpthread",
                        "-o", lib], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    L = ctypes.CDLL(lib)
    for name, (res, args) in mr._SIGS.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    L.fake_allocated.restype = ctypes.c_uint64
    yield L
    shutil.rmtree(tmp, ignore_errors=True)


def launches(L):
    out, name, v = [], ctypes.create_string_buffer(400), (ctypes.c_uint64 * 9)()
    for i in range(L.fake_launches()):
        assert L.fake_launch(i, name, 400, v) == 0
        out.append(dict(name=name.value.decode(), stream=v[0], thread=v[1], grid=tuple(v[2:5]), block=tuple(v[5:8]), refused=v[8]))
    return out


def ptrs(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def counts(*c):
    return (ctypes.c_uint64 * max(len(c), 1))(*c)


def backward(L, rows, cols, dt=BF16, wdt=FP32, dx=A[5], dgamma=A[6], dbeta=A[7], stream=None):
    return L.mr_layer_norm_backward(A[0], A[1], A[2], A[3], A[4], None, rows, cols, dt, wdt, dx, dgamma, dbeta, stream)


def forward(L, rows, cols, dt=BF16, wdt=FP32, W=1, stream=None):
    return L.mr_layer_norm_forward(ptrs(*A[5:5 + W]), W, None, A[2], A[3], rows, cols, dt, wdt, 1e-5, None, A[0], A[4], A[1], stream)


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, MOST_COLS), (3, 2 ** 26), (1, 2 ** 26 - 1), (1, 2 ** 27 + 5), (2 ** 38, 1), (2 ** 26, 4096),
                                       (2 ** 24, 8191), (2 ** 20, 40000), (1, 1)])
def test_every_norm_launch_fits_the_device(fake, dt, rows, cols):
    """The whole range of rows and columns that the header allows: a call launches all of its kernels or none."""
    for parts in ({}, dict(dx=None), dict(dgamma=None, dbeta=None)):
        fake.fake_reset(0)
        assert backward(fake, rows, cols, dt, **parts) == 0, parts
        assert fake.fake_launches() >= 1 and not any(x["refused"] for x in launches(fake))
    fake.fake_reset(0)
    assert forward(fake, rows, cols, dt) == 0
    assert fake.fake_launches() == 1 and not any(x["refused"] for x in launches(fake))


def grad_norm(L, tensors, stream=None):
    g = [A[0] + 4096 * i for i in range(tensors)]
    return L.mr_grad_norm(ptrs(*g), counts(*[64] * tensors), tensors, FP32, 1.0, 1.0, A[3], stream)


def two_shot(L, stream=None):
    return L.mr_allreduce_sum(ptrs(A[0], A[1]), 2, 4096, FP32, A[2], 1, stream)


CALLS = {"grad_norm": lambda L, st: grad_norm(L, 300, st), "backward": lambda L, st: backward(L, 5000, 1500, stream=st),
         "two_shot": two_shot}


def at_once(L, first, second, streams, hold_ms=40):
    """The launches of two calls from two threads; the second call starts once the first's first kernel is launched, and every
    launch keeps its thread for hold_ms."""
    for name, st in zip((first, second), streams):  # workspaces are there
        assert CALLS[name](L, st) == 0
    L.fake_reset(hold_ms)
    status = []
    a = threading.Thread(target=lambda: status.append(CALLS[first](L, streams[0])))
    b = threading.Thread(target=lambda: status.append(CALLS[second](L, streams[1])))
    a.start()
    end = time.monotonic() + 10
    while not L.fake_launches() and time.monotonic() < end:
        time.sleep(0.001)
    b.start()
    a.join()
    b.join()
    assert status == [0, 0]
    return launches(L)


@pytest.mark.parametrize("second", ["grad_norm", "backward", "two_shot"])
@pytest.mark.parametrize("first", ["grad_norm", "backward"])
def test_a_call_s_launches_stay_together_on_a_stream(fake, first, second):
    """The kernels of one call hand partial sums over in the stream's workspace: a call from another host thread that uses the same
    workspace must not come between them."""
    got = [x["thread"] for x in at_once(fake, first, second, (0x50, 0x50))]
    n = {"grad_norm": 3, "backward": 2, "two_shot": 1}
    assert len(got) == n[first] + n[second]
    assert len(set(got[:n[first]])) == 1 and len(set(got[n[first]:])) == 1, got


def test_streams_do_not_wait_for_one_another(fake):
    got = [x["stream"] for x in at_once(fake, "grad_norm", "backward", (0x50, 0x60), 200)]
    assert sorted(got) == [0x50] * 3 + [0x60] * 2 and got != [0x50] * 3 + [0x60] * 2


def adamw(L, eps, fmt=0):
    h = mr._AdamWHyperC(1e-3, 0.9, 0.999, eps, 0.0, 1, 0)
    st = mr._AdamWStateC(A[4], A[5], A[6] if fmt else None, A[7] if fmt else None, None)
    return L.mr_adamw_step(ptrs(A[0]), ptrs(A[1]), counts(100), 1, FP32, FP32, fmt, ctypes.byref(st), None, None, ctypes.byref(h), None, None)


def test_eps_outside_the_range_of_the_arithmetic(fake):
    """AdamW divides by a number that is at least eps, with an instruction that takes subnormal numbers as zero; layer norm takes the
    root of one.  An eps that is lost on the way would turn 0 / eps into NaN."""
    for fmt in (0, 1):
        for eps in (0.0, 2.0 ** -126, 1e-8, 1e30):
            assert adamw(fake, eps, fmt) == 0, eps
        for eps in (2.0 ** -127, 1e-39, 1e-45, 1e-300, 5e-324):
            fake.fake_reset(0)
            assert adamw(fake, eps, fmt) == -1 and fake.fake_launches() == 0, eps

    def norm(eps):
        return fake.mr_layer_norm_forward(ptrs(A[5]), 1, None, None, None, 4, 64, BF16, BF16, eps, None, A[0], None, None, None)

    for eps in (0.0, 2.0 ** -149, 1e-40, 1e-5, 3e38):
        assert norm(eps) == 0, eps
    for eps in (2.0 ** -151, 1e-300, 5e-324, 1e39, 1e300):
        fake.fake_reset(0)
        assert norm(eps) == -1 and fake.fake_launches() == 0, eps


@pytest.mark.parametrize("cols", [1, 7, 8, 31, 32, 100, 4096, 8192, 16384, 16385, 40000, 10 ** 6])
def test_a_caller_s_workspace_of_the_documented_size(fake, cols):
    """mr_workspace_bytes(1, 512 * max(cols, 32), MR_FP32) is enough for the backward pass of any number of rows."""
    bytes_ = fake.mr_workspace_bytes(1, 512 * max(cols, 32), FP32)
    assert fake.mr_set_workspace(0x70, A[8], bytes_) == 0
    before = fake.fake_allocated()
    for rows in (1, 255, 257, 3000, min(10 ** 6, 2 ** 37 // cols)):  # buffers lie 2^40 bytes apart
        for dt in (BF16, FP32):
            for parts in ({}, dict(dx=None)):
                assert backward(fake, rows, cols, dt, stream=0x70, **parts) == 0, (rows, dt, parts)
    assert fake.fake_allocated() == before
    assert fake.mr_set_workspace(0x70, None, 0) == 0


def test_a_caller_s_workspace_for_the_gradient_norm(fake):
    for tensors in (0, 1, 128, 129, 5000):
        g = [A[0] + (i << 24) for i in range(tensors)]
        bytes_ = fake.mr_workspace_bytes(1, 8 * tensors + 1024, FP32)
        assert fake.mr_set_workspace(0x70, A[8], bytes_) == 0
        before = fake.fake_allocated()
        assert fake.mr_grad_norm(ptrs(*g), counts(*[1 << 22] * tensors), tensors, FP32, 1.0, 1.0, A[7] + 4, 0x70) == 0
        assert fake.fake_allocated() == before
    small = fake.mr_workspace_bytes(1, 16, FP32)
    assert fake.mr_set_workspace(0x70, A[8], small) == 0
    assert fake.mr_grad_norm(ptrs(*g), counts(*[1 << 22] * 5000), 5000, FP32, 1.0, 1.0, A[7] + 4, 0x70) == -4
    assert backward(fake, 3000, 4096, stream=0x70) == -4
    assert fake.mr_set_workspace(0x70, None, 0) == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gdt", [BF16, FP32])
def test_the_largest_lists_fit_the_device(fake, gdt, fmt):
    """Tensors of up to 2^33 elements: a launch takes a tensor more than fills it, and still holds less than 2^32 lanes."""
    c = [2 ** 33 - 1024, 2 ** 33, 5, 2 ** 32 + 1, 2 ** 33 - 2048 * 8, 2 ** 33]
    at = [i << 36 for i in range(len(c))]
    h = mr._AdamWHyperC(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 0)
    st = mr._AdamWStateC(A[4], A[5], A[6] if fmt else None, A[7] if fmt else None, None)
    fake.fake_reset(0)
    assert fake.mr_adamw_step(ptrs(*[A[0] + a for a in at]), ptrs(*[A[2] + a for a in at]), counts(*c), len(c), gdt, gdt, fmt,
                              ctypes.byref(st), None, None, ctypes.byref(h), None, None) == 0
    got = launches(fake)
    assert len(got) >= 2 and not any(x["refused"] for x in got)
    fake.fake_reset(0)
    assert fake.mr_grad_norm(ptrs(*[A[2] + a for a in at]), counts(*c), len(c), gdt, 1.0, 1.0, A[8], None) == 0
    assert fake.fake_launches() >= 1 and not any(x["refused"] for x in launches(fake))
