"""Host-side checks of the training-step entry points (layer norm, gradient norm, AdamW): every refusal returns its
code before any HIP call, so these run without a GPU; the same checks run once more under the host sanitizers."""
import ctypes
import os
import shutil
import subprocess

import pytest

import all_gather_amd as mr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EDTYPE, EALIAS = 0, -1, -2, -3
BF16, FP16, FP32, INT32 = range(4)
A = [0x10000000 * (i + 1) for i in range(12)]  # far apart, never dereferenced


@pytest.fixture(scope="module")
def L():
    return mr.lib()


def ptrs(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def counts(*c):
    return (ctypes.c_uint64 * max(len(c), 1))(*c)


def fwd(L, bufs=(A[0],), W=None, residual=None, gamma=A[1], beta=A[2], rows=4, cols=64, dt=BF16, wdt=BF16, eps=1e-5, x_out=None,
        y=A[3], mean=A[4], rstd=A[5]):
    return L.mr_layer_norm_forward(ptrs(*bufs), len(bufs) if W is None else W, residual, gamma, beta, rows, cols, dt, wdt, eps,
                                   x_out, y, mean, rstd, None)


def test_norm_forward_refusals(L):
    assert fwd(L, W=0) == EINVAL and fwd(L, W=17) == EINVAL
    assert fwd(L, dt=INT32, wdt=INT32) == EDTYPE and fwd(L, dt=7) == EINVAL and fwd(L, wdt=-1) == EINVAL
    assert fwd(L, wdt=FP16) == EDTYPE and fwd(L, dt=FP32, wdt=BF16) == EDTYPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert fwd(L, eps=eps) == EINVAL
    assert fwd(L, bufs=(None,)) == EINVAL and fwd(L, y=None) == EINVAL
    assert L.mr_layer_norm_forward(None, 1, None, None, None, 4, 64, 0, 0, 1e-5, None, A[3], None, None, None) == EINVAL
    for kw in (dict(y=A[3] + 1), dict(bufs=(A[0] + 1,)), dict(residual=A[6] + 1), dict(gamma=A[1] + 1), dict(mean=A[4] + 2),
               dict(wdt=FP32, beta=A[2] + 2), dict(x_out=A[7] + 1)):
        assert fwd(L, **kw) == EINVAL, kw
    assert fwd(L, cols=2 ** 31) == EINVAL and fwd(L, rows=2 ** 57) == EINVAL and fwd(L, rows=2 ** 40, cols=2 ** 20) == EINVAL
    assert fwd(L, rows=0) == OK and fwd(L, cols=0) == OK  # no-ops


def test_norm_forward_alias_rules(L):
    n = 4 * 64 * 2
    assert fwd(L, y=A[0] + 2) == EALIAS and fwd(L, y=A[0] - n + 2) == EALIAS
    assert fwd(L, residual=A[6], x_out=A[6] + 16) == EALIAS
    assert fwd(L, x_out=A[3]) == EALIAS                          # two outputs in one place
    assert fwd(L, x_out=A[3] + n - 2) == EALIAS
    assert fwd(L, mean=A[3] + 16) == EALIAS and fwd(L, mean=A[5]) == EALIAS
    assert fwd(L, y=A[1]) == EALIAS and fwd(L, rstd=A[2] + 4) == EALIAS   # over the weights


def bwd(L, dy=A[0], x=A[1], gamma=A[2], mean=A[3], rstd=A[4], dres=None, rows=4, cols=64, dt=BF16, wdt=BF16, dx=A[5], dgamma=A[6],
        dbeta=A[7]):
    return L.mr_layer_norm_backward(dy, x, gamma, mean, rstd, dres, rows, cols, dt, wdt, dx, dgamma, dbeta, None)


def test_norm_backward_refusals(L):
    assert bwd(L, dt=INT32, wdt=INT32) == EDTYPE and bwd(L, dt=4) == EINVAL and bwd(L, wdt=FP16) == EDTYPE
    for k in ("dy", "x", "mean", "rstd"):
        assert bwd(L, **{k: None}) == EINVAL, k
    for kw in (dict(dy=A[0] + 1), dict(x=A[1] + 1), dict(gamma=A[2] + 1), dict(mean=A[3] + 1), dict(dres=A[8] + 1), dict(dx=A[5] + 1),
               dict(dgamma=A[6] + 1), dict(wdt=FP32, dbeta=A[7] + 2)):
        assert bwd(L, **kw) == EINVAL, kw
    assert bwd(L, cols=2 ** 31) == EINVAL
    n = 4 * 64 * 2
    assert bwd(L, dx=A[0] + 2) == EALIAS and bwd(L, dx=A[1] + n - 2) == EALIAS and bwd(L, dres=A[8], dx=A[8] - 2) == EALIAS
    assert bwd(L, dgamma=A[2]) == EALIAS and bwd(L, dgamma=A[0]) == EALIAS and bwd(L, dgamma=A[7]) == EALIAS
    assert bwd(L, dbeta=A[3]) == EALIAS and bwd(L, dx=A[4]) == EALIAS
    assert bwd(L, cols=0) == OK and bwd(L, dx=None, dgamma=None, dbeta=None) == OK
    assert bwd(L, rows=0, dgamma=None, dbeta=None, dy=None, x=None, mean=None, rstd=None) == OK


def gnorm(L, g=(A[0], A[1]), c=(8, 16), P=None, dt=BF16, scale=1.0, max_norm=1.0, out=A[2]):
    return L.mr_grad_norm(ptrs(*g), counts(*c), len(g) if P is None else P, dt, scale, max_norm, out, None)


def test_grad_norm_refusals(L):
    assert gnorm(L, P=-1) == EINVAL and gnorm(L, dt=INT32) == EDTYPE and gnorm(L, dt=9) == EINVAL
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert gnorm(L, scale=s) == EINVAL
    assert gnorm(L, max_norm=float("nan")) == EINVAL and gnorm(L, max_norm=float("inf")) == EINVAL
    assert gnorm(L, out=None) == EINVAL and gnorm(L, out=A[2] + 2) == EINVAL
    assert gnorm(L, g=(A[0], None)) == EINVAL and gnorm(L, g=(A[0] + 1, A[1])) == EINVAL
    assert gnorm(L, c=(8, 2 ** 33 + 1)) == EINVAL
    assert L.mr_grad_norm(None, counts(8), 1, BF16, 1.0, 1.0, A[2], None) == EINVAL
    assert gnorm(L, out=A[1] + 28) == EALIAS and gnorm(L, out=A[0] - 8) == EALIAS


def adam(L, params=(A[0], A[1]), grads=(A[2], A[3]), c=(100, 7), P=None, dt=BF16, gdt=BF16, fmt=0, m=A[4], v=A[5], ms=None, vs=None,
         master=None, pout=None, out=None, clip=None, **h):
    hy = mr._AdamWHyperC(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, seed=0), **h})
    st = mr._AdamWStateC(m, v, ms, vs, master)
    so = None if out is None else ctypes.byref(mr._AdamWStateC(*out))
    return L.mr_adamw_step(None if params is None else ptrs(*params), ptrs(*grads), counts(*c), len(c) if P is None else P, dt, gdt,
                           fmt, ctypes.byref(st), None if pout is None else ptrs(*pout), so, ctypes.byref(hy), clip, None)


def test_adamw_refusals(L):
    assert adam(L, dt=INT32, gdt=INT32) == EDTYPE and adam(L, dt=5) == EINVAL and adam(L, gdt=FP16) == EDTYPE
    assert adam(L, dt=FP32, gdt=BF16) == EDTYPE and adam(L, P=-1) == EINVAL and adam(L, fmt=2) == EINVAL
    for h in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-9), dict(eps=float("inf")),
              dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(step=0)):
        assert adam(L, **h) == EINVAL, h
    assert adam(L, m=None) == EINVAL and adam(L, v=None) == EINVAL and adam(L, m=A[4] + 128) == EINVAL
    assert adam(L, fmt=1) == EINVAL                                   # no scales
    assert adam(L, ms=A[6]) == EINVAL                                 # scales with fp32 moments
    assert adam(L, dt=FP32, gdt=FP32, master=A[6]) == EDTYPE          # a master copy of fp32 parameters
    assert adam(L, master=A[6] + 4) == EINVAL
    assert adam(L, master=A[6], out=(A[7], A[8], None, None, None)) == EINVAL
    assert adam(L, params=None) == EINVAL and adam(L, params=None, master=A[6]) == EINVAL
    assert adam(L, params=(A[0], None)) == EINVAL and adam(L, grads=(A[2] + 1, A[3])) == EINVAL
    assert adam(L, params=(A[0] + 1, A[1])) == EINVAL and adam(L, pout=(A[6], A[7] + 1)) == EINVAL
    assert adam(L, clip=A[9] + 2) == EINVAL and adam(L, c=(2 ** 33 + 1, 7)) == EINVAL
    assert adam(L, c=(0, 0), params=(None, None), grads=(None, None), m=None, v=None) == OK   # nothing to do
    assert L.mr_adamw_step(None, None, None, 0, FP32, FP32, 0, None, None, None, ctypes.byref(mr._AdamWHyperC(step=1)), None, None) == OK


def test_adamw_alias_rules(L):
    assert adam(L, params=(A[0], A[0] + 198)) == EALIAS               # two tensors over one another
    assert adam(L, grads=(A[0], A[3])) == EALIAS                      # a gradient where a parameter is written
    assert adam(L, pout=(A[0] + 2, A[7])) == EALIAS                   # not exactly in place
    assert adam(L, pout=(A[1], A[7])) == EALIAS                       # another tensor's place
    assert adam(L, v=A[4]) == EALIAS and adam(L, v=A[4] + 256) == EALIAS       # 160 elements: 640 bytes of state
    assert adam(L, out=(A[5], A[4], None, None, None)) == EALIAS      # exchanged
    assert adam(L, clip=A[4] + 4) == EALIAS
    assert adam(L, fmt=1, ms=A[6], vs=A[6] + 4) == EALIAS             # 5 blocks: scales overlap


def test_state_layout(L):
    n = ctypes.c_uint64()
    assert L.mr_adamw_state_elems(counts(1, 0, 32, 33), 4, ctypes.byref(n)) == OK and n.value == 32 + 0 + 32 + 64
    assert L.mr_adamw_state_elems(None, 0, ctypes.byref(n)) == OK and n.value == 0
    assert L.mr_adamw_state_elems(counts(1), 1, None) == EINVAL and L.mr_adamw_state_elems(counts(1), -1, ctypes.byref(n)) == EINVAL
    assert L.mr_adamw_state_elems(counts(*[2 ** 33] * 16), 16, ctypes.byref(n)) == EINVAL   # block numbers are 32 bits
    assert mr.adamw_offsets([1, 0, 32, 33]) == ([0, 32, 32, 64], 128)


def test_binding_refuses_wrong_tensors():
    import torch

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mr.layer_norm_forward([x], None, None, x)
    with pytest.raises(ValueError):
        mr.layer_norm_backward(x, x, None, x[:, 0], x[:, 0], x)
    with pytest.raises(ValueError):
        mr.grad_norm([x], torch.zeros(3))
    with pytest.raises(ValueError):
        mr.adamw_step([x], [x], mr.AdamWState(x, x), 1e-3, 1)
    with pytest.raises(ValueError):
        mr.adamw_init([x], bits=4)


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="ROCm toolchain not present")
def test_refusals_under_asan_and_ubsan(tmp_path):
    """The argument checks and launch tables of the training-step entry points, host code rebuilt with the sanitizers."""
    from all_gather_amd import _build

    san = "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined -Xarch_host -fno-omit-frame-pointer".split()
    obj = str(tmp_path / "train_api.o")
    r = subprocess.run([_build.hipcc(), *_build.CFLAGS, "-Xarch_host", "-g", *san, "-c", os.path.join(_build.CSRC, "train_api.hip"),
                        "-o", obj], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    others = [os.path.join(_build.OBJ, os.path.splitext(s)[0] + ".o") for s in _build.SOURCES if s != "train_api.hip"]
    lib = str(tmp_path / "libmr.so")
    r = subprocess.run([_build.hipcc(), f"--offload-arch={_build.ARCH}", "-shared", "-fPIC", *san, obj, *others, "-lhsa-runtime64",
                        "-o", lib], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    exe = str(tmp_path / "check")
    r = subprocess.run(["/opt/rocm/llvm/bin/clang", "-std=c99", "-Wall", "-Wextra", "-Werror", "-g", "-fsanitize=address,undefined", "-I",
                        os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c_abi_train_check.c"), "-L", str(tmp_path), "-lmr",
                        f"-Wl,-rpath,{tmp_path}", "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "c abi ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
    shutil.rmtree(tmp_path, ignore_errors=True)


class _OnDevice:
    """What the binding reads of a device tensor."""

    def __init__(self, n, dtype, at):
        self.n, self.dtype, self.at, self.is_cuda = n, dtype, at, True

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def test_binding_refuses_steps_that_do_not_count_from_one(monkeypatch):
    """A step of -1 would reach the library as 2^64 - 1, whose bias corrections are 1."""
    import torch

    calls, real = [], mr.lib()

    class Library:
        mr_adamw_state_elems = real.mr_adamw_state_elems

        @staticmethod
        def mr_adamw_step(*args):
            calls.append(args)
            return OK

    class Stream:
        cuda_stream = 0x50

    monkeypatch.setattr(mr, "lib", lambda: Library)
    t = [_OnDevice(32, torch.float32, a) for a in A[:4]]
    call = mr.prepare_adamw([t[0]], [t[1]], mr.AdamWState(t[2], t[3]), stream=Stream())
    call(1e-3, 1)
    call(1e-3, 2 ** 64 - 1)
    assert len(calls) == 2
    for step in (0, -1, -2 ** 63, 2 ** 64, 2 ** 64 + 1):
        with pytest.raises(ValueError):
            call(1e-3, step)
    assert len(calls) == 2
