"""Host-side checks of the losses' entry points: every refusal returns its code before any HIP call, so these run without a GPU."""
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


def fwd(L, z=A[0], rows=4, cols=64, stride=64, dt=BF16, t=A[1], temp=1.0, logp=A[2], stats=A[3]):
    return L.mr_token_logprob_forward(z, rows, cols, stride, dt, t, temp, logp, stats, None)


def bwd(L, z=A[0], rows=4, cols=64, stride=64, dt=BF16, t=A[1], temp=1.0, stats=A[3], dlogp=A[4], dz=A[5], dstride=64):
    return L.mr_token_logprob_backward(z, rows, cols, stride, dt, t, temp, stats, dlogp, dz, dstride, None)


def policy(L, z=A[0], rows=4, cols=64, stride=64, dt=BF16, t=A[1], old=A[2], ref=A[3], adv=A[4], w=A[5], record=A[6], logp=A[7], dz=A[8],
           dstride=64, hyper=True, **h):
    hy = mr._PolicyHyperC(**{**dict(temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.1, grad_scale=1.0), **h})
    return L.mr_policy_loss(z, rows, cols, stride, dt, t, old, ref, adv, w, ctypes.byref(hy) if hyper else None, record, logp, dz, dstride, None)


def pref(L, logp=A[0], ref=A[1], rows=100, off=A[2], pairs=3, record=A[3], margins=A[4], dlogp=A[5], hyper=True, **h):
    hy = mr._PreferenceHyperC(**{**dict(beta=0.1, smoothing=0.0, loss_scale=1.0, grad_scale=1.0), **h})
    return L.mr_preference_loss(logp, ref, rows, off, pairs, ctypes.byref(hy) if hyper else None, record, margins, dlogp, None)


@pytest.mark.parametrize("call", [fwd, bwd, policy])
def test_rows_types_and_temperature(L, call):
    temp = "temperature" if call is policy else "temp"
    assert call(L, dt=INT32) == EDTYPE and call(L, dt=7) == EINVAL and call(L, dt=-1) == EINVAL
    assert call(L, stride=63) == EINVAL and call(L, cols=2 ** 31, stride=2 ** 31) == EINVAL
    assert call(L, rows=2 ** 41) == EINVAL and call(L, stride=2 ** 41) == EINVAL and call(L, rows=2 ** 30, stride=2 ** 30) == EINVAL
    for t in (0.0, -1.0, NAN, INF, 1e-60, 1e60):
        assert call(L, **{temp: t}) == EINVAL, t
    assert call(L, z=None) == EINVAL and call(L, t=None) == EINVAL
    assert call(L, z=A[0] + 1) == EINVAL and call(L, t=A[1] + 4) == EINVAL and call(L, dt=FP32, z=A[0] + 2) == EINVAL


def test_forward_refusals(L):
    assert fwd(L, logp=A[2] + 2) == EINVAL and fwd(L, stats=A[3] + 1) == EINVAL
    assert fwd(L, logp=A[3]) == EALIAS and fwd(L, logp=A[0] + 64) == EALIAS and fwd(L, stats=A[1]) == EALIAS
    assert fwd(L, logp=A[0] + 4 * 64 * 2 - 4) == EALIAS                  # the last row's end
    assert fwd(L, rows=0, z=None, t=None) == OK and fwd(L, logp=None, stats=None) == OK


def test_backward_refusals(L):
    for k in ("stats", "dlogp", "dz"):
        assert bwd(L, **{k: None}) == EINVAL, k
    assert bwd(L, dz=A[5] + 1) == EINVAL and bwd(L, stats=A[3] + 2) == EINVAL and bwd(L, dlogp=A[4] + 2) == EINVAL and bwd(L, dstride=63) == EINVAL
    assert bwd(L, dz=A[0] + 2) == EALIAS and bwd(L, dz=A[0], dstride=65) == EALIAS and bwd(L, dz=A[1]) == EALIAS
    assert bwd(L, dz=A[3]) == EALIAS and bwd(L, dz=A[4] - 128) == EALIAS
    assert bwd(L, rows=0) == OK and bwd(L, cols=0) == OK


def test_policy_refusals(L):
    assert policy(L, hyper=False) == EINVAL
    for h in (dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=NAN), dict(clip_high=-0.1), dict(clip_high=INF), dict(kl_coef=NAN),
              dict(grad_scale=0.0), dict(grad_scale=INF), dict(grad_scale=-1.0)):
        assert policy(L, **h) == EINVAL, h
    assert policy(L, ref=None) == EINVAL                                   # a KL term against nothing
    assert policy(L, adv=None) == EINVAL and policy(L, record=None) == EINVAL and policy(L, dstride=63) == EINVAL
    for k, p in (("old", A[2]), ("ref", A[3]), ("adv", A[4]), ("w", A[5]), ("record", A[6]), ("logp", A[7])):
        assert policy(L, **{k: p + 2}) == EINVAL, k
    assert policy(L, dz=A[8] + 1) == EINVAL
    assert policy(L, dz=A[0] + 2) == EALIAS and policy(L, dz=A[0], dstride=80) == EALIAS and policy(L, record=A[8]) == EALIAS
    for k in ("old", "ref", "adv", "w"):
        assert policy(L, **{k: A[7]}) == EALIAS, k                         # over logp
    assert policy(L, logp=A[1]) == EALIAS and policy(L, record=A[7]) == EALIAS


def test_preference_refusals(L):
    assert pref(L, hyper=False) == EINVAL
    for h in (dict(beta=NAN), dict(smoothing=-0.1), dict(smoothing=0.6), dict(smoothing=NAN), dict(loss_scale=INF), dict(grad_scale=0.0)):
        assert pref(L, **h) == EINVAL, h
    assert pref(L, logp=None) == EINVAL and pref(L, off=None) == EINVAL and pref(L, record=None) == EINVAL
    assert pref(L, rows=2 ** 41) == EINVAL and pref(L, pairs=2 ** 41) == EINVAL
    for k, p in (("logp", A[0]), ("ref", A[1]), ("record", A[3]), ("margins", A[4]), ("dlogp", A[5])):
        assert pref(L, **{k: p + 2}) == EINVAL, k
    assert pref(L, off=A[2] + 4) == EINVAL
    assert pref(L, dlogp=A[0] + 4) == EALIAS and pref(L, dlogp=A[1]) == EALIAS and pref(L, margins=A[2]) == EALIAS
    assert pref(L, record=A[4] + 8) == EALIAS


def test_binding_refuses_wrong_tensors():
    import torch

    z, t, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError):
        mr.token_logprob_forward(z, t, f)
    with pytest.raises(ValueError):
        mr.token_logprob_backward(z, t, f, f, z)
    with pytest.raises(ValueError):
        mr.policy_loss(z, t, f, f)
    with pytest.raises(ValueError):
        mr.preference_loss(f, torch.zeros(2, dtype=torch.int64), f)
    with pytest.raises(ValueError):
        mr.preference_loss(f, torch.zeros(3, dtype=torch.int64), f)


class _OnDevice:
    """What the binding reads of a device tensor, for its checks of shapes and strides."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, k):
        return getattr(self.t, k)


def test_rows_of_logits():
    import torch

    def rows(t, ref=None):
        return mr._rows2d(_OnDevice(t), "logits", ref)

    z = torch.zeros(6, 10)
    assert rows(z) == (6, 10, 10) and rows(z[:, :7]) == (6, 7, 10) and rows(z[::2, :7]) == (3, 7, 20) and rows(z[2:3, 1:]) == (1, 9, 9)
    assert rows(torch.zeros(2, 3, 5)) == (6, 5, 5) and rows(torch.zeros(0, 5)) == (0, 5, 5) and rows(torch.zeros(5, 0)) == (5, 0, 0)
    assert rows(torch.zeros(9)) == (1, 9, 9) and rows(z[:, :1]) == (6, 1, 10)
    for bad in (z.t(), z[:1].expand(6, 10), torch.zeros(2, 3, 10)[:, :, :7], z[:, ::2]):
        with pytest.raises(ValueError):
            rows(bad)
    with pytest.raises(ValueError):
        rows(z, torch.zeros(6, 9))
    with pytest.raises(ValueError):
        rows(z, torch.zeros(6, 10, dtype=torch.float16))
