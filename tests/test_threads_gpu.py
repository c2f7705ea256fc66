"""Calls of several host threads on one stream: each call's kernels hand partial sums over in the stream's workspace."""
import threading

import pytest
import torch

import all_gather_amd as mr
from gpu_util import device

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    """A backward pass with a second launch, a gradient norm of three launches and a two-shot sum from each of two threads at once
    give the bits that they give alone."""
    rows, cols, rounds = 700, 1600, 40
    gen = torch.Generator().manual_seed(21)
    work = []
    for _ in range(2):
        x, dy = (torch.randn(rows, cols, generator=gen).to(torch.bfloat16).to(device()) for _ in range(2))
        m, r = torch.randn(rows, generator=gen).to(device()), torch.rand(rows, generator=gen).to(device())
        grads = list(torch.randn(300, 5000, generator=gen).to(device()).unbind(0))
        work.append((x, dy, m, r, grads))

    def outputs(x):
        return (torch.empty_like(x), torch.empty(cols, device=device()), torch.empty(cols, device=device()), torch.empty(3, device=device()),
                torch.empty_like(x))

    def step(w, o):
        x, dy, m, r, grads = w
        mr.layer_norm_backward(dy, x, None, m, r, o[0], dgamma=o[1], dbeta=o[2])
        mr.grad_norm(grads, o[3], max_norm=1.0)
        mr.allreduce_sum([x, dy], o[4], mode="twoshot")

    want = [outputs(w[0]) for w in work]
    for w, o in zip(work, want):
        step(w, o)
    got = [[outputs(w[0]) for _ in range(rounds)] for w in work]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def run(i):
        try:
            start.wait(timeout=30)
            for o in got[i]:
                step(work[i], o)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        for k, o in enumerate(got[i]):
            assert all(torch.equal(a, b) for a, b in zip(want[i], o)), (i, k)
    assert mr.workspace_check() == 0
