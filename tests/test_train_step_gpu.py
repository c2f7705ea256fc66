"""The example training step: gather, layer norm, reduce, clip and AdamW together learn, with 8-bit moments as with 32-bit ones."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _train():
    spec = importlib.util.spec_from_file_location("train_step_example", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.train


def test_example_learns_and_8_bit_moments_follow_32():
    train = _train()
    end = {}
    for bits in (32, 8):
        losses = train(steps=100, bits=bits)
        assert all(math.isfinite(x) for x in losses)
        end[bits] = sum(losses[-10:]) / 10
        print(f"[case] bits={bits} first {losses[0]:.4f} last {end[bits]:.4f}", flush=True)
        assert end[bits] < 0.25 * losses[0]
    # the rounding adds noise to each element's step; the loss may trail by as much as half again
    assert end[8] < 1.5 * end[32]


def test_every_run_gives_the_same_losses():
    train = _train()
    a, b = train(steps=5), train(steps=5)
    assert a[0] == b[0]  # the forward pass is this package's and torch's products of the same inputs
    assert all(abs(x - y) <= 2.0 ** -6 * abs(x) for x, y in zip(a, b))
