"""A model of how the policy loss lays a row over its lanes: for every width, alignment and start, each column is counted once and no
pack passes the row's ends."""
import random

import numpy as np
import pytest

MOST_WAVES, MOST_PACKS, CUS = 16, 16, 256


def held_row(rows, cols, V, on_grid):
    """(waves, packs a lane) of rows held in registers, or None."""
    packs, whole = (cols + (V - 1 if on_grid else 2 * V - 2)) // V, cols // V
    if whole == 0:
        return None
    order = range(min(-(-packs // 64), MOST_WAVES), 0, -1) if rows <= CUS else range(1, MOST_WAVES + 1)
    for waves in order:
        need = -(-packs // (64 * waves))
        K = need if need <= 2 else (need + 1) // 2 * 2
        if K <= MOST_PACKS and (K <= 2 or (K - 2) * 64 * waves <= whole):
            return waves, K
    return None


def check(cols, V, on_grid, off, waves, K):
    lanes, last, ends = 64 * waves, cols - V, min(K, 2)
    count = np.zeros(cols, int)
    for k in range(K):
        col = (k * lanes + np.arange(lanes)) * V - off
        at = col
        if k == 0 or k >= K - ends:
            at = np.clip(col, 0, last)
        assert at.min() >= 0 and at.max() <= last
        own = col - at
        for i in range(V):
            mine = (i >= own) & (i < own + V) if k == 0 else i >= own if k >= K - ends else np.ones(lanes, bool)
            np.add.at(count, (at + i)[mine], 1)
    assert (count == 1).all()


@pytest.mark.parametrize("V", [4, 8])
@pytest.mark.parametrize("rows", [1, 1000])
def test_every_column_once(rows, V):
    r = random.Random(V)
    widths = list(range(V, 1200, 13)) + [r.randrange(1200, V * 16500) for _ in range(60)]
    widths += [1024 * V * k + d for k in (1, 2, 5, 9, 15, 16) for d in (-V - 1, -1, 0, 1, V)]
    widths += [64 * V * k + d for k in range(1, 40, 3) for d in (-V - 1, -1, 0, 1, 2, V)]
    for cols in widths:
        for on_grid in (True, False):
            h = held_row(rows, cols, V, on_grid)
            if h is None:
                assert cols < V or (cols + 2 * V - 2) // V > 64 * MOST_WAVES * MOST_PACKS - 64 * MOST_WAVES
                continue
            assert h[0] <= MOST_WAVES and (h[1] <= 2 or h[1] % 2 == 0) and h[1] <= MOST_PACKS
            for off in [0] if on_grid else (0, 1, V - 1):
                check(cols, V, on_grid, off, *h)
