"""The model of test_logit_rows.py held against the host code: for every width, alignment and number of rows the policy loss launches
the packs a lane and the waves that the model gives, or goes over the logits twice where it gives none (fake_hip.cpp, no GPU)."""
import random
import re

import pytest

from test_launches import BF16, FP16, FP32, fake, launches, pytestmark  # noqa: F401
from test_launches_losses_muon import policy
from test_logit_rows import CUS, MOST_PACKS, MOST_WAVES, held_row

TYPES = {BF16: (8, 2, "EBf16"), FP16: (8, 2, "EFp16"), FP32: (4, 4, "EFp32")}


def launched(L, rows, cols, dt, stride, off):
    L.fake_reset(0)
    assert policy(L, rows, cols, dt, stride=stride, off=off) == 0
    out = []
    for x in launches(L):
        m = re.search(r"(policy_held|row_stats|logit_grad)INS_\d(\w{4,5}?)(?:EL|EE)", x["name"])
        if m:
            k = re.search(r"policy_held\w*?ELi(\d+)E", x["name"])
            out.append((m.group(1), m.group(2), int(k.group(1)) if k else None, x["block"][0] // 64, x["grid"][0]))
    return out


def widths(V, r):
    w = list(range(1, 3 * V)) + [r.randrange(V, V * 17000) for _ in range(60)]
    w += [1024 * V * k + d for k in (1, 2, 5, 9, 15, 16) for d in (-2 * V, -V - 1, -1, 0, 1, V)]
    return w + [64 * V * k + d for k in (*range(1, 18), 25, 39) for d in (-2 * V, -V - 1, -1, 0, 1, 2, V)]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows", [1, 8, 31, 32, CUS, CUS + 1, 5000])
def test_the_launched_shape_is_the_model_s(fake, rows, dt):
    V, es, name = TYPES[dt]
    seen = set()
    for cols in widths(V, random.Random(rows * 8 + V)):
        for stride, off in ((-(-cols // V) * V, 0), (cols, 0), (cols, es), (cols + 1, 16)):
            on_grid = off % 16 == 0 and (rows == 1 or stride * es % 16 == 0)
            h = held_row(rows, cols, V, on_grid)
            got = launched(fake, rows, cols, dt, stride, off)
            assert all(x[1] == name for x in got), got
            if h is not None and (rows >= CUS // 8 or h[1] <= 12):
                assert [x[:4] for x in got] == [("policy_held", name, h[1], h[0])], (cols, stride, off, got)
                assert 1 <= got[0][4] <= rows
                seen.add(h[1])
            else:
                assert [x[0] for x in got] == ["row_stats", "logit_grad"], (cols, stride, off, got)
    assert seen >= ({1} if rows <= CUS else {1, 2, 4, 6, 8, 10, 12, 14, 16}), seen
    assert max(seen) <= MOST_PACKS and MOST_WAVES == 16
