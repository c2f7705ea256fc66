"""How Muon's host code lays a list's matrices over its momentum launch, without a GPU (the runtime of fake_hip.cpp): each gets the
workgroups that it gets alone, so its norm is summed in the same order, and with it every bit that follows."""
import pytest

from test_launches import fake, launches, pytestmark  # noqa: F401
from test_launches_losses_muon import muon


def momentum_groups(L, shapes, products):
    L.fake_reset(0)
    assert muon(L, shapes, products) == 0
    return sum(x["grid"][0] for x in launches(L) if "momentum" in x["name"])


@pytest.mark.parametrize("products", [16, 32])
@pytest.mark.parametrize("shapes", [[(2048, 2048)] * 3, [(2048, 2048), (4096, 4096)], [(100, 100)] * 20 + [(8192, 2048)], [(4096, 4096)] * 9 + [(700, 1000)] * 30,
                                    [(1, 1), (0, 5), (3000, 2000), (2900, 2900)]])
def test_a_matrix_has_the_workgroups_that_it_has_alone(fake, shapes, products):
    alone = [momentum_groups(fake, [s], products) if s[0] * s[1] else 0 for s in shapes]
    assert momentum_groups(fake, shapes, products) == sum(alone), alone
