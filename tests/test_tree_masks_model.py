"""How far the tree attention kernel's copies run ahead of the masks of loaded keys that are still
read: the bound that the kernel asserts when it is compiled, on the model of its barriers."""
import pytest

from test_tree_protocol_model import LISTS, Model

MORE = [[(20, True)], [(20, False)], [(1, True), (30, True), (1, False), (9, False)]]
RINGS = [(5, 0), (10, 0), (3, 4), (6, 8)]


@pytest.mark.parametrize("stages,raw", RINGS)
@pytest.mark.parametrize("pieces", LISTS + MORE)
def test_the_shortest_ring_that_the_kernel_accepts(pieces, stages, raw):
    for seed in range(20):
        m = Model(pieces, stages, seed, raw, seen=(stages + raw) // 2 + 3)
        assert m.run(), "deadlock"


@pytest.mark.parametrize("stages,raw", RINGS)
def test_half_of_it_is_too_short(stages, raw):
    def fails(seen):
        for seed in range(60):
            try:
                if not Model([(40, True), (40, False)], stages, seed, raw, seen=seen).run():
                    return True
            except AssertionError:
                return True
        return False

    assert fails(((stages + raw) // 2 + 3) // 2)
