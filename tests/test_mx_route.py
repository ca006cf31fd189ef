"""The shapes of tests/_mx_kernels.py run where they say, and take in every form of both kernels."""
import pytest

from _mx_kernels import FEW, MANY, PAIRS, route


@pytest.mark.parametrize("kind", ["mx8", "mx4"])
def test_shapes_reach_their_kernels(kind):
    for (tokens, n_in, n_out), where in FEW + MANY:
        assert route(kind, tokens, n_in, n_out) == where, (tokens, n_in, n_out)
    assert {where for _, where in FEW} == {(tile, splits) for tile in (16, 32, 64) for splits in (1, 2, 4, 8)}


def test_rule_at_its_borders():
    assert route("mx8", 48, 4096, 65536) == (64, 1) and route("mx8", 49, 4096, 65536) == PAIRS
    assert route("mx8", 64, 4096, 152 * 128) == (64, 1) and route("mx8", 65, 4096, 152 * 128) == PAIRS
    assert route("mx8", 1, 128, 128) == route("mx4", 1, 768, 128) == (16, 1)     # (less than two stages a CTA)
    assert route("mx8", 1, 512, 128) == route("mx4", 1, 1024, 128) == (16, 2)
    assert route("mx8", 16, 4096, 76 * 128)[1] == 4 and route("mx8", 16, 4096, 77 * 128)[1] == 2
