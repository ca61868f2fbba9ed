"""Choices of the window attention's calls that need no GPU to be refused."""
import pytest

import chunk_routed_sparse_b200 as moc
from chunk_routed_sparse_b200 import window

P = 4096  # never dereferenced: every call here is refused first


@pytest.mark.parametrize("flags", [4, 7, -1, 1 << 30])
def test_unknown_flags_of_the_gradient_are_refused(flags):
    assert moc.lib().moc_window_attention_bwd(1, 4, 2, 300, 300, 64, P, P, P, P, P, P, 50, 0, 9, 1, None, None, flags, 0.125,
                                              P, P, P, P, 1 << 40, None) == 1


@pytest.mark.parametrize("given,want", [((-1, -1, 0), (-1, -1, 0)), ((255, -1, 64), (255, -1, 64)), ((-7, 3, 1), (-1, 3, 1)),
                                        ((1 << 70, -(1 << 70), 5), (1 << 40, -1, 5)), ((0, 0, 1 << 50), (0, 0, 1 << 40)),
                                        ((True, 2, 0), (1, 2, 0))])
def test_limits_fit_64_bits(given, want):
    got = window._limits(*given)
    assert got == want and all(type(x) is int for x in got)


def test_negative_first_keys_are_refused():
    assert window._limits(0, 0, -4) == (0, 0, -1)
    assert moc.lib().moc_window_attention(1, 4, 2, 8, 8, 64, P, P, P, 0, 0, -1, 1, None, None, 0, 0.125, P, None, None) == 1
