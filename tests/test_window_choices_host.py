"""Choices of the window attention's calls that need no GPU to be refused."""
import pytest

import chunk_routed_sparse_b200 as moc

P = 4096  # never dereferenced: every call here is refused first


@pytest.mark.parametrize("flags", [4, 7, -1, 1 << 30])
def test_unknown_flags_of_the_gradient_are_refused(flags):
    assert moc.lib().moc_window_attention_bwd(1, 4, 2, 300, 300, 64, P, P, P, P, P, P, 50, 0, 9, 1, None, None, flags, 0.125,
                                              P, P, P, P, 1 << 40, None) == 1
