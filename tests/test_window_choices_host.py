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


BIG = 1 << 24  # apart: far more than any tensor below


def _gradient(**kw):
    """Never dereferenced: every call here is refused first."""
    a = {n: BIG * (i + 1) for i, n in enumerate(("Q", "K", "V", "O", "lse", "dO", "dQ", "dK", "dV", "ws"))}
    a.update(kw)
    return moc.lib().moc_window_attention_bwd(1, 4, 2, 300, 300, 64, a["Q"], a["K"], a["V"], a["O"], a["lse"], a["dO"], 50, 0,
                                              9, 1, None, None, 0, 0.125, a["dQ"], a["dK"], a["dV"], a["ws"], BIG // 2, None)


@pytest.mark.parametrize("out,other", [(o, i) for o in ("dQ", "dK", "dV", "ws") for i in ("Q", "K", "V", "dO")] +
                         [("dQ", "dK"), ("dQ", "dV"), ("dK", "dV"), ("ws", "dQ"), ("ws", "dK"), ("ws", "O"), ("ws", "lse")])
def test_gradients_that_overlap_are_refused(out, other):
    at = {n: BIG * (i + 1) for i, n in enumerate(("Q", "K", "V", "O", "lse", "dO", "dQ", "dK", "dV", "ws"))}[other]
    assert _gradient(**{out: at}) == 1              # the same tensor
    assert _gradient(**{out: at + 256}) == 1        # part of it


@pytest.mark.parametrize("kw", [dict(O="K"), dict(O="V"), dict(lse="Q"), dict(lse="K"), dict(lse="V"), dict(lse="O")])
def test_outputs_that_overlap_are_refused(kw):
    a = dict(Q=BIG, K=2 * BIG, V=3 * BIG, O=4 * BIG, lse=5 * BIG)
    for off in (0, 256):
        b = dict(a, **{n: a[o] + off for n, o in kw.items()})
        assert moc.lib().moc_window_attention(1, 4, 2, 300, 300, 64, b["Q"], b["K"], b["V"], 50, 0, 9, 1, None, None, 0, 0.125,
                                              b["O"], b["lse"], None) == 1
    assert moc.lib().moc_window_attention(1, 4, 2, 300, 300, 64, BIG, 2 * BIG, 3 * BIG, 50, 0, 9, 1, None, None, 0, 0.125,
                                          BIG + 256, 5 * BIG, None) == 1
