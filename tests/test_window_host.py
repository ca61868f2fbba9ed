"""Argument checks and workspace sizes of the sliding-window attention, without a GPU."""
import math

import pytest
import torch

import chunk_routed_sparse_b200 as moc
import oracle.window as W

P = 4096  # never dereferenced: every call here is refused (or has nothing to do) first


def _fwd(B=1, Hq=4, Hk=2, Lq=8, Lk=8, d=64, Q=P, K=P, V=P, left=-1, right=-1, sinks=0, causal=1, ql=None, kl=None,
         fill=0, scale=0.125, O=P, lse=None):
    return moc.lib().moc_window_attention(B, Hq, Hk, Lq, Lk, d, Q, K, V, left, right, sinks, causal, ql, kl, fill,
                                          scale, O, lse, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(Hq=-4, Hk=-2), 1), (dict(Lq=-1), 1), (dict(Lk=-1), 1), (dict(d=96), 1), (dict(Hq=3), 1),
    (dict(Hk=0), 1), (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(Q=None), 1), (dict(Q=P + 8), 1), (dict(K=None), 1), (dict(V=P + 2), 1),
    (dict(O=None), 1), (dict(lse=P + 2), 1), (dict(ql=P + 1), 1), (dict(kl=P + 2), 1), (dict(Lk=1 << 28), 6),
    (dict(Lq=1 << 28), 6), (dict(B=70000, Lq=1, Lk=1), 6), (dict(B=60000, Hq=60000, Hk=60000, Lq=1, Lk=1), 6),
    (dict(B=0), 0), (dict(Hq=0, Hk=0), 0), (dict(Lq=0), 0)])
def test_bad_calls_are_refused_before_any_launch(kw, status):
    assert _fwd(**kw) == status


def test_backward_refusals_and_workspace():
    lib = moc.lib()

    def size(B=1, Hq=4, Hk=2, Lq=300, Lk=300, d=64, left=50, right=0, sinks=9, causal=1):
        return lib.moc_window_attention_bwd_workspace_bytes(B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal)

    assert size(d=96) == 0 and size(Hq=3) == 0 and size(sinks=-1) == 0
    n = size()
    assert n > 4 * 300 * 2 * 4
    # first keys seen by many rows: their tiles' rows are split, with fp32 parts
    assert size(Lq=30000, Lk=30000) > size(Lq=30000, Lk=30000, sinks=0) + 2 * 128 * 64 * 4

    def bwd(ws=P, nb=1 << 40, lse=P, dQ=P, dK=P, O=P, Lq=300):
        return lib.moc_window_attention_bwd(1, 4, 2, Lq, 300, 64, P, P, P, O, lse, P, 50, 0, 9, 1, None, None, 0, 0.125, dQ,
                                            dK, P, ws, nb, None)

    assert bwd(ws=None) == 1 and bwd(ws=P + 16) == 1 and bwd(nb=n - 1) == 3
    assert bwd(lse=None) == 1 and bwd(lse=P + 1) == 1 and bwd(dQ=P + 8) == 1 and bwd(dK=None) == 1 and bwd(O=None) == 1


def test_binding_refusals():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moc.window_attention_fwd(x, x, x)


def test_definition_counts():
    """The oracle's own mask against a direct count."""
    for n, m, left, right, sinks, causal in ((9, 9, 2, 1, 2, False), (9, 4, 3, 0, 1, True), (3, 6, 1, 1, 1, True),
                                             (7, 7, -1, 2, 0, False), (7, 7, 0, -1, 3, True)):
        see = W.visible(n, m, left, right, sinks, causal)
        for t in range(m):
            p = t + n - m
            for u in range(n):
                near = (left < 0 or p - u <= left) and (right < 0 or u - p <= right)
                assert bool(see[t, u]) == ((near or u < sinks) and (not causal or u <= p))
