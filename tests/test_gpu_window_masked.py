"""Infinities and NaN where the mask of the sliding-window attention leaves nothing: keys
that no row sees, rows that see no key, in forward and gradient. Results that do not
depend on them keep their bits."""
import math

import pytest
import torch

import chunk_routed_sparse_b200 as moc
import oracle.window as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    moc.check_window_error()


def _rand(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _step(Q, K, V, g, args, kl=None, ql=None):
    O, lse = moc.window_attention_fwd(Q, K, V, *args, q_len=ql, kv_len=kl)
    return (O, lse, *moc.window_attention_bwd(Q, K, V, O, lse, g, *args, q_len=ql, kv_len=kl))


KEYS = [  # B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal
    (1, 4, 2, 70, 500, 64, 60, 0, 5, True),       # a tile of first keys, and one that the window's start shares
    (1, 4, 2, 70, 500, 128, 60, 0, 5, True),
    (2, 2, 2, 200, 700, 64, 130, 40, 131, False),
    (2, 2, 1, 200, 700, 128, 130, 40, 0, False),
    (1, 6, 3, 17, 300, 128, 90, 0, 3, True),      # gradients of few rows
    (1, 2, 2, 3, 410, 64, 33, 0, 1, True),
    (1, 40, 40, 300, 1100, 64, 100, 7, 9, False),  # the forward's two-tile kernel
]


@pytest.mark.parametrize("case", KEYS, ids=str)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_keys_that_no_row_sees_reach_nothing(case, bad):
    B, Hq, Hk, Lq, Lk, d, *args = case
    Q, K, V, g = _rand(B, Hq, Lq, d, seed=1), _rand(B, Hk, Lk, d, seed=2), _rand(B, Hk, Lk, d, seed=3), _rand(B, Hq, Lq, d, seed=4)
    want = _step(Q, K, V, g, args)
    unseen = ~W.visible(Lk, Lq, *args).any(0).cuda()
    assert unseen.any() and not unseen.all()
    for which in ("K", "V", "KV"):
        k, v = K.clone(), V.clone()
        if "K" in which:
            k[:, :, unseen] = bad
        if "V" in which:
            v[:, :, unseen] = bad
        got = _step(Q, k, v, g, args)
        for name, x, y in zip(("O", "lse", "dQ", "dK", "dV"), got, want):
            assert torch.equal(x, y), (which, name)
        assert (got[3][:, :, unseen] == 0).all() and (got[4][:, :, unseen] == 0).all()


ROWS = [  # more rows than keys: the first rows see nothing; the first row that does is no multiple of four
    (1, 4, 2, 300, 98, 64, 20, 0, 4, True),
    (1, 4, 2, 300, 99, 128, 20, 0, 4, True),
    (2, 2, 2, 300, 100, 64, 20, 29, 0, False),
    (2, 2, 1, 301, 134, 128, 20, 6, 0, False),
    (1, 3, 1, 40, 5, 128, 90, 0, 3, True),         # gradients of few rows
    (1, 2, 1, 7, 2, 64, -1, 0, 0, True),           # the few-row kernel
    (1, 250, 1, 300, 101, 64, 20, 0, 4, True),     # the forward's two-tile kernel
]


@pytest.mark.parametrize("case", ROWS, ids=str)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_see_no_key_reach_nothing(case, bad):
    B, Hq, Hk, Lq, Lk, d, *args = case
    Q, K, V, g = _rand(B, Hq, Lq, d, seed=1), _rand(B, Hk, Lk, d, seed=2), _rand(B, Hk, Lk, d, seed=3), _rand(B, Hq, Lq, d, seed=4)
    want = _step(Q, K, V, g, args)
    blind = ~W.visible(Lk, Lq, *args).any(1).cuda()
    assert blind.any() and not blind.all()
    for which in ("Q", "dO", "Q dO"):
        q, u = Q.clone(), g.clone()
        if "Q" in which:
            q[:, :, blind] = bad
        if "dO" in which:
            u[:, :, blind] = bad
        got = _step(q, K, V, u, args)
        for name, x, y in zip(("O", "lse", "dQ", "dK", "dV"), got, want):
            assert torch.equal(x, y), (which, name)
        assert (got[0][:, :, blind] == 0).all() and (got[2][:, :, blind] == 0).all()
