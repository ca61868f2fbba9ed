"""The same window said in two ways: the same schedule, so the same bits."""
import pytest
import torch

import chunk_routed_sparse_b200 as moc

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


@pytest.mark.parametrize("B,Hq,Hk,Lq,Lk,d,left,sinks", [
    (1, 2, 2, 1, 20000, 128, 1000, 64), (1, 8, 1, 2, 9000, 64, 700, 4), (3, 12, 3, 4, 5000, 128, 255, 0),
    (1, 1, 1, 1, 60000, 64, 255, 64), (1, 2, 1, 300, 1500, 64, 200, 130), (2, 3, 3, 700, 700, 128, 100, 3)])
def test_causal_needs_no_right_limit(B, Hq, Hk, Lq, Lk, d, left, sinks):
    """Under causal no key lies right of a row: an open right side, none and a wide one are one window."""
    Q, K, V, g = (_rand(B, h, n, d, seed=i) for i, (h, n) in enumerate(((Hq, Lq), (Hk, Lk), (Hk, Lk), (Hq, Lq))))
    want = None
    for right in (0, -1, 5, 1 << 35):
        args = (left, right, sinks, True)
        O, lse = moc.window_attention_fwd(Q, K, V, *args)
        got = (O, lse, *moc.window_attention_bwd(Q, K, V, O, lse, g, *args))
        want = got if want is None else want
        for name, x, y in zip(("O", "lse", "dQ", "dK", "dV"), got, want):
            assert torch.equal(x, y), (right, name)
