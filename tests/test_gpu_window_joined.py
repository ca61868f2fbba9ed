"""Gradients of the sliding-window attention from O and lse that were joined over several
key ranges, one call a range: the usual way to keep a long cache in parts.

Tolerances as in test_gpu_window.py, with one more rounding in D = dO . O (each part's O,
then the joined one: (3 u + w) of its terms instead of (2 u + w)), so u |x| + (5 u + 2 w)
size for dQ and dK; the parts' dQ are rounded each."""
import pytest
import torch

import chunk_routed_sparse_b200 as moc
import oracle.window as W

pytestmark = pytest.mark.gpu
U, WT = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    moc.check_window_error()


def _rand(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hk,Lq,cuts,causal", [
    (1, 4, 2, 70, (0, 200, 333), False), (2, 2, 2, 300, (0, 150, 700, 1000), False), (1, 4, 1, 20, (0, 5, 90), False),
    (1, 3, 3, 200, (0, 500, 700), True), (1, 2, 1, 130, (0, 300, 430), True)])
def test_gradients_of_key_ranges_add_up(B, Hq, Hk, Lq, cuts, causal, d):
    Lk = cuts[-1]
    Q, K, V = _rand(B, Hq, Lq, d, seed=1), _rand(B, Hk, Lk, d, seed=2), _rand(B, Hk, Lk, d, seed=3)
    g = _rand(B, Hq, Lq, d, seed=4)
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        k, v = K[:, :, a:b].contiguous(), V[:, :, a:b].contiguous()
        own = causal and b == Lk  # the rows' own tokens; all of the earlier ones are visible
        parts.append((k, v, own, *moc.window_attention_fwd(Q, k, v, causal=own)))
    lse = torch.logsumexp(torch.stack([p[4] for p in parts]), 0)
    O = sum(torch.exp(p[4] - lse)[..., None] * p[3].float() for p in parts).to(torch.bfloat16)
    got = [moc.window_attention_bwd(Q, k, v, O, lse, g, causal=own, joined=True) for k, v, own, _, _ in parts]
    ref = W.attention(Q, K, V, -1, -1, 0, causal, dO=g)
    dK, dV = torch.cat([x[1] for x in got], 2).double(), torch.cat([x[2] for x in got], 2).double()
    dQ = sum(x[0].double() for x in got)
    step = U * (1 + 2 * U) * sum(x[0].double().abs() for x in got)
    for name, x, tol in (("dQ", dQ, step + (5 * U + 2 * WT) * ref["sQ"]),
                         ("dK", dK, U * ref["dK"].abs() + (5 * U + 2 * WT) * ref["sK"]),
                         ("dV", dV, U * ref["dV"].abs() + (U + WT) * ref["sV"])):
        assert ((x - ref[name]).abs() <= tol).all(), name
        # many small and independent errors: in the 2-norm, a rounding's share is u / sqrt(3); the
        # parts' O, the joined O, ds and the result: below 2 u
        assert (x - ref[name]).norm() <= 2 * U * ref[name].norm() + 1e-30, name
    again = [moc.window_attention_bwd(Q, k, v, O, lse, g, causal=own, joined=True) for k, v, own, _, _ in parts]
    assert all(torch.equal(x, y) for p, q in zip(got, again) for x, y in zip(p, q))
