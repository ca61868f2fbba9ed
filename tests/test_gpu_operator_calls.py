"""Calls of the operators around the attention that the documentation allows: a process's
first call inside a captured graph, no rows or no keys, overwritten buffers."""
import os
import subprocess
import sys

import pytest
import torch

import chunk_routed_sparse_b200 as moc
from conftest import ROOT

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


FIRST = """
import torch
import chunk_routed_sparse_b200 as moc
x = torch.randn(1, {L}, 6, 64, device="cuda").bfloat16()
q, k, v = (t.contiguous() for t in x.transpose(1, 2).split((2, 2, 2), 1))
g = torch.randn(1, 2, {L}, 64, device="cuda").bfloat16()
w = torch.ones(64, device="cuda")
n = torch.tensor([{L}], device="cuda", dtype=torch.int32)
rope = moc.Rope(64)
def step():
    {call}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
want = step()
assert all(torch.equal(a, b) for a, b in zip(held, want))
moc.check_window_error()
"""
CALLS = {
    "rotary": (9, "return (moc.rotary(rope, x.transpose(1, 2)),)"),
    "norm": (9, "return moc.qkv_norm_rope(x, 2, 2, w, w, rope)"),
    "norm gradient": (9, "return moc.qkv_norm_rope_bwd(x, 2, 2, w, w, rope, None, 1e-6, g, k, v)"),
    "few rows": (5, "return moc.window_attention_fwd(q, k, v, 3, 0, 1, True)"),
    "one tile": (300, "return moc.window_attention_fwd(q, k, v, 100, 0, 1, True)"),
    "one tile, padded": (300, "return moc.window_attention_fwd(q, k, v, 100, 0, 1, True, n, n)"),
    "two tiles": (30000, "return moc.window_attention_fwd(q, k, v, 100, 0, 1, True)"),
    "gradient": (3000, "o = moc.window_attention_fwd(q, k, v, 99, 0, 3, True); "
                       "return moc.window_attention_bwd(q, k, v, *o, g, 99, 0, 3, True)"),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_first_call_may_be_captured(name):
    L, call = CALLS[name]
    code = FIRST.format(L=L, call=call)
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, PYTHONPATH=ROOT))
    assert run.returncode == 0, run.stderr[-3000:]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Lq,Lk", [(2, 3, 0, 200), (2, 3, 200, 0), (0, 3, 20, 20), (2, 0, 20, 20), (2, 3, 0, 0)])
def test_no_rows_or_no_keys(B, H, Lq, Lk, d):
    Q, K, V, g = _rand(B, H, Lq, d, seed=1), _rand(B, H, Lk, d, seed=2), _rand(B, H, Lk, d, seed=3), _rand(B, H, Lq, d, seed=4)
    for args in ((-1, -1, 0, False), (50, 0, 130, True)):
        O, lse = moc.window_attention_fwd(Q, K, V, *args)
        grads = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
        torch.cuda.synchronize()
        for x, like in zip((O, *grads), (Q, Q, K, K)):
            assert x.shape == like.shape and (x == 0).all()
        assert lse.shape == (B, H, Lq) and (lse == -torch.inf).all()


def test_gradient_of_the_norm_into_its_inputs_and_upstream_gradients():
    """dQ over Q or over dQo, dV over dVo: a row is read before it is written."""
    B, Hq, Hk, L, d = 2, 5, 2, 333, 128
    rope = moc.Rope(d, interleaved=False)
    w = 1 + 0.1 * torch.randn(d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    Q, K = _rand(B, Hq, L, d, seed=1), _rand(B, Hk, L, d, seed=2)
    up = [_rand(B, h, L, d, seed=3 + i) for i, h in enumerate((Hq, Hk, Hk))]
    want = moc.qk_norm_rope_bwd(Q, K, w, w, rope, None, 1e-6, *up)
    for over_inputs in (True, False):
        q, k, u = Q.clone(), K.clone(), [t.clone() for t in up]
        out = (q, k, u[2]) if over_inputs else tuple(u)
        got = moc.qk_norm_rope_bwd(q, k, w, w, rope, None, 1e-6, *u, out=out)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("B,Hq,Hk,Lq,Lk,d", [(2, 4, 2, 500, 500, 64), (1, 8, 2, 3, 900, 128), (1, 30, 6, 4000, 4000, 64)])
def test_the_output_may_be_the_queries(B, Hq, Hk, Lq, Lk, d):
    Q, K, V = _rand(B, Hq, Lq, d, seed=1), _rand(B, Hk, Lk, d, seed=2), _rand(B, Hk, Lk, d, seed=3)
    args = (200, 0, 40, True)
    want = moc.window_attention_fwd(Q, K, V, *args)
    got = moc.window_attention_fwd(Q, K, V, *args, O=Q)
    assert got[0] is Q and torch.equal(Q, want[0]) and torch.equal(got[1], want[1])


def test_overlapping_outputs_are_refused():
    Q, K, V, g = (_rand(1, 2, 200, 64, seed=i) for i in range(4))
    with pytest.raises(moc.MocError):
        moc.window_attention_fwd(Q, K, V, O=K)
    O, lse = moc.window_attention_fwd(Q, K, V)
    want = moc.window_attention_bwd(Q, K, V, O, lse, g)
    for kw in (dict(dQ=Q), dict(dQ=g), dict(dK=K), dict(dV=g), dict(dK=O, dV=O)):
        with pytest.raises(moc.MocError):
            moc.window_attention_bwd(Q, K, V, O, lse, g, **kw)
    got = moc.window_attention_bwd(Q, K, V, O, lse, g, dQ=O)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
