"""Rotary plans and the row operators' argument checks, without a GPU."""
import copy
import ctypes
import math
import pickle

import pytest
import torch

import chunk_routed_sparse_b200 as moc
import oracle.rows as R
from chunk_routed_sparse_b200.rows import _RopeDesc


@pytest.mark.parametrize("axes,scaling,factor", [
    ((128,), "none", 1.0), ((64,), "linear", 4.0), ((44, 42, 42), "none", 1.0), ((24, 20), "ntk", 4.0),
    ((2, 4), "ntk", 3.0), ((128,), "yarn", 8.0), ((64,), "yarn", 1.0), ((2,), "linear", 1.0), ((32, 32, 32, 32), "none", 1.0)])
def test_plan_matches_the_definition(axes, scaling, factor):
    rope = moc.Rope(sum(axes), axes=axes, scaling=scaling, factor=factor, original_length=8192)
    freq, axis, f = rope.table()
    want, want_axis, want_f = R.frequencies(axes, scaling=scaling, factor=factor, original_length=8192.0)
    assert axis == want_axis and abs(f - want_f) <= 1e-15 * want_f
    for a, b in zip(freq, want):
        assert abs(a - b) <= 1e-14 * b  # a pow and a few products in fp64 each


def test_plan_with_its_own_factor_and_blend():
    kw = dict(scaling="yarn", factor=16.0, original_length=4096, alpha=2.0, beta=20.0, attention_factor=1.5)
    freq, _, f = moc.Rope(64, theta=500000.0, **kw).table()
    want, _, want_f = R.frequencies((64,), theta=500000.0, **kw)
    assert f == want_f == 1.5
    assert max(abs(a - b) / b for a, b in zip(freq, want)) <= 1e-14
    assert any(a != b for a, b in zip(freq, R.frequencies((64,), theta=500000.0)[0]))


@pytest.mark.parametrize("bad", [dict(dim=0, axes=()), dict(dim=3), dict(dim=130), dict(dim=64, axes=(32, 31, 1)),
                                 dict(dim=10, axes=(2,) * 5), dict(dim=64, theta=1.0), dict(dim=64, theta=math.nan),
                                 dict(dim=64, scaling="linear", factor=0.5), dict(dim=64, scaling="ntk", factor=math.inf),
                                 dict(dim=64, scaling="yarn", factor=2.0),
                                 dict(dim=64, scaling="yarn", factor=2.0, original_length=100, alpha=4, beta=4)])
def test_bad_plans_are_refused(bad):
    with pytest.raises(moc.MocError) as e:
        moc.Rope(**bad)
    assert e.value.status == 1


def test_copied_and_unpickled_plans_own_their_handles():
    rope = moc.Rope(44, axes=(24, 20), interleaved=False, scaling="yarn", factor=4.0, original_length=512)
    want = rope.table()
    others = [copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))]
    assert len({r.handle.value for r in (rope, *others)}) == 4
    rope.close()
    rope.close()
    for r in others:
        assert r.table() == want and (r.dim, r.axes, r.interleaved) == (44, (24, 20), False)


def test_bad_plan_arguments_of_the_binding():
    with pytest.raises(ValueError):
        moc.Rope(64, axes=(32, 16))
    with pytest.raises(ValueError):
        moc.Rope(64, scaling="cubic")
    with pytest.raises(ValueError):
        moc.Rope(64, scaling="yarn", factor=2, original_length=10, attention_factor=0.0)


def _call(**kw):
    """moc_rotary with never-dereferenced pointers: every case here is refused first."""
    a = dict(rope=moc.Rope(64).handle, dtype=0, B=1, H=2, L=8, d=64, X=4096, xs=(1024, 512, 64), pos=None, pb=0, pa=0,
             Y=8192, ys=(1024, 512, 64))
    keep = a["rope"]
    a.update(kw)
    s = (ctypes.c_int64 * 6)(*a["xs"], *a["ys"])
    at = ctypes.addressof(s)
    st = moc.lib().moc_rotary(a["rope"], a["dtype"], a["B"], a["H"], a["L"], a["d"], a["X"], at, a["pos"], a["pb"],
                              a["pa"], 0, a["Y"], at + 24, None)
    del keep
    return st


@pytest.mark.parametrize("kw,status", [
    (dict(rope=None), 1), (dict(dtype=3), 1), (dict(d=96), 1), (dict(B=-1), 1), (dict(L=-1), 1), (dict(X=None), 1),
    (dict(Y=None), 1), (dict(X=4097), 1), (dict(dtype=2, X=4098), 1), (dict(xs=(0, 0, -64)), 1),
    (dict(ys=(0, 0, 64)), 1), (dict(pos=4098), 1), (dict(H=70000), 6), (dict(B=1 << 20, L=1 << 20), 6),
    (dict(L=0), 0), (dict(B=0), 0), (dict(H=0), 0)])
def test_bad_calls_are_refused_before_any_launch(kw, status):
    rope = moc.Rope(64)
    kw = dict({"rope": rope.handle}, **kw)
    assert _call(**kw) == status


def test_rotation_wider_than_the_head_or_without_positions_is_refused():
    wide, three = moc.Rope(128), moc.Rope(64, axes=(32, 16, 16))
    assert _call(rope=wide.handle) == 1
    assert _call(rope=three.handle) == 1


def test_norm_calls_are_refused_before_any_launch():
    lib = moc.lib()
    s = (ctypes.c_int64 * 18)(*([1024, 512, 64] * 6))
    at = ctypes.addressof(s)

    def fwd(dtype=0, V=None, Vo=None, wq=None, wdt=2, eps=1e-6, Hq=2, Q=4096):
        return lib.moc_qk_norm_rope(None, dtype, 1, Hq, 2, 8, 64, Q, at, 4096, at, V, at, wq, None, wdt, eps, None, 0, 0,
                                    8192, at, 8192, at, Vo, at, None)

    assert fwd(eps=-1.0) == 1 and fwd(eps=math.nan) == 1 and fwd(eps=math.inf) == 1
    assert fwd(V=4096) == 1 and fwd(Vo=4096) == 1
    assert fwd(wq=4096, wdt=1) == 1 and fwd(wq=4097) == 1
    assert fwd(Hq=-1) == 1 and fwd(Q=None) == 1

    def bwd(ws=None, n=0, dwq=4096, dV=None):
        return lib.moc_qk_norm_rope_bwd(None, 0, 1, 2, 2, 8, 64, 4096, at, 4096, at, None, None, 2, 1e-6, None, 0, 0,
                                        4096, at, 4096, at, None, at, 8192, at, 8192, at, dV, at, dwq, None, ws, n, None)

    assert bwd() == 1 and bwd(ws=4097, n=1 << 30) == 1 and bwd(ws=4096, n=16) == 3 and bwd(dV=4096) == 1
    assert lib.moc_qk_norm_rope_bwd_workspace_bytes(1, 2, 2, 8, 96) == 0
    assert lib.moc_qk_norm_rope_bwd_workspace_bytes(1, 2, 2, 8, 64) > 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        moc.rotary(moc.Rope(64), x)
    with pytest.raises(ValueError):
        moc.qkv_norm_rope(torch.zeros(1, 8, 6, 64), 2, 2)
