"""Inputs that carry a forward-mode tangent go through the autograd functions, which have
no forward-mode rule: torch refuses, instead of a result whose tangent reads as zero. The
device call is replaced, so no GPU is needed."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import chunk_routed_sparse_b200 as moc
from chunk_routed_sparse_b200 import rows


@pytest.fixture(autouse=True)
def _stub(monkeypatch):
    monkeypatch.setattr(rows, "rotary_fwd", lambda rope, X, pos=None, out=None: X.clone())
    monkeypatch.setattr(rows, "qkv_norm_rope_fwd", lambda qkv, *a: (qkv.clone(), qkv.clone(), qkv.clone()))
    monkeypatch.setattr(rows, "qk_norm_rope_fwd", lambda Q, K, *a: (Q.clone(), K.clone(), None))


def _calls(x, w):
    rope = moc.Rope(64)
    yield lambda: rows.rotary(rope, x)
    yield lambda: rows.qkv_norm_rope(x, 1, 1, w, w, rope)
    yield lambda: rows.qk_norm_rope(x, x, w, w, rope)


@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused_and_never_dropped(grad):
    x, w, one = torch.randn(1, 2, 3, 64), torch.ones(64), torch.ones(1, 2, 3, 64)
    with fw.dual_level(), torch.set_grad_enabled(grad):
        for call in _calls(fw.make_dual(x, one), w):
            with pytest.raises(NotImplementedError):
                call()
        for call in list(_calls(x, fw.make_dual(w, torch.ones(64))))[1:]:
            with pytest.raises(NotImplementedError):
                call()


def test_plain_inputs_take_the_raw_calls():
    x, w = torch.randn(1, 2, 3, 64), torch.ones(64)
    with fw.dual_level():
        for call in _calls(x, w):  # a level without tangents
            out = call()
            assert not (out if isinstance(out, torch.Tensor) else out[0]).requires_grad
    for call in _calls(x, w):
        out = call()
        assert (out if isinstance(out, torch.Tensor) else out[0]).grad_fn is None
    for call in _calls(x, w.clone().requires_grad_()):
        out = call()
        assert (out if isinstance(out, torch.Tensor) else out[0]).requires_grad == (not isinstance(out, torch.Tensor))
