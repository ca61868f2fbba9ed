"""Attention with a sliding window and always-visible first keys
(``moc_window_attention`` and its gradient).

    O = window_attention(Q, K, V, left=1560, right=1560, sinks=512)        # captions and a frame either side
    O = window_attention(Q, K, V, left=4095, sinks=64, causal=True)        # a causal window
    O, lse = window_attention_fwd(q, cache_k, cache_v, 4095, 0, 64, True, kv_len=lens)   # one new token a stream

Q, O: contiguous bf16 [B, Hq, Lq, d]; K, V: [B, Hk, Lk, d], Hk dividing Hq, d 64 or
128. Row t of batch entry b is at position p = t + kv_len[b] - q_len[b] and sees key
u < kv_len[b] iff (not causal or u <= p) and (u < sinks or p - left <= u <= p + right);
a negative left or right is no limit (causal: right is not read). q_len, kv_len: int32 [B] on
the device, None for Lq, Lk. Calls run on the current stream of the tensors' device. The
_fwd and _bwd calls can be captured into graphs freely; for a captured autograd backward
torch's own rule holds, that no eager graph over the same leaves is alive.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _check, lib
from .rows import _at, _call, _workspace_bytes


_FAR = 1 << 40
_FILL_REST, _JOINED = 1, 2  # MOC_WINDOW_FILL_REST, MOC_WINDOW_JOINED


def _tensor(name, x, shape, device, dtype=torch.bfloat16):
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.shape != shape or x.device != device or \
            not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on {device}")


def _problem(Q, K, V, q_len, kv_len):
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4 or not Q.is_cuda:
        raise ValueError("Q: expected a bf16 CUDA tensor [B, Hq, Lq, d]")
    B, Hq, Lq, d = Q.shape
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("K: expected a bf16 CUDA tensor [B, Hk, Lk, d]")
    _, Hk, Lk, _ = K.shape
    if d not in (64, 128):
        raise ValueError(f"d = {d}, expected 64 or 128")
    if (Hk == 0) != (Hq == 0) or (Hk and Hq % Hk):
        raise ValueError(f"{Hk} key heads do not divide {Hq} query heads")
    device, keys = Q.device, (B, Hk, Lk, d)
    _tensor("Q", Q, Q.shape, device)
    _tensor("K", K, keys, device)
    _tensor("V", V, keys, device)
    if q_len is not None:
        _tensor("q_len", q_len, (B,), device, torch.int32)
    if kv_len is not None:
        _tensor("kv_len", kv_len, (B,), device, torch.int32)
    return B, Hq, Hk, Lq, Lk, d


def _limits(left, right, sinks):
    """The window's sizes in 64 bits: any negative limit is none, any huge one reaches every key."""
    if -1 <= left < _FAR and -1 <= right < _FAR and 0 <= sinks < _FAR:
        return int(left), int(right), int(sinks)
    return tuple(max(min(int(x), _FAR), -1) for x in (left, right, sinks))


def window_attention_fwd(Q, K, V, left: int = -1, right: int = -1, sinks: int = 0, causal: bool = False,
                         q_len: Optional[torch.Tensor] = None, kv_len: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, O: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None):
    """(O, lse) (moc_window_attention). Rows past q_len are left as they were in a
    given O or lse, and are 0 and -inf in new ones."""
    B, Hq, Hk, Lq, Lk, d = _problem(Q, K, V, q_len, kv_len)
    left, right, sinks = _limits(left, right, sinks)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    fill = O is None and lse is None
    if O is None:
        O = torch.empty_like(Q) if fill or q_len is None else torch.zeros_like(Q)
    else:
        _tensor("O", O, Q.shape, Q.device)
    if lse is None:
        lse = Q.new_empty((B, Hq, Lq), dtype=torch.float32)
        if not fill and q_len is not None:
            lse.fill_(-math.inf)
    else:
        _tensor("lse", lse, (B, Hq, Lq), Q.device, torch.float32)
    _call("moc_window_attention", Q.device, B, Hq, Hk, Lq, Lk, d, Q.data_ptr(), K.data_ptr(), V.data_ptr(), left, right,
          sinks, 1 if causal else 0, _at(q_len), _at(kv_len), fill, scale, O.data_ptr(), lse.data_ptr())
    return O, lse


def window_attention_bwd(Q, K, V, O, lse, dO, left: int = -1, right: int = -1, sinks: int = 0, causal: bool = False,
                         q_len: Optional[torch.Tensor] = None, kv_len: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, dQ: Optional[torch.Tensor] = None,
                         dK: Optional[torch.Tensor] = None, dV: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, joined: bool = False):
    """(dQ, dK, dV) for the upstream gradient dO (moc_window_attention_bwd). Rows past
    the lengths are left as they were in given tensors and are 0 in new ones.

    O and lse are window_attention_fwd's for the same arguments; with ``joined`` those of
    a softmax over more keys than this call's (O and lse joined over several key ranges,
    one call a range, whose dQ add up)."""
    B, Hq, Hk, Lq, Lk, d = _problem(Q, K, V, q_len, kv_len)
    left, right, sinks = _limits(left, right, sinks)
    _tensor("O", O, Q.shape, Q.device)
    _tensor("dO", dO, Q.shape, Q.device)
    _tensor("lse", lse, (B, Hq, Lq), Q.device, torch.float32)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    for name, x, ref in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, K)):
        if x is not None:
            _tensor(name, x, ref.shape, Q.device)
    fill = dQ is None and dK is None and dV is None
    dQ = (torch.empty_like(Q) if fill or q_len is None else torch.zeros_like(Q)) if dQ is None else dQ
    dK = (torch.empty_like(K) if fill or kv_len is None else torch.zeros_like(K)) if dK is None else dK
    dV = (torch.empty_like(K) if fill or kv_len is None else torch.zeros_like(K)) if dV is None else dV
    if ws is None:
        n = _workspace_bytes("moc_window_attention_bwd_workspace_bytes", Q.device, B, Hq, Hk, Lq, Lk, d, left, right,
                             sinks, 1 if causal else 0)
        ws = Q.new_empty(n, dtype=torch.uint8)
    elif ws.device != Q.device or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on {Q.device}")
    _call("moc_window_attention_bwd", Q.device, B, Hq, Hk, Lq, Lk, d, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
          O.data_ptr(), lse.data_ptr(), dO.data_ptr(), left, right, sinks, 1 if causal else 0, _at(q_len), _at(kv_len),
          (_FILL_REST if fill else 0) | (_JOINED if joined else 0), scale, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
          ws.data_ptr(), ws.numel() * ws.element_size())
    return dQ, dK, dV


class WindowAttention(torch.autograd.Function):
    """window_attention_fwd with its gradient for Q, K and V.
    apply(Q, K, V, left, right, sinks, causal, q_len, kv_len, scale) -> O."""

    @staticmethod
    def forward(ctx, Q, K, V, left, right, sinks, causal, q_len, kv_len, scale):
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
        O, lse = window_attention_fwd(Q, K, V, left, right, sinks, causal, q_len, kv_len, scale)
        ctx.args = (left, right, sinks, causal, scale)
        ctx.save_for_backward(Q, K, V, O, lse, q_len, kv_len)
        return O

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, lse, q_len, kv_len = ctx.saved_tensors
        left, right, sinks, causal, scale = ctx.args
        grads = window_attention_bwd(Q, K, V, O, lse, dO.contiguous().to(torch.bfloat16), left, right, sinks, causal,
                                     q_len, kv_len, scale)
        return (*grads, None, None, None, None, None, None, None)


def window_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, left: int = -1, right: int = -1, sinks: int = 0,
                     causal: bool = False, q_len: Optional[torch.Tensor] = None,
                     kv_len: Optional[torch.Tensor] = None, scale: Optional[float] = None) -> torch.Tensor:
    """Differentiable sliding-window attention: bf16 O [B, Hq, Lq, d] (0 past q_len)."""
    return WindowAttention.apply(Q, K, V, left, right, sinks, causal, q_len, kv_len, scale)


def check_window_error() -> int:
    """Read and clear the current device's error word of the window calls
    (synchronises); raises MocError on a recorded device error."""
    det = ctypes.c_int32()
    stream = torch.cuda.current_stream().cuda_stream
    _check(lib().moc_window_device_error(ctypes.byref(det), stream), "window device error word")
    return det.value
