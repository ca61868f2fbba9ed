"""Row operators in front of the attention: rotary positions, and per-head RMS
norms of queries and keys with the rotation and the re-layout to head-major in
the same pass (``moc_rotary``, ``moc_qk_norm_rope`` and its gradient).

    rope = Rope(128, axes=(44, 42, 42))                 # time, row and column of a clip
    Q, K, V = qkv_norm_rope(qkv, Hq, Hk, wq, wk, rope, pos)   # qkv [B, L, Hq + 2 Hk, d]
    O = moc_attention(layout, Q, K, V, k)

Tensors are [B, H, L, d] views in bf16, fp16 or fp32 whose last dim is dense, d 64
or 128; the other dims may have any strides (token-major projections, slots of a
cache). ``pos`` is int32 on the same device: [L] or [axes, L] for the whole batch,
or [B, axes, L]; None counts 0 .. L-1 for a one-axis rotation. Calls run on the
current stream of the tensors' device. The _fwd and _bwd calls can be captured into graphs
freely; for a captured autograd backward torch's own rule holds, that no eager graph over
the same leaves is alive. Gradients are reverse-mode: an input with a forward-mode tangent
is refused.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import MocError, _check, lib

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class _RopeDesc(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int32), ("axis_dim", ctypes.c_void_p), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double), ("alpha", ctypes.c_double), ("beta", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class Rope:
    """A rotation of the first ``dim`` dims of every head (moc_build_rope).

    axes: dims of each position axis, summing to ``dim`` (default: one axis).
    interleaved: pairs (2i, 2i + 1), else (i, i + dim / 2). scaling: "none",
    "linear", "ntk" or "yarn" by ``factor`` (yarn: trained at
    ``original_length``, blended between ``alpha`` and ``beta`` turns over it,
    the rotated part times ``attention_factor``, None for 0.1 ln(factor) + 1).
    Holds host memory only: one plan serves every device."""

    def __init__(self, dim: int, axes: Optional[Sequence[int]] = None, theta: float = 10000.0,
                 interleaved: bool = True, scaling: str = "none", factor: float = 1.0,
                 original_length: float = 0.0, alpha: float = 1.0, beta: float = 32.0,
                 attention_factor: Optional[float] = None):
        axes = (int(dim),) if axes is None else tuple(int(a) for a in axes)
        if any(abs(a) >= 1 << 31 for a in axes) or sum(axes) != dim:
            raise ValueError(f"axes {axes} do not sum to {dim} rotated dims")
        if scaling not in SCALING:
            raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(SCALING)}")
        if attention_factor is not None and not attention_factor > 0:
            raise ValueError("attention_factor is positive, or None for the default")
        arr = (ctypes.c_int32 * len(axes))(*axes)
        desc = _RopeDesc(len(axes), ctypes.cast(arr, ctypes.c_void_p), 1 if interleaved else 0, SCALING[scaling],
                         float(theta), float(factor), float(original_length), float(alpha), float(beta),
                         float(attention_factor or 0.0))
        h = ctypes.c_void_p()
        _check(lib().moc_build_rope(ctypes.byref(desc), ctypes.byref(h)), "moc_build_rope")
        self._h = h
        self._args = (dim, axes, theta, interleaved, scaling, factor, original_length, alpha, beta, attention_factor)
        self.dim, self.axes, self.interleaved = int(dim), axes, bool(interleaved)

    def __reduce__(self):  # copies and unpickled plans (a copied or saved model's) own a plan of their own
        return Rope, self._args

    @property
    def handle(self):
        return self._h

    def table(self) -> Tuple[list, list, float]:
        """(radians per position of every pair, its axis, factor on the rotated part)."""
        n, f = ctypes.c_int64(), ctypes.c_double()
        freq, axis = (ctypes.c_double * 64)(), (ctypes.c_int32 * 64)()
        _check(lib().moc_rope_table(self._h, freq, axis, 64, ctypes.byref(n), ctypes.byref(f)), "moc_rope_table")
        return list(freq)[:n.value], list(axis)[:n.value], f.value

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().moc_rope_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# (absent in a build of torch without CUDA; only CUDA tensors get here)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle, no Stream object
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(where: str, device: torch.device, *args):
    """Call lib().<where>(*args, stream) on the device and its current stream."""
    i, fn = device.index, getattr(lib(), where)
    if i == _current_device():
        status = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, _raw_stream(i))
    if status != 0:
        raise MocError(status, where)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(name: str, x: torch.Tensor, like: Optional[torch.Tensor] = None, shape=None):
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or not x.is_cuda or x.dtype not in _DTYPE:
        raise ValueError(f"{name}: expected a bf16, fp16 or fp32 CUDA tensor [B, H, L, d]")
    if x.shape[3] not in (64, 128):
        raise ValueError(f"{name}: d = {x.shape[3]}, expected 64 or 128")
    if x.stride(3) != 1 and x.numel():
        raise ValueError(f"{name}: the last dim has stride {x.stride(3)}, expected 1")
    if like is not None and (x.dtype is not like.dtype or x.device != like.device):
        raise ValueError(f"{name}: {x.dtype} on {x.device}, expected {like.dtype} on {like.device}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")


def _positions(rope: Optional[Rope], pos: Optional[torch.Tensor], B: int, L: int, d: int, device):
    """(tensor or None, batch stride, axis stride) of the positions."""
    if rope is None:
        if pos is not None:
            raise ValueError("positions without a rotation")
        return None, 0, 0
    if not isinstance(rope, Rope) or not rope._h.value:
        raise ValueError("rope: expected an open Rope")
    if rope.dim > d:
        raise ValueError(f"the rotation covers {rope.dim} dims, heads have {d}")
    n = len(rope.axes)
    if pos is None:
        if n != 1:
            raise ValueError(f"a rotation over {n} axes needs positions")
        return None, 0, 0
    if pos.dtype is not torch.int32 or pos.device != device:
        raise ValueError(f"pos: {pos.dtype} on {pos.device}, expected int32 on {device}")
    shape = pos.shape
    ok = shape == (B, n, L) or shape == (n, L) or shape == (L,) and n == 1
    if not ok:
        raise ValueError(f"pos: shape {tuple(shape)}, expected [L], [axes, L] or [B, axes, L] for B = {B}, axes = {n}, L = {L}")
    if L > 1 and pos.stride(-1) != 1:
        raise ValueError("pos: the last dim is not dense")
    dims = len(shape)
    return pos, pos.stride(0) if dims == 3 else 0, pos.stride(-2) if dims > 1 else 0


_stride_arrays: dict = {}  # strides -> their host array and its address (read during a call only)


def _stride_array(*vals):
    hit = _stride_arrays.get(vals)
    if hit is None:
        if len(_stride_arrays) >= 512:
            _stride_arrays.clear()
        buf = (ctypes.c_int64 * len(vals))(*vals)
        hit = _stride_arrays[vals] = (buf, ctypes.addressof(buf))
    return hit


def _strides(*tensors):
    """Batch, head and token strides of every tensor in one host array, and its address."""
    vals = ()
    for t in tensors:
        vals += t.stride()[:3] if t is not None else (0, 0, 0)
    return _stride_array(*vals)


def _rotary(rope, X, pos, transpose, out):
    _rows("X", X)
    B, H, L, d = X.shape
    if rope is None:
        raise ValueError("rope: expected a Rope")
    p, pb, pa = _positions(rope, pos, B, L, d, X.device)
    if out is None:
        out = torch.empty_like(X, memory_format=torch.contiguous_format)
    else:
        _rows("out", out, X, X.shape)
    buf, at = _strides(X, out)
    _call("moc_rotary", X.device, rope.handle, _DTYPE[X.dtype], B, H, L, d, X.data_ptr(), at, _at(p), pb, pa, transpose,
          out.data_ptr(), at + 24)
    return out


def rotary_fwd(rope: Rope, X: torch.Tensor, pos: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = R X (moc_rotary), head-major contiguous unless ``out`` says otherwise;
    ``out`` may be X itself."""
    return _rotary(rope, X, pos, 0, out)


def rotary_bwd(rope: Rope, dY: torch.Tensor, pos: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX = R^T dY, the gradient of rotary_fwd (moc_rotary, transposed)."""
    return _rotary(rope, dY, pos, 1, out)


def _tangent(*tensors) -> bool:
    """Whether any of them carries a forward-mode tangent. There is no rule for it here: it
    has to meet the autograd function to be refused. (Called inside a dual level alone:
    looking into a tensor costs 0.3 us.)"""
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _dense(g: torch.Tensor) -> torch.Tensor:
    return g if g.stride(-1) == 1 else g.contiguous()


class Rotary(torch.autograd.Function):
    """rotary_fwd with its gradient. apply(rope, X, pos) -> Y."""

    @staticmethod
    def forward(ctx, rope, X, pos):
        ctx.rope = rope
        ctx.save_for_backward(pos)
        ctx.like = (X.shape, X.stride())
        return rotary_fwd(rope, X, pos)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        shape, stride = ctx.like
        # the gradient in the input's own order (a broadcast input: head-major, autograd adds it up)
        dense = all(n <= 1 or s > 0 for n, s in zip(shape, stride))
        out = torch.empty_strided(shape, stride, dtype=dY.dtype, device=dY.device) if dense and _plain(shape, stride) \
            else None
        return None, rotary_bwd(ctx.rope, _dense(dY), ctx.saved_tensors[0], out), None


def _plain(shape, stride) -> bool:
    """Whether (shape, stride) tiles its storage without holes or overlap."""
    want = 1
    for s, n in sorted((s, n) for n, s in zip(shape, stride) if n > 1):
        if s != want:
            return False
        want *= n
    return True


def rotary(rope: Rope, X: torch.Tensor, pos: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable rotary positions: Y = R X, head-major contiguous."""
    if X.requires_grad and torch.is_grad_enabled() or forward_ad._current_level >= 0 and _tangent(X):
        return Rotary.apply(rope, X, pos)
    return rotary_fwd(rope, X, pos)


# ---- norm + rotation ---------------------------------------------------------
def _weights(wq, wk, X, d):
    """The weights' common type code."""
    code = 2
    if wq is not None:
        code = _weight("wq", wq, X, d)
    if wk is not None:
        code = _weight("wk", wk, X, d)
        if wq is not None and wq.dtype is not wk.dtype:
            raise ValueError("wq and wk have different types")
    return code


def _weight(name, w, X, d):
    if w.shape != (d,) or not w.is_contiguous() or w.device != X.device or \
            w.dtype is not torch.float32 and w.dtype is not X.dtype:
        raise ValueError(f"{name}: expected a contiguous [{d}] tensor in fp32 or {X.dtype} on {X.device}")
    return _DTYPE[w.dtype]


def qk_norm_rope_fwd(Q, K, V=None, wq=None, wk=None, rope: Optional[Rope] = None,
                     pos: Optional[torch.Tensor] = None, eps: float = 1e-6, out=None):
    """Queries and keys normalised per head and rotated, values re-laid
    (moc_qk_norm_rope). Q: [B, Hq, L, d], K and V: [B, Hk, L, d] views. Returns
    (Qo, Ko, Vo) - Vo None without V -, head-major contiguous, or written to the
    views of ``out`` (slots of a cache, or the inputs themselves)."""
    _rows("Q", Q)
    B, Hq, L, d = Q.shape
    Hk = K.shape[1] if isinstance(K, torch.Tensor) and K.dim() == 4 else 0
    _rows("K", K, Q, (B, Hk, L, d))
    if V is not None:
        _rows("V", V, Q, (B, Hk, L, d))
    code = _weights(wq, wk, Q, d)
    p, pb, pa = _positions(rope, pos, B, L, d, Q.device)
    if out is None:
        Qo = torch.empty_like(Q, memory_format=torch.contiguous_format)
        Ko = torch.empty_like(K, memory_format=torch.contiguous_format)
        Vo = torch.empty_like(V, memory_format=torch.contiguous_format) if V is not None else None
    else:
        Qo, Ko, Vo = out
        _rows("out Q", Qo, Q, Q.shape)
        _rows("out K", Ko, Q, K.shape)
        if (V is None) != (Vo is None):
            raise ValueError("V and its output come together")
        if V is not None:
            _rows("out V", Vo, Q, V.shape)
    buf, at = _strides(Q, K, V, Qo, Ko, Vo)
    _call("moc_qk_norm_rope", Q.device, rope.handle if rope is not None else None, _DTYPE[Q.dtype], B, Hq, Hk, L, d,
          Q.data_ptr(), at, K.data_ptr(), at + 24, _at(V), at + 48, _at(wq), _at(wk), code, eps, _at(p), pb, pa,
          Qo.data_ptr(), at + 72, Ko.data_ptr(), at + 96, _at(Vo), at + 120)
    return Qo, Ko, Vo


def qk_norm_rope_bwd(Q, K, wq, wk, rope, pos, eps, dQo, dKo, dVo=None, out=None, want_dw: bool = True):
    """Gradient of qk_norm_rope_fwd (moc_qk_norm_rope_bwd): returns (dQ, dK, dV,
    dwq, dwk); dQ, dK, dV head-major contiguous or in the views of ``out``; a
    weight that is None gets None."""
    _rows("Q", Q)
    B, Hq, L, d = Q.shape
    Hk = K.shape[1] if isinstance(K, torch.Tensor) and K.dim() == 4 else 0
    _rows("K", K, Q, (B, Hk, L, d))
    _rows("dQo", dQo, Q, Q.shape)
    _rows("dKo", dKo, Q, K.shape)
    if dVo is not None:
        _rows("dVo", dVo, Q, K.shape)
    code = _weights(wq, wk, Q, d)
    p, pb, pa = _positions(rope, pos, B, L, d, Q.device)
    if out is None:
        dQ = torch.empty_like(Q, memory_format=torch.contiguous_format)
        dK = torch.empty_like(K, memory_format=torch.contiguous_format)
        dV = torch.empty_like(K, memory_format=torch.contiguous_format) if dVo is not None else None
    else:
        dQ, dK, dV = out
        _rows("out dQ", dQ, Q, Q.shape)
        _rows("out dK", dK, Q, K.shape)
        if (dVo is None) != (dV is None):
            raise ValueError("dVo and its output come together")
        if dV is not None:
            _rows("out dV", dV, Q, K.shape)
    dwq = torch.empty_like(wq) if want_dw and wq is not None else None
    dwk = torch.empty_like(wk) if want_dw and wk is not None else None
    buf, at = _strides(Q, K, dQo, dKo, dVo, dQ, dK, dV)
    ws = _bwd_workspace(Q, B, Hq, Hk, L, d) if dwq is not None or dwk is not None else None
    _call("moc_qk_norm_rope_bwd", Q.device, rope.handle if rope is not None else None, _DTYPE[Q.dtype], B, Hq, Hk, L, d,
          Q.data_ptr(), at, K.data_ptr(), at + 24, _at(wq), _at(wk), code, eps, _at(p), pb, pa, dQo.data_ptr(), at + 48,
          dKo.data_ptr(), at + 72, _at(dVo), at + 96, dQ.data_ptr(), at + 120, dK.data_ptr(), at + 144, _at(dV),
          at + 168, _at(dwq), _at(dwk), _at(ws), ws.numel() if ws is not None else 0)
    return dQ, dK, dV, dwq, dwk


@functools.lru_cache(maxsize=256)
def _workspace_bytes(where: str, device: torch.device, *problem) -> int:
    """lib().<where>(*problem) on the device (a size depends on the problem and the device alone)."""
    if device.index == _current_device():
        n = int(getattr(lib(), where)(*problem))
    else:
        with torch.cuda.device(device):
            n = int(getattr(lib(), where)(*problem))
    if n == 0:
        raise ValueError("invalid problem for the workspace size query")
    return n


def _bwd_workspace(like, B, Hq, Hk, L, d):
    n = _workspace_bytes("moc_qk_norm_rope_bwd_workspace_bytes", like.device, B, Hq, Hk, L, d)
    return like.new_empty(n, dtype=torch.uint8)


def _packed(qkv, Hq: int, Hk: int):
    """(B, L, d) of a packed [B, L, Hq + 2 Hk, d] projection."""
    _rows("qkv", qkv)
    B, L, heads, d = qkv.shape
    if Hq < 1 or Hk < 1 or heads != Hq + 2 * Hk:
        raise ValueError(f"qkv: expected [B, L, Hq + 2 Hk, d] with Hq = {Hq}, Hk = {Hk}")
    return B, L, d


def qkv_norm_rope_fwd(qkv, Hq: int, Hk: int, wq=None, wk=None, rope=None, pos=None, eps: float = 1e-6):
    """qk_norm_rope_fwd on the packed projection [B, L, Hq + 2 Hk, d]."""
    B, L, d = _packed(qkv, Hq, Hk)
    code = _weights(wq, wk, qkv, d)
    p, pb, pa = _positions(rope, pos, B, L, d, qkv.device)
    dt, dev = qkv.dtype, qkv.device
    Q, K, V = qkv.new_empty((B, Hq, L, d)), qkv.new_empty((B, Hk, L, d)), qkv.new_empty((B, Hk, L, d))
    if not qkv.numel():
        return Q, K, V
    sb, sl, sh, _ = qkv.stride()
    buf, at = _stride_array(sb, sh, sl, sb, sh, sl, sb, sh, sl, Hq * L * d, L * d, d, Hk * L * d, L * d, d, Hk * L * d,
                            L * d, d)
    x, step = qkv.data_ptr(), sh * qkv.element_size()
    _call("moc_qk_norm_rope", dev, rope.handle if rope is not None else None, _DTYPE[dt], B, Hq, Hk, L, d, x, at,
          x + Hq * step, at + 24, x + (Hq + Hk) * step, at + 48, _at(wq), _at(wk), code, eps, _at(p), pb, pa,
          Q.data_ptr(), at + 72, K.data_ptr(), at + 96, V.data_ptr(), at + 120)
    return Q, K, V


def qkv_norm_rope_bwd(qkv, Hq: int, Hk: int, wq, wk, rope, pos, eps, dQ, dK, dV, want_dw: bool = True):
    """Gradient of qkv_norm_rope_fwd: (dqkv packed and contiguous, dwq, dwk)."""
    B, L, d = _packed(qkv, Hq, Hk)
    _rows("dQ", dQ, qkv, (B, Hq, L, d))
    _rows("dK", dK, qkv, (B, Hk, L, d))
    _rows("dV", dV, qkv, (B, Hk, L, d))
    code = _weights(wq, wk, qkv, d)
    p, pb, pa = _positions(rope, pos, B, L, d, qkv.device)
    dev = qkv.device
    dqkv = torch.empty_like(qkv, memory_format=torch.contiguous_format)
    dwq = torch.empty_like(wq) if want_dw and wq is not None else None
    dwk = torch.empty_like(wk) if want_dw and wk is not None else None
    ws = _bwd_workspace(qkv, B, Hq, Hk, L, d) if dwq is not None or dwk is not None else None
    sb, sl, sh, _ = qkv.stride()
    heads = Hq + 2 * Hk
    ob, ol = L * heads * d, heads * d
    buf, at = _stride_array(sb, sh, sl, sb, sh, sl, *dQ.stride()[:3], *dK.stride()[:3], *dV.stride()[:3], ob, d, ol, ob,
                            d, ol, ob, d, ol)
    x, y, eb = qkv.data_ptr(), dqkv.data_ptr(), qkv.element_size()
    if not qkv.numel():  # no rows: addresses mean nothing, the weights' gradients are zero
        return dqkv, *(None if w is None else w.zero_() for w in (dwq, dwk))
    _call("moc_qk_norm_rope_bwd", dev, rope.handle if rope is not None else None, _DTYPE[qkv.dtype], B, Hq, Hk, L, d,
          x, at, x + Hq * sh * eb, at + 24, _at(wq), _at(wk), code, eps, _at(p), pb, pa, dQ.data_ptr(), at + 48,
          dK.data_ptr(), at + 72, dV.data_ptr(), at + 96, y, at + 120, y + Hq * d * eb, at + 144,
          y + (Hq + Hk) * d * eb, at + 168, _at(dwq), _at(dwk), _at(ws), ws.numel() if ws is not None else 0)
    return dqkv, dwq, dwk


class QKVNormRope(torch.autograd.Function):
    """apply(qkv, wq, wk, Hq, Hk, rope, pos, eps) -> Q, K, V with gradients for the
    projection and the weights."""

    @staticmethod
    def forward(ctx, qkv, wq, wk, Hq, Hk, rope, pos, eps):
        ctx.args = (Hq, Hk, rope, eps)
        ctx.save_for_backward(qkv, wq, wk, pos)
        return qkv_norm_rope_fwd(qkv, Hq, Hk, wq, wk, rope, pos, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dQ, dK, dV):
        qkv, wq, wk, pos = ctx.saved_tensors
        Hq, Hk, rope, eps = ctx.args
        want = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dqkv, dwq, dwk = qkv_norm_rope_bwd(qkv, Hq, Hk, wq, wk, rope, pos, eps, _dense(dQ), _dense(dK), _dense(dV), want)
        return dqkv, dwq, dwk, None, None, None, None, None


def qkv_norm_rope(qkv: torch.Tensor, Hq: int, Hk: int, wq: Optional[torch.Tensor] = None,
                  wk: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                  pos: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Differentiable: the packed projection [B, L, Hq + 2 Hk, d] to head-major Q
    (normalised, rotated), K (the same) and V in one pass."""
    if (qkv.requires_grad or wq is not None and wq.requires_grad or wk is not None and wk.requires_grad) and \
            torch.is_grad_enabled() or forward_ad._current_level >= 0 and _tangent(qkv, wq, wk):
        return QKVNormRope.apply(qkv, wq, wk, Hq, Hk, rope, pos, eps)
    return qkv_norm_rope_fwd(qkv, Hq, Hk, wq, wk, rope, pos, eps)


class QKNormRope(torch.autograd.Function):
    """apply(Q, K, wq, wk, rope, pos, eps) -> Qo, Ko with gradients for all four tensors."""

    @staticmethod
    def forward(ctx, Q, K, wq, wk, rope, pos, eps):
        ctx.args = (rope, eps)
        ctx.save_for_backward(Q, K, wq, wk, pos)
        return qk_norm_rope_fwd(Q, K, None, wq, wk, rope, pos, eps)[:2]

    @staticmethod
    @once_differentiable
    def backward(ctx, dQo, dKo):
        Q, K, wq, wk, pos = ctx.saved_tensors
        rope, eps = ctx.args
        want = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        dQ, dK, _, dwq, dwk = qk_norm_rope_bwd(Q, K, wq, wk, rope, pos, eps, _dense(dQo), _dense(dKo), want_dw=want)
        return dQ, dK, dwq, dwk, None, None, None


def qk_norm_rope(Q: torch.Tensor, K: torch.Tensor, wq: Optional[torch.Tensor] = None,
                 wk: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                 pos: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Differentiable norm and rotation of separate Q and K views: (Qo, Ko)."""
    if any(t is not None and t.requires_grad for t in (Q, K, wq, wk)) and torch.is_grad_enabled() or \
            forward_ad._current_level >= 0 and _tangent(Q, K, wq, wk):
        return QKNormRope.apply(Q, K, wq, wk, rope, pos, eps)
    return qk_norm_rope_fwd(Q, K, None, wq, wk, rope, pos, eps)[:2]
