"""fp64 definitions of the row operators (rotary positions, per-head RMS norm with
the rotation, and their gradients) for [B, H, L, d] torch tensors on any device.

Written from the formulas, independent of the package: a pair (a, b) turns by the
angle position * frequency as the complex number a + ib; the norm divides by the
root mean square over d.
"""
from __future__ import annotations

import math

import torch


def frequencies(axes, theta=10000.0, scaling="none", factor=1.0, original_length=0.0, alpha=1.0, beta=32.0,
                attention_factor=None):
    """([radians per position], [axis], factor on the rotated part)."""
    freq, axis = [], []
    for a, n in enumerate(axes):
        for j in range(n // 2):
            base = theta * factor ** (n / (n - 2)) if scaling == "ntk" and n > 2 else theta
            w = base ** (-2.0 * j / n)
            if scaling == "linear":
                w = w / factor
            if scaling == "yarn":
                t = original_length * w / (2 * math.pi)
                if t <= alpha:
                    w = w / factor
                elif t < beta:
                    blend = (t - alpha) / (beta - alpha)
                    w = blend * w + (1 - blend) * w / factor
            freq.append(w)
            axis.append(a)
    f = 1.0
    if scaling == "yarn":
        f = attention_factor if attention_factor is not None else 1.0 + 0.1 * math.log(factor)
    return freq, axis, f


def angles(freq, axis, pos, B, L):
    """fp64 [B, L, pairs]; pos int tensor [B, axes, L], or None for 0 .. L-1."""
    if pos is None:
        pos = torch.arange(L).expand(B, 1, L)
    return torch.stack([pos[:, a].double() * w for w, a in zip(freq, axis)], -1)


def rotate(x, ang, factor, interleaved, sign=1):
    """R x (sign 1) or R^T x (sign -1) in fp64; ang [B, L, pairs]."""
    x = x.double()
    n = ang.shape[-1]
    i = torch.arange(n, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.full_like(ang, factor), sign * ang)[:, None]
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def norm_rope(x, w, eps, ang, factor, interleaved):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    return rotate(y, ang, factor, interleaved) if ang is not None else y


def norm_rope_bwd(x, w, eps, ang, factor, interleaved, dy):
    """(dx, dw, sum |g xhat| per weight, row-wise size of dx's terms)."""
    x = x.double()
    g = rotate(dy, ang, factor, interleaved, -1) if ang is not None else dy.double()
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    gw = g * w.double() if w is not None else g
    m = (gw * xh).mean(-1, keepdim=True)
    dx = r * (gw - xh * m)
    size = r * (gw.abs().amax(-1, keepdim=True) + xh.abs().amax(-1, keepdim=True) *
                (gw * xh).abs().mean(-1, keepdim=True))
    return dx, (g * xh).sum((0, 1, 2)), (g * xh).abs().sum((0, 1, 2)), size
