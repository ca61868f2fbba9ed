"""fp64 definition of the sliding-window attention and its gradient, dense per
head, for [B, H, L, d] torch tensors on any device. Independent of the package."""
from __future__ import annotations

import math

import torch


def visible(n, m, left, right, sinks, causal, device="cpu"):
    """bool [m, n]: which of n keys the m last tokens see."""
    p = (torch.arange(m, device=device) + n - m)[:, None]
    u = torch.arange(n, device=device)[None]
    near = torch.ones(m, n, dtype=torch.bool, device=device)
    if left >= 0:
        near &= u >= p - left
    if right >= 0:
        near &= u <= p + right
    see = near | (u < sinks)
    return see & (u <= p) if causal else see


def attention(Q, K, V, left, right, sinks, causal, q_len=None, kv_len=None, scale=None, dO=None):
    """dict of O, lse (rows past q_len: 0, -inf); with dO also dQ, dK, dV and, per
    element, sizes of the terms behind them (sQ, sK, sV) for error bounds."""
    B, Hq, Lq, d = Q.shape
    Hk, Lk = K.shape[1], K.shape[2]
    G, dev = Hq // Hk, Q.device
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    f = dict(dtype=torch.float64, device=dev)
    out = dict(O=torch.zeros(B, Hq, Lq, d, **f), lse=torch.full((B, Hq, Lq), -math.inf, **f),
               sO=torch.zeros(B, Hq, Lq, d, **f))
    for name, ref in (("dQ", Q), ("dK", K), ("dV", V), ("sQ", Q), ("sK", K), ("sV", V)):
        out[name] = torch.zeros(*ref.shape, **f)
    for b in range(B):
        n = Lk if kv_len is None else min(max(int(kv_len[b]), 0), Lk)
        m = Lq if q_len is None else min(max(int(q_len[b]), 0), Lq)
        if m == 0:
            continue
        see = visible(n, m, left, right, sinks, causal, dev)
        for h in range(Hq):
            q, k, v = Q[b, h, :m].double(), K[b, h // G, :n].double(), V[b, h // G, :n].double()
            s = (q @ k.T * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, 1) if n else torch.full((m,), -math.inf, **f)
            p = torch.where(see, torch.exp(s - lse[:, None]), torch.zeros((), **f))
            o = p @ v
            out["O"][b, h, :m], out["lse"][b, h, :m] = o, lse
            out["sO"][b, h, :m] = (p @ v.abs())
            if dO is None:
                continue
            g = dO[b, h, :m].double()
            dp = g @ v.T - (g * o).sum(1, keepdim=True)
            ds = p * dp * scale
            out["dQ"][b, h, :m] = ds @ k
            out["dK"][b, h // G, :n] += ds.T @ q
            out["dV"][b, h // G, :n] += p.T @ g
            # |p| (|g| . |v| + |D|): what dp is a difference of
            t = p * scale * (g.abs() @ v.abs().T + (g * o).sum(1, keepdim=True).abs())
            out["sQ"][b, h, :m] = t @ k.abs()
            out["sK"][b, h // G, :n] += t.T @ q.abs()
            out["sV"][b, h // G, :n] += p.T @ g.abs()
    return out
