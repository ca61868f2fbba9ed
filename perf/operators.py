"""Cases of the operators around the attention: rotary positions, per-head RMS
norms of queries and keys with the rotation in the same pass, and attention with
a sliding window and always-visible first tokens.

``run`` computes each operator in plain torch operations in fp32 (angles in
fp64), or with ``own`` set through the package's public calls. ``exact`` holds
the definitions in fp64.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------
def _rotary(name, B, H, L, d, axes, layout, dtype, scaling="none", factor=1.0, start=0, frame=0, width=1,
            token_major=True, train=False):
    return dict(name=name, op="rotary", B=B, H=H, L=L, d=d, axes=axes, layout=layout, dtype=dtype,
                scaling=scaling, factor=factor, start=start, frame=frame, width=width, token_major=token_major,
                train=train)


def _norm(name, B, Hq, Hk, L, d, axes, layout, dtype, wdtype="fp32", scaling="none", factor=1.0, start=0, frame=0,
          width=1, train=False):
    return dict(name=name, op="norm", B=B, Hq=Hq, Hk=Hk, L=L, d=d, axes=axes, layout=layout, dtype=dtype,
                wdtype=wdtype, scaling=scaling, factor=factor, start=start, frame=frame, width=width, train=train)


def _window(name, B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, ragged=False, train=False):
    return dict(name=name, op="window", B=B, Hq=Hq, Hk=Hk, Lq=Lq, Lk=Lk, d=d, left=left, right=right, sinks=sinks,
                causal=causal, ragged=ragged, train=train)


def listed():
    return [
        # one new token of each of eight streams, at far positions under a stretched context
        _rotary("rotary_token", 8, 24, 1, 128, "128", "half", "bf16", "yarn", 8.0, 180000),
        # the tiny scene in fp32, half of every head rotated, head-major input
        _rotary("rotary_tiny", 1, 2, 2112, 64, "32", "half", "fp32", "linear", 4.0, token_major=False),
        # the single-shot clip: time, row and column axes, and the gradient
        _rotary("rotary_single_train", 1, 12, 33272, 128, "44,42,42", "interleaved", "bf16", frame=1560, width=52,
                train=True),
        # the packed projection of one new token of each of eight streams
        _norm("norm_token", 8, 24, 24, 1, 128, "128", "half", "bf16", start=22563),
        # an odd-sized padded batch in fp16 with shared key heads and a partly rotated head, and its gradient
        _norm("norm_odd_train", 3, 12, 4, 1237, 64, "24,20", "half", "fp16", "fp16", "ntk", 4.0, frame=187, width=11,
              train=True),
        # one layer's training step of the single-shot clip
        _norm("norm_single_train", 1, 12, 12, 33272, 128, "44,42,42", "interleaved", "bf16", frame=1560, width=52,
              train=True),
        # the eight-shot scene's projection to head-major Q, K, V
        _norm("norm_eight", 1, 24, 24, 180512, 128, "44,42,42", "interleaved", "bf16", frame=1500, width=50),
        # one new token of each stream against its cache: captions and the last frames stay visible
        _window("window_token", 8, 24, 24, 1, 22563, 128, 8191, 0, 64, True, ragged=True),
        # the tiny scene: captions and one frame on either side
        _window("window_tiny", 1, 2, 2, 2112, 2112, 64, 256, 256, 64, False),
        # an odd padded batch with shared key heads, and its gradient
        _window("window_odd_train", 3, 12, 4, 2501, 2501, 64, 700, 0, 5, True, ragged=True, train=True),
        # the single-shot clip: all captions and one frame on either side of each token
        _window("window_single", 1, 12, 12, 33272, 33272, 128, 1560, 1560, 512, False),
        # one layer's training step, causal over the last four frames
        _window("window_single_train", 1, 12, 12, 33272, 33272, 128, 6239, 0, 512, True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _place(rng, d):
    """Axes, pair layout, stretch and grid of a drawn rotation."""
    axes = rng.choice({64: ["64", "32", "24,20,20", "24,20", "20"], 128: ["128", "64", "44,42,42", "32,48,48", "96"]}[d])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    width = _log(rng, 3, 90)
    return dict(axes=axes, layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                factor=1.0 if scaling == "none" else round(rng.uniform(1.5, 16.0), 2),
                start=rng.choice([0, _log(rng, 1, 1000000)]), frame=width * _log(rng, 2, 60), width=width)


def draw(rng):
    op = rng.choice(["rotary", "norm", "window"])
    d = rng.choice([64, 128])
    if op in ("rotary", "norm"):
        B = rng.choice([1, 1, 2, 3, 8])
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 24])
        H = Hk * rng.choice([1, 1, 2, 3]) if op == "norm" else rng.choice([1, 2, 5, 12, 24])
        heads = H + 2 * Hk if op == "norm" else H
        L = 1 if rng.random() < 0.15 else _log(rng, 2, max(4, min(180512, 1.2e9 / (B * heads * d))))
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        p = _place(rng, d)
        train = rng.random() < 0.5
        if op == "rotary":
            return {k: v for k, v in _rotary("", B, H, L, d, dtype=dtype, token_major=rng.random() < 0.6, train=train,
                                             **p).items() if k != "name"}
        return {k: v for k, v in _norm("", B, H, Hk, L, d, dtype=dtype, wdtype=rng.choice(["fp32", dtype]), train=train,
                                       **p).items() if k != "name"}
    B = rng.choice([1, 2, 3, 8])
    Hk = rng.choice([1, 2, 3, 4, 12])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4])
    causal = rng.random() < 0.6
    if rng.random() < 0.35:  # a few new tokens against a cache
        Lq, train = rng.choice([1, 1, 1, 2, 3, 7]), False
        Lk = _log(rng, Lq, 60000)
        left = rng.choice([-1, _log(rng, 1, 20000)])
        causal = True
    else:
        train = rng.random() < 0.5
        Lq = _log(rng, 2, max(8, min(20000, 4.0e5 / (B * Hq))))
        Lk = Lq + rng.choice([0, 0, _log(rng, 1, 2000)])
        left = rng.choice([_log(rng, 1, 3000), _log(rng, 1, 3000), -1 if B * Hq * Lq * Lk < 4e8 else 1000])
    right = 0 if causal else rng.choice([left, max(0, left // 2), _log(rng, 1, 1000)])
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 600)])
    return {k: v for k, v in _window("", B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, rng.random() < 0.4,
                                     train).items() if k != "name"}


# ---- inputs --------------------------------------------------------------------
def _dims(case):
    return [int(x) for x in case["axes"].split(",")]


ORIGINAL = 8192  # context length that a stretched rotation was trained at


def _freq(case):
    """Angle per position of every pair, fp64, and the factor on the rotated part."""
    out = []
    s, kind = float(case["factor"]), case["scaling"]
    for D in _dims(case):
        i = torch.arange(D // 2, dtype=torch.float64)
        theta = 10000.0
        if kind == "ntk" and D > 2:
            theta = theta * s ** (D / (D - 2))
        w = theta ** (-2.0 * i / D)
        if kind == "linear":
            w = w / s
        if kind == "yarn":
            g = ((ORIGINAL * w / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
            w = w / s * (1 - g) + w * g
        out.append(w)
    return torch.cat(out), (0.1 * math.log(s) + 1.0 if kind == "yarn" and s > 1 else 1.0)


def _positions(case):
    """int32 [B, axes, L]: a running index, or frame / row / column of a grid of frames."""
    B, L, n = case["B"], case["L"], len(_dims(case))
    i = torch.arange(L, device="cuda", dtype=torch.int64)
    start = case["start"] + 17 * torch.arange(B, device="cuda", dtype=torch.int64)[:, None, None]
    if n == 1:
        ax = i[None]
    else:
        f, w = max(case["frame"], 1), max(case["width"], 1)
        ax = torch.stack([i // f, (i % f) // w, (i % f) % w][:n])
    first = torch.zeros(n, 1, device="cuda", dtype=torch.int64)
    first[0] = 1
    return (ax[None] + start * first[None]).to(torch.int32).contiguous()


def _lens(case, g):
    """Lengths of a padded batch (int32 [B]): one full, the rest shorter, the last of three or more empty."""
    B, n = case["B"], case["Lk"]
    frac = torch.rand(B, device="cuda", generator=g) * 0.7 + 0.3
    lens = (frac * n).to(torch.int32).clamp(1, n)
    lens[0] = n
    if B >= 3 and case["Lq"] == n:
        lens[-1] = 0
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype, scale=1.0):
        x = torch.empty(*shape, device="cuda", dtype=dtype)
        x.normal_(0.0, scale, generator=g)
        return x

    st = {"case": case}
    B, d = case["B"], case["d"]
    if case["op"] in ("rotary", "norm"):
        dt = DT[case["dtype"]]
        f, m = _freq(case)
        st["freq"], st["mscale"], st["pos"] = f.cuda(), m, _positions(case)
        if own:
            import chunk_routed_sparse_b200 as moc
            st["rope"] = moc.Rope(sum(_dims(case)), axes=_dims(case), interleaved=case["layout"] == "interleaved",
                                  scaling=case["scaling"], factor=case["factor"], original_length=ORIGINAL)
    if case["op"] == "rotary":
        H, L = case["H"], case["L"]
        st["x"] = normal(B, L, H, d, dtype=dt).transpose(1, 2) if case["token_major"] else normal(B, H, L, d, dtype=dt)
        if case["train"]:
            st["dy"] = normal(B, H, L, d, dtype=dt)
    elif case["op"] == "norm":
        Hq, Hk, L = case["Hq"], case["Hk"], case["L"]
        st["qkv"] = normal(B, L, Hq + 2 * Hk, d, dtype=dt, scale=1.5)
        wdt = DT[case["wdtype"]]
        st["wq"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(wdt)
        st["wk"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(wdt)
        if case["train"]:
            st["dQ"], st["dK"], st["dV"] = (normal(B, h, L, d, dtype=dt) for h in (Hq, Hk, Hk))
    else:
        Hq, Hk, Lq, Lk = case["Hq"], case["Hk"], case["Lq"], case["Lk"]
        bf = torch.bfloat16
        st["Q"], st["K"], st["V"] = normal(B, Hq, Lq, d, dtype=bf), normal(B, Hk, Lk, d, dtype=bf), normal(B, Hk, Lk, d, dtype=bf)
        st["kv_len"] = st["q_len"] = None
        if case["ragged"]:
            st["kv_len"] = _lens(case, g)
            if Lq == Lk:  # a padded batch; otherwise the last Lq tokens of each stream are new
                st["q_len"] = st["kv_len"]
            else:
                st["kv_len"] = st["kv_len"].clamp(min=min(Lq, Lk))
        if case["train"]:
            st["dO"] = normal(B, Hq, Lq, d, dtype=bf)
    return st


# ---- plain forms ---------------------------------------------------------------
def _cos_sin(st):
    """cos and sin of every token's pairs, fp32 [B, 1, L, pairs], with the rotation's factor."""
    pos, f = st["pos"], st["freq"]
    axis = torch.repeat_interleave(torch.arange(pos.shape[1], device=pos.device),
                                   torch.tensor([n // 2 for n in _dims(st["case"])], device=pos.device))
    ang = pos.double()[:, axis].transpose(1, 2) * f
    return (ang.cos() * st["mscale"]).float()[:, None], (ang.sin() * st["mscale"]).float()[:, None]


def _turn(x, c, s, layout):
    """The rotation of the first 2 * pairs columns of x by the angles of c and s."""
    n = c.shape[-1]
    if layout == "interleaved":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((r, x[..., 2 * n:]), -1)


def _run_rotary(st):
    case = st["case"]
    if own:
        import chunk_routed_sparse_b200 as moc
        y = moc.rotary(st["rope"], st["x"], st["pos"])
        if not case["train"]:
            return {"y": y}
        return {"y": y, "dx": moc.rotary_bwd(st["rope"], st["dy"], st["pos"])}
    c, s = _cos_sin(st)
    out = {"y": _turn(st["x"].float(), c, s, case["layout"]).to(st["x"].dtype)}
    if case["train"]:
        out["dx"] = _turn(st["dy"].float(), c, -s, case["layout"]).to(st["dy"].dtype)
    return out


EPS = 1e-6


def _run_norm(st):
    case = st["case"]
    Hq, Hk = case["Hq"], case["Hk"]
    if own:
        import chunk_routed_sparse_b200 as moc
        Q, K, V = moc.qkv_norm_rope(st["qkv"], Hq, Hk, st["wq"], st["wk"], st["rope"], st["pos"], EPS)
        out = {"Q": Q, "K": K, "V": V}
        if case["train"]:
            out["dqkv"], out["dwq"], out["dwk"] = moc.qkv_norm_rope_bwd(
                st["qkv"], Hq, Hk, st["wq"], st["wk"], st["rope"], st["pos"], EPS, st["dQ"], st["dK"], st["dV"])
        return out
    c, s = _cos_sin(st)
    x = st["qkv"].transpose(1, 2)
    dt = x.dtype

    def head(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return x * r, r, w.float()

    hq, rq, wq = head(x[:, :Hq], st["wq"])
    hk, rk, wk = head(x[:, Hq:Hq + Hk], st["wk"])
    out = {"Q": _turn(hq * wq, c, s, case["layout"]).to(dt), "K": _turn(hk * wk, c, s, case["layout"]).to(dt),
           "V": x[:, Hq + Hk:].contiguous()}
    if case["train"]:

        def back(h, r, w, g):
            g = _turn(g.float(), c, -s, case["layout"])
            dw = (g * h).sum((0, 1, 2))
            g = g * w
            return ((g - h * (g * h).mean(-1, keepdim=True)) * r).to(dt), dw

        dq, dwq = back(hq, rq, wq, st["dQ"])
        dk, dwk = back(hk, rk, wk, st["dK"])
        out["dqkv"] = torch.cat((dq, dk, st["dV"]), 1).transpose(1, 2).contiguous()
        out["dwq"], out["dwk"] = dwq.to(st["wq"].dtype), dwk.to(st["wk"].dtype)
    return out


def _run_window(st):
    case = st["case"]
    left, right, sinks, causal = case["left"], case["right"], case["sinks"], case["causal"]
    if own:
        import chunk_routed_sparse_b200 as moc
        O, lse = moc.window_attention_fwd(st["Q"], st["K"], st["V"], left, right, sinks, causal, q_len=st["q_len"],
                                          kv_len=st["kv_len"])
        out = {"O": O, "lse": lse}
        if case["train"]:
            out["dQ"], out["dK"], out["dV"] = moc.window_attention_bwd(
                st["Q"], st["K"], st["V"], O, lse, st["dO"], left, right, sinks, causal, q_len=st["q_len"],
                kv_len=st["kv_len"])
        return out
    B, Hk, G, Lq, Lk, d = case["B"], case["Hk"], case["Hq"] // case["Hk"], case["Lq"], case["Lk"], case["d"]
    dev = st["Q"].device
    n = st["kv_len"].long() if st["kv_len"] is not None else torch.full((B,), Lk, device=dev)
    m = st["q_len"].long() if st["q_len"] is not None else torch.full((B,), Lq, device=dev)
    # queries in blocks; each block reads the keys its window can reach (one block over every key for an open window)
    reach = Lk if left < 0 or right < 0 else min(Lk, left + right + 1)
    blk = Lq if reach == Lk else min(Lq, max(reach // 2, 64))
    nb = -(-Lq // blk)
    row = torch.arange(nb * blk, device=dev).view(nb, blk)                        # query rows of every block
    p = row[None] + (n - m)[:, None, None]                                        # their positions [B, nb, blk]
    slab = min(Lk, blk + reach - 1)
    lo = torch.zeros_like(p[..., :1]) if slab == Lk else (p[..., :1] - left).clamp(0, Lk - slab)
    u = lo + torch.arange(slab, device=dev)                                       # keys of every block [B, nb, slab]
    first = torch.arange(min(sinks, Lk), device=dev)
    pq = p[..., :, None]

    def keep(u, p):
        ok = (u < n[:, None, None, None]) & (row[..., :, None][None] < m[:, None, None, None])
        return ok & (u <= p) if causal else ok

    near = keep(u[..., None, :], pq) & (u[..., None, :] >= len(first))
    if left >= 0:
        near = near & (u[..., None, :] >= pq - left)
    if right >= 0:
        near = near & (u[..., None, :] <= pq + right)
    mask = torch.cat((keep(first, pq), near), -1)[:, None, None]                  # [B, 1, 1, nb, blk, keys]

    def blocks(x):  # [B, Hk * G, Lq, d] -> fp32 [B, Hk, G, nb, blk, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * blk - Lq))
        return x.view(B, Hk, G, nb, blk, d)

    at = u.view(B, 1, nb * slab, 1).expand(B, Hk, nb * slab, d)

    def keys(x):    # [B, Hk, Lk, d] -> fp32 [B, Hk, 1, nb, keys, d]
        x = x.float()
        w = x.gather(2, at).view(B, Hk, nb, slab, d)
        return torch.cat((x[:, :, None, :len(first)].expand(B, Hk, nb, len(first), d), w), -2)[:, :, None]

    scale = 1.0 / math.sqrt(d)
    q, k, v = blocks(st["Q"]), keys(st["K"]), keys(st["V"])
    s = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = s.sub_(top).exp_()
    z = e.sum(-1, keepdim=True)
    pr = e.div_(torch.where(z == 0, torch.ones_like(z), z))
    o = pr @ v

    def rows(x):    # back to [B, Hq, Lq, ...]
        return x.reshape(B, Hk * G, nb * blk, -1)[:, :, :Lq]

    out = {"O": rows(o).to(st["Q"].dtype), "lse": rows(top + z.log())[..., 0].contiguous()}
    if case["train"]:
        g = blocks(st["dO"])
        ds = g @ v.transpose(-1, -2)
        ds = ds.sub_((g * o).sum(-1, keepdim=True)).mul_(pr).mul_(scale)
        out["dQ"] = rows(ds @ k).to(st["Q"].dtype)

        def scatter(x):  # fp32 [B, Hk, nb, keys, d] -> gradient of the keys
            acc = torch.zeros(B, Hk, Lk, d, device=dev)
            acc.scatter_add_(2, at, x[..., len(first):, :].reshape(B, Hk, nb * slab, d))
            acc[:, :, :len(first)] += x[..., :len(first), :].sum(2)
            return acc.to(st["K"].dtype)

        out["dK"] = scatter((ds.transpose(-1, -2) @ q).sum(2))
        out["dV"] = scatter((pr.transpose(-1, -2) @ g).sum(2))
    return out


def run(state):
    return {"rotary": _run_rotary, "norm": _run_norm, "window": _run_window}[state["case"]["op"]](state)


# ---- work ----------------------------------------------------------------------
def _pairs(case, n, m):
    """(visible pairs, keys that some row sees) of one sequence of n keys and m query rows."""
    p = np.arange(m, dtype=np.int64) + (n - m)
    lo = np.maximum(p - case["left"], 0) if case["left"] >= 0 else np.zeros_like(p)
    hi = np.minimum(p + case["right"] + 1, n) if case["right"] >= 0 else np.full_like(p, n)
    end = np.minimum(p + 1, n) if case["causal"] else np.full_like(p, n)
    end, hi = np.maximum(end, 0), np.maximum(np.minimum(hi, end), 0)
    s = np.minimum(case["sinks"], end)
    pairs = s + np.maximum(hi - np.maximum(lo, s), 0)
    if not m:
        return 0, 0
    seen = s.max() + max(0, hi.max() - max(lo.min(), s.max()))
    return int(pairs.sum()), int(seen)


def work(case):
    B, d = case["B"], case["d"]
    if case["op"] == "rotary":
        n = B * case["H"] * case["L"] * d
        size = 4 if case["dtype"] == "fp32" else 2
        k = 2 if case["train"] else 1
        return {"bytes": k * 2 * n * size, "flops": k * 3 * n}
    if case["op"] == "norm":
        n = B * (case["Hq"] + 2 * case["Hk"]) * case["L"] * d
        size = 4 if case["dtype"] == "fp32" else 2
        dots = B * (case["Hq"] + case["Hk"]) * case["L"] * d
        # the gradient reads the Q and K parts again (V's is a copy) and the upstream gradients, and writes dqkv
        return {"bytes": 2 * n * size + (size * (2 * n + dots) if case["train"] else 0),
                "flops": 7 * dots + (15 * dots if case["train"] else 0)}
    Hq, Hk = case["Hq"], case["Hk"]
    lens = [case["Lk"]] * B
    if case["ragged"]:
        lens = [case["Lk"]] + [int(0.65 * case["Lk"])] * (B - 1)
        if B >= 3 and case["Lq"] == case["Lk"]:
            lens[-1] = 0
    got = [_pairs(case, n, n if case["ragged"] and case["Lq"] == case["Lk"] else case["Lq"]) for n in lens]
    pairs, seen = sum(x for x, _ in got) * Hq, sum(x for _, x in got) * Hk
    q = B * Hq * case["Lq"]
    fwd = 2 * q * d * 2 + 4 * q + 2 * seen * d * 2
    bwd = 4 * q * d * 2 + 4 * q + 2 * seen * d * 2 + 2 * B * Hk * case["Lk"] * d * 2
    return {"bytes": fwd + (bwd if case["train"] else 0), "flops": pairs * d * (14 if case["train"] else 4)}


# ---- the definitions in 64 bits ------------------------------------------------
def _angles64(case, pos):
    """fp64 [B, L, pairs], and the factor, from the positions alone."""
    cols, f = [], 1.0
    s = float(case["factor"])
    if case["scaling"] == "yarn" and s > 1:
        f = 1.0 + math.log(s) / 10.0
    for a, D in enumerate(_dims(case)):
        for i in range(D // 2):
            base = 10000.0
            if case["scaling"] == "ntk" and D > 2:
                base *= math.pow(s, D / (D - 2.0))
            w = math.pow(base, -2.0 * i / D)
            if case["scaling"] == "linear":
                w /= s
            elif case["scaling"] == "yarn":
                turns = ORIGINAL * w / (2.0 * math.pi)  # over the original context: below 1 stretched, above 32 kept
                keep = min(max((turns - 1.0) / 31.0, 0.0), 1.0)
                w = keep * w + (1.0 - keep) * w / s
            cols.append(pos[:, a].double() * w)
    return torch.stack(cols, -1), f


def _rotate64(x, ang, f, layout):
    """x: fp64 [B, L, d] of one head."""
    n = ang.shape[-1]
    y = x.clone()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + n)
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(ang, f), ang)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rotary(st):
    case = st["case"]
    ang, f = _angles64(case, st["pos"])
    out = {"y": torch.stack([_rotate64(st["x"][:, h].double(), ang, f, case["layout"]) for h in range(case["H"])], 1)}
    if case["train"]:
        out["dx"] = torch.stack([_rotate64(st["dy"][:, h].double(), -ang, f, case["layout"]) for h in range(case["H"])], 1)
    return out


def _exact_norm(st):
    case = st["case"]
    Hq, Hk, d, lay = case["Hq"], case["Hk"], case["d"], case["layout"]
    ang, f = _angles64(case, st["pos"])
    out = {"Q": [], "K": [], "V": st["qkv"][:, :, Hq + Hk:].transpose(1, 2).double()}
    grad, dw = [], {"wq": 0.0, "wk": 0.0}
    for h in range(Hq + Hk):
        name, other, j = ("wq", "Q", h) if h < Hq else ("wk", "K", h - Hq)
        x, w = st["qkv"][:, :, h].double(), st[name].double()
        rms = ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
        out[other].append(_rotate64(x / rms * w, ang, f, lay))
        if case["train"]:
            g = _rotate64(st["d" + other][:, j].double(), -ang, f, lay)
            dw[name] = dw[name] + (g * x / rms).sum((0, 1))
            gw = g * w
            grad.append(gw / rms - x * (gw * x).sum(-1, keepdim=True) / (d * rms ** 3))
    out["Q"], out["K"] = torch.stack(out["Q"], 1), torch.stack(out["K"], 1)
    if case["train"]:
        grad += [st["dV"][:, j].double() for j in range(Hk)]
        out["dqkv"] = torch.stack(grad, 2)
        out["dwq"], out["dwk"] = dw["wq"], dw["wk"]
    return out


def _exact_window(st):
    case = st["case"]
    B, Hq, Hk, Lq, Lk, d = (case[k] for k in ("B", "Hq", "Hk", "Lq", "Lk", "d"))
    dev, dbl = st["Q"].device, torch.float64
    out = {"O": torch.zeros(B, Hq, Lq, d, device=dev, dtype=dbl),
           "lse": torch.full((B, Hq, Lq), -math.inf, device=dev, dtype=dbl)}
    if case["train"]:
        out["dQ"] = torch.zeros_like(out["O"])
        out["dK"], out["dV"] = (torch.zeros(B, Hk, Lk, d, device=dev, dtype=dbl) for _ in range(2))
    for b in range(B):
        n = Lk if st["kv_len"] is None else int(st["kv_len"][b])
        m = Lq if st["q_len"] is None else int(st["q_len"][b])
        for h in range(Hq):
            k, v = st["K"][b, h // (Hq // Hk), :n].double(), st["V"][b, h // (Hq // Hk), :n].double()
            for r in range(0, m, 4096):
                e = min(m, r + 4096)
                t = torch.arange(r, e, device=dev)[:, None] + (n - m)
                u = torch.arange(n, device=dev)[None]
                see = torch.ones(e - r, n, dtype=torch.bool, device=dev)
                if case["left"] >= 0:
                    see &= t - u <= case["left"]
                if case["right"] >= 0:
                    see &= u - t <= case["right"]
                see |= u < case["sinks"]
                if case["causal"]:
                    see &= u <= t
                q = st["Q"][b, h, r:e].double()
                s = torch.where(see, q @ k.T / math.sqrt(d), torch.full((), -math.inf, device=dev, dtype=dbl))
                lse = torch.logsumexp(s, -1) if n else torch.full((e - r,), -math.inf, device=dev, dtype=dbl)
                p = torch.where(see, torch.exp(s - lse[:, None]), torch.zeros((), device=dev, dtype=dbl))
                o = p @ v
                out["lse"][b, h, r:e], out["O"][b, h, r:e] = lse, o
                if case["train"]:
                    g = st["dO"][b, h, r:e].double()
                    ds = p * (g @ v.T - (g * o).sum(-1, keepdim=True)) / math.sqrt(d)
                    out["dQ"][b, h, r:e] = ds @ k
                    out["dK"][b, h // (Hq // Hk), :n] += ds.T @ q
                    out["dV"][b, h // (Hq // Hk), :n] += p.T @ g
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "norm": _exact_norm, "window": _exact_window}[case["op"]](st)
