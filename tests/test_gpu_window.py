"""Sliding-window attention on the GPU against the fp64 definition in
oracle/window.py.

Tolerances. Rounding to bf16 is off by at most u = 2^-8 of the value. Scores are
fp32 sums of d products: off by at most d 2^-24 scale |q||k|, and |q||k| stays below
d + 9 sqrt(2 d) for d normal values a row (below 300 at d = 128): under
128 * 2^-24 * 300 / sqrt(128) = 2.1e-4 of exponent; the exponential adds 2^-22. So a
weight is within w = 2^-11 of itself before its rounding, and the log-sum-exp
within 3e-4.
  O: u |O| + (u + w) sum p |v|.
  dQ, dK, dV: u of the value, and u + w of the terms (oracle: sQ, sK, sV) for the
    rounding of ds or p before the last product. ds = p (dO . v - D) goes by what it is
    a difference of: dO . v is an fp32 sum of d products (within d 2^-24 of |dO||v|) and
    D = dO . O has O rounded by u (and its weights, u + w), so up to (2 u + w) sum
    |dO||O| of D's terms: the oracle's sizes hold |dO| . |v| for the one and, as
    |O| <= sum p |v|, an average of such for the other, which the shared size stands for
    over a row. In all u |x| + (4 u + 2 w) size for dQ and dK, u |x| + (u + w) size for
    dV; and, the errors being many, independent and mostly far smaller, 2 u in the
    2-norm over a batch entry (a rounding's own share is u / sqrt(3)).
"""
import math

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


def _qkv(B, Hq, Hk, Lq, Lk, d, seed=0):
    return _rand(B, Hq, Lq, d, seed=seed), _rand(B, Hk, Lk, d, seed=seed + 1), _rand(B, Hk, Lk, d, seed=seed + 2)


def _lens(x):
    return None if x is None else torch.tensor(x, device="cuda", dtype=torch.int32)


def _check_fwd(O, lse, ref):
    assert torch.equal(torch.isinf(lse), torch.isinf(ref["lse"]))
    fin = torch.isfinite(ref["lse"])
    assert (lse.double() - ref["lse"])[fin].abs().max() <= 3e-4 if fin.any() else True
    tol = U * ref["O"].abs() + (U + WT) * ref["sO"]
    err = (O.double() - ref["O"]).abs()
    assert (err <= tol).all(), float((err - tol).max())


CASES = [  # B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, q_len, kv_len
    (1, 1, 1, 1, 1, 64, -1, -1, 0, False, None, None),
    (1, 1, 1, 1, 1, 128, 0, 0, 0, True, None, None),
    (1, 2, 2, 300, 300, 64, 40, 7, 5, False, None, None),
    (1, 2, 1, 257, 257, 128, 0, 0, 0, True, None, None),
    (2, 4, 2, 513, 513, 64, 100, 0, 3, True, None, None),
    (1, 2, 2, 700, 700, 128, 129, 129, 200, False, None, None),
    (1, 1, 1, 1100, 1100, 64, 10, 0, 131, True, None, None),      # sinks apart from the window
    (1, 3, 1, 640, 640, 128, -1, 0, 0, True, None, None),
    (1, 2, 2, 384, 384, 64, -1, -1, 0, False, None, None),
    (2, 2, 1, 200, 900, 128, 300, 20, 64, False, None, None),     # last rows of a longer stream
    (2, 2, 2, 130, 1025, 64, 200, 0, 9, True, None, None),
    (1, 2, 2, 300, 100, 64, 20, 0, 4, True, None, None),          # more rows than keys: the first see nothing
    (1, 2, 2, 300, 100, 128, 20, 30, 0, False, None, None),
    (1, 2, 2, 300, 0, 64, -1, -1, 3, False, None, None),          # no keys
    (4, 2, 1, 333, 333, 128, 50, 0, 2, True, [333, 0, 1, 200], [333, 0, 1, 200]),
    (3, 2, 2, 333, 500, 64, 64, 64, 7, False, [333, 10, 256], [500, 3, 129]),
    (2, 1, 1, 140, 140, 64, 30, 0, 500, True, [-5, 999], [999, 999]),  # lengths outside the tensors are clamped
    (1, 1, 1, 2112, 2112, 64, 256, 256, 64, False, None, None),   # the tiny scene: captions and a frame either side
]

FEW = [  # few rows against a cache: one tile of up to 16 rows (query heads of a key head x rows)
    (1, 1, 1, 1, 1000, 64, -1, 0, 0, True, None, None),
    (8, 24, 24, 1, 777, 128, 255, 0, 64, True, None, [777, 1, 0, 64, 65, 320, 500, 700]),
    (2, 16, 1, 1, 3000, 128, -1, 0, 4, True, None, [3000, 2999]),
    (2, 8, 2, 4, 515, 64, 100, 0, 7, True, None, None),
    (3, 6, 2, 5, 1025, 128, 300, 40, 9, False, [5, 0, 3], [1025, 600, 2]),
    (1, 3, 3, 16, 4100, 128, 1000, 0, 200, True, None, None),
    (1, 2, 2, 17, 4100, 128, 1000, 0, 200, True, None, None),          # one row too many: the many-row kernel
    (2, 5, 5, 2, 63, 64, 0, 0, 0, True, None, None),
    (1, 4, 2, 3, 2, 64, -1, -1, 0, True, None, None),                  # more rows than keys
    (40, 4, 4, 1, 130, 64, 64, 0, 1, True, None, None),
    (1, 1, 1, 1, 70000, 128, -1, 0, 0, True, None, None),
]
CASES += FEW


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_matches_the_definition(case):
    B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, ql, kl = case
    Q, K, V = _qkv(B, Hq, Hk, Lq, Lk, d)
    ql, kl = _lens(ql), _lens(kl)
    O = torch.full_like(Q, 5.0)
    lse = torch.full((B, Hq, Lq), 5.0, device="cuda")
    moc.window_attention_fwd(Q, K, V, left, right, sinks, causal, ql, kl, O=O, lse=lse)
    ref = W.attention(Q, K, V, left, right, sinks, causal, ql, kl)
    for b in range(B):
        m = Lq if ql is None else min(max(int(ql[b]), 0), Lq)
        assert (O[b, :, m:] == 5).all() and (lse[b, :, m:] == 5).all()  # rows behind the last: as they were
        O[b, :, m:], lse[b, :, m:] = 0, -math.inf
    _check_fwd(O, lse, ref)
    O2, lse2 = moc.window_attention_fwd(Q, K, V, left, right, sinks, causal, ql, kl)
    assert torch.equal(O2, O) and torch.equal(lse2, lse)
    lse2 = moc.window_attention_fwd(Q, K, V, left, right, sinks, causal, ql, kl, O=O2)[1]
    assert torch.equal(O2, O) and torch.equal(lse2, lse)
    moc.check_window_error()


def test_garbage_past_the_lengths_is_not_read():
    B, H, L, d = 2, 2, 400, 128
    Q, K, V = _qkv(B, H, H, L, L, d)
    n = _lens([170, 301])
    want = moc.window_attention_fwd(Q, K, V, 60, 0, 4, True, n, n)
    for bad in (math.nan, math.inf):
        q, k, v = Q.clone(), K.clone(), V.clone()
        for b in range(B):
            for t in (q, k, v):
                t[b, :, int(n[b]):] = bad
        got = moc.window_attention_fwd(q, k, v, 60, 0, 4, True, n, n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_few_rows_ignore_garbage_past_the_lengths():
    B, Hq, Hk, L, d = 3, 8, 2, 500, 128
    Q, K, V = _qkv(B, Hq, Hk, 2, L, d)
    n = _lens([170, 500, 33])
    want = moc.window_attention_fwd(Q, K, V, 60, 0, 4, True, None, n)
    for bad in (math.nan, math.inf):
        k, v = K.clone(), V.clone()
        for b in range(B):
            k[b, :, int(n[b]):] = v[b, :, int(n[b]):] = bad
            lo = max(4, int(n[b]) - 2 - 60)  # between the first keys and the window of both rows
            k[b, :, 4:lo] = v[b, :, 4:lo] = bad
        got = moc.window_attention_fwd(Q, k, v, 60, 0, 4, True, None, n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_large_scores_and_scale():
    """Scores up to some thousands: the running maximum moves by far more than the
    lazy rescale's 2^8 and the softmax is nearly one-hot."""
    Q, K, V = _qkv(1, 1, 1, 300, 300, 64)
    Q, K = Q * 16, K * 16
    ref = W.attention(Q, K, V, 100, 100, 0, False, scale=1.0)
    O, lse = moc.window_attention_fwd(Q, K, V, 100, 100, 0, False, scale=1.0)
    # scores of size 16 * 16 * 8: fp32 sums within 64 * 2^-24 * 16 * 16 * 130 = 0.13 in the worst order;
    # rows whose two largest scores are 8 apart have every other weight below e^-7.8
    s = (Q.double() @ K.double().transpose(-1, -2))
    s = s.masked_fill(~W.visible(300, 300, 100, 100, 0, False, "cuda"), -math.inf)
    top = s.topk(2, -1).values
    clear = (top[..., 0] - top[..., 1]) > 8
    assert clear.float().mean() > 0.9
    assert ((lse.double() - ref["lse"]).abs() <= 0.13 + 1e-6 * ref["lse"].abs()).all()
    err = (O.double() - ref["O"]).abs()[clear]
    assert (err <= 2 * U * 5 + 100 * math.exp(-7.8) * 0.13 * 10).all()


def _check_bwd(got, ref, ql, kl, Lq, Lk, rest=0):
    for name, size, k, lens, L in (("dQ", "sQ", 4 * U + 2 * WT, ql, Lq), ("dK", "sK", 4 * U + 2 * WT, kl, Lk),
                                   ("dV", "sV", U + WT, kl, Lk)):
        x, want = got[name].double(), ref[name]
        for b in range(x.shape[0]):
            n = L if lens is None else min(max(int(lens[b]), 0), L)
            err = (x[b, :, :n] - want[b, :, :n]).abs()
            tol = U * want[b, :, :n].abs() + k * ref[size][b, :, :n] + 1e-30
            assert (err <= tol).all(), (name, b, float((err - tol).max()))
            if n and want[b].abs().max() > 0 and want[b, :, :n].numel() > 1000:
                rel = (err.square().sum() / want[b, :, :n].square().sum()).sqrt()
                assert rel <= 2 * U, (name, b, float(rel))
            if lens is not None:
                assert (x[b, :, n:] == rest).all(), name


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradient_matches_the_definition(case):
    B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, ql, kl = case
    Q, K, V = _qkv(B, Hq, Hk, Lq, Lk, d)
    g = _rand(B, Hq, Lq, d, seed=9)
    ql, kl = _lens(ql), _lens(kl)
    args = (left, right, sinks, causal, ql, kl)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    ref = W.attention(Q, K, V, *args, dO=g)
    got = {n: torch.full_like(t, 5.0) for n, t in (("dQ", Q), ("dK", K), ("dV", V))}
    moc.window_attention_bwd(Q, K, V, O, lse, g, *args, **got)
    moc.check_window_error()
    _check_bwd(got, ref, ql, kl, Lq, Lk, rest=5)  # as they were
    new = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
    _check_bwd(dict(zip(("dQ", "dK", "dV"), new)), ref, ql, kl, Lq, Lk)
    some = moc.window_attention_bwd(Q, K, V, O, lse, g, *args, dK=got["dK"])
    assert torch.equal(some[0], new[0]) and torch.equal(some[2], new[2])


MANY = [  # more row tiles than the one-tile kernel takes; the last: several of its items a CTA
    (6, 24, 8, 513, 513, 64, 100, 0, 3, True, [513, 0, 1, 200, 256, 400], [513, 0, 1, 200, 256, 400]),
    (3, 25, 5, 700, 900, 128, 129, 129, 200, False, None, None),
    (2, 40, 40, 577, 577, 128, -1, 0, 0, True, None, None),
    (1, 250, 1, 300, 100, 64, 20, 0, 4, True, None, None),
    (8, 30, 10, 130, 700, 64, 64, 64, 7, False, [130, 1, 0, 129, 128, 7, 64, 130], [700, 1, 3, 0, 128, 699, 64, 130]),
    (3, 9, 3, 1425, 1425, 64, 256, 256, 64, False, None, [1425, 0, 700]),
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_forward_and_gradient_of_many_row_tiles(case):
    test_forward_matches_the_definition(case)
    test_gradient_matches_the_definition(case)


def test_many_row_tiles_ignore_garbage_past_the_lengths():
    B, H, L, d = 4, 32, 400, 128
    Q, K, V = _qkv(B, H, H, L, L, d)
    n = _lens([170, 301, 0, 400])
    want = moc.window_attention_fwd(Q, K, V, 60, 0, 4, True, n, n)
    for bad in (math.nan, math.inf):
        q, k, v = Q.clone(), K.clone(), V.clone()
        for b in range(B):
            for t in (q, k, v):
                t[b, :, int(n[b]):] = bad
        for _ in range(5):
            got = moc.window_attention_fwd(q, k, v, 60, 0, 4, True, n, n)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_both_forward_kernels_give_a_row_the_same_weights():
    """One head of many against the head by itself: other tiles and another order of the
    sums, so within the rounding of P and O (each of the two within its bound)."""
    B, H, L, d = 1, 120, 500, 64
    Q, K, V = _qkv(B, H, H, L, L, d)
    Q[:, 7] *= 16
    args = (130, 40, 9, False)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    for h in (0, 7, 119):
        o, l1 = moc.window_attention_fwd(*(t[:, h:h + 1].contiguous() for t in (Q, K, V)), *args)
        ref = W.attention(*(t[:, h:h + 1] for t in (Q, K, V)), *args)
        # scores of head 7 are 16 times larger: so is the error of the exponents
        w = WT * (16 if h == 7 else 1)
        tol = U * ref["O"].abs() + (U + w) * ref["sO"]
        for x, y in ((O[:, h:h + 1], lse[:, h:h + 1]), (o, l1)):
            assert ((x.double() - ref["O"]).abs() <= tol).all()
            assert ((y.double() - ref["lse"]).abs() <= 3e-4 * (16 if h == 7 else 1)).all()


@pytest.mark.parametrize("case", [
    (1, 1, 1, 2, 2, 64, -1, -1, 0, False, None, None), (8, 1, 1, 5, 7, 128, -1, 0, 1, True, None, None),
    (2, 2, 2, 4, 184, 64, 201, 0, 0, True, None, None), (1, 12, 4, 3, 1434, 128, 18, 18, 4, False, None, [1100]),
    (3, 6, 2, 17, 300, 64, 90, 0, 130, True, [17, 0, 9], [300, 20, 150]), (2, 4, 4, 64, 64, 128, -1, -1, 0, False, None, None)],
    ids=str)
def test_gradients_of_few_rows_lose_little_more_than_their_own_rounding(case):
    """Up to 64 rows a head, p and ds enter the products as two bf16: 2^-16 of each is lost
    (u of u), not u. The rows' spans stay below 384 keys, so that D is exact in dQ too.
    Left of the bounds above: u |x| + (2^-16 + 2 w) size for dQ and dK, + (2^-16 + w) for dV."""
    B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, ql, kl = case
    Q, K, V = _qkv(B, Hq, Hk, Lq, Lk, d)
    g = _rand(B, Hq, Lq, d, seed=9)
    ql, kl = _lens(ql), _lens(kl)
    args = (left, right, sinks, causal, ql, kl)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    ref = W.attention(Q, K, V, *args, dO=g)
    got = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
    for name, size, x, k in (("dQ", "sQ", got[0], 2 * WT), ("dK", "sK", got[1], 2 * WT), ("dV", "sV", got[2], WT)):
        err = (x.double() - ref[name]).abs()
        tol = U * ref[name].abs() + (2.0 ** -16 + k) * ref[size] + 1e-30
        assert (err <= tol).all(), (name, float((err / tol).max()))
    for x, y in zip(got, moc.window_attention_bwd(Q, K, V, O, lse, g, *args)):
        assert torch.equal(x, y)
    moc.check_window_error()


def test_gradients_with_shared_first_keys_split_over_many_rows():
    """First keys seen by thousands of rows of six query heads: their tiles' rows are
    split over units and joined."""
    B, Hq, Hk, L, d = 1, 6, 2, 3333, 64
    Q, K, V = _qkv(B, Hq, Hk, L, L, d)
    g = _rand(B, Hq, L, d, seed=9)
    args = (60, 0, 150, True)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    got = dict(zip(("dQ", "dK", "dV"), moc.window_attention_bwd(Q, K, V, O, lse, g, *args)))
    _check_bwd(got, W.attention(Q, K, V, *args, dO=g), None, None, L, L)
    again = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
    for a, b in zip(got.values(), again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", [(3, 8, 2, 1225, 128, 161, 2, 1, False), (2, 6, 3, 1500, 64, 40, 0, 3, True),
                                  (1, 12, 12, 2500, 128, 700, 300, 200, False), (1, 16, 2, 900, 128, -1, 0, 0, True)], ids=str)
def test_repeatable_bit_for_bit(case):
    """Nothing depends on which warps run ahead or on the order of the work units."""
    B, Hq, Hk, L, d, *args = case
    Q, K, V = _qkv(B, Hq, Hk, L, L, d)
    g = _rand(B, Hq, L, d, seed=9)
    want = None
    for _ in range(20):
        O, lse = moc.window_attention_fwd(Q, K, V, *args)
        got = (O, lse, *moc.window_attention_bwd(Q, K, V, O, lse, g, *args))
        want = got if want is None else want
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_gradient_ignores_garbage_past_the_lengths():
    B, H, L, d = 2, 2, 400, 128
    Q, K, V = _qkv(B, H, H, L, L, d)
    g = _rand(B, H, L, d, seed=9)
    n = _lens([170, 301])
    args = (60, 0, 4, True, n, n)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    want = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
    for bad in (math.nan, math.inf):
        t = [x.clone() for x in (Q, K, V, O, g)]
        l2 = lse.clone()
        for b in range(B):
            for x in t:
                x[b, :, int(n[b]):] = bad
            l2[b, :, int(n[b]):] = bad
        for a, b in zip(moc.window_attention_bwd(*t[:4], l2, t[4], *args), want):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """<grad, v> against central differences of the definition's sum(dO * O) in fp64 along
    v = grad / |grad| (h = 1e-4: truncation and rounding below 1e-6 of it). The gradient is
    within 2 u of itself in the 2-norm, so is its product with a unit vector
    (Cauchy-Schwarz)."""
    Q, K, V = _qkv(1, 2, 1, 96, 96, 64)
    g = _rand(1, 2, 96, 64, seed=9)
    args = (30, 0, 4, True)
    O, lse = moc.window_attention_fwd(Q, K, V, *args)
    grads = moc.window_attention_bwd(Q, K, V, O, lse, g, *args)
    x = [t.double() for t in (Q, K, V)]
    for i in range(3):
        v = grads[i].double() / grads[i].double().norm()
        f = []
        for h in (1e-4, -1e-4):
            y = list(x)
            y[i] = x[i] + h * v
            f.append((g.double() * W.attention(*y, *args)["O"]).sum())
        want = float(f[0] - f[1]) / 2e-4
        assert abs(float((grads[i].double() * v).sum()) - want) <= (2 * U + 1e-6) * want


def test_autograd_and_capture():
    B, Hq, Hk, L, d = 2, 4, 2, 700, 64
    Q, K, V = (x.requires_grad_() for x in _qkv(B, Hq, Hk, L, L, d))
    n = _lens([700, 123])
    O = moc.window_attention(Q, K, V, 200, 0, 16, True, n, n)
    assert (O[1, :, 123:] == 0).all()
    g = _rand(B, Hq, L, d, seed=3)
    O.backward(g)
    q, k, v = (x.detach() for x in (Q, K, V))
    args = (200, 0, 16, True, n, n)
    o, lse = moc.window_attention_fwd(q, k, v, *args)
    want = moc.window_attention_bwd(q, k, v, o, lse, g, *args)
    for x, w in zip((Q, K, V), want):
        assert torch.equal(x.grad, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = moc.window_attention_fwd(q, k, v, *args)
        grads = moc.window_attention_bwd(q, k, v, *held, g, *args)
    for _ in range(2):
        for t in (*held, *grads):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], o)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
    moc.check_window_error()
