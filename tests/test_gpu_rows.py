"""Row operators on the GPU (rotary positions, norm + rotation + re-layout, their
gradients) against the fp64 definitions in oracle/rows.py.

Tolerances, with e = 2^-24 (half an fp32 step) and u = eps(type) / 2:
  forward: one rounding to the type, u |y|, and the fp32 work before it. Angle:
    the half-turn fraction is rounded once (e/2 of 1, pi e / 2 in radians),
    sincospif is within 2 steps (4 e), factor, norm (12 additions, a square root
    within 2 steps, 2 products) and the two products of the turn: below 40 e of
    the row's largest value.
  gradient: the same with the mean of 128 products on top: below 80 e of the size
    of the terms (oracle: r (max|gw| + max|xhat| mean|gw xhat|)).
  weight gradient: at most N + 200 fp32 additions and products, (N + 200) e of the
    sum of the terms' magnitudes, and one rounding to its type. A term g * xhat has
    g = R^T dy, whose error goes by the turned pair's size and not by g, which may
    cancel: 40 e f sqrt(2) max|dy| of the row, times |xhat|, summed.
  fp16 results below 2^-14 are spaced 2^-24: half a step is 2^-25 there.
"""
import math

import pytest
import torch

import chunk_routed_sparse_b200 as moc
import oracle.rows as R

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def _plan(axes, interleaved, **kw):
    rope = moc.Rope(sum(axes), axes=axes, interleaved=interleaved, **kw)
    freq, axis, f = R.frequencies(axes, **{k: float(v) if k != "scaling" else v for k, v in kw.items()})
    return rope, freq, axis, f


def _pos(B, n, L, seed, far=50000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-far, far, (B, n, L), generator=g, device="cuda", dtype=torch.int32)


def _close(got, want, size, steps):
    u = torch.finfo(got.dtype).eps / 2
    tol = u * want.abs() * (1 + 1e-6) + steps * E * size
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of fp16's subnormals
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()))


def _row(x):
    return x.double().abs().amax(-1, keepdim=True)


SHAPES = [(1, 1, 1), (1, 5, 3), (2, 3, 17), (3, 1, 33), (8, 24, 1), (1, 2, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("d,axes", [(64, (64,)), (64, (2,)), (64, (20,)), (64, (24, 20)), (128, (128,)), (128, (44, 42, 42)),
                                    (128, (16, 48, 48)), (128, (6, 4, 2, 2)), (128, (126,)), (64, (34, 16))])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_matches_the_definition(dtype, d, axes, interleaved):
    rope, freq, axis, f = _plan(axes, interleaved)
    for i, (B, H, L) in enumerate(SHAPES):
        x = _rand(B, L, H, d, dtype=dtype, seed=i).transpose(1, 2)
        pos = _pos(B, len(axes), L, i)
        ang = R.angles(freq, axis, pos, B, L)
        _close(moc.rotary_fwd(rope, x, pos), R.rotate(x, ang, f, interleaved), _row(x), 40)
        _close(moc.rotary_bwd(rope, x, pos), R.rotate(x, ang, f, interleaved, -1), _row(x), 40)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=8), dict(scaling="ntk", factor=2.5),
                                dict(scaling="yarn", factor=8, original_length=8192),
                                dict(scaling="yarn", factor=4, original_length=2000, attention_factor=0.75)])
def test_stretched_rotations_at_far_positions(kw):
    """Positions up to 2^31 - 1: the fp64 product itself is off by |angle| 2^-53."""
    rope, freq, axis, f = _plan((64,), False, **kw)
    x = _rand(2, 3, 9, 64, dtype=torch.float32, seed=3)
    pos = torch.tensor([0, 1, -1, 180511, 1 << 20, (1 << 31) - 1, -(1 << 31), 12345678, -999], device="cuda",
                       dtype=torch.int32)
    ang = R.angles(freq, axis, pos.expand(2, 1, 9), 2, 9)
    want = R.rotate(x, ang, f, False)
    _close(moc.rotary(rope, x, pos), want, f * _row(x) * (1 + 2.0 ** 31 * 2.0 ** -53 / (40 * E)), 40)


def test_default_positions_shared_positions_and_batch_positions_agree():
    rope = moc.Rope(64)
    x = _rand(3, 2, 11, 64, dtype=torch.bfloat16, seed=1)
    p = torch.arange(11, device="cuda", dtype=torch.int32)
    a = moc.rotary(rope, x)
    for pos in (p, p[None], p.expand(3, 1, 11), p.expand(3, 1, 11).contiguous()):
        assert torch.equal(moc.rotary(rope, x, pos), a)


def test_unrotated_columns_and_position_zero_pass_through_exactly():
    """Infinities and NaN among the dims that are not rotated stay where they are
    (a NaN as some NaN: the conversions to and from fp32 keep no payload)."""

    def same(y, x):
        n = x.isnan()
        return torch.equal(n, y.isnan()) and torch.equal(y[~n].view(torch.int16), x[~n].view(torch.int16))

    for interleaved in (True, False):
        rope = moc.Rope(24, interleaved=interleaved)
        x = _rand(1, 2, 5, 64, dtype=torch.bfloat16, seed=2)
        x[..., 24:30] = math.inf
        x[..., 31] = math.nan
        y = moc.rotary(rope, x, torch.full((5,), 7, device="cuda", dtype=torch.int32))
        assert torch.isfinite(y[..., :24]).all()
        assert same(y[..., 24:], x[..., 24:])
        y = moc.rotary(rope, x, torch.zeros(5, device="cuda", dtype=torch.int32))
        assert same(y, x)


def test_layouts_alignment_in_place_and_broadcast_inputs_agree():
    rope, d = moc.Rope(64, interleaved=False), 64
    for dtype in (torch.bfloat16, torch.float32):
        x = _rand(2, 3, 13, d, dtype=dtype, seed=4)
        want = moc.rotary(rope, x)
        wide = torch.zeros(2, 13, 3, d + 9, device="cuda", dtype=dtype)
        for off in (0, 1, 3, 8):  # rows on and off 16-byte boundaries
            v = wide[..., off:off + d].transpose(1, 2)
            v.copy_(x)
            assert torch.equal(moc.rotary(rope, v), want)
            before = wide.clone()
            moc.rotary_fwd(rope, x, out=v)
            assert torch.equal(v, want)
            wide[..., off:off + d] = before[..., off:off + d]
            assert torch.equal(wide, before)  # nothing around the rows was written
        y = x.clone()
        assert moc.rotary_fwd(rope, y, out=y) is y and torch.equal(y, want)
        one = x[:, :1].expand(2, 3, 13, d)
        assert torch.equal(moc.rotary(rope, one), want[:, :1].expand(2, 3, 13, d))
    with pytest.raises(moc.MocError):
        moc.rotary_fwd(rope, x, out=x[:, :1].expand(2, 3, 13, d))


def test_empty_tensors():
    rope = moc.Rope(64)
    for shape in ((0, 2, 3, 64), (2, 0, 3, 64), (2, 3, 0, 64)):
        assert moc.rotary(rope, torch.empty(shape, device="cuda")).shape == shape
    qkv = torch.empty(2, 0, 4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    sum(t.sum() for t in moc.qkv_norm_rope(qkv, 2, 1, w, w)).backward()
    assert qkv.grad.shape == qkv.shape and torch.equal(w.grad, torch.zeros_like(w))


NORM = [  # B, Hq, Hk, L, d, axes, interleaved
    (1, 1, 1, 1, 64, (64,), True), (2, 4, 2, 7, 64, (24, 20), False), (3, 12, 4, 37, 128, (44, 42, 42), True),
    (1, 5, 5, 130, 128, (128,), False), (2, 3, 1, 65, 128, (20,), False), (8, 24, 24, 1, 128, (96,), True),
    (1, 2, 2, 1500, 64, (64,), False)]


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                          (torch.float16, torch.float16), (torch.float32, torch.float32),
                                          (torch.float16, None)], ids=str)
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_rope_and_gradient_match_the_definition(dtype, wdtype, case):
    B, Hq, Hk, L, d, axes, inter = case
    rope, freq, axis, f = _plan(axes, inter, scaling="yarn", factor=4, original_length=1000)
    pos = _pos(B, len(axes), L, 5)
    ang = R.angles(freq, axis, pos, B, L)
    qkv = _rand(B, L, Hq + 2 * Hk, d, dtype=dtype, seed=6, scale=2.0)
    wq = wk = None
    if wdtype is not None:
        wq = (1 + 0.3 * _rand(d, dtype=torch.float32, seed=7)).to(wdtype)
        wk = (1 + 0.3 * _rand(d, dtype=torch.float32, seed=8)).to(wdtype)
    eps = 1e-5
    Q, K, V = moc.qkv_norm_rope(qkv, Hq, Hk, wq, wk, rope, pos, eps)
    x = qkv.transpose(1, 2)
    g = [_rand(B, h, L, d, dtype=dtype, seed=9 + i) for i, h in enumerate((Hq, Hk, Hk))]
    dqkv, dwq, dwk = moc.qkv_norm_rope_bwd(qkv, Hq, Hk, wq, wk, rope, pos, eps, *g)
    assert torch.equal(V, x[:, Hq + Hk:]) and torch.equal(dqkv.transpose(1, 2)[:, Hq + Hk:], g[2])
    for y, lo, hi, w, gy, dw in ((Q, 0, Hq, wq, g[0], dwq), (K, Hq, Hq + Hk, wk, g[1], dwk)):
        want = R.norm_rope(x[:, lo:hi], w, eps, ang, f, inter)
        plain = R.norm_rope(x[:, lo:hi], w, eps, None, f, inter)
        _close(y, want, f * _row(plain), 40)
        dx, wsum, wabs, size = R.norm_rope_bwd(x[:, lo:hi], w, eps, ang, f, inter, gy)
        _close(dqkv.transpose(1, 2)[:, lo:hi], dx, 1.5 * size, 80)  # a turned pair is at most sqrt(2) its larger part
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == wdtype
            xh = R.norm_rope(x[:, lo:hi], None, eps, None, 1.0, inter).abs()
            turn = 40 * E * (xh * f * math.sqrt(2) * _row(gy)).sum((0, 1, 2))
            tol = torch.finfo(wdtype).eps / 2 * wsum.abs() + (B * L * (hi - lo) + 200) * E * wabs + turn
            if wdtype == torch.float16:
                tol = tol + 2.0 ** -25
            assert ((dw.double() - wsum).abs() <= tol).all()


def test_norm_without_rotation_zero_rows_and_large_values():
    x = _rand(1, 2, 6, 64, dtype=torch.float32, seed=11)
    x[0, 0, 0] = 0
    x[0, 1, 2] *= 1e15
    Q, K, V = moc.qk_norm_rope_fwd(x, x, eps=1e-6)
    assert V is None and torch.equal(Q, K) and (Q[0, 0, 0] == 0).all()
    _close(Q, R.norm_rope(x, None, 1e-6, None, 1.0, True), _row(R.norm_rope(x, None, 1e-6, None, 1.0, True)), 40)
    # a zero row: dx = g w / sqrt(eps)
    dQ, _, _, _, _ = moc.qk_norm_rope_bwd(x, x, None, None, None, None, 1e-6, torch.ones_like(x), torch.ones_like(x))
    assert torch.allclose(dQ[0, 0, 0], torch.full((64,), 1000.0, device="cuda"), rtol=1e-6)


def test_outputs_into_a_cache_leave_its_other_slots():
    """New tokens' keys and values written at their slots of a longer cache, queries in place."""
    B, Hq, Hk, L, d, cap, at = 2, 4, 2, 3, 128, 16, 5
    qkv = _rand(B, L, Hq + 2 * Hk, d, dtype=torch.bfloat16, seed=12)
    rope = moc.Rope(d, interleaved=False)
    pos = torch.arange(at, at + L, device="cuda", dtype=torch.int32)
    want = moc.qkv_norm_rope(qkv, Hq, Hk, None, None, rope, pos)
    kc, vc = (torch.full((B, Hk, cap, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    x = qkv.transpose(1, 2)
    moc.qk_norm_rope_fwd(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], None, None, rope, pos,
                         out=(x[:, :Hq], kc[:, :, at:at + L], vc[:, :, at:at + L]))
    assert torch.equal(x[:, :Hq], want[0])
    for c, w in ((kc, want[1]), (vc, want[2])):
        assert torch.equal(c[:, :, at:at + L], w)
        assert (c[:, :, :at] == 7).all() and (c[:, :, at + L:] == 7).all()


def test_gradients_against_differences():
    """<grad, v> against (f(x + hv) - f(x - hv)) / 2h in fp32, f = sum(u * y) over 10
    rows of 64, h = 2^-7. Rounding: 640 outputs, each within 40 e of a row maximum
    below 4 and weighted by |u| below 4: under 640 * 40 e * 16 / h = 3.2 if all had
    the same sign; they have random signs, so under 3.2 / sqrt(640) = 0.13 a sigma,
    0.4 at three. Truncation: h^2 / 6 times a third derivative below 15 |u y| a
    value: 640 * 15 * 1e-5 = 0.1. Together 0.5 of a derivative of about 25."""
    rope = moc.Rope(44, axes=(24, 20), interleaved=False)
    B, Hq, Hk, L, d, h = 1, 2, 1, 5, 64, 2.0 ** -7
    pos = _pos(B, 2, L, 1, far=100)
    qkv = _rand(B, L, Hq + 2 * Hk, d, dtype=torch.float32, seed=1).requires_grad_()
    wq = (1 + 0.1 * _rand(d, dtype=torch.float32, seed=2)).requires_grad_()
    wk = (1 + 0.1 * _rand(d, dtype=torch.float32, seed=3)).requires_grad_()
    u = [_rand(B, n, L, d, dtype=torch.float32, seed=4 + n) for n in (Hq, Hk, Hk)]

    def f(a, b, c):
        return sum((y.double() * t.double()).sum() for y, t in zip(moc.qkv_norm_rope(a, Hq, Hk, b, c, rope, pos), u))

    f(qkv, wq, wk).backward()
    for t in (qkv, wq, wk):
        v = _rand(*t.shape, dtype=torch.float32, seed=20)
        args = [qkv.detach(), wq.detach(), wk.detach()]
        i = 0 if t is qkv else 1 if t is wq else 2
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * v, args[i] - h * v
        diff = (f(*hi) - f(*lo)) / (2 * h)
        assert abs(float((t.grad.double() * v.double()).sum() - diff)) <= 0.5


def test_autograd_layouts_and_needs():
    rope = moc.Rope(64)
    base = _rand(2, 9, 3, 64, dtype=torch.bfloat16, seed=30).requires_grad_()
    g = _rand(2, 3, 9, 64, dtype=torch.bfloat16, seed=31)
    moc.rotary(rope, base.transpose(1, 2)).backward(g)
    assert torch.equal(base.grad.transpose(1, 2), moc.rotary_bwd(rope, g))
    one = _rand(2, 1, 9, 64, dtype=torch.float32, seed=32).requires_grad_()  # broadcast over heads
    moc.rotary(rope, one.expand(2, 3, 9, 64)).backward(g.float())
    want = moc.rotary_bwd(rope, g.float()).double().sum(1, keepdim=True)
    assert (one.grad.double() - want).abs().max() <= 8 * E * want.abs().max() + 8 * E * 4
    Q = _rand(2, 3, 9, 64, dtype=torch.bfloat16, seed=33).requires_grad_()
    K = _rand(2, 3, 9, 64, dtype=torch.bfloat16, seed=34)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    Qo, Ko = moc.qk_norm_rope(Q, K, w, w, rope)
    (Qo.float().sum() + Ko.float().sum()).backward()  # a gradient of stride 0
    ones = torch.ones_like(Q)
    assert torch.equal(Q.grad, moc.qk_norm_rope_bwd(Q.detach(), K, w, w, rope, None, 1e-6, ones, ones)[0])
    with torch.no_grad():
        assert not moc.qk_norm_rope(Q, K, w, w, rope)[0].requires_grad


def test_repeatable_and_on_another_stream_and_captured():
    rope = moc.Rope(128, axes=(44, 42, 42))
    B, Hq, Hk, L, d = 1, 6, 2, 3001, 128
    qkv = _rand(B, L, Hq + 2 * Hk, d, dtype=torch.bfloat16, seed=40)
    w = _rand(d, dtype=torch.float32, seed=41)
    pos = _pos(1, 3, L, 42)
    g = [_rand(B, n, L, d, dtype=torch.bfloat16, seed=43 + n) for n in (Hq, Hk, Hk)]

    def step():
        return (*moc.qkv_norm_rope_fwd(qkv, Hq, Hk, w, w, rope, pos),
                *moc.qkv_norm_rope_bwd(qkv, Hq, Hk, w, w, rope, pos, 1e-6, *g))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for x in held:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, held):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals_of_the_binding():
    rope = moc.Rope(64)
    x = torch.zeros(1, 2, 4, 64, device="cuda")
    p = torch.zeros(4, device="cuda", dtype=torch.int32)
    for bad in (dict(pos=p.long()), dict(pos=p[:3]), dict(pos=p.cpu()), dict(pos=p.expand(2, 4)),
                dict(X=x[..., ::2]), dict(X=x.double()), dict(X=x[0]), dict(X=torch.zeros(1, 2, 4, 32, device="cuda")),
                dict(out=x.bfloat16()), dict(out=x[:, :1]), dict(rope=None), dict(rope=moc.Rope(128))):
        kw = dict(rope=rope, X=x, pos=None, out=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            moc.rotary_fwd(**kw)
    w = torch.ones(64, device="cuda")
    for bad in (dict(wq=w[:32]), dict(wq=w.double()), dict(wq=w.cpu()), dict(K=x[:, :, :2]), dict(K=x.half()),
                dict(pos=p), dict(V=x[..., :32]), dict(wq=w, wk=w.half()), dict(rope=moc.Rope(64, axes=(32, 32)))):
        kw = dict(Q=x, K=x, V=x)
        kw.update(bad)
        with pytest.raises(ValueError):
            moc.qk_norm_rope_fwd(**kw)
    with pytest.raises(ValueError):
        moc.qkv_norm_rope(x, 1, 1)
    closed = moc.Rope(64)
    closed.close()
    with pytest.raises(ValueError):
        moc.rotary(closed, x)
