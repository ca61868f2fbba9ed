"""The operators of an attention layer run together as they would be used: the
packed projection through norm, rotation and re-layout into the routed attention or
the sliding window, with gradients; a stream of new tokens against its cache; calls
on several streams, captured graphs that share a workspace, far offsets."""
import math

import pytest
import torch

import chunk_routed_sparse_b200 as moc
import moc_workloads as W
import oracle.rows as R
import oracle.window as OW

pytestmark = pytest.mark.gpu
U = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    moc.check_window_error()


def _rand(*shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def _clip(B, frames, rows, cols):
    """Time, row and column of every token, int32 [3, L]."""
    t, r, c = torch.meshgrid(torch.arange(frames), torch.arange(rows), torch.arange(cols), indexing="ij")
    return torch.stack([t, r, c]).reshape(3, -1).to(torch.int32).cuda()


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_projection_to_window_attention_and_back():
    """O and the gradients of the projection and of both weights against the fp64 chain.
    Q, K, V, the weights p, O, ds, the three gradients and dqkv are each rounded to bf16
    once: ten independent errors of at most u in the 2-norm, none amplified by more than
    two (a softmax's and a norm's derivatives are contractions of their inputs' relative
    errors at these sizes): 20 u, and for O, behind five of them, 10 u."""
    B, Hq, Hk, d, axes = 1, 4, 2, 64, (24, 20, 20)
    pos = _clip(B, 5, 12, 9)
    L = pos.shape[1]
    rope = moc.Rope(64, axes=axes)
    freq, axis, f = R.frequencies(axes)
    qkv = _rand(B, L, Hq + 2 * Hk, d, seed=1).requires_grad_()
    wq = (1 + 0.1 * _rand(d, seed=2, dtype=torch.float32)).requires_grad_()
    wk = (1 + 0.1 * _rand(d, seed=3, dtype=torch.float32)).requires_grad_()
    g = _rand(B, Hq, L, d, seed=4)
    args = (108, 108, 20, False)
    Q, K, V = moc.qkv_norm_rope(qkv, Hq, Hk, wq, wk, rope, pos)
    O = moc.window_attention(Q, K, V, *args)
    O.backward(g)
    # the same chain in fp64
    x = qkv.detach().transpose(1, 2)
    ang = R.angles(freq, axis, pos[None], B, L)
    q, k = (R.norm_rope(x[:, a:b], w.detach(), 1e-6, ang, f, True) for a, b, w in ((0, Hq, wq), (Hq, Hq + Hk, wk)))
    ref = OW.attention(q, k, x[:, Hq + Hk:].double(), *args, dO=g)
    assert _rel(O.detach(), ref["O"]) <= 10 * U
    dq, dwq, _, _ = R.norm_rope_bwd(x[:, :Hq], wq.detach(), 1e-6, ang, f, True, ref["dQ"])
    dk, dwk, _, _ = R.norm_rope_bwd(x[:, Hq:Hq + Hk], wk.detach(), 1e-6, ang, f, True, ref["dK"])
    want = torch.cat([dq, dk, ref["dV"]], 1).transpose(1, 2)
    for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)):
        assert _rel(qkv.grad[:, :, a:b], want[:, :, a:b]) <= 20 * U
    assert _rel(wq.grad, dwq) <= 20 * U and _rel(wk.grad, dwk) <= 20 * U
    # and the raw calls are what autograd ran
    with torch.no_grad():
        o, lse = moc.window_attention_fwd(Q, K, V, *args)
        grads = moc.window_attention_bwd(Q, K, V, o, lse, g, *args)
        dqkv, rwq, rwk = moc.qkv_norm_rope_bwd(qkv.detach(), Hq, Hk, wq.detach(), wk.detach(), rope, pos, 1e-6, *grads)
    assert torch.equal(o, O) and torch.equal(dqkv, qkv.grad) and torch.equal(rwq, wq.grad) and torch.equal(rwk, wk.grad)


def test_projection_to_routed_attention_and_back():
    """The same front end feeding the routed attention: autograd through both is the raw calls, bit for bit."""
    wl = W.tiny()
    B, H, L, d = wl.B, wl.H, wl.L, wl.d
    lay = moc.Layout.from_workload(wl)
    rope = moc.Rope(64, axes=(24, 20, 20))
    i = torch.arange(L, dtype=torch.int32, device="cuda")
    pos = torch.stack([i // 256, (i % 256) // 16, i % 16])
    qkv = _rand(B, L, 3 * H, d, seed=11).requires_grad_()
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16).requires_grad_()
    Q, K, V = moc.qkv_norm_rope(qkv, H, H, w, w, rope, pos)
    O = moc.moc_attention(lay, Q, K, V, wl.k, wl.causal)
    g = _rand(B, H, L, d, seed=12)
    O.backward(g)
    with torch.no_grad():
        o, lse, sel, _ = moc.forward(lay, Q, K, V, wl.k, wl.causal)
        grads = moc.attention_bwd(lay, Q, K, V, o, lse, g, sel, wl.k)
        dqkv, a, b = moc.qkv_norm_rope_bwd(qkv.detach(), H, H, w.detach(), w.detach(), rope, pos, 1e-6, *grads)
    assert torch.equal(O, o) and torch.equal(qkv.grad, dqkv)
    assert torch.equal(w.grad, a + b)


def test_a_stream_of_new_tokens_against_its_cache():
    """A prompt, then tokens one and three at a time: keys and values written to their
    cache slots by the front end, attention over the cache up to the present length - the
    rows of the whole stream's attention at once. The two kernels round the same weights
    (u + 2^-11 of them) and the result once."""
    B, Hq, Hk, d, cap, n0 = 2, 8, 2, 128, 900, 600
    rope = moc.Rope(d, interleaved=False, scaling="yarn", factor=4.0, original_length=256)
    w = 1 + 0.1 * _rand(d, seed=20, dtype=torch.float32)
    steps = [n0, 1, 1, 3, 1, 2]
    total = sum(steps)
    qkv = _rand(B, total, Hq + 2 * Hk, d, seed=21)
    win = (150, 0, 10, True)
    kc, vc = (torch.full((B, Hk, cap, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    outs, at = [], 0
    for n in steps:
        x = qkv[:, at:at + n].transpose(1, 2)
        pos = torch.arange(at, at + n, device="cuda", dtype=torch.int32)
        q = torch.empty(B, Hq, n, d, device="cuda", dtype=torch.bfloat16)
        moc.qk_norm_rope_fwd(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], w, w, rope, pos,
                             out=(q, kc[:, :, at:at + n], vc[:, :, at:at + n]))
        at += n
        lens = torch.full((B,), at, device="cuda", dtype=torch.int32)
        outs.append(moc.window_attention_fwd(q, kc, vc, *win, kv_len=lens)[0])
    Q, K, V = moc.qkv_norm_rope(qkv, Hq, Hk, w, w, rope)
    assert torch.equal(kc[:, :, :total], K) and torch.equal(vc[:, :, :total], V)
    assert kc[:, :, total:].isnan().all()
    ref = OW.attention(Q, K, V, *win)
    got = torch.cat(outs, 2).double()
    tol = U * ref["O"].abs() + (U + 2.0 ** -11) * ref["sO"]
    assert ((got - ref["O"]).abs() <= tol).all()


def test_calls_on_two_streams_at_once():
    a = [_rand(1, 6, 3000, 128, seed=30 + i) for i in range(4)]
    b = [_rand(2, 4, 1500, 128, seed=40 + i) for i in range(4)]

    def step(t, args):
        o, lse = moc.window_attention_fwd(*t[:3], *args)
        return (o, lse, *moc.window_attention_bwd(*t[:3], o, lse, t[3], *args))

    wa, wb = (400, 0, 130, True), (64, 64, 3, False)
    want = step(a, wa), step(b, wb)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for st, t, args in zip(s, (a, b), (wa, wb)):
            with torch.cuda.stream(st):
                got.append(step(t, args))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, want[i % 2]):
            assert torch.equal(x, y)


def test_padded_batches_on_two_streams_and_in_a_graph():
    """Their row tiles go to CTAs as these become free: in another order every time, with
    the same bits, next to another call or replayed."""
    L = [2501, 1900]
    lens = [torch.tensor(x, device="cuda", dtype=torch.int32) for x in ([2501, 0, 1311], [3, 1900, 1024, 127])]
    t = [[_rand(len(n), 12, l, 64, seed=70 + 4 * i + j) for j in range(4)] for i, (n, l) in enumerate(zip(lens, L))]
    args = [(700, 0, 5, True), (64, 64, 300, False)]

    def step(i):
        q, k, v, g = t[i]
        o, lse = moc.window_attention_fwd(q, k, v, *args[i], lens[i], lens[i])
        return (o, lse, *moc.window_attention_bwd(q, k, v, o, lse, g, *args[i], lens[i], lens[i]))

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, step(i)))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(0)
    for _ in range(3):
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want[0]))
    moc.check_window_error()


def test_two_graphs_that_share_a_workspace():
    Q, K, V, g = (_rand(1, 4, 2000, 64, seed=50 + i) for i in range(4))
    cases = [(300, 0, 140, True), (40, 0, 7, True)]
    n = max(moc.lib().moc_window_attention_bwd_workspace_bytes(1, 4, 4, 2000, 2000, 64, *c[:3], 1) for c in cases)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, held, want, kept = [], [], [], []
    for c in cases:
        o, lse = moc.window_attention_fwd(Q, K, V, *c)
        kept.append((o, lse))  # the graphs read them
        want.append(moc.window_attention_bwd(Q, K, V, o, lse, g, *c))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(moc.window_attention_bwd(Q, K, V, o, lse, g, *c, ws=ws))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1, 0):
        for t in held[i]:
            t.zero_()
        ws.fill_(0xff)  # nothing of the last run is needed
        graphs[i].replay()
        torch.cuda.synchronize()
        for x, y in zip(held[i], want[i]):
            assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """24 heads of a cache of 2^20 slots: element offsets up to 3.2e9; and a token-major
    projection of 3.4e9 elements."""
    H, cap, d = 24, 1 << 20, 128
    K, V = (torch.zeros(1, H, cap, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    n = cap - 5
    K[:, :, n - 300:n], V[:, :, n - 300:n] = _rand(1, H, 300, d, seed=60), _rand(1, H, 300, d, seed=61)
    K[:, :, :4], V[:, :, :4] = _rand(1, H, 4, d, seed=62), _rand(1, H, 4, d, seed=63)
    kl = torch.tensor([n], device="cuda", dtype=torch.int32)
    for Lq in (1, 200):  # the few-row and the many-row kernel
        Q = _rand(1, H, Lq, d, seed=64)
        O, lse = moc.window_attention_fwd(Q, K, V, 99, 0, 4, True, None, kl)
        k = torch.cat([K[:, :, :4], K[:, :, n - 300:n]], 2)
        v = torch.cat([V[:, :, :4], V[:, :, n - 300:n]], 2)
        ref = OW.attention(Q, k, v, 99, 0, 4, True)  # the last 300 tokens hold both windows; first keys in front
        tol = U * ref["O"].abs() + (U + 2.0 ** -11) * ref["sO"]
        assert ((O.double() - ref["O"]).abs() <= tol).all()
    del K, V
    L, heads = 370000, 72
    qkv = torch.empty(1, L, heads, d, device="cuda", dtype=torch.bfloat16)
    qkv[:, -3:] = _rand(1, 3, heads, d, seed=65)
    qkv[:, :-3] = 0
    rope = moc.Rope(d)
    Q, K, V = moc.qkv_norm_rope(qkv, 24, 24, None, None, rope)
    pos = torch.arange(L - 3, L, device="cuda", dtype=torch.int32)
    small = moc.qkv_norm_rope(qkv[:, -3:], 24, 24, None, None, rope, pos)
    for x, y in zip((Q, K, V), small):
        assert torch.equal(x[:, :, -3:], y) and (x[:, :, :-3] == 0).all()


def test_kernels_that_start_early_wait_for_all_that_they_depend_on():
    """Front end, attention and gradients on two streams that fork and join, buffers
    overwritten right before and right after, eagerly and in a captured graph: the same
    bits as one call after the other."""
    B, Hq, Hk, L, d = 2, 8, 4, 1300, 64
    rope = moc.Rope(d, interleaved=False)
    w = 1 + 0.1 * _rand(d, seed=60, dtype=torch.float32)
    src = [_rand(B, L, Hq + 2 * Hk, d, seed=61 + i) for i in range(2)]
    up = _rand(B, Hq, L, d, seed=64)
    args = (200, 0, 140, True)
    qkv, half = torch.empty_like(src[0]), torch.empty_like(src[0])

    def chain(x):
        Q, K, V = moc.qkv_norm_rope(x, Hq, Hk, w, w, rope)
        O, lse = moc.window_attention_fwd(Q, K, V, *args)
        g = moc.window_attention_bwd(Q, K, V, O, lse, up, *args)
        return (O, lse, *g, *moc.qkv_norm_rope_bwd(x, Hq, Hk, w, w, rope, None, 1e-6, *g))

    want = []
    for s in src:
        torch.cuda.synchronize()
        out = []
        for step in range(2):
            out.append([t.clone() for t in chain(s if step == 0 else s * 0.5)])
            torch.cuda.synchronize()
        want.append(out)
    other = torch.cuda.Stream()

    def both(x):
        qkv.copy_(x)
        torch.mul(qkv, 0.5, out=half)
        other.wait_stream(torch.cuda.current_stream())
        a = chain(qkv)
        with torch.cuda.stream(other):
            b = chain(half)
        torch.cuda.current_stream().wait_stream(other)
        joined = moc.window_attention_fwd(a[2], b[3], b[4], *args)  # from both streams' last kernels
        qkv.zero_()
        half.zero_()
        return (*a, *b, *joined)

    joined = []
    for i, x in enumerate(src):
        (dq, dk, dv) = want[i][0][2], want[i][1][3], want[i][1][4]
        joined.append([t.clone() for t in moc.window_attention_fwd(dq, dk, dv, *args)])
    torch.cuda.synchronize()

    def check(got, i):
        torch.cuda.synchronize()
        for x, y in zip(got, (*want[i][0], *want[i][1], *joined[i])):
            assert torch.equal(x, y)

    for r in range(6):
        check(both(src[r & 1]), r & 1)
    x = src[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(x)
    for r in range(6):
        x.copy_(src[r & 1])
        for t in held:
            t.zero_()
        graph.replay()
        if r % 3 == 2:
            graph.replay()  # one right after the other
        check(held, r & 1)
    moc.check_window_error()
