"""Sliding window with sinks: forward, backward (default and deterministic) and
decode against the 64-bit form."""

import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu

fa = pytest.importorskip("io_aware_exact_forward_b200")


def _rand(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


CASES = [
    # B, Hq, Hkv, Tq, Tk, d, W, sinks
    (1, 1, 1, 1, 1, 64, 1, 1),
    (1, 2, 2, 300, 300, 64, 1, 1),            # the diagonal key and one sink
    (1, 2, 1, 517, 517, 64, 100, 4),          # sink tile beside window tiles, ragged tail, GQA 2
    (1, 2, 2, 384, 384, 128, 128, 128),       # sinks of exactly one tile
    (2, 4, 2, 517, 517, 128, 200, 130),       # sinks into a second tile
    (1, 2, 2, 200, 450, 64, 130, 3),          # Tq < Tk
    (1, 2, 2, 450, 200, 128, 64, 5),          # Tq > Tk: early rows see no key
    (1, 4, 1, 640, 640, 64, 1000, 7),         # window wider than the sequence
    (1, 8, 1, 512, 512, 64, 257, 1024),       # more sinks than keys, G = 8
    (1, 1, 1, 1500, 1500, 128, 64, 2),        # sink tile in pieces (12 query tiles, 4 each)
    (1, 2, 1, 1100, 2300, 64, 60, 200),       # pieces of two sink tiles, Tq < Tk
]


def _inputs(B, Hq, Hkv, Tq, Tk, d, W, S):
    s = 17 + Tq + 3 * Tk + d + W + 5 * S
    return (_rand((B, Tq, Hq, d), s), _rand((B, Tk, Hkv, d), s + 1), _rand((B, Tk, Hkv, d), s + 2),
            _rand((B, Tq, Hq, d), s + 3))


@pytest.mark.parametrize("B,Hq,Hkv,Tq,Tk,d,W,S", CASES)
def test_sink_forward(B, Hq, Hkv, Tq, Tk, d, W, S):
    q, k, v, _ = _inputs(B, Hq, Hkv, Tq, Tk, d, W, S)
    o, lse = fa.forward(q.cuda(), k.cuda(), v.cuda(), window=W, sinks=S)
    assert fa.check() == 0
    ref, tol, rl = P.sink_forward(q, k, v, W, S, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,Tk,d,W,S", CASES)
def test_sink_backward(B, Hq, Hkv, Tq, Tk, d, W, S, deterministic):
    q, k, v, do = _inputs(B, Hq, Hkv, Tq, Tk, d, W, S)
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    got = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=deterministic)
    assert fa.check() == 0
    ref = P.sink_backward(q, k, v, do, W, S, d ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        P.check(x, *ref[n], n)
    if deterministic:
        again = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=True)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,Tk,d,W,S", [
    (2, 32, 32, 300, 700, 64, 40, 3),         # key tiles that no query sees among a block's items
    (3, 20, 20, 520, 520, 64, 130, 140),
    (2, 40, 20, 640, 640, 128, 60, 5),
])
def test_sink_backward_many_items(B, Hq, Hkv, Tq, Tk, d, W, S, deterministic):
    """More work items than multiprocessors: blocks walk several."""
    q, k, v, do = _inputs(B, Hq, Hkv, Tq, Tk, d, W, S)
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    got = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=deterministic)
    assert fa.check() == 0
    fo, ft, fl = P.sink_forward(q, k, v, W, S, d ** -0.5)
    P.check(o, fo, ft, "O")
    P.check_lse(lse, fl)
    ref = P.sink_backward(q, k, v, do, W, S, d ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        P.check(x, *ref[n], n)


def test_sink_gradient_against_differences():
    """Directional derivatives of L = sum(dO * O): the 64-bit loss's central
    difference along u against the kernel's gradients."""
    B, Hq, Hkv, T, d, W, S = 1, 4, 2, 300, 64, 40, 3
    q, k, v, do = _inputs(B, Hq, Hkv, T, T, d, W, S)
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    got = dict(zip("qkv", fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S)))
    tol = P.sink_backward(q, k, v, do, W, S, d ** -0.5)
    G = do.double()

    def loss(q, k, v):
        return float((P.sink_forward(q, k, v, W, S, d ** -0.5)[0] * G).sum())

    h = 1e-5
    x = dict(q=q.double(), k=k.double(), v=v.double())
    for n in "qkv":
        u = torch.randn(x[n].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        up, dn = dict(x), dict(x)
        up[n], dn[n] = x[n] + h * u, x[n] - h * u
        diff = (loss(**up) - loss(**dn)) / (2 * h)
        bound = float((tol["d" + n][1] * u.abs()).sum())   # the gradients' own bound, along u
        assert abs(float((got[n].double().cpu() * u).sum()) - diff) <= bound + 1e-3, n   # h^2 term


def test_zero_sinks_is_the_window():
    q, k, v, do = (x.cuda() for x in _inputs(1, 2, 2, 300, 300, 64, 100, 0))
    a, b = fa.forward(q, k, v, window=100), fa.forward(q, k, v, window=100, sinks=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_every_key_visible_is_causal():
    """A window and sinks that leave nothing out: the causal result, bit for bit."""
    q, k, v, _ = (x.cuda() for x in _inputs(1, 2, 2, 500, 500, 128, 400, 120))
    a, b = fa.forward(q, k, v, causal=True), fa.forward(q, k, v, window=400, sinks=120)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sink_forward_persistent_items():
    """More items than SMs: later items of a CTA, and sampled long rows."""
    H, T, d, W, S = 16, 4096, 64, 300, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((1, T, H, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    o, lse = fa.forward(q, k, v, window=W, sinks=S)
    assert fa.check() == 0
    rows = torch.tensor([0, 3, 127, 128, 299, 300, 304, 2047, 2048, 4095])
    mask = P.visible(T, T, W, S)[rows]
    for h in (0, 7, 15):
        Q, K, V = (x[0, :, h].double().cpu() for x in (q, k, v))
        ref, rl, _, a = P.attention(Q[rows], K, V, mask, d ** -0.5)
        P.check(o[0, rows.cuda(), h], ref, (2 * P.H + P.R32) * a + P.H * ref.abs(), f"head {h}")
        P.check_lse(lse[0, h, rows.cuda()], rl)


@pytest.mark.parametrize("Hq,Hkv,d,chunk,W,S,seqlens", [
    (8, 2, 128, 256, 300, 4, [0, 1, 4, 255, 304, 305, 1000]),
    (4, 4, 64, 256, 1, 1, [1, 2, 64, 65, 777]),
    (16, 2, 128, 512, 513, 600, [3, 1000, 513, 514]),    # sinks beyond a chunk
    (2, 2, 64, 64, 5000, 70, [1, 63, 64, 65, 500]),      # wider than every sequence
    (8, 1, 64, 64, 64, 64, [1000, 129, 128, 127]),
    (8, 1, 64, 64, 64, 64, [1 << 20, -5]),               # lengths outside the cache are clamped
])
def test_sink_decode(Hq, Hkv, d, chunk, W, S, seqlens):
    B, Tk = len(seqlens), 1000
    q, k, v = _rand((B, Hq, d), 50 + W), _rand((B, Tk, Hkv, d), 51 + W), _rand((B, Tk, Hkv, d), 52 + W)
    lens = [min(max(n, 0), Tk) for n in seqlens]
    kk, vv = k.cuda(), v.cuda()
    for b, n in enumerate(lens):
        # rows that the query does not see hold NaN
        lo = max(0, n - W)
        for t in (kk, vv):
            t[b, n:] = float("nan")
            t[b, min(S, lo):lo] = float("nan")
    o, lse = fa.decode_splitkv(q.cuda(), kk, vv, torch.tensor(seqlens, dtype=torch.int32).cuda(), chunk=chunk, window=W,
                               sinks=S)
    assert fa.check() == 0
    ref, tol, rl = P.decode(q, k.double().transpose(1, 2), v.double().transpose(1, 2), None, lens, W, S, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)


def test_sink_decode_is_the_last_row_of_the_forward():
    q, k, v = _rand((1, 700, 4, 128), 1), _rand((1, 700, 2, 128), 2), _rand((1, 700, 2, 128), 3)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    o, lse = fa.forward(q, k, v, window=150, sinks=9)
    od, ld = fa.decode_splitkv(q[:, -1].contiguous(), k, v, torch.tensor([700], dtype=torch.int32).cuda(), window=150,
                               sinks=9)
    # each within the bound of the same exact row
    ref, tol, _ = P.sink_forward(q.cpu()[:, -1:], k.cpu(), v.cpu(), 150, 9, 128 ** -0.5)
    P.check(o[:, -1:], ref, tol, "forward")
    P.check(od[:, None], ref, tol, "decode")
    assert float((lse[0, :, -1] - ld[0]).abs().max()) <= 2 * P.LSE_TOL


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("B,Tq,Tk", [(0, 5, 5), (1, 0, 200), (1, 200, 0)])
def test_sink_empty_calls(B, Tq, Tk, deterministic):
    q, do = (torch.ones(B, Tq, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.ones(B, Tk, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o, lse = fa.forward(q, k, v, window=10, sinks=3)
    assert not o.any() and bool(torch.isneginf(lse).all())
    for x in fa.backward(q, k, v, o, lse, do, window=10, sinks=3, deterministic=deterministic):
        assert not x.any()
    assert fa.check() == 0


def test_sink_decode_without_keys():
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.full((2, 64, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.decode_splitkv(q, c, c, torch.zeros(2, dtype=torch.int32, device="cuda"), window=5, sinks=2)
    assert not o.any() and bool(torch.isneginf(lse).all())
    assert fa.check() == 0


def test_sink_decode_many_sequences():
    """More sequences than a block keeps the lengths of."""
    B, T, W, S = 1300, 64, 20, 3
    q, k, v = _rand((B, 2, 64), 61), _rand((B, T, 1, 64), 62), _rand((B, T, 1, 64), 63)
    lens = [i * 7 % 65 for i in range(B)]
    o, lse = fa.decode_splitkv(q.cuda(), k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), chunk=64,
                               window=W, sinks=S)
    assert fa.check() == 0
    ref, tol, rl = P.decode(q, k.double().transpose(1, 2), v.double().transpose(1, 2), None, lens, W, S, 64 ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)


def test_sink_decode_streams_and_graphs():
    """Two graphs with one workspace, replayed in turn after their inputs changed,
    and two calls at once on streams of their own."""
    B, T, W, S = 4, 1000, 300, 5
    k, v = _rand((B, T, 2, 128), 64).cuda(), _rand((B, T, 2, 128), 65).cuda()
    qs = [_rand((B, 8, 128), 66 + i).cuda() for i in range(2)]
    lens = torch.tensor([1000, 3, 305, 0], dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def call(q, **kw):
        return fa.decode_splitkv(q, k, v, lens, window=W, sinks=S, **kw)

    want = [call(q) for q in qs]
    streams, got = [torch.cuda.Stream() for _ in qs], []
    for s, q in zip(streams, qs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(call(q))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(q, workspace=ws))
        graphs.append(g)
    lens.copy_(torch.tensor([17, 1000, 0, 640], dtype=torch.int32))
    k.copy_(k.flip(0))
    for _ in range(2):
        for g in graphs:
            g.replay()
    want = [call(q) for q in qs]
    assert fa.check() == 0
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
def test_sink_training_step_in_a_graph(d):
    T, W, S = 900, 130, 4
    q, do = (_rand((1, T, 4, d), 70 + i).cuda() for i in range(2))
    k, v = (_rand((1, T, 2, d), 72 + i).cuda() for i in range(2))
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")

    def step(**kw):
        o, lse = fa.forward(q, k, v, window=W, sinks=S)
        return (o, lse, *fa.backward(q, k, v, o, lse, do, window=W, sinks=S, deterministic=True, **kw))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(workspace=ws)
    for t in (q, k, v, do):
        t.copy_(t.flip(1))
    ws.fill_(255)
    g.replay()
    want = step()
    assert fa.check() == 0
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("above", [12.0, 16.0, 20.0, 40.0])
def test_sink_backward_where_the_sink_takes_the_weight(above, d, deterministic):
    """The sink's score lies far above the window's, as trained sinks' do: the
    other keys' probabilities are e^-12 to e^-40, and their dK is as exact as any."""
    B, Hq, Hkv, T, W, S = 1, 2, 1, 600, 128, 1
    q, k, v, do = _inputs(B, Hq, Hkv, T, T, d, W, S)
    # the first dim of q is 4, and 0 in every key but the sink's
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, 0, :, 0] = above * d ** 0.5 / 4.0
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    got = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=deterministic)
    assert fa.check() == 0
    ref = P.sink_backward_by_rounding(q, k, v, do, W, S, d ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        P.check(x, *ref[n], n)


@pytest.mark.parametrize("deterministic", [False, True])
def test_sink_workspaces_as_asked_for(deterministic):
    """Workspaces of just the sizes that the library names: the same results, nothing
    written behind them, and one byte less is refused."""
    T, W, S, d = 1500, 64, 200, 64
    q, k, v, do = (x.cuda() for x in _inputs(1, 4, 2, T, T, d, W, S))
    o, lse = fa.forward(q, k, v, window=W, sinks=S)
    need = fa.backward_workspace_bytes(1, 4, 2, T, T, d, window=W, sinks=S)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    kw = dict(window=W, sinks=S, deterministic=deterministic)
    want = fa.backward(q, k, v, o, lse, do, **kw)
    got = fa.backward(q, k, v, o, lse, do, workspace=ws[:need], **kw)
    assert bool((ws[need:] == 0x5A).all())
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])     # dQ's order is free by default
    with pytest.raises(fa.FAError):
        fa.backward(q, k, v, o, lse, do, workspace=ws[:need - 1], **kw)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    need = fa.decode_workspace_bytes(1, 4, T, d, window=W, sinks=S)
    ws.fill_(0x5A)
    a = fa.decode_splitkv(q[:, -1].contiguous(), k, v, lens, window=W, sinks=S)
    b = fa.decode_splitkv(q[:, -1].contiguous(), k, v, lens, window=W, sinks=S, workspace=ws[:need])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool((ws[need:] == 0x5A).all())
    with pytest.raises(fa.FAError):
        fa.decode_splitkv(q[:, -1].contiguous(), k, v, lens, window=W, sinks=S, workspace=ws[:need - 1])
    assert fa.check() == 0


@pytest.mark.parametrize("deterministic", [False, True])
def test_sink_backward_with_many_sink_tiles(deterministic):
    """Eight sink tiles, cut into fewer pieces than one would be."""
    B, Hq, Hkv, T, d, W, S = 1, 1, 1, 2048, 64, 64, 1024
    q, k, v, do = _inputs(B, Hq, Hkv, T, T, d, W, S)
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    got = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=deterministic)
    assert fa.check() == 0
    ref = P.sink_backward(q, k, v, do, W, S, d ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        P.check(x, *ref[n], n)


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_sink_prefill_does_not_read_behind_the_window(d, deterministic):
    """The last 256 rows of a long sequence: key tiles between the sinks' and the
    window's may hold NaN, and K may wherever no row sees it (in the forward)."""
    Tq, Tk, W, S = 256, 2048, 300, 4
    q, k, v, do = _inputs(1, 4, 2, Tq, Tk, d, W, S)
    first = Tk - Tq - W + 1                    # of the window of the first row
    c = [x.cuda() for x in (q, k, v, do)]
    for t in c[1:3]:
        t[:, 128:first // 128 * 128] = float("nan")
    kn = c[1].clone()
    kn[:, S:first] = float("nan")
    o, lse = fa.forward(c[0], kn, c[2], window=W, sinks=S)
    assert fa.check() == 0
    ref, tol, rl = P.sink_forward(q, k, v, W, S, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)
    got = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S, deterministic=deterministic)
    assert fa.check() == 0
    ref = P.sink_backward(q, k, v, do, W, S, d ** -0.5)
    for n, x in zip(("dq", "dk", "dv"), got):
        P.check(x, *ref[n], n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W,S", [(16, 4), (30, 5), (300, 4)])
def test_sink_backward_rounds_once_before_the_products(d, W, S):
    """The error of dQ and dK as a whole is that of dS rounded to bf16 once, D from the
    rounded O, and the result rounded: P reaches dS with more bits than bf16 has, in
    windows of a few keys too.  A rounding to bf16 is off by 2^-8 / sqrt(3) times the root
    mean square of 1 / mantissa, sqrt(0.541) for mantissas spread evenly in their
    logarithm: 0.00166 of the value.  8% are left for other spreads; a second
    rounding, of P, would add 20%."""
    B, H, T, rho = 1, 4, 600, 2.0 ** -8 * (0.541 / 3) ** 0.5
    q, k, v, do = _inputs(B, H, H, T, T, d, W, S)
    c = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*c[:3], window=W, sinks=S)
    dq, dk, _ = fa.backward(*c[:3], o, lse, c[3], window=W, sinks=S)
    assert fa.check() == 0
    Q, K, V, G = (P.split_heads(x, H) for x in (q, k, v, do))
    O, _, w, _ = P.attention(Q, K, V, P.visible(T, T, W, S), d ** -0.5)
    ds = w * (G @ V.transpose(-1, -2) - (G * O).sum(-1, keepdim=True))
    D2 = (G ** 2 * O ** 2).sum(-1, keepdim=True)            # of D's error, in rho
    for got, ref, var in (
            (dq, ds @ K, ds ** 2 @ K ** 2 + D2 * (w @ K) ** 2),
            (dk, ds.transpose(-1, -2) @ Q,
             (ds ** 2).transpose(-1, -2) @ Q ** 2 + (w ** 2 * D2).transpose(-1, -2) @ Q ** 2)):
        ref, var = ref * d ** -0.5, var / d
        err = float((P.split_heads(got, H) - ref).norm())
        want = rho * float((ref ** 2 + var).sum() ** 0.5)
        assert err <= 1.08 * want, (err / float(ref.norm()), want / float(ref.norm()))
