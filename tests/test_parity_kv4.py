"""The 4-bit cache: append and read bit for bit, decode against the 64-bit form."""

import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu

fa = pytest.importorskip("io_aware_exact_forward_b200")


def _rand(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _filled(B, Hkv, Tk, d, seed):
    """A cache of quantised rows (keys with offsets by channel), and its values in 64 bits."""
    k = (_rand((B, Hkv, Tk, d), seed).float() + _rand((Hkv, 1, d), seed + 1).float()).to(torch.bfloat16)
    v = _rand((B, Hkv, Tk, d), seed + 2)
    cache = fa.KV4Cache(*(t.cuda() for x in (k, v) for t in P.pack4(x)))
    return cache, P.values4(cache.k_codes, cache.k_params), P.values4(cache.v_codes, cache.v_params)


@pytest.mark.parametrize("B,T,Hkv,d,Tk,start,count", [
    (1, 1, 1, 64, 64, [0], None),
    (3, 1, 8, 128, 192, [0, 77, 191], None),
    (2, 50, 2, 64, 128, [3, 100], None),            # the second runs past the cache's end
    (2, 50, 3, 128, 128, [-10, 60], [50, 17]),      # the first begins before it
    (2, 5, 2, 128, 64, [1, 2], [0, 9]),             # nothing of the first; a count above T
    (1, 700, 4, 64, 704, [4], None),
])
def test_append_and_read(B, T, Hkv, d, Tk, start, count):
    k, v = _rand((B, T, Hkv, d), 1), _rand((B, T, Hkv, d), 2)
    k[:, :, :, 0] *= 30          # an outlier channel
    k[0, 0, 0, :32] = 1.5        # a group of one value: step 0
    v[0, 0, 0, :32] = 0
    cache = fa.kv4_cache(B, Hkv, Tk, d)
    for t in cache:
        t.view(torch.uint8).fill_(0xA5)
    before = [t.cpu().clone() for t in cache]
    fa.kv4_append(k.cuda(), v.cuda(), cache, _i32(start), None if count is None else _i32(count))
    assert fa.check() == 0
    want = [t.clone() for t in before]
    for b in range(B):
        for t in range(min(T, T if count is None else count[b])):
            at = start[b] + t
            if 0 <= at < Tk:
                for x, c, p in ((k, 0, 1), (v, 2, 3)):
                    want[c][b, :, at], want[p][b, :, at] = P.pack4(x[b, t])
    for got, w in zip(cache, want):
        assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8))
    rk, rv = fa.kv4_read(cache, _i32(start), T, None if count is None else _i32(count))
    assert fa.check() == 0
    for got, codes, params in ((rk, want[0], want[1]), (rv, want[2], want[3])):
        ref = torch.zeros((B, T, Hkv, d), dtype=torch.float64)
        vals = P.values4(codes, params)[0]
        for b in range(B):
            for t in range(min(T, T if count is None else count[b])):
                if 0 <= start[b] + t < Tk:
                    ref[b, t] = vals[b, :, start[b] + t]
        assert torch.equal(got.cpu(), ref.float().to(torch.bfloat16))


def test_append_takes_slices_and_odd_values():
    """k and v out of a packed projection; the largest bf16 values, denormals,
    NaN and infinities keep to their group."""
    B, T, Hkv, d = 2, 3, 2, 64
    x = _rand((B, T, 4 + 2 * Hkv, d), 3)
    big = torch.finfo(torch.bfloat16).max
    x[0, 0, 4, :32] = (torch.linspace(-1, 1, 32) * big).to(torch.bfloat16)
    x[0, 1, 4, :32] = torch.arange(32).to(torch.bfloat16) * 2.0 ** -133
    x[0, 2, 4, 5] = float("nan")
    x[1, 0, 4, 40] = float("inf")
    x[1, 1, 4, :32] = 100 + torch.arange(32) * 0.5          # a range far smaller than the offset
    dev = x.cuda()
    k, v = dev[:, :, 4:4 + Hkv], dev[:, :, 4 + Hkv:]
    a, b = fa.kv4_cache(B, Hkv, 64, d), fa.kv4_cache(B, Hkv, 64, d)
    fa.kv4_append(k, v, a, _i32([0, 9]))
    fa.kv4_append(k.contiguous(), v.contiguous(), b, _i32([0, 9]))
    ra, rb = fa.kv4_read(a, _i32([0, 9]), T), fa.kv4_read(b, _i32([0, 9]), T)
    assert fa.check() == 0
    for m, n in zip(ra, rb):
        assert torch.equal(m.view(torch.int16), n.view(torch.int16))
    got = ra[0].cpu()
    fine = torch.isfinite(got)
    bad = torch.zeros_like(fine)
    bad[0, 2, 0, :32] = True
    bad[1, 0, 0, 32:] = True
    assert torch.equal(fine, ~bad)
    c, s, z = P.split4(x[:, :, 4:4 + Hkv])
    val = (s.double().repeat_interleave(32, -1) * (c - 8) + z.double().repeat_interleave(32, -1))
    assert torch.equal(got[fine], val[fine].float().to(torch.bfloat16))
    # half a step, and the roundings of step and centre, from the input
    xs = x[:, :, 4:4 + Hkv].double()
    step = s.double().repeat_interleave(32, -1)
    lim = (0.5 + 8 * P.H) * step + 2 * P.H * z.double().abs().repeat_interleave(32, -1) + P.H * val.abs() + 2.0 ** -133
    assert bool(((got.double() - xs).abs() <= lim)[fine].all())


DECODE = [
    # Hq, Hkv, d, Tk, W, S, seqlens
    (1, 1, 64, 64, 0, 0, [1]),
    (8, 2, 128, 1024, 0, 0, [0, 1, 15, 16, 63, 64, 65, 128, 1000, 1024]),
    (4, 4, 64, 576, 0, 0, [575, 576, 3, 512]),
    (16, 2, 128, 704, 0, 0, [700, 129]),
    (8, 4, 64, 704, 0, 0, [700, 129]),
    (8, 2, 128, 1024, 300, 4, [0, 1, 4, 255, 304, 305, 1000]),
    (4, 4, 64, 1024, 1, 1, [1, 2, 64, 65, 777]),
    (8, 1, 64, 1024, 64, 130, [1000, 129, 128, 127]),
    (16, 2, 128, 1024, 513, 0, [3, 1000, 513, 514]),
    (2, 2, 128, 1024, 5000, 70, [1, 63, 64, 65, 500]),
    (8, 1, 64, 64, 16, 4, [1 << 20, -5]),                 # lengths outside the cache are clamped
    (32, 8, 128, 4096, 0, 0, [4096, 2049, 31]),
]


@pytest.mark.parametrize("Hq,Hkv,d,Tk,W,S,seqlens", DECODE)
def test_decode(Hq, Hkv, d, Tk, W, S, seqlens):
    B = len(seqlens)
    cache, (kv, _), (vv, vp) = _filled(B, Hkv, Tk, d, 60 + W + d)
    q = _rand((B, Hq, d), 61)
    lens = [min(max(n, 0), Tk) for n in seqlens]
    for b, n in enumerate(lens):
        # rows that the query does not see hold NaN steps and centres
        lo = max(0, n - W) if W else 0
        for p in (cache.k_params, cache.v_params):
            p[b, :, n:] = float("nan")
            p[b, :, min(S, lo):lo] = float("nan")
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32(seqlens), window=W or None, sinks=S)
    assert fa.check() == 0
    ref, tol, rl = P.decode(q, kv, vv, vp, lens, W, S, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)
    o2, lse2 = fa.kv4_decode(q.cuda(), cache, _i32(seqlens), window=W or None, sinks=S)
    assert torch.equal(o, o2) and torch.equal(lse, lse2), "the same inputs give the same bits"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scales", [
    [1e-6], [1e4], [3e4, 1.0], [1e-3, 1e3],       # per third of the sequence, values of V
    [1.0, 300.0, 1e5], [1e5, 300.0, 1.0], [1e-12, 1e-9, 1e-10],
])
def test_decode_value_ranges(d, scales):
    """Values of other sizes, growing and falling along the sequence: the
    probabilities' scaling follows them."""
    Hkv, Hq, Tk = 2, 8, 704
    k = _rand((1, Hkv, Tk, d), 90)
    f = torch.tensor([scales[min(len(scales) - 1, 3 * i // Tk * len(scales) // 3)] for i in range(Tk)])
    v = (_rand((1, Hkv, Tk, d), 91).float() * f[:, None]).to(torch.bfloat16)
    cache = fa.KV4Cache(*(t.cuda() for x in (k, v) for t in P.pack4(x)))
    q = (_rand((1, Hq, d), 92).float() * 2).to(torch.bfloat16)
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32([700]))
    assert fa.check() == 0
    vv, vp = P.values4(cache.v_codes, cache.v_params)
    ref, tol, rl = P.decode(q, P.values4(cache.k_codes, cache.k_params)[0], vv, vp, [700], 0, 0, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)


def test_decode_query_ranges():
    """Rows of q of very different sizes, zero, and with a NaN or an infinity."""
    cache, (kv, _), (vv, vp) = _filled(1, 1, 128, 128, 95)
    q = _rand((1, 8, 128), 96).float()
    q[0, 1] *= 1e-20
    q[0, 2] = 0
    q[0, 3] *= torch.logspace(0, -12, 128)      # 40 binades within a row
    q[0, 4, 7] = float("nan")
    q[0, 5, 9] = float("inf")
    q[0, 6] *= 5
    q = q.to(torch.bfloat16)
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32([128]))
    assert fa.check() == 0
    rows = [0, 1, 2, 3, 6, 7]
    ref, tol, rl = P.decode(q[:, rows], kv, vv, vp, [128], 0, 0, 128 ** -0.5)
    P.check(o[:, rows], ref, tol, "O")
    P.check_lse(lse[:, rows], rl)
    assert bool(torch.isnan(o[0, [4, 5]].float()).all()) and bool(torch.isnan(lse[0, [4, 5]]).all())


def test_decode_many_sequences():
    """More sequences than a block plans at once."""
    B, Hkv, d, Tk = 1500, 1, 64, 64
    cache, (kv, _), (vv, vp) = _filled(B, Hkv, Tk, d, 70)
    q = _rand((B, 2, d), 71)
    lens = [i * 7 % 65 for i in range(B)]
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32(lens))
    assert fa.check() == 0
    ref, tol, rl = P.decode(q, kv, vv, vp, lens, 0, 0, d ** -0.5)
    P.check(o, ref, tol, "O")
    P.check_lse(lse, rl)


def test_decode_on_its_own_stream_and_in_graphs():
    """Two graphs over one cache, replayed in turn after its contents changed,
    and a call on a side stream."""
    B, Hkv, Hq, d, Tk = 3, 2, 8, 128, 1024
    cache, _, _ = _filled(B, Hkv, Tk, d, 80)
    q1, q2 = _rand((B, Hq, d), 81).cuda(), _rand((B, Hq, d), 82).cuda()
    lens = _i32([1000, 5, 640])
    fa.kv4_decode(q1, cache, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s1 = fa.kv4_decode(q1, cache, lens)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for q in (q1, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.kv4_decode(q, cache, lens))
        graphs.append(g)
    lens.copy_(_i32([17, 1024, 0]))
    cache.v_codes.copy_(cache.v_codes.flip(0))
    for _ in range(2):
        for g in graphs:
            g.replay()
    want = [fa.kv4_decode(q, cache, lens) for q in (q1, q2)]
    assert fa.check() == 0
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(torch.isfinite(s1[0].float()).all())


def test_bad_calls():
    cache = fa.kv4_cache(2, 2, 64, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = _i32([1, 1])
    for bad in (dict(q=q[:1]), dict(q=q[:, :3]), dict(seqlens=n[:1]), dict(sinks=2000, window=4),
                dict(out=q[:, :2]), dict(lse=torch.zeros(1, device="cuda")), dict(scale=float("nan")),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        kw = dict(dict(q=q, cache=cache, seqlens=n), **bad)
        with pytest.raises((ValueError, fa.FAError)):
            fa.kv4_decode(**kw)
    with pytest.raises(TypeError):
        fa.kv4_decode(q, cache, n.long())
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        fa.kv4_append(x[:1], x[:1], cache, n)
    with pytest.raises(ValueError):
        fa.kv4_append(x, x[:, :2], cache, n)
    with pytest.raises(TypeError):
        fa.kv4_append(x, x, cache, None)
    with pytest.raises(ValueError):
        fa.kv4_read(fa.KV4Cache(cache[0], cache[1][:, :, :32], cache[2], cache[3]), n, 1)


def test_empty_calls():
    """No sequences, no rows, no keys."""
    c0 = fa.kv4_cache(0, 2, 64, 64)
    o, lse = fa.kv4_decode(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), c0, _i32([]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    c1 = fa.kv4_cache(2, 2, 0, 64)
    o, lse = fa.kv4_decode(torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda"), c1, _i32([0, 3]))
    assert not o.any() and bool(torch.isneginf(lse).all())
    c2 = fa.kv4_cache(2, 2, 64, 64)
    x = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    fa.kv4_append(x, x, c2, _i32([0, 0]))
    k, v = fa.kv4_read(c2, _i32([0, 0]), 0)
    assert k.shape == (2, 0, 2, 64)
    k, v = fa.kv4_read(c1, _i32([0, 0]), 3)
    assert not k.any() and not v.any()
    assert fa.check() == 0


def test_append_and_read_in_a_graph():
    B, T, Hkv, d, Tk = 2, 3, 2, 128, 128
    x = _rand((B, T, Hkv, d), 83).cuda()
    start, count = _i32([5, 60]), _i32([3, 2])
    cache = fa.kv4_cache(B, Hkv, Tk, d)
    fa.kv4_append(x, x, cache, start, count)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.kv4_append(x, x, cache, start, count)
        k, v = fa.kv4_read(cache, start, T, count)
    for b in range(2):  # the second replay appends behind the first's rows
        x.copy_(_rand((B, T, Hkv, d), 84 + b))
        g.replay()
        values, _ = P.values4(*(t.cuda() for t in P.pack4(x.cpu().transpose(1, 2).contiguous())))
        want = values.transpose(1, 2).to(torch.bfloat16)
        want[1, 2] = 0
        assert torch.equal(k.cpu(), want.cpu()) and torch.equal(v.cpu(), want.cpu())
        start += 3
    assert fa.check() == 0


def test_offsets_past_32_bits():
    """The last sequence of a cache whose codes alone pass 2^31 bytes, with all
    rows but its last ones unwritten."""
    B, Hkv, Tk, d, n = 66, 8, 65536, 128, 300
    cache = fa.kv4_cache(B, Hkv, Tk, d)
    assert cache.k_codes.numel() > 1 << 31
    k, v = _rand((B, n, Hkv, d), 86), _rand((B, n, Hkv, d), 87)
    count = [0] * (B - 1) + [n]
    fa.kv4_append(k.cuda(), v.cuda(), cache, _i32([Tk - n] * B), _i32(count))
    want = [P.values4(*(t.cuda() for t in P.pack4(x[-1:].transpose(1, 2).contiguous()))) for x in (k, v)]
    rk, rv = fa.kv4_read(cache, _i32([Tk - n] * B), n, _i32(count))
    for x, (y, _) in zip((rk, rv), want):
        assert torch.equal(x[-1:].cpu(), y.transpose(1, 2).to(torch.bfloat16).cpu())
    q = _rand((B, 16, d), 88)
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32([0] * (B - 1) + [Tk]), window=n)
    assert fa.check() == 0
    assert not o[:-1].any() and bool(torch.isneginf(lse[:-1]).all())
    (kv, _), (vv, vp) = want
    ref, tol, rl = P.decode(q[-1:], kv, vv, vp, [n], 0, 0, d ** -0.5)
    P.check(o[-1:], ref, tol, "O")
    P.check_lse(lse[-1:], rl)


def _appended(k, v):
    """A cache filled by append from bf16 k, v [1,Hkv,T,d], and its values."""
    _, Hkv, T, d = k.shape
    cache = fa.kv4_cache(1, Hkv, T, d)
    fa.kv4_append(k.transpose(1, 2).contiguous().cuda(), v.transpose(1, 2).contiguous().cuda(), cache, _i32([0]))
    return cache, P.values4(cache.k_codes, cache.k_params)[0], P.values4(cache.v_codes, cache.v_params)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [
    # values of V in the first half of the keys, those of the second, by group
    (None, 1.0), (None, 1e30), (1e30, None), (1e-30, 1e30), (1e30, 1e-30), (None, 1e-30), (1e-30, None), (1e33, 1.0)])
def test_decode_lse_does_not_depend_on_v(d, first):
    """Constant groups (steps of 0), very small and very large steps one after the
    other: the denominator and LSE keep every key."""
    Hkv, Hq, Tk = 1, 8, 704
    k, v = _rand((1, Hkv, Tk, d), 97), _rand((1, Hkv, Tk, d), 98).float()
    for x, at in zip(first, (slice(0, 352), slice(352, 704))):
        v[:, :, at] = 0.75 if x is None else v[:, :, at] * x
    cache, kv, (vv, vp) = _appended(k, v.to(torch.bfloat16))
    q = _rand((1, Hq, d), 99)
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32([700]))
    assert fa.check() == 0
    ref, tol, rl = P.decode(q, kv, vv, vp, [700], 0, 0, d ** -0.5)
    P.check_lse(lse, rl)
    P.check(o, ref, tol, "O")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("key", [3, 500])
@pytest.mark.parametrize("x", [float("inf"), float("-inf"), float("nan"), 3e38, 1e30, -1e12])
def test_decode_keeps_a_group_s_values_to_itself(d, key, x):
    """An infinity, a NaN or a very large value in one group of a visible row of
    V: the other groups of that head are as without it."""
    Hkv, Hq, Tk, g = 2, 8, 704, 1
    k, v = _rand((1, Hkv, Tk, d), 100), _rand((1, Hkv, Tk, d), 101)
    v[0, 1, key, 32 * g + 7] = x
    cache, kv, (vv, vp) = _appended(k, v)
    q = _rand((1, Hq, d), 102)
    o, lse = fa.kv4_decode(q.cuda(), cache, _i32([700]))
    assert fa.check() == 0
    hit = torch.zeros(1, Hq, d, dtype=torch.bool)
    hit[0, Hq // 2:, 32 * g:32 * g + 32] = True
    if abs(x) < float("inf"):
        ref, tol, rl = P.decode(q, kv, vv, vp, [700], 0, 0, d ** -0.5)
        P.check(o, ref, tol, "O")
    else:
        assert not bool(torch.isfinite(o.cpu()[hit]).any())
        vv[0, 1, key, 32 * g:32 * g + 32] = vp[0, 1, key, 32 * g:32 * g + 32] = 0
        ref, tol, rl = P.decode(q, kv, vv, vp, [700], 0, 0, d ** -0.5)
        P.check(o.cpu()[~hit], ref[~hit], tol[~hit], "O")
    P.check_lse(lse, rl)
