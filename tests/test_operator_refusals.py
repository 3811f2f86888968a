"""Host-side checks of the rotary, sink and 4-bit-cache entry points: bad calls
are refused before anything is launched (no GPU needed)."""

import ctypes
import math

import pytest
import torch

import io_aware_exact_forward_b200 as fa

N = None
INVALID, UNSUPPORTED, ALIGN, WS = 1, 2, 3, 4


@pytest.fixture
def mem():
    buf = (ctypes.c_uint8 * 8192)()
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    yield lambda off=0: ctypes.c_void_p(base + off)
    del buf


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


def test_sink_entry_points():
    lib = fa.load_library()
    f = lambda w, s, d=64, Tq=16: lib.fa_forward_sinks(N, N, N, N, N, 1, 1, 1, Tq, 16, d, 1.0, w, s, N)  # noqa: E731
    assert f(0, 4) == INVALID and f(-1, 4) == INVALID
    assert f(4, -1) == INVALID and f(4, 1025) == INVALID
    assert f(4, 4, d=96) == UNSUPPORTED
    assert f(4, 4) == INVALID            # null pointers
    assert f(4, 4, Tq=0) == 0
    b = lambda w, s, det=0, d=64, B=1: lib.fa_backward_sinks(  # noqa: E731
        *([N] * 9), N, 0, B, 1, 1, 16, 16, d, 1.0, w, s, det, N)
    assert b(0, 4) == INVALID and b(4, -1) == INVALID and b(4, 1025) == INVALID and b(4, 4, det=2) == INVALID
    assert b(4, 4, d=80) == UNSUPPORTED
    assert b(4, 4) == INVALID
    assert b(4, 4, B=0) == 0
    c = lambda w, s: lib.fa_decode_splitkv_sinks(*([N] * 6), N, 0, 2, 32, 8, 1024, 128, 0.1, 256, w, s, N)  # noqa: E731
    assert c(0, 4) == INVALID and c(8, -2) == INVALID and c(8, 1025) == INVALID and c(8, 4) == INVALID
    assert lib.fa_decode_splitkv_sinks(*([N] * 6), N, 0, 2, 32, 2, 1024, 128, 0.1, 256, 8, 4, N) == UNSUPPORTED


def test_sink_backward_workspace(mem):
    lib = fa.load_library()
    base = lib.fa_backward_workspace_bytes(1, 4, 2, 4096, 4096, 64)
    more = lib.fa_backward_sinks_workspace_bytes(1, 4, 2, 4096, 4096, 64, 256, 4)
    # 32 query tiles in pieces of max(4, 256 / 128 + 1) = 4: 8 pieces of one 128-key tile and 2 KV heads
    assert more - base == 2 * 8 * 2 * 128 * 64 * 4
    assert lib.fa_backward_sinks_workspace_bytes(1, 4, 2, 256, 256, 64, 256, 4) == \
        lib.fa_backward_workspace_bytes(1, 4, 2, 256, 256, 64)
    # a workspace that only the plain backward could do with
    args = [mem()] * 9
    assert lib.fa_backward_sinks(*args, mem(), base, 1, 4, 2, 4096, 4096, 64, 1.0, 256, 4, 0, N) == WS
    assert lib.fa_backward_sinks(*args, N, more, 1, 4, 2, 4096, 4096, 64, 1.0, 256, 4, 0, N) == WS


def test_sinks_need_a_window():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="window"):
        fa.forward(q, q, q, sinks=4)
    with pytest.raises(ValueError, match="window"):
        fa.backward(q, q, q, q, q, q, sinks=4)
    with pytest.raises(ValueError, match="window"):
        fa.decode_splitkv(q[0], q, q, q, sinks=4)
    with pytest.raises(ValueError, match="window"):
        fa.kv4_decode(q[0], None, None, sinks=4)


def test_rope_arguments(mem):
    lib = fa.load_library()
    T, H, d = 2, 2, 64
    dense = (T * H * d, H * d, d)
    st = strides(*dense * 4)

    def call(q=0, q_out=1024, k=2048, k_out=3200, st=st, freqs=4096, rot=64, inter=0, amp=1.0, B=1, T=T, Hq=H,
             Hkv=H, d=d, pos=N):
        p = lambda x: N if x is None else mem(x)  # noqa: E731
        return lib.fa_rope(p(q), p(q_out), p(k), p(k_out), st, pos, p(freqs), rot, inter, amp, B, T, Hq, Hkv, d, N)

    assert call(d=96) == UNSUPPORTED
    for rot in (0, 8, 24, 80, -16):
        assert call(rot=rot) == INVALID, rot
    assert call(inter=2) == INVALID
    assert call(amp=math.nan) == INVALID
    assert call(Hq=0, Hkv=0) == INVALID
    assert call(B=-1) == INVALID
    assert call(B=0) == 0 and call(T=0) == 0
    assert call(freqs=None) == INVALID and call(q=None) == INVALID and call(k_out=None) == INVALID
    assert call(st=N) == INVALID
    assert call(q=8) == ALIGN and call(freqs=4100) == ALIGN
    assert call(pos=mem(4098)) == ALIGN
    # the output overlaps its input without being it
    assert call(q_out=256) == INVALID
    # token strides: not a multiple of 8, negative, and outputs whose elements share places
    assert call(st=strides(*dense, *dense, *dense, T * H * d, H * d + 4, d)) == ALIGN
    assert call(st=strides(-8, H * d, d, *dense * 3)) == INVALID
    assert call(st=strides(*dense, 0, 0, d, *dense * 2)) == INVALID
    assert call(st=strides(*dense, T * H * d, d, d, *dense * 2)) == INVALID
    # one output for both; q's output over k; k's output over q
    assert call(k_out=1024) == INVALID and call(q_out=2048) == INVALID and call(k_out=128) == INVALID
    # packed rows of 6 heads: q is heads 0, 1 and k heads 2, 3 of the same rows.  In
    # place and into heads of another packed tensor the ranges interleave, which is
    # no collision: the call gets as far as the device (there is none here)
    row = 6 * d
    packed = strides(*(T * row, row, d) * 4)
    tokens_out = strides(*(row, 2 * row, d) * 4)  # [T, B, heads, d]
    heads_out = strides(*(6 * T * d, d, T * d) * 4)  # [B, heads, T, d]
    if not torch.cuda.is_available():
        for st, k in ((packed, 2 * d * 2), (tokens_out, 2 * d * 2), (heads_out, 2 * T * d * 2)):
            assert call(q=0, q_out=0, k=k, k_out=k, st=st, B=2) != INVALID
            assert call(q=0, q_out=k // 2, k=k, k_out=k, st=st, B=2) == INVALID
            # two heads further
            assert call(q=0, q_out=2 * k, k=k, k_out=k, st=st, B=2) != INVALID
    # heads 1, 2 for k overlap q's heads 0, 1
    assert call(q=0, q_out=0, k=2 * d, k_out=2 * d, st=packed) == INVALID
    # broadcast inputs step by nothing; steps that would leave 64 bits
    assert call(q=0, q_out=0, k=256, k_out=1024, st=strides(*dense * 2, 0, 0, d, *dense), B=2) == INVALID
    assert call(st=strides(*dense * 3, 1 << 60, H * d, d), B=2) == INVALID
    # k's output one token further than k
    assert call(q=0, q_out=0, k=2 * d * 2, k_out=2 * d * 2 + 2 * row, st=packed) == INVALID
    for f in (lib.fa_rope_backward,):
        assert f(N, N, N, N, st, N, mem(0), 64, 0, 1.0, 1, T, H, H, 96, N) == UNSUPPORTED


def test_kv4_arguments(mem):
    lib = fa.load_library()
    st = strides(*(2 * 64, 2 * 64, 64) * 2)

    def append(k=0, v=512, codes=1024, start=2048, count=N, B=1, T=1, Hkv=2, Tk=64, d=64, st=st):
        p = lambda x: N if x is None else mem(x)  # noqa: E731
        return lib.fa_kv4_append(p(k), p(v), st, *([p(codes)] * 4), p(start), count, B, T, Hkv, Tk, d, N)

    assert append(d=96) == UNSUPPORTED
    assert append(Tk=65) == INVALID and append(Tk=-64) == INVALID and append(T=-1) == INVALID
    assert append(Hkv=0) == INVALID and append(T=(1 << 30) + 1) == INVALID
    assert append(B=0) == 0 and append(T=0) == 0 and append(Tk=0) == 0
    assert append(k=None) == INVALID and append(codes=None) == INVALID and append(start=None) == INVALID
    assert append(k=8) == ALIGN and append(codes=1032) == ALIGN and append(start=2049) == ALIGN
    assert append(st=strides(128, 128, 60, 128, 128, 64)) == ALIGN
    assert append(st=strides(-128, 128, 64, 128, 128, 64)) == INVALID

    def read(k=0, codes=1024, start=2048, Tk=64, d=64, T=1):
        p = lambda x: N if x is None else mem(x)  # noqa: E731
        return lib.fa_kv4_read(p(k), p(k), *([p(codes)] * 4), p(start), N, 1, T, 2, Tk, d, N)

    assert read(d=32) == UNSUPPORTED and read(Tk=100) == INVALID and read(T=-2) == INVALID and read(T=0) == 0
    assert read(k=None) == INVALID and read(codes=None) == INVALID and read(start=None) == INVALID
    assert read(k=4) == ALIGN

    def decode(q=0, codes=1024, lens=2048, ws=4096, wsb=1 << 20, B=1, Hq=4, Hkv=2, Tk=64, d=64, scale=1.0, window=0,
               sinks=0):
        p = lambda x: N if x is None else mem(x)  # noqa: E731
        return lib.fa_kv4_decode(p(q), *([p(codes)] * 4), p(lens), p(0), p(0), p(ws), wsb, B, Hq, Hkv, Tk, d, scale,
                                 window, sinks, N)

    assert decode(d=96) == UNSUPPORTED and decode(Hq=6) == UNSUPPORTED and decode(Hq=32) == UNSUPPORTED
    assert decode(Hq=3) == INVALID and decode(Tk=96) == INVALID and decode(scale=math.inf) == INVALID
    assert decode(window=-1) == INVALID and decode(sinks=4) == INVALID and decode(window=4, sinks=1025) == INVALID
    assert decode(B=0) == 0
    assert decode(q=None) == INVALID and decode(lens=None) == INVALID and decode(codes=None) == INVALID
    assert decode(q=4) == ALIGN
    assert decode(ws=None) == WS and decode(wsb=16) == WS and decode(ws=4100) == WS
    assert lib.fa_kv4_decode_workspace_bytes(1, 4, 2, 64, 96) == 0


def test_bindings_refuse():
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(x, x, f)
    with pytest.raises(ValueError, match="q must be"):
        fa.rope(x[0], x[0], f)
    with pytest.raises(ValueError):
        fa.kv4_cache(1, 2, 100, 96, device="cpu")
    c = fa.kv4_cache(1, 2, 100, 64, device="cpu")
    assert c.k_codes.shape == (1, 2, 128, 32) and c.v_params.shape == (1, 2, 128, 4)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_append(x, x, c, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv4_read(c, torch.zeros(1, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="window"):
        fa.kv4_decode(x[0], c, torch.zeros(1, dtype=torch.int32), window=0)


def test_rope_frequencies():
    """Against the definitions, pair by pair."""
    f, a = fa.rope_frequencies(64, 10000.0)
    assert a == 1.0 and f.dtype == torch.float64
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert max(abs(float(f[i]) / want[i] - 1) for i in range(32)) < 1e-14
    f4, _ = fa.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.allclose(f4 * 4, f, rtol=1e-14, atol=0)
    # ntk: the fastest pair stays, the slowest is stretched by the factor
    fn, _ = fa.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert float(fn[0]) == 1.0 and abs(float(f[-1] / fn[-1]) - 4.0) < 1e-12
    # within the trained length nothing changes; beyond it the factor follows the length
    same, _ = fa.rope_frequencies(64, 10000.0, "ntk", 2.0, trained_length=4096, length=4096)
    assert torch.allclose(same, f, rtol=1e-14, atol=0)
    longer, _ = fa.rope_frequencies(64, 10000.0, "ntk", 2.0, trained_length=4096, length=8192)
    assert abs(float(f[-1] / longer[-1]) - 3.0) < 1e-12
    # yarn: many turns kept, few turns interpolated, monotone between; amplitude from the factor
    fy, ay = fa.rope_frequencies(128, 10000.0, "yarn", 8.0, trained_length=4096)
    f0, _ = fa.rope_frequencies(128, 10000.0)
    ratio = f0 / fy
    turns = 4096 * f0 / (2 * math.pi)
    assert torch.allclose(ratio[turns > 40], torch.ones(()).double())
    assert torch.allclose(ratio[turns < 0.8], torch.full((), 8.0).double())
    assert bool((ratio[1:] >= ratio[:-1] - 1e-12).all())
    assert abs(ay - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, factor=0.5, scaling="linear"), dict(rotary_dim=64, factor=2.0),
                dict(rotary_dim=64, scaling="yarn", factor=2.0), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, scaling="ntk", factor=2.0, length=8192)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad)


def test_chunks_of_the_longest_sequences():
    """Decode with sinks finds a key's chunk without a division: right for every
    chunk size up to the longest lengths that the checks let through, and past them."""
    f = fa.load_library().fa_selftest_chunk_of
    keys = [0, 1, 63, 64, (1 << 31) - 1]
    keys += [(1 << e) + x for e in range(7, 31) for x in (-65, -64, -63, -1, 0, 1, 62, 63, 64)]
    for chunk in range(64, 4097, 64):
        edges = [chunk * (k // chunk) + x for k in keys for x in (-1, 0, 1)]
        for key in keys + edges:
            if 0 <= key < 1 << 31:
                assert f(key, chunk) == key // chunk, (key, chunk)
    assert f(-1, 64) == -1 and f(5, 0) == -1 and f(5, 100) == -1 and f(5, 8192) == -1


@pytest.fixture
def cuda_tensors():
    """Tensors that say they are on a CUDA device and have no memory: what a binding
    does not refuse by itself ends at their data_ptr()."""
    mode = torch._subclasses.fake_tensor.FakeTensorMode(allow_non_fake_inputs=True)
    with mode:
        yield lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda:0")


def test_sink_forward_checks_its_outputs(cuda_tensors):
    t, f32 = cuda_tensors, torch.float32
    q, k = t(2, 40, 4, 64), t(2, 50, 2, 64)
    for out in (t(2, 39, 4, 64), t(1, 40, 4, 64), t(2, 40, 4, 32), t(2, 40, 256)):
        with pytest.raises(ValueError, match="out must have shape"):
            fa.forward(q, k, k, window=8, sinks=2, out=out)
    for lse in (t(2, 4, 39, dtype=f32), t(1, 4, 40, dtype=f32), t(2, 40, 4, dtype=f32), t(4, dtype=f32)):
        with pytest.raises(ValueError, match="lse must have shape"):
            fa.forward(q, k, k, window=8, sinks=2, lse=lse)


def test_prefill_calls_refuse_short_buffers(cuda_tensors):
    """forward() and backward() without sinks: what does not hold the elements that the
    kernels read or write, or is elsewhere, is refused; shapes stay the caller's."""
    t, f32 = cuda_tensors, torch.float32
    q, k, o, lse = t(2, 40, 4, 64), t(2, 50, 2, 64), t(2, 40, 4, 64), t(2, 4, 40, dtype=f32)
    for kw in (dict(out=t(2, 39, 4, 64)), dict(lse=t(2, 4, 39, dtype=f32)), dict(v=t(2, 49, 2, 64)),
               dict(k=t(1, 50, 2, 64))):
        for mask in (dict(), dict(causal=True), dict(window=8)):
            a = dict(dict(q=q, k=k, v=k), **kw)
            with pytest.raises(ValueError, match="the call needs"):
                fa.forward(a.pop("q"), a.pop("k"), a.pop("v"), **a, **mask)
    ws = t(1 << 20, dtype=torch.uint8)
    short = dict(dq=t(2, 39, 4, 64), dk=t(2, 49, 2, 64), dv=t(2, 49, 2, 64))
    for n, x in short.items():
        for mask in (dict(), dict(deterministic=True), dict(window=8)):
            with pytest.raises(ValueError, match="the call needs"):
                fa.backward(q, k, k, o, lse, o, workspace=ws, **{n: x}, **mask)
    with pytest.raises(ValueError, match="the call needs"):
        fa.backward(q, k, k, o, t(2, 4, 39, dtype=f32), o, workspace=ws)
    with pytest.raises(ValueError, match="the call needs"):
        fa.backward(q, k, k, o, lse, t(2, 39, 4, 64), workspace=ws)
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        fa.backward(q, k, k, o, lse, o, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cpu"))
    for sinks in (dict(), dict(window=8, sinks=2)):
        with pytest.raises(TypeError, match="dq must be"):
            fa.backward(q, k, k, o, lse, o, workspace=ws, dq=t(2, 40, 4, 64, dtype=f32), **sinks)


def test_workspace_sizes_with_sinks():
    lib = fa.load_library()
    sizes = (1, 4, 2, 4096, 4096, 64)
    assert fa.backward_workspace_bytes(*sizes, window=256, sinks=4) == \
        lib.fa_backward_sinks_workspace_bytes(*sizes, 256, 4) > fa.backward_workspace_bytes(*sizes)
    assert fa.backward_workspace_bytes(*sizes, window=256) == lib.fa_backward_workspace_bytes(*sizes)
    sizes = (2, 8, 4096, 128, 256)
    assert fa.decode_workspace_bytes(*sizes, window=300, sinks=4) == \
        lib.fa_decode_sinks_workspace_bytes(*sizes, 300, 4) < fa.decode_workspace_bytes(*sizes)
    for f, s in ((fa.backward_workspace_bytes, (1, 4, 2, 16, 16, 64)), (fa.decode_workspace_bytes, sizes)):
        with pytest.raises(ValueError, match="window"):
            f(*s, sinks=4)


@pytest.mark.parametrize("B,Hq,Hkv,T,d,W,S", [(16, 16, 16, 16384, 64, 256, 1024), (1, 8, 1, 65536, 128, 16, 1024),
                                             (2, 4, 4, 700, 64, 1, 600), (1, 1, 1, 1 << 20, 64, 64, 129)])
def test_sink_partial_sums_stay_within_twice_the_accumulator(B, Hq, Hkv, T, d, W, S):
    base = fa.backward_workspace_bytes(B, Hq, Hkv, T, T, d)
    more = fa.backward_workspace_bytes(B, Hq, Hkv, T, T, d, window=W, sinks=S) - base
    assert 0 <= more <= 2 * B * T * Hq * d * 4


def test_sink_forward_needs_a_positive_scale():
    """With a scale of 0 or below, the masked scores would turn the row's sum to NaN."""
    lib = fa.load_library()
    for scale in (0.0, -0.0, -0.125, -math.inf, math.inf, math.nan):
        assert lib.fa_forward_sinks(N, N, N, N, N, 1, 1, 1, 0, 16, 64, scale, 4, 4, N) == INVALID, scale
    assert lib.fa_forward_sinks(N, N, N, N, N, 1, 1, 1, 0, 16, 64, 1e-3, 4, 4, N) == 0


def test_numbers_past_32_bits_are_refused(cuda_tensors):
    """Their low 32 bits, which a C int would take, are a window, sinks or a chunk of
    their own."""
    t = cuda_tensors
    q, k, n = t(2, 40, 4, 64), t(2, 64, 2, 64), t(2, dtype=torch.int32)
    cache = fa.kv4_cache(2, 2, 64, 64, device="cuda:0")
    big = 1 << 32
    for kw in (dict(window=big + 8), dict(window=big + 8, sinks=2), dict(window=8, sinks=big + 2),
               dict(window=-big + 8, sinks=2)):
        with pytest.raises(ValueError, match="32 bits"):
            fa.forward(q, k, k, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            fa.backward(q, k, k, q, t(2, 4, 40, dtype=torch.float32), q, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            fa.decode_splitkv(q[:, 0], k, k, n, **kw)
        with pytest.raises(ValueError, match="32 bits|at least 1"):
            fa.kv4_decode(q[:, 0], cache, n, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            fa.backward_workspace_bytes(2, 4, 2, 40, 64, 64, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        fa.decode_splitkv(q[:, 0], k, k, n, chunk=big + 64)
    with pytest.raises(ValueError, match="32 bits"):
        fa.decode_workspace_bytes(2, 4, 64, 64, chunk=big + 64)


def test_kv4_outputs_share_no_memory(mem):
    """K and V are written by blocks that run in any order."""
    lib = fa.load_library()
    st = strides(*(2 * 64, 2 * 64, 64) * 2)
    p = lambda *x: [mem(v) for v in x]  # noqa: E731
    codes, params = 2 * 64 * 32, 2 * 64 * 8         # bytes of one buffer, at [1, 2, 64]

    def append(kc, kp, vc, vp):
        return lib.fa_kv4_append(*p(0, 512), st, *p(kc, kp, vc, vp), mem(256), N, 1, 1, 2, 64, 64, N)

    apart = (0, 2 * codes, codes, 2 * codes + params)
    for i in range(4):
        for j in range(4):
            if i != j:
                bad = list(apart)
                bad[i] = bad[j] + 16 * (i > j)
                assert append(*bad) == INVALID, (i, j)
    read = lambda k, v, T: lib.fa_kv4_read(*p(k, v), *p(*apart), mem(256), N, 1, T, 2, 64, 64, N)  # noqa: E731
    assert read(0, 0, 1) == INVALID and read(0, 240, 1) == INVALID and read(1008, 0, 4) == INVALID
    if not torch.cuda.is_available():
        # apart: the call gets as far as the device (there is none here)
        assert append(*apart) not in (0, INVALID)
        assert read(0, 256, 1) not in (0, INVALID) and read(1024, 0, 4) not in (0, INVALID)
