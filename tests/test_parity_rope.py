"""Rotary positions (fa_rope, fa_rope_backward) against the 64-bit form."""

import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu

fa = pytest.importorskip("io_aware_exact_forward_b200")


def _rand(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


CASES = [
    # B, T, Hq, Hkv, d, rot, interleaved, first position
    (1, 1, 1, 1, 64, 16, False, 0),
    (2, 7, 3, 1, 64, 64, True, 5),
    (3, 5, 4, 2, 128, 128, False, 1000003),      # far positions: 10^6 radians in the first pair
    (1, 33, 8, 8, 128, 96, True, 131072),
    (2, 130, 2, 1, 128, 48, False, 0),
    (1, 4100, 2, 1, 64, 32, False, 0),           # several tokens per block, the last block short
    (64, 1, 32, 8, 128, 128, False, 30000),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,rot,inter,first", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_rope(B, T, Hq, Hkv, d, rot, inter, first, backward):
    q, k = _rand((B, T, Hq, d), 1), _rand((B, T, Hkv, d), 2)
    pos = (first + torch.arange(B * T).view(B, T) * 3 % 977).to(torch.int32)
    freqs, _ = fa.rope_frequencies(rot, 10000.0)
    f = fa.rope_backward if backward else fa.rope
    oq, ok = f(q.cuda(), k.cuda(), freqs.cuda(), pos.cuda(), interleaved=inter, amplitude=1.25)
    assert fa.check() == 0
    for x, y, n in ((q, oq, "q"), (k, ok, "k")):
        ref = P.rope(x, freqs, pos, rot, inter, 1.25, inverse=backward)
        P.check(y, ref, P.rope_tol(x, ref, rot, inter, 1.25), n)
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:]), "dims behind the rotated ones are copied"


def test_rope_without_positions_and_without_k():
    q = _rand((2, 9, 4, 64), 3)
    freqs, _ = fa.rope_frequencies(64)
    oq, ok = fa.rope(q.cuda(), None, freqs.cuda())
    assert ok is None and fa.check() == 0
    pos = torch.arange(9).expand(2, 9)
    ref = P.rope(q, freqs, pos, 64)
    P.check(oq, ref, P.rope_tol(q, ref, 64, False, 1.0), "q")


@pytest.mark.parametrize("inter", [False, True])
def test_rope_packed_and_in_place(inter):
    """q and k as slices of a packed projection, into dense outputs, in place,
    and into slices of the packed gradient, whose v part stays as it was."""
    B, T, Hq, Hkv, d, rot = 2, 11, 4, 2, 128, 64
    qkv = _rand((B, T, Hq + 2 * Hkv, d), 4)
    freqs, _ = fa.rope_frequencies(rot)
    pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(0)).to(torch.int32)
    dev = qkv.cuda()
    want_q, want_k = fa.rope(dev[:, :, :Hq].contiguous(), dev[:, :, Hq:Hq + Hkv].contiguous(), freqs.cuda(),
                             pos.cuda(), interleaved=inter)
    got_q, got_k = fa.rope(dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv], freqs.cuda(), pos.cuda(), interleaved=inter)
    assert got_q.is_contiguous() and torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    sq, sk = dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv]
    fa.rope(sq, sk, freqs.cuda(), pos.cuda(), interleaved=inter, out_q=sq, out_k=sk)
    assert torch.equal(dev[:, :, :Hq], want_q) and torch.equal(dev[:, :, Hq:Hq + Hkv], want_k)
    assert torch.equal(dev[:, :, Hq + Hkv:].cpu(), qkv[:, :, Hq + Hkv:])
    # heads before tokens: [B, H, T, d] memory
    hq = want_q.transpose(1, 2).contiguous().transpose(1, 2)
    back_q, _ = fa.rope_backward(hq, None, freqs.cuda(), pos.cuda(), interleaved=inter)
    ref = P.rope(want_q, freqs, pos, rot, inter, inverse=True)
    P.check(back_q, ref, P.rope_tol(want_q, ref, rot, inter, 1.0), "back")
    assert fa.check() == 0


def test_rope_refuses_on_the_device():
    q = _rand((1, 8, 2, 64), 5).cuda()
    f = fa.rope_frequencies(64)[0].cuda()
    with pytest.raises(TypeError):
        fa.rope(q.float(), None, f)
    with pytest.raises(TypeError):
        fa.rope(q, None, f.float())
    with pytest.raises(ValueError):
        fa.rope(q, q[:, :4], f)
    with pytest.raises(ValueError):
        fa.rope(q, None, f, torch.zeros(1, 7, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fa.rope(q.transpose(2, 3), None, f)
    with pytest.raises(fa.FAError):      # overlaps its input one token further
        buf = torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16, device="cuda")
        fa.rope(buf[:, :8], None, f, out_q=buf[:, 1:])
    with pytest.raises(fa.FAError):      # one row for every token
        fa.rope(q, None, f, out_q=torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(1, 8, 2, 64))


def test_rope_gradient_against_differences():
    """<rope_backward(g), u> is the change of <g, rope(x)> along u: rope is
    linear, so the difference quotient of the 64-bit form is exact."""
    B, T, H, d, rot = 1, 6, 2, 64, 32
    x, g, u = (_rand((B, T, H, d), s) for s in (6, 7, 8))
    freqs, amp = fa.rope_frequencies(rot, 10000.0, "yarn", 4.0, trained_length=2048)
    pos = torch.arange(100, 100 + T).expand(B, T)
    y, _ = fa.rope_backward(g.cuda(), None, freqs.cuda(), pos.to(torch.int32).cuda().contiguous(), amplitude=amp)
    up = P.rope(x.double() + u.double(), freqs, pos, rot, amplitude=amp)
    dn = P.rope(x.double() - u.double(), freqs, pos, rot, amplitude=amp)
    diff = float((g.double() * (up - dn)).sum() / 2)
    ref = P.rope(g, freqs, pos, rot, amplitude=amp, inverse=True)
    bound = float((P.rope_tol(g, ref, rot, False, amp) * u.double().abs()).sum())
    assert abs(float((y.double().cpu() * u.double()).sum()) - diff) <= bound + 1e-9


def test_rope_empty_and_graph():
    f = fa.rope_frequencies(64)[0].cuda()
    x = torch.zeros(2, 0, 3, 64, dtype=torch.bfloat16, device="cuda")
    assert fa.rope(x, x, f)[0].shape == (2, 0, 3, 64)
    q, pos = _rand((3, 1, 4, 64), 11).cuda(), torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    fa.rope(q, None, f, pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _ = fa.rope(q, None, f, pos)
    pos.fill_(77)
    g.replay()
    assert torch.equal(y, fa.rope(q, None, f, pos)[0])
    assert fa.check() == 0


def test_rope_strides_past_32_bits():
    T, step = 200, 1 << 24
    big = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, T, 3, 64), (T * step, step, 64, 1))
    x.copy_(_rand((1, T, 3, 64), 12))
    f = fa.rope_frequencies(64)[0].cuda()
    want, _ = fa.rope(x.contiguous(), None, f)
    got, _ = fa.rope(x, None, f)
    assert torch.equal(got, want)
    fa.rope(x, None, f, out_q=x)
    assert torch.equal(x, want) and fa.check() == 0
