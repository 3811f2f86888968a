"""The rotary, sink and 4-bit-cache operators together, as a serving loop and a
training step use them, against the 64-bit forms chained the same way."""

import pytest
import torch

import _plain as P

pytestmark = pytest.mark.gpu

fa = pytest.importorskip("io_aware_exact_forward_b200")


def _rand(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def test_prompt_then_tokens():
    """A prompt's packed projection: rotate, attend with window and sinks, fill
    the 4-bit cache; then single tokens: rotate, append, decode."""
    B, T, Hq, Hkv, d, W, S, steps = 2, 150, 4, 2, 128, 60, 4, 3
    qkv = _rand((B, T + steps, Hq + 2 * Hkv, d), 1)
    dev = qkv.cuda()
    freqs, amp = fa.rope_frequencies(d, 10000.0, "yarn", 4.0, trained_length=128, device="cuda")
    cache = fa.kv4_cache(B, Hkv, T + steps, d)
    for t in cache:
        t.view(torch.uint8).fill_(0xFF)      # as unwritten memory may be: NaN steps
    start = torch.zeros(B, dtype=torch.int32, device="cuda")

    q, k = fa.rope(dev[:, :T, :Hq], dev[:, :T, Hq:Hq + Hkv], freqs, amplitude=amp)
    v = dev[:, :T, Hq + Hkv:].contiguous()
    o, lse = fa.forward(q, k, v, window=W, sinks=S)
    fa.kv4_append(k, dev[:, :T, Hq + Hkv:], cache, start)
    ref, tol, rl = P.sink_forward(q.cpu(), k.cpu(), v.cpu(), W, S, d ** -0.5)
    P.check(o, ref, tol, "prompt O")
    P.check_lse(lse, rl)

    keys, vals = [k.cpu()], [v.cpu()]
    for i in range(steps):
        n = T + i
        pos = torch.full((B, 1), n, dtype=torch.int32, device="cuda")
        q1, k1 = fa.rope(dev[:, n:n + 1, :Hq], dev[:, n:n + 1, Hq:Hq + Hkv], freqs, pos, amplitude=amp)
        fa.kv4_append(k1, dev[:, n:n + 1, Hq + Hkv:], cache, start + n)
        lens = start + n + 1
        o1, l1 = fa.kv4_decode(q1[:, 0], cache, lens, window=W, sinks=S)
        assert fa.check() == 0
        want = P.rope(qkv[:, n:n + 1, :Hq], freqs, pos, d, amplitude=amp)
        P.check(q1, want, P.rope_tol(qkv[:, n:n + 1, :Hq], want, d, False, amp), "q")
        keys.append(k1.cpu())
        vals.append(qkv[:, n:n + 1, Hq + Hkv:])
        kv = P.values4(*P.pack4(torch.cat(keys, 1).transpose(1, 2)))[0]
        vv, vp = P.values4(*P.pack4(torch.cat(vals, 1).transpose(1, 2)))
        ref, tol, rl = P.decode(q1[:, 0].cpu(), kv, vv, vp, [n + 1] * B, W, S, d ** -0.5)
        P.check(o1, ref, tol, f"token {i} O")
        P.check_lse(l1, rl)

    # the next chunk's prefill over the values read back
    rk, rv = fa.kv4_read(cache, start, T + steps)
    assert torch.equal(rk.cpu(), kv.transpose(1, 2).float().to(torch.bfloat16))
    o2, _ = fa.forward(q1, rk, rv, window=W, sinks=S)
    ref, tol, _ = P.sink_forward(q1.cpu(), rk.cpu(), rv.cpu(), W, S, d ** -0.5)
    P.check(o2, ref, tol, "chunk O")


@pytest.mark.parametrize("inter", [False, True])
def test_training_step(inter):
    """Gradient of the packed projection through rotation and attention."""
    B, T, Hq, Hkv, d, rot, W, S = 2, 200, 4, 2, 64, 32, 50, 4
    qkv, do = _rand((B, T, Hq + 2 * Hkv, d), 5), _rand((B, T, Hq, d), 6)
    dev = qkv.cuda()
    freqs, _ = fa.rope_frequencies(rot, device="cuda")
    q, k = fa.rope(dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv], freqs, interleaved=inter)
    v = dev[:, :, Hq + Hkv:].contiguous()
    o, lse = fa.forward(q, k, v, window=W, sinks=S)
    dq, dk, dv = fa.backward(q, k, v, o, lse, do.cuda(), window=W, sinks=S)
    grad = torch.empty_like(dev)
    fa.rope_backward(dq, dk, freqs, interleaved=inter, out_q=grad[:, :, :Hq], out_k=grad[:, :, Hq:Hq + Hkv])
    grad[:, :, Hq + Hkv:] = dv
    assert fa.check() == 0
    ref = P.sink_backward(q.cpu(), k.cpu(), v.cpu(), do, W, S, d ** -0.5)
    pos = torch.arange(T).expand(B, T)
    for n, at in (("dq", slice(0, Hq)), ("dk", slice(Hq, Hq + Hkv))):
        g, t = ref[n]
        want = P.rope(g, freqs, pos, rot, inter, inverse=True)
        # the turned bound (|cos|, |sin| <= 1: both parts of a pair), and the rotation's own
        both = P.rope_tol(t, torch.zeros_like(t), rot, inter, 2.0 ** 24 / 8)
        both[..., rot:] = t[..., rot:]
        P.check(grad[:, :, at], want, both + P.rope_tol(g.abs() + t, want.abs() + both, rot, inter, 1.0), n)
    P.check(grad[:, :, Hq + Hkv:], *ref["dv"], "dv")
