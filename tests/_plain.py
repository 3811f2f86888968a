"""Plain 64-bit forms of the rotary, sink-attention and 4-bit-cache operators,
and the error bounds that their kernels are held to.

H is half a step of bf16 relative to the value, torch.finfo(bfloat16).eps / 2:
what rounding a result or an operand to bf16 can move it by.  R32 bounds the
relative error of a probability from everything done in 32 bits: scores of d <=
128 products (their sums' error is at most 128 * 2^-24 of sum |q k| scale, under
20 on N(0,1) inputs: 1.6e-4), the log-sum-exp and the exponential (both well
below that)."""

import math

import torch

H = torch.finfo(torch.bfloat16).eps / 2
R32 = 2e-4
LSE_TOL = 2e-4   # the scores' bound above, in log units
GROUP = 32


# ------------------------------------------------------------------- rotary
def rope(x, freqs, positions, rot, interleaved=False, amplitude=1.0, inverse=False):
    """x [B,T,H,d] in float64, positions [B,T]."""
    x = x.double().cpu()
    theta = positions.double().cpu()[..., None] * freqs.double().cpu()
    c, s = torch.cos(theta)[:, :, None] * amplitude, torch.sin(theta)[:, :, None] * amplitude
    if inverse:
        s = -s
    y = x.clone()
    h = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    ya, yb = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    else:
        y[..., :h], y[..., h:rot] = ya, yb
    return y


def rope_tol(x, ref, rot, interleaved, amplitude):
    """One rounding to bf16, and in 32 bits: cos and sin to 2 steps, their
    product with the amplitude, two products and a sum (8 half steps in all) of
    |x| + |y|."""
    x = x.double().cpu().abs()
    mag = torch.zeros_like(x)
    h = rot // 2
    if interleaved:
        m = x[..., 0:rot:2] + x[..., 1:rot:2]
        mag[..., 0:rot:2], mag[..., 1:rot:2] = m, m
    else:
        m = x[..., :h] + x[..., h:rot]
        mag[..., :h], mag[..., h:rot] = m, m
    return H * ref.abs() + 8 * 2.0 ** -24 * abs(amplitude) * mag + 1e-38


# --------------------------------------------------------------------- sinks
def visible(Tq, Tk, window, sinks):
    i = torch.arange(Tq)[:, None] + (Tk - Tq)
    j = torch.arange(Tk)[None, :]
    return (j <= i) & ((j > i - window) | (j < sinks))


def attention(q, k, v, mask, scale):
    """float64 O, LSE, P and the |V|-weighted sum A of [.., Tq, d], [.., Tk, d]
    rows; rows that see no key have O = 0, LSE = -inf."""
    s = torch.einsum("...id,...jd->...ij", q, k) * scale
    s = s.masked_fill(~mask, -math.inf)
    m = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full(s.shape[:-1] + (1,), -math.inf, dtype=s.dtype)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    w = p / torch.where(l > 0, l, torch.ones_like(l))
    return w @ v, (m + torch.log(l))[..., 0], w, w @ v.abs()


def split_heads(x, Hkv):
    """[B,T,H,d] to float64 [B,Hkv,H/Hkv,T,d] on the CPU."""
    return x.double().cpu().transpose(1, 2).unflatten(1, (Hkv, -1))


def join_heads(x):
    return x.flatten(1, 2).transpose(1, 2)


def sink_forward(q, k, v, window, sinks, scale):
    """(O, tolerance of O, LSE).  The kernel rounds each probability to bf16 and
    normalises by the rounded ones' sum (2 H of sum w |v|), then rounds O."""
    Hkv = k.shape[2]
    Q, K, V = split_heads(q, Hkv), split_heads(k, Hkv), split_heads(v, Hkv)
    o, lse, _, a = attention(Q, K, V, visible(q.shape[1], k.shape[1], window, sinks), scale)
    tol = (2 * H + R32) * a + H * o.abs() + 1e-30
    return join_heads(o), join_heads(tol), lse.flatten(1, 2)


def sink_backward(q, k, v, do, window, sinks, scale):
    """{name: (gradient, tolerance)}.  Roundings to bf16: P (in dV, and in dS),
    dS, the result; D = sum dO O is formed from the rounded O."""
    Hkv = k.shape[2]
    Q, K, V, G = (split_heads(x, Hkv) for x in (q, k, v, do))
    o, _, w, a = attention(Q, K, V, visible(q.shape[1], k.shape[1], window, sinks), scale)
    dv = w.transpose(-1, -2) @ G
    tv = (H + R32) * (w.transpose(-1, -2) @ G.abs())
    dp = G @ V.transpose(-1, -2)
    D = (G * o).sum(-1, keepdim=True)
    dD = (G.abs() * ((2 * H + R32) * a + H * o.abs())).sum(-1, keepdim=True)
    ds = w * (dp - D)
    tds = w * ((2 * H + R32) * (dp.abs() + D.abs()) + dD)
    dq, tq = ds @ K * scale, tds @ K.abs() * scale
    dk, tk = ds.transpose(-1, -2) @ Q * scale, tds.transpose(-1, -2) @ Q.abs() * scale
    out = {"dq": (join_heads(dq), join_heads(tq + H * dq.abs()))}
    for n, x, t in (("dk", dk, tk), ("dv", dv, tv)):
        x, t = x.sum(2), t.sum(2)
        out[n] = (x.transpose(1, 2), (t + H * x.abs()).transpose(1, 2))
    return {n: (x, t + 1e-30) for n, (x, t) in out.items()}


def check(x, ref, tol, what):
    d = (x.double().cpu() - ref).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                                 f"{float((d / tol)[bad].max()):.3g} times it")


def check_lse(x, ref, what="LSE"):
    x = x.double().cpu()
    assert torch.equal(torch.isneginf(x), torch.isneginf(ref)), f"{what}: rows without keys differ"
    f = ~torch.isneginf(ref)
    if f.any():
        d = float((x - ref)[f].abs().max())
        assert d <= LSE_TOL, f"{what}: {d:.3g}"


# ----------------------------------------------------------------- 4-bit rows
def split4(x):
    """codes int64 [..., d], steps and centres bf16 [..., d/32] of bf16 x, with
    the format's own roundings in 32 bits."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((0.5 * hi - 0.5 * lo) / 7.5).to(torch.bfloat16)
    z = (lo.double() + 8.0 * s.double()).float().to(torch.bfloat16)  # 8 s alone may overflow
    sf, zf = s.float()[..., None], z.float()[..., None]
    c = torch.round((g - zf) / sf).clamp(-8, 7)
    c = torch.where(sf > 0, c, torch.zeros_like(c)).to(torch.int64) + 8
    return c.flatten(-2), s, z


def pack4(x):
    c, s, z = split4(x)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8), torch.cat([s, z], -1)


def values4(codes, params):
    """float64 values, and the codes' part s (c - 8) of them."""
    codes, params = codes.cpu(), params.cpu()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
    s, z = params.double().chunk(2, -1)
    part = s.repeat_interleave(GROUP, -1) * c
    return part + z.repeat_interleave(GROUP, -1), part


def decode(q, k, v, parts, lens, window, sinks, scale):
    """(O, tolerance, LSE) of q [B,Hq,d] against float64 k, v [B,Hkv,T,d]: rows
    beyond lens, or outside window and sinks, are not looked at.  Bound: p (times
    the step, for 4-bit values) rounded to bf16 against the unrounded sum, or
    against the rounded one (2 H), and O rounded."""
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    o = torch.zeros((B, Hq, d), dtype=torch.float64)
    t = torch.full((B, Hq, d), 1e-30, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        keep = [j for j in range(n) if j >= lo or j < sinks]
        if not keep:
            continue
        Q = q[b].double().cpu().view(Hkv, -1, d)
        V = v[b][:, keep]
        O, L, w, a = attention(Q, k[b][:, keep], V, torch.ones(1, len(keep), dtype=torch.bool), scale)
        if parts is not None:
            a = a + w @ parts[b][:, keep].abs() + w @ (V - parts[b][:, keep]).abs()
        o[b], lse[b] = O.reshape(Hq, d), L.reshape(Hq)
        t[b] += ((2 * H + R32) * a + H * O.abs()).reshape(Hq, d)
    return o, t, lse


def sink_backward_by_rounding(q, k, v, do, window, sinks, scale):
    """{name: (gradient, tolerance)} for scores of any size, from the roundings
    that the kernels make: P to bf16 for dV (H) and, at worst, for dS (H; the
    deterministic dQ pass does not round it), dS to bf16 (H), the result (H), D =
    sum dO O from the rounded O.  r bounds what the scores' sums
    in 32 bits, 128 steps of 2^-24 of their sizes, do to a probability, with
    2^-20 for the log-sum-exp and the exponential."""
    Hkv = k.shape[2]
    Q, K, V, G = (split_heads(x, Hkv) for x in (q, k, v, do))
    o, _, w, a = attention(Q, K, V, visible(q.shape[1], k.shape[1], window, sinks), scale)
    r = 2 * 128 * 2.0 ** -24 * float((Q.abs() @ K.abs().transpose(-1, -2)).max()) * scale + 2.0 ** -20
    n = (q.shape[1] * q.shape[2] // Hkv + k.shape[1]) * 2.0 ** -24   # sums over queries or keys
    dv, gw = w.transpose(-1, -2) @ G, w.transpose(-1, -2) @ G.abs()
    tv = (H + r + n) * gw
    dp, dpa = G @ V.transpose(-1, -2), G.abs() @ V.abs().transpose(-1, -2)
    D = (G * o).sum(-1, keepdim=True)
    dD = (G.abs() * ((2 * H + r) * a + H * o.abs())).sum(-1, keepdim=True)
    ds = w * (dp - D)
    tds = (2 * H + H * H + r + n) * ds.abs() + 1.01 * w * (dD + 128 * 2.0 ** -24 * dpa)
    dq, tq = ds @ K * scale, tds @ K.abs() * scale
    dk, tk = ds.transpose(-1, -2) @ Q * scale, tds.transpose(-1, -2) @ Q.abs() * scale
    out = {"dq": (join_heads(dq), join_heads(tq + H * (dq.abs() + tq)))}
    for name, x, t in (("dk", dk, tk), ("dv", dv, tv)):
        x, t = x.sum(2), t.sum(2)
        out[name] = (x.transpose(1, 2), (t + H * (x.abs() + t)).transpose(1, 2))
    return {name: (x, t + 1e-36) for name, (x, t) in out.items()}
