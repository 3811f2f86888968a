"""Rotary positions: the frequencies of a model's pairs, and the calls that turn
q and k before attention and their gradients after it (fa_rope,
fa_rope_backward).

    freqs, amplitude = rope_frequencies(rotary_dim, base, device=q.device)
    q, k = rope(q, k, freqs, positions, amplitude=amplitude)
    o, lse = forward(q, k, v, causal=True)
    ...
    dq, dk, dv = backward(q, k, v, o, lse, do, causal=True)
    dq, dk = rope_backward(dq, dk, freqs, positions, amplitude=amplitude)
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._binding import _check_dev, _cuda_index, _demand, _on_device, _raise, _stream_of, load_library

__all__ = ["rope_frequencies", "rope", "rope_backward"]


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, trained_length=None, length=None,
                     fast_turns=32.0, slow_turns=1.0, device=None):
    """(freqs, amplitude): float64 [rotary_dim / 2] radians per position, and the
    factor on the rotated values.  Without ``scaling``, pair i has
    f_i = base^(-2i / rotary_dim) and the amplitude is 1.  For contexts longer
    than the ``trained_length``:

    "linear"  f_i / factor: positions interpolated into the trained range.
    "ntk"     the base grows so that the slowest pair is stretched by the factor
              and the fastest stays: base * s^(r / (r - 2)), r = rotary_dim, with
              s = factor, or, where ``length`` is given too, the factor that
              this length needs, factor * length / trained_length - (factor - 1)
              (never below 1).
    "yarn"    per pair between the two (Peng et al., "YaRN: Efficient Context
              Window Extension of Large Language Models"): pairs that make more
              than ``fast_turns`` turns over the trained length stay, those with
              fewer than ``slow_turns`` are interpolated, with a linear ramp over
              the pair index between; the amplitude is 0.1 ln(factor) + 1.

    A plan that a program makes once; all of it in 64 bits on the host."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be above 1, got {base}")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor must be at least 1, got {factor}")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)

    def plain(b):
        return torch.pow(torch.tensor(float(b), dtype=torch.float64), -2.0 * i / rotary_dim)

    amplitude = 1.0
    if scaling is None:
        if factor != 1.0:
            raise ValueError("a factor needs a scaling")
        f = plain(base)
    elif scaling == "linear":
        f = plain(base) / factor
    elif scaling == "ntk":
        if rotary_dim < 4:
            raise ValueError("ntk scaling needs a rotary_dim of at least 4")
        s = float(factor)
        if length is not None:
            if not trained_length or trained_length < 1:
                raise ValueError("a length needs the trained_length")
            s = max(1.0, factor * length / trained_length - (factor - 1.0))
        f = plain(base * s ** (rotary_dim / (rotary_dim - 2.0)))
    elif scaling == "yarn":
        if not trained_length or trained_length < 1:
            raise ValueError("yarn scaling needs the trained_length")
        if not fast_turns > slow_turns > 0:
            raise ValueError("yarn scaling needs fast_turns > slow_turns > 0")

        def pair_of(turns):  # the (real) pair index that makes so many turns over the trained length
            return rotary_dim * math.log(trained_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        lo = max(0, math.floor(pair_of(fast_turns)))
        hi = min(rotary_dim - 1, math.ceil(pair_of(slow_turns)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)  # 0: kept, 1: interpolated
        f = plain(base) * (1.0 - ramp) + plain(base) / factor * ramp
        amplitude = 0.1 * math.log(factor) + 1.0
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device) if device is not None else f, amplitude


def _check_rows(name, t, index, B, T, d):
    """(heads, batch, token and head stride) of bf16 [B,T,H,d] rows that are
    contiguous in the last dim."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on a CUDA device (libfa has no CPU path)")
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != d:
        raise ValueError(f"{name} must be [{B}, {T}, H, {d}], got {tuple(shape)}")
    if st[3] != 1:
        raise ValueError(f"{name} must be contiguous in its last dim")
    # no address depends on the stride of a dim of size 1
    return shape[2], 0 if B == 1 else st[0], 0 if T == 1 else st[1], 0 if shape[2] == 1 else st[2]


_STRIDES = ctypes.c_longlong * 12


def _rope(fn, q, k, freqs, positions, interleaved, amplitude, out_q, out_k):
    lib = load_library()
    index = _cuda_index("q", q)
    if q.dim() != 4:
        raise ValueError(f"q must be [B, T, Hq, d], got {tuple(q.shape)}")
    B, T, _, d = q.shape
    Hq, *sq = _check_rows("q", q, index, B, T, d)
    if out_q is None:
        out_q = q.new_empty((B, T, Hq, d))
        soq = T * Hq * d, Hq * d, d
    else:
        h, *soq = _check_rows("out_q", out_q, index, B, T, d)
        if h != Hq:
            raise ValueError(f"out_q must be {tuple(q.shape)}, got {tuple(out_q.shape)}")
    Hkv, kp, okp = 0, 0, 0
    sk = sok = (0, 0, 0)
    if k is not None:
        Hkv, *sk = _check_rows("k", k, index, B, T, d)
        if out_k is None:
            out_k = q.new_empty((B, T, Hkv, d))
            sok = T * Hkv * d, Hkv * d, d
        else:
            h, *sok = _check_rows("out_k", out_k, index, B, T, d)
            if h != Hkv:
                raise ValueError(f"out_k must be {tuple(k.shape)}, got {tuple(out_k.shape)}")
        kp, okp = k.data_ptr(), out_k.data_ptr()
    elif out_k is not None:
        raise ValueError("out_k without k")
    if freqs.dim() != 1:
        raise ValueError(f"freqs must be [rotary_dim / 2], got {tuple(freqs.shape)}")
    _demand("freqs", freqs, torch.float64, index, freqs.shape)
    if positions is not None:
        _demand("positions", positions, torch.int32, index, (B, T))
    with _on_device(index):
        st = getattr(lib, fn)(q.data_ptr(), out_q.data_ptr(), kp, okp, _STRIDES(*sq, *soq, *sk, *sok),
                              0 if positions is None else positions.data_ptr(), freqs.data_ptr(), 2 * freqs.shape[0],
                              1 if interleaved else 0, amplitude, B, T, Hq, Hkv, d, _stream_of(index))
    if st:
        _raise(fn, st)
    return out_q, out_k


def rope(q, k, freqs, positions=None, interleaved=False, amplitude=1.0, out_q=None, out_k=None):
    """Rotated q and k (fa_rope).  q bf16 [B,T,Hq,d] and k [B,T,Hkv,d] (or None)
    on a CUDA device, contiguous in the last dim: slices of a packed projection
    will do.  freqs float64 [rotary_dim / 2] (rope_frequencies), positions int32
    [B,T] or None for 0 .. T - 1.  ``interleaved``: pairs (2i, 2i + 1) instead of
    (i, i + rotary_dim / 2).  The outputs are new dense tensors unless given; an
    output may be its own input (in place)."""
    return _rope("fa_rope", q, k, freqs, positions, interleaved, amplitude, out_q, out_k)


def rope_backward(dq, dk, freqs, positions=None, interleaved=False, amplitude=1.0, out_q=None, out_k=None):
    """Gradients of rope()'s inputs from those of its outputs (fa_rope_backward);
    arguments as rope().  out_q and out_k may be slices of the packed
    projection's gradient."""
    return _rope("fa_rope_backward", dq, dk, freqs, positions, interleaved, amplitude, out_q, out_k)
