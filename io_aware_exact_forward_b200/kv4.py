"""A KV cache held in 4 bits (fa_kv4_append, fa_kv4_read, fa_kv4_decode).

    cache = kv4_cache(B, Hkv, Tk_max, d, device)
    kv4_append(k, v, cache, start)              # a prompt, or one token
    o, lse = kv4_decode(q1, cache, seqlens)     # one query token per sequence
    k, v = kv4_read(cache, start, T)            # values back, in bf16

Values are held in groups of 32 dims with a bf16 step and centre each; see
include/fa.h for the format.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._binding import (_check_decode_out, _check_dev, _check_out, _on_device, _ptr, _raise, _stream_ptr,
                       load_library)

__all__ = ["KV4Cache", "kv4_cache", "kv4_append", "kv4_read", "kv4_decode", "kv4_decode_workspace_bytes"]

GROUP = 32


class KV4Cache(NamedTuple):
    """The cache's buffers: codes uint8 [B,Hkv,Tk_max,d/2], params bf16
    [B,Hkv,Tk_max,2 d/32] (steps, then centres)."""

    k_codes: torch.Tensor
    k_params: torch.Tensor
    v_codes: torch.Tensor
    v_params: torch.Tensor


def kv4_cache(B, Hkv, Tk_max, d, device="cuda"):
    """An empty cache for Tk_max keys a sequence (rounded up to a multiple of
    64).  Its contents are not initialised: rows that were never appended may hold
    anything, and no decode within seqlens looks at them."""
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    T = -(-int(Tk_max) // 64) * 64

    def codes():
        return torch.empty((B, Hkv, T, d // 2), dtype=torch.uint8, device=device)

    def params():
        return torch.empty((B, Hkv, T, 2 * (d // GROUP)), dtype=torch.bfloat16, device=device)

    return KV4Cache(codes(), params(), codes(), params())


def _cache_sizes(cache, dev):
    kc, kp, vc, vp = cache
    if kc.dim() != 4:
        raise ValueError(f"k_codes must be [B, Hkv, Tk_max, d/2], got {tuple(kc.shape)}")
    B, Hkv, Tk, d = kc.shape[0], kc.shape[1], kc.shape[2], 2 * kc.shape[3]
    for n, t, dt, w in (("k_codes", kc, torch.uint8, d // 2), ("k_params", kp, torch.bfloat16, 2 * (d // GROUP)),
                        ("v_codes", vc, torch.uint8, d // 2), ("v_params", vp, torch.bfloat16, 2 * (d // GROUP))):
        _check_dev(n, t, dt, dev)
        _check_out(n, t, (B, Hkv, Tk, w))
    return B, Hkv, Tk, d


def _check_counts(name, t, B, dev):
    if t is not None:
        _check_dev(name, t, torch.int32, dev)
        _check_out(name, t, (B,))


def kv4_append(k, v, cache, start, count=None):
    """Quantise rows k, v bf16 [B,T,Hkv,d] (contiguous in the last dim; slices
    of a packed projection will do) into the cache at positions start[b] + t.
    ``start`` int32 [B] (CUDA); ``count`` int32 [B]: only rows t < count[b] are
    written.  Rows outside the cache are dropped."""
    lib = load_library()
    dev = k.device
    B, Hkv, Tk, d = _cache_sizes(cache, dev)
    for n, t in (("k", k), ("v", v)):
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError(f"{n} must be on {dev}, a CUDA device")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{n} must be {torch.bfloat16}, got {t.dtype}")
        if t.dim() != 4 or t.shape != (B, k.shape[1], Hkv, d):
            raise ValueError(f"{n} must be [{B}, T, {Hkv}, {d}], got {tuple(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"{n} must be contiguous in its last dim")
    if start is None:
        raise TypeError("start must be an int32 tensor")
    _check_counts("start", start, B, dev)
    _check_counts("count", count, B, dev)
    strides = (ctypes.c_longlong * 6)(*(0 if t.shape[i] == 1 else t.stride(i) for t in (k, v) for i in range(3)))
    with _on_device(dev):
        st = lib.fa_kv4_append(k.data_ptr(), v.data_ptr(), strides, *(t.data_ptr() for t in cache), start.data_ptr(),
                               _ptr(count), B, k.shape[1], Hkv, Tk, d, _stream_ptr(dev))
    _raise("fa_kv4_append", st)


def kv4_read(cache, start, T, count=None, out_k=None, out_v=None):
    """k, v bf16 [B,T,Hkv,d]: the cache's values at positions start[b] + t.
    Rows t >= count[b], or outside the cache, read as zeros."""
    lib = load_library()
    dev = cache[0].device
    B, Hkv, Tk, d = _cache_sizes(cache, dev)
    if start is None:
        raise TypeError("start must be an int32 tensor")
    _check_counts("start", start, B, dev)
    _check_counts("count", count, B, dev)
    out_k = torch.empty((B, T, Hkv, d), dtype=torch.bfloat16, device=dev) if out_k is None else out_k
    out_v = torch.empty((B, T, Hkv, d), dtype=torch.bfloat16, device=dev) if out_v is None else out_v
    for n, t in (("out_k", out_k), ("out_v", out_v)):
        _check_dev(n, t, torch.bfloat16, dev)
        _check_out(n, t, (B, T, Hkv, d))
    with _on_device(dev):
        st = lib.fa_kv4_read(out_k.data_ptr(), out_v.data_ptr(), *(t.data_ptr() for t in cache), start.data_ptr(),
                             _ptr(count), B, int(T), Hkv, Tk, d, _stream_ptr(dev))
    _raise("fa_kv4_read", st)
    return out_k, out_v


def kv4_decode_workspace_bytes(B, Hq, Hkv, Tk_max, d) -> int:
    return int(load_library().fa_kv4_decode_workspace_bytes(B, Hq, Hkv, Tk_max, d))


def kv4_decode(q, cache, seqlens, scale=None, window=None, sinks=0, workspace=None, out=None, lse=None):
    """Split-KV decode over the 4-bit cache: O bf16 [B,Hq,d] and LSE fp32 [B,Hq]
    of q [B,Hq,d] against the first seqlens[b] keys (int32 [B]) of each sequence;
    ``window`` and ``sinks`` as in decode_splitkv()."""
    lib = load_library()
    if sinks and window is None:
        raise ValueError("sinks need a window (without one every key is visible)")
    if window is not None and window < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    dev = q.device
    _check_dev("q", q, torch.bfloat16, dev)
    B, Hkv, Tk, d = _cache_sizes(cache, dev)
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != d:
        raise ValueError(f"q must be [{B}, Hq, {d}], got {tuple(q.shape)}")
    Hq = q.shape[1]
    _check_dev("seqlens", seqlens, torch.int32, dev)
    if scale is None:
        scale = d ** -0.5
    need = kv4_decode_workspace_bytes(B, Hq, Hkv, Tk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    else:
        _check_dev("workspace", workspace, torch.uint8, dev)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    _check_decode_out(q, seqlens, out, lse)
    with _on_device(dev):
        st = lib.fa_kv4_decode(q.data_ptr(), *(t.data_ptr() for t in cache), seqlens.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), workspace.data_ptr(), workspace.numel(), B, Hq, Hkv, Tk, d,
                               float(scale), 0 if window is None else int(window), int(sinks), _stream_ptr(dev))
    _raise("fa_kv4_decode", st)
    return out, lse
