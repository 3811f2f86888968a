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

from ._binding import _check_dev, _cuda_index, _demand, _need_window, _on_device, _raise, _stream_of, load_library

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


def _cache_sizes(cache, index):
    kc, kp, vc, vp = cache
    if kc.dim() != 4:
        raise ValueError(f"k_codes must be [B, Hkv, Tk_max, d/2], got {tuple(kc.shape)}")
    B, Hkv, Tk, w = codes = kc.shape
    params = (B, Hkv, Tk, 4 * w // GROUP)
    _demand("k_codes", kc, torch.uint8, index, codes)
    _demand("k_params", kp, torch.bfloat16, index, params)
    _demand("v_codes", vc, torch.uint8, index, codes)
    _demand("v_params", vp, torch.bfloat16, index, params)
    return B, Hkv, Tk, 2 * w


def _counts(start, count, B, index):
    """Pointers of start and count (0 for none)."""
    if start is None:
        raise TypeError("start must be an int32 tensor")
    _demand("start", start, torch.int32, index, (B,))
    if count is None:
        return start.data_ptr(), 0
    _demand("count", count, torch.int32, index, (B,))
    return start.data_ptr(), count.data_ptr()


_STRIDES = ctypes.c_longlong * 6


def kv4_append(k, v, cache, start, count=None):
    """Quantise rows k, v bf16 [B,T,Hkv,d] (contiguous in the last dim; slices
    of a packed projection will do) into the cache at positions start[b] + t.
    ``start`` int32 [B] (CUDA); ``count`` int32 [B]: only rows t < count[b] are
    written.  Rows outside the cache are dropped."""
    lib = load_library()
    index = _cuda_index("k", k)
    B, Hkv, Tk, d = _cache_sizes(cache, index)
    T = k.shape[1] if k.dim() == 4 else 0
    strides = []
    for n, t in (("k", k), ("v", v)):
        if _cuda_index(n, t) != index:
            raise ValueError(f"{n} is on {t.device}, expected cuda:{index}")
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{n} must be {torch.bfloat16}, got {t.dtype}")
        if t.shape != (B, T, Hkv, d):
            raise ValueError(f"{n} must be [{B}, T, {Hkv}, {d}], got {tuple(t.shape)}")
        st = t.stride()
        if st[3] != 1:
            raise ValueError(f"{n} must be contiguous in its last dim")
        # no address depends on the stride of a dim of size 1
        strides += (0 if B == 1 else st[0], 0 if T == 1 else st[1], 0 if Hkv == 1 else st[2])
    start_ptr, count_ptr = _counts(start, count, B, index)
    kc, kp, vc, vp = cache
    with _on_device(index):
        st = lib.fa_kv4_append(k.data_ptr(), v.data_ptr(), _STRIDES(*strides), kc.data_ptr(), kp.data_ptr(),
                               vc.data_ptr(), vp.data_ptr(), start_ptr, count_ptr, B, T, Hkv, Tk, d, _stream_of(index))
    if st:
        _raise("fa_kv4_append", st)


def kv4_read(cache, start, T, count=None, out_k=None, out_v=None):
    """k, v bf16 [B,T,Hkv,d]: the cache's values at positions start[b] + t.
    Rows t >= count[b], or outside the cache, read as zeros."""
    lib = load_library()
    index = _cuda_index("k_codes", cache[0])
    B, Hkv, Tk, d = _cache_sizes(cache, index)
    start_ptr, count_ptr = _counts(start, count, B, index)
    shape = (B, T, Hkv, d)
    kc, kp, vc, vp = cache
    if out_k is None:
        out_k = kp.new_empty(shape)
    else:
        _demand("out_k", out_k, torch.bfloat16, index, shape)
    if out_v is None:
        out_v = torch.empty_like(out_k)
    else:
        _demand("out_v", out_v, torch.bfloat16, index, shape)
    with _on_device(index):
        st = lib.fa_kv4_read(out_k.data_ptr(), out_v.data_ptr(), kc.data_ptr(), kp.data_ptr(), vc.data_ptr(),
                             vp.data_ptr(), start_ptr, count_ptr, B, T, Hkv, Tk, d, _stream_of(index))
    if st:
        _raise("fa_kv4_read", st)
    return out_k, out_v


def kv4_decode_workspace_bytes(B, Hq, Hkv, Tk_max, d) -> int:
    return int(load_library().fa_kv4_decode_workspace_bytes(B, Hq, Hkv, Tk_max, d))


def kv4_decode(q, cache, seqlens, scale=None, window=None, sinks=0, workspace=None, out=None, lse=None):
    """Split-KV decode over the 4-bit cache: O bf16 [B,Hq,d] and LSE fp32 [B,Hq]
    of q [B,Hq,d] against the first seqlens[b] keys (int32 [B]) of each sequence;
    ``window`` and ``sinks`` as in decode_splitkv()."""
    lib = load_library()
    _need_window(window, sinks)
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError(f"window must be at least 1, got {window}")
    index = _cuda_index("q", q)
    B, Hkv, Tk, d = _cache_sizes(cache, index)
    if q.dim() != 3:
        raise ValueError(f"q must be [{B}, Hq, {d}], got {tuple(q.shape)}")
    Hq = q.shape[1]
    _demand("q", q, torch.bfloat16, index, (B, Hq, d))
    _demand("seqlens", seqlens, torch.int32, index, (B,))
    if workspace is None:
        need = lib.fa_kv4_decode_workspace_bytes(B, Hq, Hkv, Tk, d)
        workspace = cache[0].new_empty(max(need, 16))
    else:
        _check_dev("workspace", workspace, torch.uint8, q.device)
    if out is None:
        out = torch.empty_like(q)
    else:
        _demand("out", out, torch.bfloat16, index, (B, Hq, d))
    if lse is None:
        lse = q.new_empty((B, Hq), dtype=torch.float32)
    else:
        _demand("lse", lse, torch.float32, index, (B, Hq))
    kc, kp, vc, vp = cache
    with _on_device(index):
        st = lib.fa_kv4_decode(q.data_ptr(), kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(),
                               seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                               workspace.numel(), B, Hq, Hkv, Tk, d, d ** -0.5 if scale is None else scale, window,
                               sinks, _stream_of(index))
    if st:
        _raise("fa_kv4_decode", st)
    return out, lse
