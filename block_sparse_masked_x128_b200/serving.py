"""Rotary positions, the paged K/V cache, and attention of one new token over it.

The Python side of fa_rotary, fa_cache_append, fa_cache_read and fa_decode.  A decode step makes
these calls back to back and each kernel takes a few microseconds, so the host's part is kept
short: a tensor's description is packed in one go, devices are compared by index, and the current
stream is asked for as a bare pointer.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Tuple

import torch

from . import (FA_DTYPE_BF16, FA_DTYPE_E4M3, FA_DTYPE_F16, FA_DTYPE_S8, FA_OK, FA_ROTARY_HALF,
               FA_ROTARY_INTERLEAVED, FA_ROTARY_SCALE_NONE, FA_SCORE_NONE, FaError, FaKvCache, FaRotaryScaling,
               FaScoreParams, _check, _check_alibi, _lib, _stream_ptr)

_CODES = {torch.float16: FA_DTYPE_F16, torch.bfloat16: FA_DTYPE_BF16, torch.float8_e4m3fn: FA_DTYPE_E4M3,
          torch.int8: FA_DTYPE_S8}
_INT32, _FLOAT32, _FLOAT64 = torch.int32, torch.float32, torch.float64
_pack_tensor = struct.Struct("=Qi4x8q").pack      # fa_tensor_t: address, dtype, padding, extents, strides
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _packed(t) -> bytes:
    """t's fa_tensor_t (t: (B, H, S, D))."""
    B, H, S, D = t.shape
    return _pack_tensor(t.data_ptr(), _CODES.get(t.dtype, -1), B, H, S, D, *t.stride())


def _call(function, index: int, stream, *args) -> None:
    """function(*args, stream) with device `index` current."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(function, index, stream, *args)
    stream = _current_stream(index) if stream is None else getattr(stream, "cuda_stream", stream)
    status = function(*args, stream)
    if status != FA_OK:
        raise FaError(status, function.__name__)


def _int32_rows(t, name: str, index: int, n: int) -> int:
    """The address of a contiguous int32 tensor of n values on device `index`; else ValueError."""
    if t.dtype is not _INT32 or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({n},) on cuda:{index}")
    return t.data_ptr()


# ---------------------------------------------------------------- rotary positions

def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: int = FA_ROTARY_SCALE_NONE,
                       factor: float = 1.0, original_len: float = 0.0, low_turns: float = 1.0,
                       high_turns: float = 32.0, device=None):
    """Angles a position (radians) of the rot_dim / 2 pairs, for rotary(): base^(-2i / rot_dim), scaled
    for long contexts as the FA_ROTARY_SCALE_* kind says.  A float64 tensor on `device` (default: the
    current CUDA device)."""
    out = torch.empty(max(0, int(rot_dim)) // 2, dtype=_FLOAT64)
    sc = FaRotaryScaling(int(scaling), float(factor), float(original_len), float(low_turns), float(high_turns))
    _check(_lib.fa_rotary_frequencies(int(rot_dim), float(base), ctypes.byref(sc), out.data_ptr()),
           "fa_rotary_frequencies")
    return out.to(device if device is not None else torch.device("cuda", torch.cuda.current_device()))


def rotary(q, k, positions, frequencies, *, interleaved: bool = False, factor: float = 1.0, q_out=None,
           k_out=None, inverse: bool = False, stream=None) -> Tuple:
    """Rotary positions of q (B, Hq, S, D) and k (B, Hk, S, D; may be None): the pairs of the first
    2 * len(frequencies) elements of each head turn by position * frequency, times `factor`; the rest
    is copied.  positions: int32 CUDA tensor (B, S) or (S,), or the int position of row 0.  q_out and
    k_out may be q and k (in place).  Returns (q_out, k_out)."""
    index = q.get_device()
    if index < 0 or (k is not None and k.get_device() != index):
        raise ValueError("q and k must be CUDA tensors of one device")
    if (frequencies.dtype is not _FLOAT64 or frequencies.get_device() != index or frequencies.dim() != 1
            or not frequencies.is_contiguous()):
        raise ValueError("frequencies must be a contiguous 1-D float64 tensor on q's device")
    if isinstance(positions, int):
        pos, pos_stride, first = None, 0, positions
    else:
        B, _, S, _ = q.shape
        shape = positions.shape
        if (positions.dtype is not _INT32 or positions.get_device() != index or (shape != (B, S) and shape != (S,))
                or (S > 1 and positions.stride(-1) != 1)):
            raise ValueError("positions must be an int or an int32 tensor (B, S) or (S,) with contiguous rows on "
                             "q's device")
        pos, pos_stride, first = positions.data_ptr(), positions.stride(0) if len(shape) == 2 and B > 1 else 0, 0
    if q_out is None:
        q_out = torch.empty_like(q)
    elif q_out.get_device() != index:
        raise ValueError("q_out must be on q's device")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        packed_k = packed_out = None
    else:
        if k_out is None:
            k_out = torch.empty_like(k)
        elif k_out.get_device() != index:
            raise ValueError("k_out must be on q's device")
        packed_k, packed_out = _packed(k), _packed(k_out)
    _call(_lib.fa_rotary, index, stream, _packed(q), packed_k, pos, pos_stride, first, frequencies.data_ptr(),
          2 * frequencies.numel(), FA_ROTARY_INTERLEAVED if interleaved else FA_ROTARY_HALF, factor, inverse,
          _packed(q_out), packed_out)
    return q_out, k_out


def rotary_backward(dq, dk, positions, frequencies, *, interleaved: bool = False, factor: float = 1.0,
                    q_out=None, k_out=None, stream=None) -> Tuple:
    """Gradients of rotary() with respect to its q and k, given those of its outputs."""
    return rotary(dq, dk, positions, frequencies, interleaved=interleaved, factor=factor, q_out=q_out, k_out=k_out,
                  inverse=True, stream=stream)


# ---------------------------------------------------------------- the cache

class PagedKVCache:
    """The pools of a paged K/V cache: k and v (n_pages, H, page_size, D) of float16, bfloat16,
    float8_e4m3fn or int8, any strides whose last is 1 (a transposed (n_pages, page_size, H, D) pool
    fits), and for the 8-bit types the float32 scales (n_pages, H, page_size).  The tensors stay the
    caller's; the object keeps them alive and describes them to the library."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in _CODES:
            raise TypeError(f"unsupported cache dtype {k.dtype}")
        if not (k.dim() == 4 and k.is_cuda and k.stride(3) == 1 and v.dtype == k.dtype and v.shape == k.shape
                and v.stride() == k.stride() and v.device == k.device):
            raise ValueError("k and v must be (n_pages, H, page_size, D) CUDA tensors of one dtype, shape, stride and "
                             "device, contiguous in D")
        eight = k.dtype in (torch.float8_e4m3fn, torch.int8)
        st = (0, 0, 0)
        if eight:
            for t in (k_scale, v_scale):
                if not (t is not None and t.dtype == _FLOAT32 and t.shape == k.shape[:3] and t.device == k.device
                        and t.stride() == k_scale.stride()):
                    raise ValueError("an 8-bit cache needs float32 scales (n_pages, H, page_size) of one stride on "
                                     "its device")
            st = k_scale.stride()
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a 16-bit cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device, self.quantised = k.dtype, k.device, eight
        self.n_pages, self.H, self.page_size, self.D = k.shape
        self._index = k.get_device()
        self._c = FaKvCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if eight else None,
                            v_scale.data_ptr() if eight else None, _CODES[k.dtype], self.page_size, self.n_pages, self.H,
                            self.D, (ctypes.c_int64 * 3)(*k.stride()[:3]), (ctypes.c_int64 * 3)(*st))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, H: int, page_size: int, D: int, dtype, device=None):
        """Fresh pools (zeros), with scales where the type has them."""
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        k, v = (torch.zeros(n_pages, H, page_size, D, dtype=dtype, device=dev) for _ in range(2))
        if dtype in (torch.float8_e4m3fn, torch.int8):
            return cls(k, v, *(torch.zeros(n_pages, H, page_size, dtype=_FLOAT32, device=dev) for _ in range(2)))
        return cls(k, v)

    def _table(self, table, B: int) -> Tuple[int, int, int]:
        """Address, row stride and width of a page table for B sequences; else ValueError."""
        shape = table.shape
        if len(shape) == 2 and shape[0] == B and table.dtype is _INT32 and table.get_device() == self._index:
            width = shape[1]
            stride, step = table.stride()
            if width <= 1 or step == 1:
                return table.data_ptr(), (stride if B > 1 else width), width
        raise ValueError(f"page_table must be an int32 tensor ({B}, n) with contiguous rows on the cache's device")


def cache_append(cache: PagedKVCache, k, v, page_table, start, *, count=None, stream=None) -> None:
    """Write the new rows k, v (B, H, S, D) of each sequence at positions start[b] + s of the cache
    (quantised for 8-bit caches); count (int32, B) says how many of a padded batch's S rows are real."""
    index, B = cache._index, k.shape[0]
    if k.get_device() != index or v.get_device() != index:
        raise ValueError("k and v must be on the cache's device")
    table, stride, width = cache._table(page_table, B)
    _call(_lib.fa_cache_append, index, stream, _packed(k), _packed(v), cache._ref, table, stride, width,
          _int32_rows(start, "start", index, B), None if count is None else _int32_rows(count, "count", index, B))


def cache_read(cache: PagedKVCache, page_table, kv_lens, S: int, *, start=None, dtype=None, k_out=None,
               v_out=None, stream=None) -> Tuple:
    """Rows start[b] .. start[b] + S - 1 (start None: from 0) of each sequence as (k, v) of shape
    (B, H, S, D); rows at or past kv_lens[b] are zero.  dtype: of the result (a 16-bit cache's own;
    bfloat16 by default for 8-bit caches)."""
    index, B = cache._index, page_table.shape[0]
    shape = (B, cache.H, S, cache.D)
    if k_out is None:
        if dtype is None:
            dtype = torch.bfloat16 if cache.quantised else cache.dtype
        k_out = torch.empty(shape, dtype=dtype, device=cache.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    for t in (k_out, v_out):
        if t.get_device() != index or t.shape != shape:
            raise ValueError("k_out and v_out must be (B, H, S, D) tensors on the cache's device")
    table, stride, width = cache._table(page_table, B)
    _call(_lib.fa_cache_read, index, stream, cache._ref, table, stride, width,
          None if start is None else _int32_rows(start, "start", index, B), _int32_rows(kv_lens, "kv_lens", index, B),
          _packed(k_out), _packed(v_out))
    return k_out, v_out


def cache_status(stream=None) -> int:
    """Synchronise the stream and return FA_OK, or FA_ERR_INVALID_ARG when a call on a cache of the
    current device met a page, position or length out of range since the last look."""
    return _lib.fa_cache_status(_stream_ptr(stream))


# ---------------------------------------------------------------- decode

def decode_workspace_bytes(B: int, HQ: int, H: int, D: int) -> int:
    """Bytes of device scratch that decode_attention needs on the current device."""
    return int(_lib.fa_decode_workspace_bytes(B, HQ, H, D))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index: int, B: int, HQ: int, H: int, D: int) -> int:
    with torch.cuda.device(index):
        return decode_workspace_bytes(B, HQ, H, D)


def decode_attention(q, cache: PagedKVCache, page_table, kv_lens, *, window: int = 0,
                     score_mod: int = FA_SCORE_NONE, softcap: float = 30.0, alibi_slopes=None,
                     scale: Optional[float] = None, out=None, lse=None, return_lse: bool = True, workspace=None,
                     stream=None) -> Tuple:
    """Attention of one new token a sequence: q (B, HQ, 1, D) over the kv_lens[b] (int32, the new one
    among them) tokens that page_table maps, or the last `window` of them; HQ a multiple of the cache's
    heads.  The lengths are read on the device.  Returns (out, lse), lse (B, HQ, 1) or None."""
    index = cache._index
    if q.get_device() != index:
        raise ValueError("q must be on the cache's device")
    B, HQ, _, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    elif out.get_device() != index:
        raise ValueError("out must be on the cache's device")
    if lse is not None:
        if lse.dtype is not _FLOAT32 or lse.get_device() != index or lse.shape != (B, HQ, 1) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 tensor (B, HQ, 1) on the cache's device")
    elif return_lse:
        lse = torch.empty((B, HQ, 1), device=cache.device, dtype=_FLOAT32)
    table, stride, width = cache._table(page_table, B)
    if workspace is None:
        nbytes = _workspace_bytes(index, B, HQ, cache.H, cache.D)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    elif workspace.get_device() != index:
        raise ValueError("workspace must be on the cache's device")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    params = ctypes.byref(FaScoreParams(softcap, _check_alibi(alibi_slopes, q))) if score_mod else None
    _call(_lib.fa_decode, index, stream, _packed(q), cache._ref, table, stride, width,
          _int32_rows(kv_lens, "kv_lens", index, B), window, score_mod, params, -1.0 if scale is None else scale,
          _packed(out), None if lse is None else lse.data_ptr(), workspace.data_ptr(), nbytes)
    return out, lse
