"""Rotary positions, the paged K/V cache, and attention of one new token over it.

The Python side of fa_rotary, fa_cache_append, fa_cache_read and fa_decode.  A decode step makes
these calls back to back and each kernel takes a few microseconds, so their argument checks and
allocations are compiled (csrc/binding.cpp); the computation is the C library's, by the addresses
of its entry points.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import (FA_DTYPE_BF16, FA_DTYPE_E4M3, FA_DTYPE_F16, FA_DTYPE_S8, FA_ROTARY_HALF, FA_ROTARY_INTERLEAVED,
               FA_ROTARY_SCALE_NONE, FA_SCORE_NONE, FaError, FaKvCache, FaRotaryScaling, FaScoreParams, _check,
               _check_alibi, _lib, _stream_ptr)

_CODES = {torch.float16: FA_DTYPE_F16, torch.bfloat16: FA_DTYPE_BF16, torch.float8_e4m3fn: FA_DTYPE_E4M3,
          torch.int8: FA_DTYPE_S8}


def _load_binding():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "fa_b200_torch.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python block_sparse_masked_x128_b200/build.py`")
    loader = importlib.machinery.ExtensionFileLoader("fa_b200_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("fa_b200_torch", loader))
    loader.exec_module(module)
    module.bind(*(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in
                  ("fa_rotary", "fa_cache_append", "fa_cache_read", "fa_decode", "fa_decode_workspace_bytes")))
    return module


_binding = _load_binding()


def _address(stream):
    """A stream as the binding takes it: None for the current one, else the cudaStream_t's address."""
    return None if stream is None else int(getattr(stream, "cuda_stream", stream))


# ---------------------------------------------------------------- rotary positions

def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: int = FA_ROTARY_SCALE_NONE,
                       factor: float = 1.0, original_len: float = 0.0, low_turns: float = 1.0,
                       high_turns: float = 32.0, device=None):
    """Angles a position (radians) of the rot_dim / 2 pairs, for rotary(): base^(-2i / rot_dim), scaled
    for long contexts as the FA_ROTARY_SCALE_* kind says.  A float64 tensor on `device` (default: the
    current CUDA device)."""
    out = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
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
    first = 0
    if isinstance(positions, int):
        positions, first = None, positions
    r = _binding.rotary(q, k, positions, first, frequencies, FA_ROTARY_INTERLEAVED if interleaved else FA_ROTARY_HALF,
                        factor, inverse, q_out, k_out, None if stream is None else _address(stream))
    if type(r) is int:
        raise FaError(r, "fa_rotary")
    return r


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
                if not (t is not None and t.dtype == torch.float32 and t.shape == k.shape[:3] and t.device == k.device
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
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, n_pages: int, H: int, page_size: int, D: int, dtype, device=None):
        """Fresh pools (zeros), with scales where the type has them."""
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        k, v = (torch.zeros(n_pages, H, page_size, D, dtype=dtype, device=dev) for _ in range(2))
        if dtype in (torch.float8_e4m3fn, torch.int8):
            return cls(k, v, *(torch.zeros(n_pages, H, page_size, dtype=torch.float32, device=dev) for _ in range(2)))
        return cls(k, v)


def cache_append(cache: PagedKVCache, k, v, page_table, start, *, count=None, stream=None) -> None:
    """Write the new rows k, v (B, H, S, D) of each sequence at positions start[b] + s of the cache
    (quantised for 8-bit caches); count (int32, B) says how many of a padded batch's S rows are real."""
    r = _binding.append(cache._at, cache._index, k, v, page_table, start, count,
                        None if stream is None else _address(stream))
    if r is not None:
        raise FaError(r, "fa_cache_append")


def cache_read(cache: PagedKVCache, page_table, kv_lens, S: int, *, start=None, dtype=None, k_out=None,
               v_out=None, stream=None) -> Tuple:
    """Rows start[b] .. start[b] + S - 1 (start None: from 0) of each sequence as (k, v) of shape
    (B, H, S, D); rows at or past kv_lens[b] are zero.  dtype: of the result (a 16-bit cache's own;
    bfloat16 by default for 8-bit caches)."""
    if dtype is None:
        dtype = torch.bfloat16 if cache.quantised else cache.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"unsupported dtype {dtype}: use torch.float16 or torch.bfloat16")
    r = _binding.read(cache._at, cache._index, page_table, kv_lens, S, start, dtype is torch.bfloat16, k_out, v_out,
                      None if stream is None else _address(stream))
    if type(r) is int:
        raise FaError(r, "fa_cache_read")
    return r


def cache_status(stream=None) -> int:
    """Synchronise the stream and return FA_OK, or FA_ERR_INVALID_ARG when a call on a cache of the
    current device met a page, position or length out of range since the last look."""
    return _lib.fa_cache_status(_stream_ptr(stream))


# ---------------------------------------------------------------- decode

def decode_workspace_bytes(B: int, HQ: int, H: int, D: int) -> int:
    """Bytes of device scratch that decode_attention needs on the current device."""
    return int(_lib.fa_decode_workspace_bytes(B, HQ, H, D))


def decode_attention(q, cache: PagedKVCache, page_table, kv_lens, *, window: int = 0,
                     score_mod: int = FA_SCORE_NONE, softcap: float = 30.0, alibi_slopes=None,
                     scale: Optional[float] = None, out=None, lse=None, return_lse: bool = True, workspace=None,
                     stream=None) -> Tuple:
    """Attention of one new token a sequence: q (B, HQ, 1, D) over the kv_lens[b] (int32, the new one
    among them) tokens that page_table maps, or the last `window` of them; HQ a multiple of the cache's
    heads.  The lengths are read on the device.  Returns (out, lse), lse (B, HQ, 1) or None."""
    params = at = None
    if score_mod:
        params = FaScoreParams(softcap, _check_alibi(alibi_slopes, q))
        at = ctypes.addressof(params)
    r = _binding.decode(cache._at, cache._index, q, page_table, kv_lens, window, score_mod, at,
                        -1.0 if scale is None else scale, out, lse, return_lse, workspace,
                        None if stream is None else _address(stream))
    if type(r) is int:
        raise FaError(r, "fa_decode")
    return r
