"""The paged cache of the target's attention: rotation with the page write, 4-bit and 8-bit pages, and
attention of a round's tokens over the pages (the cache calls of ``include/specdec.h``).

Pages are caller-owned CUDA tensors ``[num_pages, page_size, kv_heads, head_dim]`` of bfloat16
or float16 (the layout ``compact_kv`` takes), or, held in 4 bits, uint8 codes
``[num_pages, page_size, kv_heads, head_dim / 2]`` with scales ``[..., head_dim / 16]`` (uint8
or float8_e4m3fn bytes), or, held in 8 bits, float8_e4m3fn codes ``[num_pages, page_size, kv_heads, head_dim]``
with scales ``[num_pages, blocks, kv_heads]`` (uint8 or float8_e8m0fnu bytes), one for each head and each
``page_size / blocks`` slots, a multiple of 16.  They may be views with any strides of whole 16-byte rows (4-bit
scales: ``head_dim / 16`` bytes; 8-bit scales: any), keys and values with the same strides.  Slot s of sequence b is
entry ``s % page_size`` of page ``block_table[b, s // page_size]``.
"""
from __future__ import annotations

import ctypes
import math

import torch

F16, KV4, KV8 = 2, 3, 4
_CODES = (torch.bfloat16, torch.float16)


class _KvPages(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("k", "v", "k_scales", "v_scales", "block_table")]
                + [(f, ctypes.c_int64) for f in ("page_stride", "slot_stride", "head_stride", "scale_page_stride",
                                                 "scale_slot_stride", "scale_head_stride")]
                + [(f, ctypes.c_int32) for f in ("num_pages", "page_size", "max_pages", "kv_heads", "head_dim",
                                                 "format")]
                + [(f, ctypes.c_float) for f in ("k_scale", "v_scale")] + [("scale_block", ctypes.c_int32)])


def declare(lib) -> None:
    """The argument types of the library's cache calls."""
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    st, pg = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(_KvPages)
    lib.specdec_rotate_qk.argtypes = [vp, st, vp, st, vp, st, i32, vp, vp, f32, vp, i32, i32, vp, vp, vp, i32, i32,
                                      i32, i32, i32, vp, vp, pg, vp, vp]
    for f in (lib.specdec_append_kv4, lib.specdec_append_kv8):
        f.argtypes = [vp, st, vp, st, i32, vp, vp, i32, i32, pg, vp, vp]
    for f in (lib.specdec_read_kv4, lib.specdec_read_kv8):
        f.argtypes = [vp, vp, i32, i32, pg, i32, vp, vp, vp, vp]
    lib.specdec_attend_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.specdec_attend_workspace_bytes.restype = sz
    lib.specdec_attend.argtypes = [vp, st, i32, pg, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, sz,
                                   vp]
    for f in (lib.specdec_rotate_qk, lib.specdec_append_kv4, lib.specdec_read_kv4, lib.specdec_append_kv8, lib.specdec_read_kv8,
              lib.specdec_attend):
        f.restype = i32


_calls = None


def _module():
    """The compiled argument marshalling (csrc/cache_calls.cpp)."""
    global _calls
    if _calls is None:
        from . import load_library
        load_library()
        from . import _cache_calls
        _calls = _cache_calls
    return _calls


def _failed(rc, what, detail):
    from . import SpecdecError, _ERR_NAMES
    raise SpecdecError(f"{what}: {_ERR_NAMES.get(rc, rc)} (code {rc}): {detail}")


def rotation_turns(inv_freq, device=None) -> torch.Tensor:
    """Rotation frequencies (radians for a position, any sequence of floats) as the 64-bit
    counts of 2^-64 turns that ``rotate_qk`` takes."""
    out = []
    for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq):
        t = int(round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64)) % (1 << 64)
        out.append(t - (1 << 64) if t >= 1 << 63 else t)
    return torch.tensor(out, dtype=torch.int64, device=device)


def rotate_qk(q, k, turns, context_len, *, query_len=None, depth=None, q_weight=None, k_weight=None, eps: float = 1e-6,
              interleaved: bool = False, v=None, k_pages=None, v_pages=None, block_table=None, stream=None) -> dict:
    """Norms of queries and keys for each head and the position rotation, in one pass
    (specdec_rotate_qk).

    q [B, n, q_heads, D], k and v [B, n, kv_heads, D] bfloat16 or float16, views with contiguous
    rows (of a fused projection's output, say); turns [rot/2] int64 (``rotation_turns``);
    context_len [B] int32, the new tokens included; query_len [B] int32 (default n); depth [n]
    int32 for tree nodes; q_weight, k_weight [D] (None: no norm).  With k_pages, v_pages and
    block_table the keys and values are written to their pages, else the rotated keys are
    returned.  Returns q [B, n, q_heads, D], k (without pages) and status [B]."""
    call = (_calls or _module()).rotate_qk
    if stream is None:
        return call(q, k, turns, context_len, query_len, depth, q_weight, k_weight, eps, interleaved, v, k_pages, v_pages,
                    block_table)
    with torch.cuda.stream(stream):
        return call(q, k, turns, context_len, query_len, depth, q_weight, k_weight, eps, interleaved, v, k_pages, v_pages,
                    block_table)



def append_kv4(k, v, k_pages, v_pages, block_table, context_len, *, k_scales, v_scales, k_scale: float = 1.0,
               v_scale: float = 1.0, query_len=None, stream=None) -> dict:
    """Keys and values [B, n, kv_heads, D] of the new tokens written to 4-bit pages
    (specdec_append_kv4).  Returns status [B]."""
    call = (_calls or _module()).append_kv4
    if stream is None:
        return call(k, v, k_pages, v_pages, block_table, context_len, query_len, k_scales, v_scales, k_scale, v_scale)
    with torch.cuda.stream(stream):
        return call(k, v, k_pages, v_pages, block_table, context_len, query_len, k_scales, v_scales, k_scale, v_scale)



def read_kv4(k_pages, v_pages, block_table, context_len, n: int, *, k_scales, v_scales, k_scale: float = 1.0,
             v_scale: float = 1.0, query_len=None, dtype=torch.bfloat16, stream=None) -> dict:
    """The values that 4-bit pages hold for the last n tokens (query_len[b] <= n) of each
    sequence (specdec_read_kv4): k, v [B, n, kv_heads, D] of dtype, and status [B]."""
    if dtype not in _CODES:
        raise ValueError("dtype must be bfloat16 or float16")
    call = (_calls or _module()).read_kv4
    brain = dtype is torch.bfloat16
    if stream is None:
        return call(k_pages, v_pages, block_table, context_len, n, query_len, k_scales, v_scales, k_scale, v_scale, brain)
    with torch.cuda.stream(stream):
        return call(k_pages, v_pages, block_table, context_len, n, query_len, k_scales, v_scales, k_scale, v_scale, brain)



def append_kv8(k, v, k_pages, v_pages, block_table, context_len, *, k_scales, v_scales, k_scale: float = 1.0,
               v_scale: float = 1.0, query_len=None, stream=None) -> dict:
    """Keys and values [B, n, kv_heads, D] of the new tokens written to 8-bit pages, with a scale for each block of
    slots and head (specdec_append_kv8).  A block's scale grows with the tokens appended to it, and its earlier codes
    follow; it stays when a draft that raised it is rejected, unless the caller puts the block back as it was (its codes
    and scales) before the accepted tokens are appended again.  Returns status [B]."""
    call = (_calls or _module()).append_kv8
    if stream is None:
        return call(k, v, k_pages, v_pages, block_table, context_len, query_len, k_scales, v_scales, k_scale, v_scale)
    with torch.cuda.stream(stream):
        return call(k, v, k_pages, v_pages, block_table, context_len, query_len, k_scales, v_scales, k_scale, v_scale)


def read_kv8(k_pages, v_pages, block_table, context_len, n: int, *, k_scales, v_scales, k_scale: float = 1.0,
             v_scale: float = 1.0, query_len=None, dtype=torch.bfloat16, stream=None) -> dict:
    """The values that 8-bit pages hold for the last n tokens (query_len[b] <= n) of each
    sequence (specdec_read_kv8): k, v [B, n, kv_heads, D] of dtype, and status [B]."""
    if dtype not in _CODES:
        raise ValueError("dtype must be bfloat16 or float16")
    call = (_calls or _module()).read_kv8
    brain = dtype is torch.bfloat16
    if stream is None:
        return call(k_pages, v_pages, block_table, context_len, n, query_len, k_scales, v_scales, k_scale, v_scale, brain)
    with torch.cuda.stream(stream):
        return call(k_pages, v_pages, block_table, context_len, n, query_len, k_scales, v_scales, k_scale, v_scale, brain)


def attend(q, k_pages, v_pages, block_table, context_len, *, query_len=None, tree_mask=None, depth=None,
           window: int = 0, sinks: int = 0, scale=None, k_scales=None, v_scales=None, k_scale: float = 1.0,
           v_scale: float = 1.0, with_lse: bool = False, stream=None) -> dict:
    """Attention of the new tokens over a paged cache that holds their keys and values already
    (specdec_attend): chain or tree, a sliding window with a few first tokens that stay
    visible, 16-bit, 8-bit or 4-bit pages.

    q [B, n, q_heads, D] bfloat16 or float16, a view with contiguous rows; context_len [B] int32,
    the new tokens included; query_len [B] int32 (default n); tree_mask [n, n] uint8 and depth [n]
    int32: ``build_tree_mask(parents, 0)``'s mask and depth; scale: default 1 / sqrt(D).
    Returns out [B, n, q_heads, D], status [B] and, with_lse, lse [B, n, q_heads] fp32."""
    call = (_calls or _module()).attend
    if stream is None:
        return call(q, k_pages, v_pages, block_table, context_len, query_len, tree_mask, depth, window, sinks, scale,
                    k_scales, v_scales, k_scale, v_scale, with_lse)
    with torch.cuda.stream(stream):
        return call(q, k_pages, v_pages, block_table, context_len, query_len, tree_mask, depth, window, sinks, scale,
                    k_scales, v_scales, k_scale, v_scale, with_lse)
