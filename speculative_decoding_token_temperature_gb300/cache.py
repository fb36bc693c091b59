"""The paged cache of the target's attention: rotation with the page write, 4-bit pages, and
attention of a round's tokens over the pages (the cache calls of ``include/specdec.h``).

Pages are caller-owned CUDA tensors ``[num_pages, page_size, kv_heads, head_dim]`` of bfloat16
or float16 (the layout ``compact_kv`` takes), or, held in 4 bits, uint8 codes
``[num_pages, page_size, kv_heads, head_dim / 2]`` with scales ``[..., head_dim / 16]`` (uint8
or float8_e4m3fn bytes).  They may be views with any strides of whole 16-byte rows (scales:
``head_dim / 16`` bytes), keys and values with the same strides.  Slot s of sequence b is
entry ``s % page_size`` of page ``block_table[b, s // page_size]``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

F16, KV4 = 2, 3
_CODES = {torch.bfloat16: 1, torch.float16: F16}
_SCALE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


class _KvPages(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("k", "v", "k_scales", "v_scales", "block_table")]
                + [(f, ctypes.c_int64) for f in ("page_stride", "slot_stride", "head_stride", "scale_page_stride",
                                                 "scale_slot_stride", "scale_head_stride")]
                + [(f, ctypes.c_int32) for f in ("num_pages", "page_size", "max_pages", "kv_heads", "head_dim",
                                                 "format")]
                + [(f, ctypes.c_float) for f in ("k_scale", "v_scale")])


_Strides = ctypes.c_int64 * 3


def declare(lib) -> None:
    """The argument types of the library's cache calls."""
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    st, pg = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(_KvPages)
    lib.specdec_rotate_qk.argtypes = [vp, st, vp, st, vp, st, i32, vp, vp, f32, vp, i32, i32, vp, vp, vp, i32, i32,
                                      i32, i32, i32, vp, vp, pg, vp, vp]
    lib.specdec_append_kv4.argtypes = [vp, st, vp, st, i32, vp, vp, i32, i32, pg, vp, vp]
    lib.specdec_read_kv4.argtypes = [vp, vp, i32, i32, pg, i32, vp, vp, vp, vp]
    lib.specdec_attend_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.specdec_attend_workspace_bytes.restype = sz
    lib.specdec_attend.argtypes = [vp, st, i32, pg, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp, sz,
                                   vp]
    for f in (lib.specdec_rotate_qk, lib.specdec_append_kv4, lib.specdec_read_kv4, lib.specdec_attend):
        f.restype = i32


def _steps(t):
    """Strides, 0 for dimensions of one entry (whose stride means nothing)."""
    return tuple(0 if n == 1 else s for n, s in zip(t.shape, t.stride()))


def _call_stream(device, stream):
    """The call's stream, and a context in which its outputs belong to that stream."""
    if device.type != "cuda":
        raise ValueError(f"the cache calls take CUDA tensors, got {device}")
    current = torch.cuda.current_stream(device)
    if stream is None:
        stream = current
    if stream == current and device.index == torch.cuda.current_device():
        return stream, contextlib.nullcontext()
    return stream, torch.cuda.stream(stream)


def _view(t, name, dtype, shape, device):
    """A [B, n, heads, D] view with contiguous rows; its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    s = _steps(t)
    if s[3] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _Strides(s[0], s[1], s[2])


def _small(t, name, dtype, shape, device):
    """The address of a contiguous tensor (None: no tensor)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pages(k, v, block_table, B, device, head_dim=None, k_scales=None, v_scales=None, k_scale=1.0, v_scale=1.0):
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("k_pages and v_pages must be torch.Tensors")
    four = k.dtype == torch.uint8
    if (k.dtype not in _CODES and not four) or k.dim() != 4:
        raise ValueError("pages must be [num_pages, page_size, kv_heads, head_dim] of bfloat16 or float16, or uint8 "
                         "codes [..., head_dim / 2]")
    if v.dtype != k.dtype or v.shape != k.shape or _steps(v) != _steps(k) or k.device != device or v.device != device:
        raise ValueError("k_pages and v_pages must have the same type, shape and strides, on the call's device")
    st, es = _steps(k), k.element_size()
    if st[3] != 1:
        raise ValueError("the pages' last dimension must be contiguous")
    pg = _KvPages()
    pg.num_pages, pg.page_size, pg.kv_heads = k.shape[0], k.shape[1], k.shape[2]
    pg.head_dim = k.shape[3] * 2 if four else k.shape[3]
    if head_dim is not None and pg.head_dim != head_dim:
        raise ValueError(f"the pages hold heads of {pg.head_dim}, the call has {head_dim}")
    pg.k, pg.v = k.data_ptr(), v.data_ptr()
    pg.page_stride, pg.slot_stride, pg.head_stride = st[0] * es, st[1] * es, st[2] * es
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages] int32")
    pg.max_pages = block_table.shape[1]
    pg.block_table = _small(block_table, "block_table", torch.int32, (B, pg.max_pages), device)
    if four:
        want = (*k.shape[:3], pg.head_dim // 16)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"pages held in 4 bits need {name}")
            if t.dtype not in _SCALE_DTYPES or t.shape != want or t.device != device or t.stride(3) != 1:
                raise ValueError(f"{name} must be E4M3 bytes of shape {want} on {device}, the last dimension contiguous")
        if _steps(k_scales) != _steps(v_scales):
            raise ValueError("k_scales and v_scales must have the same strides")
        st = _steps(k_scales)
        pg.k_scales, pg.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        pg.scale_page_stride, pg.scale_slot_stride, pg.scale_head_stride = st[0], st[1], st[2]
        pg.k_scale, pg.v_scale, pg.format = k_scale, v_scale, KV4
    else:
        if k_scales is not None or v_scales is not None:
            raise ValueError("16-bit pages have no scales")
        pg.format = _CODES[k.dtype]
    return pg


def _checked(rc, what):
    if rc != 0:
        from . import SpecdecError, _ERR_NAMES, load_library
        detail = load_library().specdec_last_error().decode(errors="replace")
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
    from . import load_library
    lib = load_library()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.dtype not in _CODES:
        raise ValueError("q must be [B, n, q_heads, D] bfloat16 or float16")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, n, kv_heads, D]")
    B, n, hq, D = q.shape
    hkv, dev, dt = k.shape[2], q.device, q.dtype
    s, own = _call_stream(dev, stream)
    qs = _view(q, "q", dt, q.shape, dev)
    ks = _view(k, "k", dt, (B, n, hkv, D), dev)
    if not isinstance(turns, torch.Tensor) or turns.dim() != 1:
        raise ValueError("turns must be [rot / 2] int64")
    args = (_small(q_weight, "q_weight", dt, (D,), dev), _small(k_weight, "k_weight", dt, (D,), dev), float(eps),
            _small(turns, "turns", torch.int64, (turns.shape[0],), dev), 2 * turns.shape[0], 1 if interleaved else 0,
            _small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev), _small(depth, "depth", torch.int32, (n,), dev))
    pages = vs = None
    if k_pages is not None or v_pages is not None or block_table is not None:
        vs = _view(v, "v", dt, (B, n, hkv, D), dev)
        pages = _pages(k_pages, v_pages, block_table, B, dev, D)
    with own:
        out = {"q": torch.empty((B, n, hq, D), dtype=dt, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
        if pages is None:
            out["k"] = torch.empty((B, n, hkv, D), dtype=dt, device=dev)
    _checked(lib.specdec_rotate_qk(q.data_ptr(), qs, k.data_ptr(), ks, None if vs is None else v.data_ptr(), vs,
                                   _CODES[dt], *args, B, n, hq, hkv, D, out["q"].data_ptr(),
                                   out["k"].data_ptr() if pages is None else None, pages, out["status"].data_ptr(),
                                   s.cuda_stream), "specdec_rotate_qk")
    return out


def append_kv4(k, v, k_pages, v_pages, block_table, context_len, *, k_scales, v_scales, k_scale: float = 1.0,
               v_scale: float = 1.0, query_len=None, stream=None) -> dict:
    """Keys and values [B, n, kv_heads, D] of the new tokens written to 4-bit pages
    (specdec_append_kv4).  Returns status [B]."""
    from . import load_library
    lib = load_library()
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.dtype not in _CODES:
        raise ValueError("k must be [B, n, kv_heads, D] bfloat16 or float16")
    B, n, hkv, D = k.shape
    dev, dt = k.device, k.dtype
    s, own = _call_stream(dev, stream)
    ks, vs = _view(k, "k", dt, k.shape, dev), _view(v, "v", dt, k.shape, dev)
    pages = _pages(k_pages, v_pages, block_table, B, dev, D, k_scales, v_scales, k_scale, v_scale)
    if pages.kv_heads != hkv:
        raise ValueError(f"the pages hold {pages.kv_heads} heads, k has {hkv}")
    lens = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev))
    with own:
        status = torch.empty(B, dtype=torch.int32, device=dev)
    _checked(lib.specdec_append_kv4(k.data_ptr(), ks, v.data_ptr(), vs, _CODES[dt], *lens, B, n, pages,
                                    status.data_ptr(), s.cuda_stream), "specdec_append_kv4")
    return {"status": status}


def read_kv4(k_pages, v_pages, block_table, context_len, n: int, *, k_scales, v_scales, k_scale: float = 1.0,
             v_scale: float = 1.0, query_len=None, dtype=torch.bfloat16, stream=None) -> dict:
    """The values that 4-bit pages hold for the last n tokens (query_len[b] <= n) of each
    sequence (specdec_read_kv4): k, v [B, n, kv_heads, D] of dtype, and status [B]."""
    from . import load_library
    lib = load_library()
    if dtype not in _CODES:
        raise ValueError("dtype must be bfloat16 or float16")
    if not isinstance(k_pages, torch.Tensor) or not isinstance(context_len, torch.Tensor):
        raise TypeError("k_pages and context_len must be torch.Tensors")
    dev, B = k_pages.device, context_len.shape[0]
    s, own = _call_stream(dev, stream)
    pages = _pages(k_pages, v_pages, block_table, B, dev, None, k_scales, v_scales, k_scale, v_scale)
    lens = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev))
    n = int(n)
    with own:
        shape = (B, max(n, 0), pages.kv_heads, pages.head_dim)
        out = {"k": torch.empty(shape, dtype=dtype, device=dev), "v": torch.empty(shape, dtype=dtype, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
    _checked(lib.specdec_read_kv4(*lens, B, n, pages, _CODES[dtype], out["k"].data_ptr(), out["v"].data_ptr(),
                                  out["status"].data_ptr(), s.cuda_stream), "specdec_read_kv4")
    return out


def attend(q, k_pages, v_pages, block_table, context_len, *, query_len=None, tree_mask=None, depth=None,
           window: int = 0, sinks: int = 0, scale=None, k_scales=None, v_scales=None, k_scale: float = 1.0,
           v_scale: float = 1.0, with_lse: bool = False, stream=None) -> dict:
    """Attention of the new tokens over a paged cache that holds their keys and values already
    (specdec_attend): chain or tree, a sliding window with a few first tokens that stay
    visible, 16-bit or 4-bit pages.

    q [B, n, q_heads, D] bfloat16 or float16, a view with contiguous rows; context_len [B] int32,
    the new tokens included; query_len [B] int32 (default n); tree_mask [n, n] uint8 and depth [n]
    int32: ``build_tree_mask(parents, 0)``'s mask and depth; scale: default 1 / sqrt(D).
    Returns out [B, n, q_heads, D], status [B] and, with_lse, lse [B, n, q_heads] fp32."""
    from . import _workspace, load_library
    lib = load_library()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.dtype not in _CODES:
        raise ValueError("q must be [B, n, q_heads, D] bfloat16 or float16")
    B, n, hq, D = q.shape
    dev, dt = q.device, q.dtype
    s, own = _call_stream(dev, stream)
    qs = _view(q, "q", dt, q.shape, dev)
    pages = _pages(k_pages, v_pages, block_table, B, dev, D, k_scales, v_scales, k_scale, v_scale)
    if pages.format != KV4 and k_pages.dtype != dt:
        raise ValueError(f"q is {dt}, the pages are {k_pages.dtype}")
    args = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev),
            _small(tree_mask, "tree_mask", torch.uint8, (n, n), dev), _small(depth, "depth", torch.int32, (n,), dev))
    need = int(lib.specdec_attend_workspace_bytes(B, n, hq, pages.kv_heads, D))
    with own:
        out = {"out": torch.empty((B, n, hq, D), dtype=dt, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
        if with_lse:
            out["lse"] = torch.empty((B, n, hq), dtype=torch.float32, device=dev)
        if torch.cuda.is_current_stream_capturing():
            # a graph keeps its own workspace: the shared one may be replaced by a larger one
            ws, wsb = torch.empty(need, dtype=torch.uint8, device=dev), need
        else:
            ws, wsb = _workspace(need, dev, s.cuda_stream)
    _checked(lib.specdec_attend(q.data_ptr(), qs, _CODES[dt], pages, *args, B, n, hq, int(window), int(sinks),
                                1.0 / math.sqrt(D) if scale is None else float(scale), out["out"].data_ptr(),
                                out["lse"].data_ptr() if with_lse else None, out["status"].data_ptr(),
                                None if ws is None else ws.data_ptr(), wsb, s.cuda_stream), "specdec_attend")
    return out
