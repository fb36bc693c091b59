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


# One call marshals some twenty values for kernels of a few microseconds, so the checks below
# are written for few attribute reads: about 0.1 us each on a GB300 host.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _call_stream(t, name, stream):
    """The device, the handle of the call's stream, and a context in which new tensors belong
    to that stream (None: the current one, nothing to switch)."""
    if not t.is_cuda:
        raise ValueError(f"the cache calls take CUDA tensors, {name} is on {t.device}")
    dev = t.device
    if stream is None:
        if dev.index == torch._C._cuda_getDevice():
            return dev, _raw_stream(dev.index), None
        stream = torch.cuda.current_stream(dev)
    return dev, stream.cuda_stream, torch.cuda.stream(stream)


def _strides(t, unit=1):
    """The first three strides of a 4-dimensional tensor, 0 for dimensions of one entry (whose
    stride means nothing); None where the last dimension is not contiguous."""
    a, b, c, d = t.stride()
    if d != 1:
        return None
    x, y, z, _ = t.shape
    return (a * unit if x != 1 else 0, b * unit if y != 1 else 0, c * unit if z != 1 else 0)


def _view(t, name, dtype, shape, device):
    """A [B, n, heads, D] view with contiguous rows; its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    s = _strides(t)
    if s is None:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _Strides(*s)


def _small(t, name, dtype, shape, device):
    """The address of a contiguous tensor (None: no tensor)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pages(k, v, block_table, B, device, head_dim=None, k_scales=None, v_scales=None, k_scale=1.0, v_scale=1.0):
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("k_pages and v_pages must be torch.Tensors")
    dt, shape = k.dtype, k.shape
    four = dt is torch.uint8
    if (not four and dt not in _CODES) or len(shape) != 4:
        raise ValueError("pages must be [num_pages, page_size, kv_heads, head_dim] of bfloat16 or float16, or uint8 "
                         "codes [..., head_dim / 2]")
    if v.dtype is not dt or v.shape != shape or k.device != device or v.device != device:
        raise ValueError("k_pages and v_pages must have the same type and shape, on the call's device")
    st = _strides(k, 1 if four else 2)
    if st is None or _strides(v, 1 if four else 2) != st:
        raise ValueError("k_pages and v_pages must have the same strides and a contiguous last dimension")
    num, page, heads, width = shape
    if four:
        width *= 2
    if head_dim is not None and width != head_dim:
        raise ValueError(f"the pages hold heads of {width}, the call has {head_dim}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages] int32")
    per = block_table.shape[1]
    table = _small(block_table, "block_table", torch.int32, (B, per), device)
    if not four:
        if k_scales is not None or v_scales is not None:
            raise ValueError("16-bit pages have no scales")
        return _KvPages(k.data_ptr(), v.data_ptr(), None, None, table, *st, 0, 0, 0, num, page, per, heads, width,
                        _CODES[dt], 1.0, 1.0)
    want = (num, page, heads, width // 16)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"pages held in 4 bits need {name}")
        if t.dtype not in _SCALE_DTYPES or t.shape != want or t.device != device:
            raise ValueError(f"{name} must be E4M3 bytes of shape {want} on {device}")
    sst = _strides(k_scales)
    if sst is None or _strides(v_scales) != sst:
        raise ValueError("k_scales and v_scales must have the same strides and a contiguous last dimension")
    return _KvPages(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), table, *st, *sst, num, page, per,
                    heads, width, KV4, k_scale, v_scale)


_NO_SWITCH = contextlib.nullcontext()
_lib = _workspace = None


def _library():
    global _lib, _workspace
    if _lib is None:
        from . import _workspace as workspace, load_library
        _lib, _workspace = load_library(), workspace
    return _lib


def _failed(rc, what):
    from . import SpecdecError, _ERR_NAMES
    detail = _library().specdec_last_error().decode(errors="replace")
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
    lib = _library()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.dtype not in _CODES:
        raise ValueError("q must be [B, n, q_heads, D] bfloat16 or float16")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, n, kv_heads, D]")
    B, n, hq, D = q.shape
    hkv, dt = k.shape[2], q.dtype
    dev, s, switch = _call_stream(q, "q", stream)
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
    with switch or _NO_SWITCH:
        out = {"q": torch.empty((B, n, hq, D), dtype=dt, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
        if pages is None:
            out["k"] = torch.empty((B, n, hkv, D), dtype=dt, device=dev)
        rc = lib.specdec_rotate_qk(q.data_ptr(), qs, k.data_ptr(), ks, None if vs is None else v.data_ptr(), vs,
                                   _CODES[dt], *args, B, n, hq, hkv, D, out["q"].data_ptr(),
                                   out["k"].data_ptr() if pages is None else None, pages, out["status"].data_ptr(),
                                   s)
    if rc:
        _failed(rc, "specdec_rotate_qk")
    return out


def append_kv4(k, v, k_pages, v_pages, block_table, context_len, *, k_scales, v_scales, k_scale: float = 1.0,
               v_scale: float = 1.0, query_len=None, stream=None) -> dict:
    """Keys and values [B, n, kv_heads, D] of the new tokens written to 4-bit pages
    (specdec_append_kv4).  Returns status [B]."""
    lib = _library()
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.dtype not in _CODES:
        raise ValueError("k must be [B, n, kv_heads, D] bfloat16 or float16")
    B, n, hkv, D = k.shape
    dt = k.dtype
    dev, s, switch = _call_stream(k, "k", stream)
    ks, vs = _view(k, "k", dt, k.shape, dev), _view(v, "v", dt, k.shape, dev)
    pages = _pages(k_pages, v_pages, block_table, B, dev, D, k_scales, v_scales, k_scale, v_scale)
    if pages.kv_heads != hkv:
        raise ValueError(f"the pages hold {pages.kv_heads} heads, k has {hkv}")
    lens = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev))
    with switch or _NO_SWITCH:
        status = torch.empty(B, dtype=torch.int32, device=dev)
        rc = lib.specdec_append_kv4(k.data_ptr(), ks, v.data_ptr(), vs, _CODES[dt], *lens, B, n, pages,
                                    status.data_ptr(), s)
    if rc:
        _failed(rc, "specdec_append_kv4")
    return {"status": status}


def read_kv4(k_pages, v_pages, block_table, context_len, n: int, *, k_scales, v_scales, k_scale: float = 1.0,
             v_scale: float = 1.0, query_len=None, dtype=torch.bfloat16, stream=None) -> dict:
    """The values that 4-bit pages hold for the last n tokens (query_len[b] <= n) of each
    sequence (specdec_read_kv4): k, v [B, n, kv_heads, D] of dtype, and status [B]."""
    lib = _library()
    if dtype not in _CODES:
        raise ValueError("dtype must be bfloat16 or float16")
    if not isinstance(k_pages, torch.Tensor) or not isinstance(context_len, torch.Tensor):
        raise TypeError("k_pages and context_len must be torch.Tensors")
    B = context_len.shape[0]
    dev, s, switch = _call_stream(k_pages, "k_pages", stream)
    pages = _pages(k_pages, v_pages, block_table, B, dev, None, k_scales, v_scales, k_scale, v_scale)
    lens = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev))
    n = int(n)
    with switch or _NO_SWITCH:
        shape = (B, max(n, 0), pages.kv_heads, pages.head_dim)
        out = {"k": torch.empty(shape, dtype=dtype, device=dev), "v": torch.empty(shape, dtype=dtype, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
        rc = lib.specdec_read_kv4(*lens, B, n, pages, _CODES[dtype], out["k"].data_ptr(), out["v"].data_ptr(),
                                  out["status"].data_ptr(), s)
    if rc:
        _failed(rc, "specdec_read_kv4")
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
    lib = _library()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.dtype not in _CODES:
        raise ValueError("q must be [B, n, q_heads, D] bfloat16 or float16")
    B, n, hq, D = q.shape
    dt = q.dtype
    dev, s, switch = _call_stream(q, "q", stream)
    qs = _view(q, "q", dt, q.shape, dev)
    pages = _pages(k_pages, v_pages, block_table, B, dev, D, k_scales, v_scales, k_scale, v_scale)
    if pages.format != KV4 and k_pages.dtype != dt:
        raise ValueError(f"q is {dt}, the pages are {k_pages.dtype}")
    args = (_small(context_len, "context_len", torch.int32, (B,), dev),
            _small(query_len, "query_len", torch.int32, (B,), dev),
            _small(tree_mask, "tree_mask", torch.uint8, (n, n), dev), _small(depth, "depth", torch.int32, (n,), dev))
    need = int(lib.specdec_attend_workspace_bytes(B, n, hq, pages.kv_heads, D))
    with switch or _NO_SWITCH:
        out = {"out": torch.empty((B, n, hq, D), dtype=dt, device=dev),
               "status": torch.empty(B, dtype=torch.int32, device=dev)}
        if with_lse:
            out["lse"] = torch.empty((B, n, hq), dtype=torch.float32, device=dev)
        if torch._C._cuda_isCurrentStreamCapturing():
            # a graph keeps its own workspace: the shared one may be replaced by a larger one
            ws, wsb = torch.empty(need, dtype=torch.uint8, device=dev), need
        else:
            ws, wsb = _workspace(need, dev, s)
        rc = lib.specdec_attend(q.data_ptr(), qs, _CODES[dt], pages, *args, B, n, hq, int(window), int(sinks),
                                1.0 / math.sqrt(D) if scale is None else float(scale), out["out"].data_ptr(),
                                out["lse"].data_ptr() if with_lse else None, out["status"].data_ptr(),
                                None if ws is None else ws.data_ptr(), wsb, s)
    if rc:
        _failed(rc, "specdec_attend")
    return out
