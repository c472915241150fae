"""The microscaled key/value cache: a thin binding over the entry points of include/mx_kv.h.

    import microscaling_fp4_weight_amd as mx
    cache = mx.mxkv_alloc(pages, heads, page_size, dim)             # E2M1 elements, E8M0 blocks of 32
    table = mx.mxkv_rope_table(max_pos, dim)
    q = mx.mxkv_rope(q, positions, table)                           # (tokens, q_heads, dim)
    mx.mxkv_write(k, v, cache, slots, positions=positions, table=table)
    out = mx.mxkv_attention(q.view(batch, new, q_heads, dim), cache, block_table, lens)

As elsewhere in this package every function only checks and marshals tensors; the arithmetic runs
in the library's HIP kernels, on the current stream unless one is given.  With a stream given, results that are
not passed in and the workspace are memory of that stream, and the caller orders it with others.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from .streams import made_on

ELEMENT = {"fp4": 0, "fp8": 1}
SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3}
_FMT = {"e4m3": 0, "ue5m3": 1, "e8m0": 2}
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_TYPE = {_F32: 0, _BF16: 1}


class KVCache(NamedTuple):
    """A pool's four byte tensors: codes (pages, heads, page, dim / 2 or dim), scales (pages,
    heads, page, dim / block), for keys and for values."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


# mxkv_cache: four pointers, pages, then heads, page size, dim, block, element, format and the two
# per-tensor scales
_POOL = struct.Struct("=4Qq6i2f")


class _Pool(NamedTuple):
    heads: int
    dim: int
    packed: bytes


_lib = None


def _entry():
    """The library with the argument types of these entry points set."""
    global _lib
    if _lib is None:
        from . import lib
        L = lib()
        i32, i64, f32, f64, vp, sz = (ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p,
                                      ctypes.c_size_t)
        pool = ctypes.c_char_p  # the packed mxkv_cache
        L.mxkv_rope_table.argtypes = [vp, i64, i32, f64, i32, f64, f64, f64, f64, f64, vp]
        L.mxkv_rope.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, vp, i64, i32, i32, i32, vp, i64, i64, vp]
        L.mxkv_write.argtypes = [pool, vp, vp, i32, i64, i64, i64, i64, i64, vp, vp, vp, i64, i32, i32, vp, vp, vp]
        L.mxkv_read.argtypes = [pool, vp, i64, vp, vp, i32, vp]
        L.mxkv_attention_workspace_size.argtypes = [pool, i64, i64, i64, i64]
        L.mxkv_attention.argtypes = [pool, vp, i64, i64, i64, i64, i64, i64, vp, i64, i64, vp, vp, vp, i64, i64, f32, vp,
                                     vp, vp, sz, vp]
        for f in (L.mxkv_rope_table, L.mxkv_rope, L.mxkv_write, L.mxkv_read, L.mxkv_attention):
            f.restype = i32
        L.mxkv_attention_workspace_size.restype = sz
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        from . import MXError
        raise MXError(status, where)


def _stream(stream, device: int) -> int:
    """The stream's handle.  A null handle means the current device's null stream, so the tensors'
    device has to be current."""
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"the tensors are on GPU {device}, the current device is {torch._C._cuda_getDevice()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the tensors are on GPU {device}, the stream on GPU {stream.device_index}")
    return stream.cuda_stream


def _on_gpu(t: torch.Tensor) -> int:
    """The index of the GPU that holds t."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"the tensors must be on a GPU (device {t.device})")
    return device


def _same_device(device: int, *tensors):
    """The tensors, which may be None, are on that GPU; dtypes and sizes have been checked before."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, the others on GPU {device}")


def _indices(t: torch.Tensor, name: str, n: int) -> int:
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be of dtype {_I32}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _dense(t: torch.Tensor, name: str):
    """Shape and strides of a (tokens, heads, dim) bf16 / fp32 tensor with unit stride along dim."""
    if t.dtype is not _BF16 and t.dtype is not _F32:
        raise TypeError(f"{name} must be of dtype {_BF16} or {_F32}, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or (strides[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be a 3-D tensor (tokens, heads, dim) with unit stride along dim")
    return shape, strides


def _like(t: torch.Tensor, name: str, shape, dtype) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be of dtype {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and of shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _pool(cache, block: int, fmt: str, element: str, k_scale: float, v_scale: float) -> _Pool:
    kc, ks, vc, vs = cache
    for name, t in (("k_codes", kc), ("k_scales", ks), ("v_codes", vc), ("v_scales", vs)):
        if t.dtype is not _U8:
            raise TypeError(f"cache {name} must be of dtype {_U8}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"cache {name} must be contiguous")
    shape = kc.shape
    if len(shape) != 4:
        raise ValueError("cache tensors must be 4-D (pages, heads, page, bytes)")
    pages, heads, page, width = shape
    kind = ELEMENT[element]
    dim = width if kind else width * 2
    if block < 1 or dim % block:
        raise ValueError(f"a head of {dim} elements is no whole number of blocks of {block}")
    if vc.shape != shape:
        raise ValueError(f"v_codes has shape {tuple(vc.shape)}, k_codes {tuple(shape)}")
    want = (pages, heads, page, dim // block)
    if ks.shape != want or vs.shape != want:
        raise ValueError(f"cache scales must have shape {want}, got {tuple(ks.shape)} and {tuple(vs.shape)}")
    return _Pool(heads, dim, _POOL.pack(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, heads, page, dim,
                                        block, kind, _FMT[fmt], k_scale, v_scale))


def _rope_args(positions, table, tokens: int, dim: int):
    """(positions pointer, table pointer, max_pos, rot_dim) of a checked rotation."""
    if table is None:
        return None, None, 0, 0
    if positions is None:
        raise ValueError("a table needs positions")
    where = _indices(positions, "positions", tokens)
    if table.dtype is not _F32:
        raise TypeError(f"table must be of dtype {_F32}, got {table.dtype}")
    shape = table.shape
    if len(shape) != 2 or shape[0] < 1 or not table.is_contiguous():
        raise ValueError("table must be a contiguous 2-D tensor (max_pos, rot_dim)")
    if shape[1] > dim:
        raise ValueError(f"table rotates {shape[1]} elements of a head of {dim}")
    return where, table.data_ptr(), shape[0], shape[1]


def mxkv_alloc(num_pages: int, heads: int, page_size: int, dim: int, block: int = 32, element: str = "fp4",
               device="cuda") -> KVCache:
    """An empty pool of num_pages pages of page_size tokens."""
    if block < 1 or dim % block:
        raise ValueError(f"a head of {dim} elements is no whole number of blocks of {block}")
    width = dim // 2 if ELEMENT[element] == 0 else dim
    return KVCache(*(torch.zeros((num_pages, heads, page_size, w), dtype=_U8, device=device)
                     for w in (width, dim // block, width, dim // block)))


def mxkv_rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                    original_len: float = 0.0, low: float = 1.0, high: float = 32.0, magnitude: float = 1.0,
                    device="cuda", stream=None) -> torch.Tensor:
    """cos | sin of position * frequency, (max_pos, rot_dim) fp32.  `scaling` stretches the
    frequencies for long contexts: "linear" divides them by factor, "base" enlarges the base,
    "parts" divides only those that make few turns (between low and high) in original_len positions."""
    table = made_on(stream, torch.empty, (max_pos, rot_dim), dtype=_F32, device=device)
    _check(_entry().mxkv_rope_table(table.data_ptr(), max_pos, rot_dim, base, SCALING[scaling], factor, original_len, low,
                                    high, magnitude, _stream(stream, _on_gpu(table))), "mxkv_rope_table")
    return table


def mxkv_rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, interleaved: bool = False,
              transpose: bool = False, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x (tokens, heads, dim; bf16 or fp32): the first table.size(1) elements
    of each head are turned by their token's angles, in pairs (i, i + rot / 2) or, interleaved,
    (2 i, 2 i + 1).  `transpose` turns back: the gradient dx of dy.  y may be x."""
    shape, ld = _dense(x, "x")
    tokens, heads, dim = shape
    pos, tab, max_pos, rot = _rope_args(positions, table, tokens, dim)
    if y is not None:
        yshape, ldy = _dense(y, "y")
        if yshape != shape or y.dtype is not x.dtype:
            raise ValueError("y must have the shape and dtype of x")
    device = _on_gpu(x)
    _same_device(device, positions, table, y)
    where = _stream(stream, device)
    if y is None:
        y = made_on(stream, torch.empty_like, x)  # as dense as x: unit stride along dim
        ldy = y.stride()
    st = _entry().mxkv_rope(x.data_ptr(), _TYPE[x.dtype], tokens, heads, dim, ld[0], ld[1], pos, tab, max_pos, rot, interleaved,
                            transpose, y.data_ptr(), ldy[0], ldy[1], where)
    if st:
        _check(st, "mxkv_rope")
    return y


def mxkv_write(k: torch.Tensor, v: torch.Tensor, cache, slots: torch.Tensor, block: int = 32, fmt: str = "e8m0",
               element: str = "fp4", k_scale: float = 1.0, v_scale: float = 1.0, positions: torch.Tensor | None = None,
               table: torch.Tensor | None = None, interleaved: bool = False, k_hat: torch.Tensor | None = None,
               v_hat: torch.Tensor | None = None, stream=None):
    """Quantize the keys and values (tokens, heads, dim; bf16 or fp32) of `tokens` tokens into their
    slots (int32; one outside the pool is passed over, and no two tokens of a call may share one).  With a
    table the keys are rotated first, as mxkv_rope does.  k_hat and v_hat, if given (both), receive the
    values that the codes stand for."""
    heads, dim, pool = _pool(cache, block, fmt, element, k_scale, v_scale)
    shape, ldk = _dense(k, "k")
    vshape, ldv = _dense(v, "v")
    tokens = shape[0]
    if shape[1] != heads or shape[2] != dim:
        raise ValueError(f"k must have shape (tokens, {heads}, {dim}), got {tuple(shape)}")
    if vshape != shape or v.dtype is not k.dtype:
        raise ValueError("v must have the shape and dtype of k")
    where = _indices(slots, "slots", tokens)
    pos, tab, max_pos, rot = _rope_args(positions, table, tokens, dim)
    if (k_hat is None) != (v_hat is None):
        raise ValueError("k_hat and v_hat go together")
    kh = vh = None
    if k_hat is not None:
        kh, vh = _like(k_hat, "k_hat", shape, k.dtype), _like(v_hat, "v_hat", shape, k.dtype)
    device = _on_gpu(k)
    _same_device(device, v, *cache, slots, positions, table, k_hat, v_hat)
    st = _entry().mxkv_write(pool, k.data_ptr(), v.data_ptr(), _TYPE[k.dtype], tokens, ldk[0], ldk[1], ldv[0], ldv[1], where,
                             pos, tab, max_pos, rot, interleaved, kh, vh, _stream(stream, device))
    if st:
        _check(st, "mxkv_write")


def mxkv_read(cache, slots: torch.Tensor, block: int = 32, fmt: str = "e8m0", element: str = "fp4", k_scale: float = 1.0,
              v_scale: float = 1.0, out_dtype: torch.dtype = torch.bfloat16, k: torch.Tensor | None = None,
              v: torch.Tensor | None = None, stream=None):
    """The keys and values that the slots (int32) hold, as (tokens, heads, dim) tensors of out_dtype;
    zeros for a slot outside the pool."""
    heads, dim, pool = _pool(cache, block, fmt, element, k_scale, v_scale)
    tokens = slots.numel()
    where = _indices(slots, "slots", tokens)
    if out_dtype not in _TYPE:
        raise TypeError(f"unsupported dtype {out_dtype}")
    shape = (tokens, heads, dim)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _like(t, name, shape, out_dtype)
    device = _on_gpu(slots)
    _same_device(device, *cache, k, v)
    on = _stream(stream, device)
    if k is None:
        k = made_on(stream, torch.empty, shape, dtype=out_dtype, device=slots.device)
    if v is None:
        v = made_on(stream, torch.empty, shape, dtype=out_dtype, device=slots.device)
    st = _entry().mxkv_read(pool, where, tokens, k.data_ptr(), v.data_ptr(), _TYPE[out_dtype], on)
    if st:
        _check(st, "mxkv_read")
    return k, v


def mxkv_attention_workspace_size(cache, batch: int, new_tokens: int, q_heads: int, max_pages: int, block: int = 32,
                                  element: str = "fp4") -> int:
    pool = _pool(cache, block, "e8m0", element, 1.0, 1.0)
    return int(_entry().mxkv_attention_workspace_size(pool.packed, batch, new_tokens, q_heads, max_pages))


def mxkv_attention(q: torch.Tensor, cache, block_table: torch.Tensor, lens: torch.Tensor, block: int = 32,
                   fmt: str = "e8m0", element: str = "fp4", k_scale: float = 1.0, v_scale: float = 1.0,
                   n_new: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                   softmax_scale: float | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None,
                   stream=None):
    """Attention of the new tokens q (batch, new, q_heads, dim; bf16) over the cache, whose pages
    block_table (batch, pages; int32) lists for each sequence.  A sequence has lens[b] tokens
    before its n_new[b] (default: all) new ones, which are in the cache already.  New token i sees
    all tokens before, and new token j where mask (batch or 1, new, new; bool or uint8) is true, or
    j <= i without a mask.  Returns out (as q), with return_lse also lse (batch, new, q_heads; fp32).
    softmax_scale defaults to dim ** -0.5."""
    heads, dim, pool = _pool(cache, block, fmt, element, k_scale, v_scale)
    if q.dtype is not _BF16:
        raise TypeError(f"q must be of dtype {_BF16}, got {q.dtype}")
    shape, ldq = q.shape, q.stride()
    if len(shape) != 4 or shape[3] != dim or (ldq[3] != 1 and dim > 1):
        raise ValueError(f"q must be a 4-D tensor (batch, new, q_heads, {dim}) with unit stride along dim")
    batch, new, q_heads, _ = shape
    if block_table.dtype is not _I32:
        raise TypeError(f"block_table must be of dtype {_I32}, got {block_table.dtype}")
    tshape, ldt = block_table.shape, block_table.stride()
    if len(tshape) != 2 or tshape[0] != batch or (ldt[1] != 1 and tshape[1] > 1):
        raise ValueError(f"block_table must be a 2-D tensor ({batch}, pages) with unit stride along pages")
    max_pages = tshape[1]
    lp = _indices(lens, "lens", batch)
    np = None if n_new is None else _indices(n_new, "n_new", batch)
    mp, mb, mr = None, 0, 0
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not _U8:
            raise TypeError(f"mask must be of dtype {torch.bool} or {_U8}, got {mask.dtype}")
        mshape, ldm = mask.shape, mask.stride()
        if mshape != (batch, new, new) and mshape != (1, new, new) or (ldm[2] != 1 and new > 1):
            raise ValueError(f"mask must be a 3-D tensor ({batch} or 1, {new}, {new}) with unit stride along the last")
        mp, mb, mr = mask.data_ptr(), 0 if mshape[0] == 1 else ldm[0], ldm[1]
    if out is not None:
        _like(out, "out", shape, _BF16)
    if lse is not None:
        _like(lse, "lse", (batch, new, q_heads), _F32)
    L = _entry()
    need = L.mxkv_attention_workspace_size(pool, batch, new, q_heads, max_pages)
    if workspace is not None and (workspace.dtype is not _U8 or not workspace.is_contiguous() or workspace.numel() < need):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes")
    device = _on_gpu(q)
    _same_device(device, *cache, block_table, lens, n_new, mask, out, lse, workspace)
    where = _stream(stream, device)
    if out is None:
        out = made_on(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
    if return_lse and lse is None:
        lse = made_on(stream, torch.empty, (batch, new, q_heads), dtype=_F32, device=q.device)
    if workspace is None and need:
        workspace = made_on(stream, lens.new_empty, need, dtype=_U8)
    op, ep = out.data_ptr(), None if lse is None else lse.data_ptr()
    wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    st = L.mxkv_attention(pool, q.data_ptr(), batch, new, q_heads, ldq[0], ldq[1], ldq[2], block_table.data_ptr(), max_pages,
                          ldt[0], lp, np, mp, mb, mr, dim ** -0.5 if softmax_scale is None else softmax_scale, op, ep, wp, wn,
                          where)
    if st:
        _check(st, "mxkv_attention")
    return (out, lse) if return_lse else out
