"""The 8-bit block cache of ``include/fa_cache.h``: planning its block tables,
appending keys and values, and the attention that reads it.

    cache = fa.cache_empty(num_blocks, heads, block, d)
    slots, cu, kv_lens, pos = fa.cache_plan(lens, new_lens, table, free, pos, T, block)
    fa.cache_append(k, v, slots, cache)                  # k, v: [T, heads, d]
    o, lse = fa.attention_forward_cache(q, cache, table, kv_lens, cu)   # q: [T, H, d]

Like the rest of the binding this only marshals arguments.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

from . import (FA_DTYPE_BF16, FA_DTYPE_FP16, FA_OK, FaError, FaStrides, _allocating_on, _build,
               load_library)

HEADER = os.path.join(_build.INCLUDE, "fa_cache.h")


class FaCache(ctypes.Structure):
    """fa_cache: pointers, sizes and byte strides of a block cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int), ("block", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("block_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong)]


class Cache(NamedTuple):
    """A block cache as torch tensors: k and v [num_blocks, heads, block, d] of
    e4m3 codes (float8_e4m3fn or uint8; equal strides, unit along d, the others
    multiples of 16), k_scales and v_scales contiguous float32
    [num_blocks, heads]. Any tuple of the four serves as one."""
    k: object
    v: object
    k_scales: object
    v_scales: object


def bind(lib) -> None:
    """Argument types of the cache's entry points."""
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_cache_plan.argtypes = [vp, vp, vp, i, vp, i, vp, vp, i, vp, vp, vp, i, i, vp]
    lib.fa_cache_plan.restype = i
    lib.fa_cache_append.argtypes = [vp, vp, ctypes.POINTER(FaStrides), vp, i,
                                    ctypes.POINTER(FaCache), i, vp]
    lib.fa_cache_append.restype = i
    lib.fa_fwd_cache.argtypes = [vp, ctypes.POINTER(FaCache), vp, i, vp, vp, vp, vp, i, i, i,
                                 ctypes.POINTER(FaStrides), i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_cache.restype = i
    lib.fa_fwd_cache_workspace_size.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_fwd_cache_workspace_size.restype = i


# ------------------------------------------------------------ raw C ABI

def fa_cache_plan(lens: int, new_lens: int, block_table: int, table_width: int, free_blocks: int,
                  n_free: int, free_pos: int, slots: int, T: int, cu_new: int, kv_lens: int,
                  free_next: int, B: int, block: int, stream: int = 0) -> int:
    """Same arguments as the C function (device pointers as ints); returns the status."""
    return load_library().fa_cache_plan(lens, new_lens, block_table, table_width, free_blocks,
                                        n_free, free_pos, slots, T, cu_new, kv_lens, free_next, B,
                                        block, stream)


def fa_cache_append(k: int, v: int, strides, slots: int, T: int, cache: FaCache, dtype: int,
                    stream: int = 0) -> int:
    """Same arguments as the C function; strides: 2 (b, h, n) element-stride
    triples of k and v, cache: an FaCache (None passes a null pointer)."""
    return load_library().fa_cache_append(k, v, _strides2(strides), slots, T,
                                          None if cache is None else ctypes.byref(cache),
                                          int(dtype), stream)


def fa_fwd_cache(q: int, cache: FaCache, block_table: int, table_width: int, kv_lens: int,
                 cu_q: int, o: int, lse: int, B: int, T: int, H: int, strides, causal: bool,
                 scale: float, dtype: int, workspace: int, workspace_size: int,
                 stream: int = 0) -> int:
    """Same arguments as the C function; strides: 2 (b, h, n) element-stride
    triples of q and o, cache: an FaCache (None passes a null pointer)."""
    return load_library().fa_fwd_cache(q, None if cache is None else ctypes.byref(cache),
                                       block_table, table_width, kv_lens, cu_q, o, lse, B, T, H,
                                       _strides2(strides), int(bool(causal)), float(scale),
                                       int(dtype), workspace, int(workspace_size), stream)


def fa_fwd_cache_workspace_size(B: int, T: int, H: int, Hkv: int, d: int) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().fa_fwd_cache_workspace_size(B, T, H, Hkv, d, ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_cache_workspace_size")
    return int(n.value)


def _strides2(strides):
    if strides is None:
        return None
    (b0, h0, n0), (b1, h1, n1) = strides
    return (FaStrides * 2)(FaStrides(b0, h0, n0), FaStrides(b1, h1, n1))


# ------------------------------------------------------------ torch helpers

def _dtype16(t) -> int:
    import torch
    if t.dtype is torch.float16:
        return FA_DTYPE_FP16
    if t.dtype is torch.bfloat16:
        return FA_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (fp16 or bf16)")


def _describe(cache, device: int) -> FaCache:
    """The FaCache of a Cache whose tensors are on CUDA device `device`."""
    import torch
    k, v, ks, vs = cache
    st, shape = k.stride(), k.shape
    if not (len(shape) == 4 and shape == v.shape and st == v.stride() and st[3] == 1
            and k.element_size() == 1 and v.element_size() == 1
            and ks.shape == shape[:2] and vs.shape == shape[:2]
            and ks.dtype is torch.float32 and vs.dtype is torch.float32
            and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache: k, v must be [blocks, heads, block, d] 8-bit tensors of equal "
                         "strides (1 along d) and k_scales, v_scales contiguous float32 "
                         "[blocks, heads]")
    if not k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == device:
        raise ValueError("cache: tensors must be on the same CUDA device as the other arguments")
    n, heads, block, d = shape
    # an axis of length one has no stride of its own
    return FaCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n, block, heads, d,
                   st[0] if n > 1 else 16, st[1] if heads > 1 else 16, st[2])


def _index(t, device: int, *shape) -> int:
    """The address of a contiguous int32 tensor of this shape on CUDA device `device`."""
    import torch
    if not (t.dtype is torch.int32 and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        raise ValueError(f"expected a contiguous int32 tensor of shape {tuple(shape)} on CUDA "
                         f"device {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cuda_index(t, what: str) -> int:
    """The CUDA device index of a tensor; raises for one elsewhere."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    return i


def _call(fn, what: str, device: int, stream, *args) -> None:
    """fn(*args, stream handle) with the tensors' device current; raises on a status."""
    import torch
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device_index != device:
        raise ValueError(f"{what}: the stream is on CUDA device {stream.device_index}, the "
                         f"tensors on {device}")
    else:
        handle = stream.cuda_stream
    if device == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != FA_OK:
        raise FaError(rc, what)


def cache_empty(num_blocks: int, heads: int, block: int, d: int, device=None) -> Cache:
    """A cache of num_blocks blocks on `device` (default: the current CUDA
    device): codes zero, scales one."""
    import torch
    device = torch.device("cuda") if device is None else torch.device(device)
    k, v = (torch.zeros(num_blocks, heads, block, d, dtype=torch.uint8, device=device)
            .view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(num_blocks, heads, dtype=torch.float32, device=device) for _ in range(2))
    return Cache(k, v, ks, vs)


def cache_plan_into(lens, new_lens, block_table, free_blocks, free_pos, slots, cu_new, kv_lens,
                    free_next, block: int, stream=None) -> None:
    """Enqueues fa_cache_plan on contiguous int32 CUDA tensors: lens, new_lens,
    kv_lens [B], block_table [B, width] (in and out), free_blocks [n], free_pos
    and free_next [1], slots [T], cu_new [B + 1]."""
    dev = _cuda_index(lens, "fa_cache_plan")
    (B,), (T,), (n,), width = lens.shape, slots.shape, free_blocks.shape, block_table.shape[1]
    _call(load_library().fa_cache_plan, "fa_cache_plan", dev, stream,
          _index(lens, dev, B), _index(new_lens, dev, B), _index(block_table, dev, B, width),
          width, _index(free_blocks, dev, n), n, _index(free_pos, dev, 1), _index(slots, dev, T),
          T, _index(cu_new, dev, B + 1), _index(kv_lens, dev, B), _index(free_next, dev, 1), B,
          block)


def cache_plan(lens, new_lens, block_table, free_blocks, free_pos, n_tokens: int, block: int,
               stream=None):
    """Plans a step that appends new_lens[b] tokens to request b, which holds
    lens[b]: writes the block table entries that they open and returns (slots
    [n_tokens], cu_new [B + 1], kv_lens [B], free_next [1]), int32. n_tokens is
    the number of rows to plan, at least the sum of new_lens (slots behind the
    last token are -1). Requests that cannot be served keep their length and
    get slots -1 (see fa_cache.h)."""
    import torch
    _cuda_index(lens, "fa_cache_plan")
    B, dev, i32 = lens.shape[0], lens.device, torch.int32
    with _allocating_on(stream):
        kv_lens, slots = torch.empty_like(lens), torch.empty(n_tokens, dtype=i32, device=dev)
        cu_new = torch.empty(B + 1, dtype=i32, device=dev)
        free_next = torch.empty_like(free_pos)
    cache_plan_into(lens, new_lens, block_table, free_blocks, free_pos, slots, cu_new, kv_lens,
                    free_next, block, stream)
    return slots, cu_new, kv_lens, free_next


def cache_append(k, v, slots, cache, stream=None) -> None:
    """Enqueues fa_cache_append: k, v [T, heads, d] fp16 / bf16 CUDA tensors
    (unit stride along d, the others multiples of 8) into the slots [T] of a
    Cache, in 8 bits, with its blocks' scales."""
    dev = _cuda_index(k, "fa_cache_append")
    desc = _describe(cache, dev)
    T, heads, d = k.shape
    ks, vs = k.stride(), v.stride()
    if not (v.shape == k.shape and v.dtype is k.dtype and v.get_device() == dev
            and heads == desc.Hkv and d == desc.d and ks[2] == 1 and vs[2] == 1):
        raise ValueError("k, v must be [T, heads, d] tensors of one dtype with the cache's heads "
                         "and d, and unit d stride")
    code, sl = _dtype16(k), _index(slots, dev, T)
    if T == 0:
        return
    one = heads == 1  # an axis of length one has no stride of its own
    st = (FaStrides * 2)((0, d if one else ks[1], ks[0] if T > 1 else d),
                         (0, d if one else vs[1], vs[0] if T > 1 else d))
    _call(load_library().fa_cache_append, "fa_cache_append", dev, stream,
          k.data_ptr(), v.data_ptr(), st, sl, T, ctypes.byref(desc), code)


def attention_forward_cache_into(q, cache, block_table, kv_lens, o, lse, workspace, cu_q=None,
                                 causal: bool = True, scale: float | None = None,
                                 stream=None) -> None:
    """Enqueues fa_fwd_cache. With cu_q ([B + 1] int32): q, o [T, H, d], lse
    [T, H]. Without: q, o [B, H, n, d] and lse [B, H, n] (n query tokens for
    each sequence), or [B, H, d] and [B, H] (one). q and o have unit stride
    along d, the other strides are multiples of 8; lse is contiguous float32.
    block_table [B, width] and kv_lens [B] are contiguous int32; workspace: a
    uint8 tensor of fa_fwd_cache_workspace_size bytes."""
    import torch
    dev = _cuda_index(q, "fa_fwd_cache")
    desc = _describe(cache, dev)
    shape, qs, os_ = q.shape, q.stride(), o.stride()
    B, width = block_table.shape
    d = desc.d
    if not (o.shape == shape and o.dtype is q.dtype and qs[-1] == 1 and os_[-1] == 1
            and lse.shape == shape[:-1] and lse.dtype is torch.float32 and lse.is_contiguous()
            and shape[-1] == d and workspace.dtype is torch.uint8 and workspace.is_contiguous()
            and o.get_device() == lse.get_device() == workspace.get_device() == dev):
        raise ValueError("q, o must be [T, H, d], [B, H, d] or [B, H, n, d] tensors of one dtype "
                         "with the cache's d and unit d stride, lse contiguous float32 of their "
                         "shape without d, workspace contiguous uint8, all on one device")
    # (an axis of length one has no stride of its own)
    if cu_q is not None and len(shape) == 3:
        T, H = shape[0], shape[1]
        cu = _index(cu_q, dev, B + 1)
        q3 = (8, qs[1] if H > 1 else d, qs[0] if T > 1 else d)
        o3 = (8, os_[1] if H > 1 else d, os_[0] if T > 1 else d)
    elif cu_q is None and len(shape) in (3, 4) and shape[0] == B:
        H, n = shape[1], shape[2] if len(shape) == 4 else 1
        T, cu = B * n, None
        q3 = (qs[0] if B > 1 else 8, qs[1] if H > 1 else d, qs[2] if n > 1 else d)
        o3 = (os_[0] if B > 1 else 8, os_[1] if H > 1 else d, os_[2] if n > 1 else d)
    else:
        raise ValueError("q must be [T, H, d] with cu_q, or [B, H, d] or [B, H, n, d] without")
    tab, kv, code = _index(block_table, dev, B, width), _index(kv_lens, dev, B), _dtype16(q)
    if H == 0 or H % desc.Hkv:
        raise ValueError(f"{H} query heads do not share {desc.Hkv} K / V heads evenly")
    if T == 0:
        return
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _call(load_library().fa_fwd_cache, "fa_fwd_cache", dev, stream,
          q.data_ptr(), ctypes.byref(desc), tab, width, kv, cu, o.data_ptr(), lse.data_ptr(), B, T,
          H, (FaStrides * 2)(q3, o3), 1 if causal else 0, scale, code, workspace.data_ptr(),
          workspace.numel())


def attention_forward_cache(q, cache, block_table, kv_lens, cu_q=None, causal: bool = True,
                            scale: float | None = None, stream=None):
    """(O, LSE) of the last query tokens of each sequence over its cached keys:
    see attention_forward_cache_into for the shapes. O has q's shape and dtype;
    rows that belong to no sequence are not written."""
    import torch
    index, dev = _cuda_index(q, "fa_fwd_cache"), q.device
    shape = q.shape
    H, heads, d = shape[1], cache[0].shape[1], shape[-1]
    if H == 0 or heads == 0 or H % heads:
        raise ValueError(f"{H} query heads do not share {heads} K / V heads evenly")
    if d != cache[0].shape[-1]:
        raise ValueError(f"q has d = {d}, the cache {cache[0].shape[-1]}")
    B, T = block_table.shape[0], math.prod(shape[:-1]) // H
    if index == torch.cuda.current_device():
        size = fa_fwd_cache_workspace_size(B, T, H, heads, d)
    else:
        with torch.cuda.device(index):
            size = fa_fwd_cache_workspace_size(B, T, H, heads, d)
    with _allocating_on(stream):
        o = torch.empty(shape, dtype=q.dtype, device=dev)
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    attention_forward_cache_into(q, cache, block_table, kv_lens, o, lse, ws, cu_q, causal, scale,
                                 stream)
    return o, lse
