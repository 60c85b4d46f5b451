"""The 8-bit block cache of ``include/fa_cache.h``: planning its block tables,
appending keys and values, and the attention that reads it.

    cache = fa.cache_empty(num_blocks, heads, block, d)
    slots, cu, kv_lens, pos = fa.cache_plan(lens, new_lens, table, free, pos, T, block)
    fa.cache_append(k, v, slots, cache)                  # k, v: [T, heads, d]
    o, lse = fa.attention_forward_cache(q, cache, table, kv_lens, cu)   # q: [T, H, d]

Like the rest of the binding this only marshals arguments; it does so in host
code (_build/_fa_cache_torch.so), because a decoding step's calls are so short
that the same checks and allocations in Python would take longer than they do.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
from typing import NamedTuple

from . import FA_OK, FaError, FaStrides, _build, load_library

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

_lock = threading.Lock()
_native = None


def _module():
    """The host code of the torch calls (built in-tree by build.build()). Raises if absent."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries, before the module that uses them)
        load_library()
        with _lock:
            if _native is None:
                p = _build.torch_path()
                if not os.path.exists(p):
                    raise RuntimeError(f"torch module not built: {p} (run __graft_entry__.build())")
                loader = importlib.machinery.ExtensionFileLoader("_fa_cache_torch", p)
                m = importlib.util.module_from_spec(
                    importlib.util.spec_from_file_location("_fa_cache_torch", p, loader=loader))
                loader.exec_module(m)
                _native = m
    return _native


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
    r = _module().cache_plan(lens, new_lens, block_table, free_blocks, free_pos,
                             (slots, cu_new, kv_lens, free_next), 0, block, stream)
    if type(r) is int:
        raise FaError(r, "fa_cache_plan")


def cache_plan(lens, new_lens, block_table, free_blocks, free_pos, n_tokens: int, block: int,
               stream=None):
    """Plans a step that appends new_lens[b] tokens to request b, which holds
    lens[b]: writes the block table entries that they open and returns (slots
    [n_tokens], cu_new [B + 1], kv_lens [B], free_next [1]), int32. n_tokens is
    the number of rows to plan, at least the sum of new_lens (slots behind the
    last token are -1), parts of one allocation. Requests that cannot be served
    keep their length and get slots -1 (see fa_cache.h)."""
    r = (_native or _module()).cache_plan(lens, new_lens, block_table, free_blocks, free_pos, None,
                                          n_tokens, block, stream)
    if type(r) is int:
        raise FaError(r, "fa_cache_plan")
    return r


def cache_append(k, v, slots, cache, stream=None) -> None:
    """Enqueues fa_cache_append: k, v [T, heads, d] fp16 / bf16 CUDA tensors
    (unit stride along d, the others multiples of 8) into the slots [T] of a
    Cache, in 8 bits, with its blocks' scales."""
    r = (_native or _module()).cache_append(k, v, slots, cache, stream)
    if r is not None:
        raise FaError(r, "fa_cache_append")


def attention_forward_cache_into(q, cache, block_table, kv_lens, o, lse, workspace, cu_q=None,
                                 causal: bool = True, scale: float | None = None,
                                 stream=None) -> None:
    """Enqueues fa_fwd_cache. With cu_q ([B + 1] int32): q, o [T, H, d], lse
    [T, H]. Without: q, o [B, H, n, d] and lse [B, H, n] (n query tokens for
    each sequence), or [B, H, d] and [B, H] (one). q and o have unit stride
    along d, the other strides are multiples of 8; lse is contiguous float32.
    block_table [B, width] and kv_lens [B] are contiguous int32; workspace: a
    uint8 tensor of fa_fwd_cache_workspace_size bytes."""
    r = _module().attention_forward_cache(q, cache, block_table, kv_lens, cu_q, (o, lse, workspace),
                                          causal, scale, stream)
    if type(r) is int:
        raise FaError(r, "fa_fwd_cache")


def attention_forward_cache(q, cache, block_table, kv_lens, cu_q=None, causal: bool = True,
                            scale: float | None = None, stream=None):
    """(O, LSE) of the last query tokens of each sequence over its cached keys:
    see attention_forward_cache_into for the shapes. O has q's shape and dtype;
    rows that belong to no sequence are not written."""
    r = (_native or _module()).attention_forward_cache(q, cache, block_table, kv_lens, cu_q, None,
                                                       causal, scale, stream)
    if type(r) is int:
        raise FaError(r, "fa_fwd_cache")
    return r
