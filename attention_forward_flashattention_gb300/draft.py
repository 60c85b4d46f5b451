"""Trees of drafted tokens over the block cache (``include/fa_draft.h``).

    masks, positions = fa.cache_tree(parents, cu, lens)
    o, lse = fa.attention_forward_cache_tree(q, cache, table, kv_lens, masks, cu)

Masks are int64 tensors whose bits are a set of 64 * words drafted tokens. Like
the rest of the binding this only marshals arguments.
"""
from __future__ import annotations

import ctypes
import os

from . import FaError, FaStrides, _build, cache, load_library

HEADER = os.path.join(_build.INCLUDE, "fa_draft.h")


def bind(lib) -> None:
    """Argument types of the entry points."""
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_cache_tree.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp]
    lib.fa_cache_tree.restype = i
    lib.fa_fwd_cache_tree.argtypes = [vp, ctypes.POINTER(cache.FaCache), vp, i, vp, vp, vp, i, vp, vp, i, i,
                                      i, ctypes.POINTER(FaStrides), f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_cache_tree.restype = i


# ------------------------------------------------------------ raw C ABI

def fa_cache_tree(parents: int, cu: int, lens: int, masks: int, positions: int, B: int, T: int,
                  words: int, stream: int = 0) -> int:
    """Same arguments as the C function (device pointers as ints); returns the status."""
    return load_library().fa_cache_tree(parents, cu, lens, masks, positions, B, T, words, stream)


def fa_fwd_cache_tree(q: int, cache_: cache.FaCache, block_table: int, table_width: int, kv_lens: int,
                      cu_q: int, masks: int, words: int, o: int, lse: int, B: int, T: int, H: int,
                      strides, scale: float, dtype: int, workspace: int, workspace_size: int,
                      stream: int = 0) -> int:
    """Same arguments as the C function; strides: 2 (b, h, n) element-stride
    triples of q and o, cache_: an FaCache (None passes a null pointer)."""
    return load_library().fa_fwd_cache_tree(q, None if cache_ is None else ctypes.byref(cache_),
                                            block_table, table_width, kv_lens, cu_q, masks, words, o,
                                            lse, B, T, H, cache._strides2(strides), float(scale),
                                            int(dtype), workspace, int(workspace_size), stream)


# ------------------------------------------------------------ torch helpers

def cache_tree(parents, cu, lens, words: int | None = None, stream=None):
    """(masks int64 [T, words], positions int32 [T]) of drafted tokens: parents [T] are
    the numbers of their parents among their request's tokens (-1: the context), cu
    [B + 1] the requests' rows (cache_plan's cu_new) and lens [B] the lengths of their
    contexts (before the drafted tokens), all int32. A request's tokens from 64 * words on
    are seen by none, themselves neither; by default there are words for T tokens of
    one request, at most 16 (1024 tokens): a program that knows its requests to be
    smaller says how many it needs. Rows that belong to no request are not written.
    The two are parts of one allocation."""
    r = (cache._native or cache._module()).cache_tree(parents, cu, lens, words, None, stream)
    if type(r) is int:
        raise FaError(r, "fa_cache_tree")
    return r


def cache_tree_into(parents, cu, lens, masks, positions, stream=None) -> None:
    """cache_tree into masks [T, words] and positions [T]."""
    r = cache._module().cache_tree(parents, cu, lens, masks.shape[-1], (masks, positions), stream)
    if type(r) is int:
        raise FaError(r, "fa_cache_tree")


def attention_forward_cache_tree(q, cache_, block_table, kv_lens, masks, cu_q=None,
                                 scale: float | None = None, stream=None):
    """attention_forward_cache of drafted tokens: the last query tokens of each
    sequence see its keys before them, and of themselves those whose bits are set in
    their masks (int64 [rows, words], or without cu_q [B, n, words])."""
    r = cache._module().attention_forward_cache_tree(q, cache_, block_table, kv_lens, cu_q, None, masks,
                                                     scale, stream)
    if type(r) is int:
        raise FaError(r, "fa_fwd_cache_tree")
    return r


def attention_forward_cache_tree_into(q, cache_, block_table, kv_lens, masks, o, lse, workspace,
                                      cu_q=None, scale: float | None = None, stream=None) -> None:
    """attention_forward_cache_into with masks."""
    r = cache._module().attention_forward_cache_tree(q, cache_, block_table, kv_lens, cu_q,
                                                     (o, lse, workspace), masks, scale, stream)
    if type(r) is int:
        raise FaError(r, "fa_fwd_cache_tree")
