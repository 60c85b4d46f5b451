"""Upkeep of the block cache (``include/fa_pages.h``): dropping drafted tokens that
were not accepted, handing blocks back, sharing them between requests.

    # after the drafts have been verified: `keep` is the mask of the last accepted token
    kv_lens_after = fa.cache_keep(cache, table, kv_lens, cu, keep)            # each layer's cache
    pos = fa.cache_release(table, kv_lens, kv_lens_after, free, pos, block)   # once

    # samples of a prompt, a beam: row k of the new table goes on from request src[k]
    table, lens, copies, pos = fa.cache_fork(table, lens, src, free, pos, shares, block)   # once
    fa.cache_copy(cache, copies)                                              # each layer's cache

Shared blocks must not be written: drafts are dropped before a fork, and a request that goes back to
a token inside a block that it may share goes on as a fork of itself, after which its old row ends:

    row, back, copies, pos = fa.cache_fork(table, shorter, src, free, pos, shares, block)
    fa.cache_copy(cache, copies)                                              # each layer's cache
    pos = fa.cache_release(table, lens, zeros, free, pos, block, shares)

Like the rest of the binding this only marshals arguments.
"""
from __future__ import annotations

import ctypes
import os

from . import FaError, _build, cache, load_library

HEADER = os.path.join(_build.INCLUDE, "fa_pages.h")


def bind(lib) -> None:
    """Argument types of the entry points."""
    vp, i, c = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(cache.FaCache)
    lib.fa_cache_keep.argtypes = [c, vp, i, vp, vp, vp, i, vp, i, vp]
    lib.fa_cache_release.argtypes = [vp, i, vp, vp, vp, i, vp, i, vp, vp, i, i, vp]
    lib.fa_cache_fork.argtypes = [vp, i, vp, i, vp, i, vp, i, vp, i, vp, vp, vp, vp, vp, i, vp]
    lib.fa_cache_copy.argtypes = [c, vp, i, vp]
    for f in (lib.fa_cache_keep, lib.fa_cache_release, lib.fa_cache_fork, lib.fa_cache_copy):
        f.restype = i


# ------------------------------------------------------------ raw C ABI

def _ref(c):
    return None if c is None else ctypes.byref(c)


def fa_cache_keep(cache_: cache.FaCache, block_table: int, table_width: int, kv_lens: int, cu: int,
                  keep: int, words: int, lens_out: int, B: int, stream: int = 0) -> int:
    """Same arguments as the C function (device pointers as ints); returns the status."""
    return load_library().fa_cache_keep(_ref(cache_), block_table, table_width, kv_lens, cu, keep, words,
                                        lens_out, B, stream)


def fa_cache_release(block_table: int, table_width: int, lens: int, new_lens: int, shares: int,
                     num_blocks: int, free_blocks: int, n_free: int, free_pos: int, free_next: int,
                     B: int, block: int, stream: int = 0) -> int:
    """Same arguments as the C function; returns the status."""
    return load_library().fa_cache_release(block_table, table_width, lens, new_lens, shares, num_blocks,
                                           free_blocks, n_free, free_pos, free_next, B, block, stream)


def fa_cache_fork(block_table: int, table_width: int, lens: int, B: int, src: int, n: int, shares: int,
                  num_blocks: int, free_blocks: int, n_free: int, free_pos: int, new_table: int,
                  new_lens: int, copies: int, free_next: int, block: int, stream: int = 0) -> int:
    """Same arguments as the C function; returns the status."""
    return load_library().fa_cache_fork(block_table, table_width, lens, B, src, n, shares, num_blocks,
                                        free_blocks, n_free, free_pos, new_table, new_lens, copies,
                                        free_next, block, stream)


def fa_cache_copy(cache_: cache.FaCache, copies: int, n: int, stream: int = 0) -> int:
    """Same arguments as the C function; returns the status."""
    return load_library().fa_cache_copy(_ref(cache_), copies, n, stream)


# ------------------------------------------------------------ torch helpers

def _result(r, what: str):
    if type(r) is int:
        raise FaError(r, what)
    return r


def cache_keep(cache_, block_table, kv_lens, cu, keep, out=None, stream=None):
    """Moves the kept ones of each sequence's last tokens together in one layer's
    cache; returns the lengths after, int32 [B] (`out` where it is given). block_table
    [B, width], kv_lens [B] and cu [B + 1] (rows of the tokens at stake) int32, keep
    int64 [B, words]: bit c for the c-th of them. With one cache per layer each
    layer's call takes the same kv_lens; see fa_pages.h for scales and refusals."""
    return _result(cache._module().cache_keep(cache_, block_table, kv_lens, cu, keep, out, stream),
                   "fa_cache_keep")


def cache_release(block_table, lens, new_lens, free_blocks, free_pos, block: int, shares=None, out=None,
                  stream=None):
    """Puts the blocks behind new_lens [B] of requests that hold lens [B] tokens back in
    front of free_pos [1] in free_blocks (in place); returns the next free_pos. shares
    [num_blocks]: counts of cache_fork, where blocks may have several holders. All
    int32."""
    return _result(cache._module().cache_release(block_table, lens, new_lens, free_blocks, free_pos, block,
                                                 shares, out, stream), "fa_cache_release")


def cache_fork(block_table, lens, src, free_blocks, free_pos, shares, block: int, out=None, stream=None):
    """(new_table [n, width], new_lens [n], copies [n, 3], free_next [1]), int32, of
    requests that start as copies of requests src [n]: full blocks are shared (their
    counts in shares [num_blocks] go up, in place), a last one that is not full gets a
    free block in its place, which cache_copy fills. `out`: those four, to be written
    (otherwise they are parts of one allocation)."""
    return _result(cache._module().cache_fork(block_table, lens, src, free_blocks, free_pos, shares, block,
                                              out, stream), "fa_cache_fork")


def cache_copy(cache_, copies, stream=None) -> None:
    """Enqueues fa_cache_copy: copies int32 [n, 3] (from, to, rows), cache_fork's."""
    _result(cache._module().cache_copy(cache_, copies, stream), "fa_cache_copy")
