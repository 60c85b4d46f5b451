"""fa_pages.h: exported symbols, every refusal of bad arguments before a GPU is
touched, and the tests' own implementation against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import cache_util as U
import pages_util as P
from attention_forward_flashattention_gb300 import build as fabuild
from attention_forward_flashattention_gb300 import cache as fc
from attention_forward_flashattention_gb300 import pages as fp

GOOD = 0x100000  # aligned stand-in addresses: never dereferenced by the checks


def addr(i):
    return GOOD + 0x10000 * i


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


def test_header_and_exports(lib):
    names = fa.header_functions(fp.HEADER)
    assert names == ["fa_cache_keep", "fa_cache_release", "fa_cache_fork", "fa_cache_copy"]
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


def cache(**kw):
    d = dict(k=addr(20), v=addr(21), k_scales=addr(22), v_scales=addr(23), num_blocks=9, block=32,
             Hkv=2, d=128, block_stride=2 * 32 * 128, head_stride=32 * 128, token_stride=128)
    d.update(kw)
    return fc.FaCache(*d.values())


KEEP = dict(c=cache(), table=addr(0), width=8, kv=addr(1), cu=addr(2), keep=addr(3), words=1, out=addr(4), B=3)
RELEASE = dict(table=addr(0), width=8, lens=addr(1), new=addr(2), shares=addr(3), num_blocks=9, free=addr(4),
               n_free=9, pos=addr(5), next=addr(6), B=3, block=32)
FORK = dict(table=addr(0), width=8, lens=addr(1), B=3, src=addr(2), n=2, shares=addr(3), num_blocks=9,
            free=addr(4), n_free=9, pos=addr(5), rows=addr(6), out=addr(7), copies=addr(8), next=addr(9), block=32)
COPY = dict(c=cache(), copies=addr(0), n=3)


def rc(fn, base, **kw):
    return fn(*{**base, **kw}.values())


BAD = [
    *[(fa.fa_cache_keep, KEEP, kw) for kw in (
        *({n: 0} for n in ("table", "kv", "cu", "keep", "out")), dict(keep=addr(3) + 4), dict(cu=addr(2) + 2),
        dict(out=addr(1)), dict(out=addr(0)), dict(words=0), dict(B=0), dict(width=0), dict(c=cache(k=0)),
        dict(c=None), dict(c=cache(token_stride=120)))],
    *[(fa.fa_cache_release, RELEASE, kw) for kw in (
        *({n: 0} for n in ("table", "lens", "new", "free", "pos", "next")), dict(shares=addr(3) + 2),
        dict(num_blocks=0), dict(n_free=-1), dict(B=0), dict(width=-1), dict(next=addr(5)), dict(free=addr(3)),
        dict(free=addr(0)), dict(next=addr(4)))],
    *[(fa.fa_cache_fork, FORK, kw) for kw in (
        *({n: 0} for n in ("table", "lens", "src", "shares", "free", "pos", "rows", "out", "copies", "next")),
        dict(rows=addr(6) + 1), dict(B=0), dict(n=0), dict(n=-1), dict(width=0), dict(num_blocks=0),
        dict(n_free=-2), dict(rows=addr(0)), dict(out=addr(1)), dict(next=addr(5)), dict(copies=addr(7)))],
    *[(fa.fa_cache_copy, COPY, kw) for kw in (dict(copies=0), dict(copies=addr(0) + 2), dict(n=-1), dict(c=None),
                                              dict(c=cache(num_blocks=0)))],
]


@pytest.mark.parametrize("fn,base,kw", BAD)
def test_refused(fn, base, kw):
    assert rc(fn, base, **kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("fn,base,kw", [
    (fa.fa_cache_keep, KEEP, dict(words=17)), (fa.fa_cache_keep, KEEP, dict(B=(1 << 20) + 1)),
    (fa.fa_cache_keep, KEEP, dict(width=1 << 26)), (fa.fa_cache_keep, KEEP, dict(c=cache(d=96))),
    (fa.fa_cache_keep, KEEP, dict(c=cache(block=48))),
    (fa.fa_cache_release, RELEASE, dict(block=8)), (fa.fa_cache_release, RELEASE, dict(B=(1 << 20) + 1)),
    (fa.fa_cache_release, RELEASE, dict(B=1 << 20, width=1 << 11)),
    (fa.fa_cache_fork, FORK, dict(block=100)), (fa.fa_cache_fork, FORK, dict(n=(1 << 20) + 1)),
    (fa.fa_cache_fork, FORK, dict(width=1 << 26)), (fa.fa_cache_fork, FORK, dict(B=(1 << 20) + 1)),
    (fa.fa_cache_copy, COPY, dict(n=(1 << 20) + 1)), (fa.fa_cache_copy, COPY, dict(c=cache(Hkv=40000)))])
def test_unsupported(fn, base, kw):
    assert rc(fn, base, **kw) == fa.FA_ERR_UNSUPPORTED


def test_no_device_is_an_error_not_a_fallback():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for r in (rc(fa.fa_cache_keep, KEEP), rc(fa.fa_cache_release, RELEASE),
              rc(fa.fa_cache_release, RELEASE, shares=0, num_blocks=0, n_free=0, free=0),
              rc(fa.fa_cache_fork, FORK), rc(fa.fa_cache_fork, FORK, n_free=0, free=0), rc(fa.fa_cache_copy, COPY),
              rc(fa.fa_cache_copy, COPY, n=0)):
        assert r in (fa.FA_ERR_CUDA, fa.FA_ERR_ARCH)


def test_binding_refuses_cpu_tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c = fa.cache_empty(4, 2, 16, 64, device="cpu")
    for call in (lambda: fa.cache_keep(c, i(2, 3), i(2), i(3), torch.zeros(2, 1, dtype=torch.int64)),
                 lambda: fa.cache_release(i(2, 3), i(2), i(2), i(4), i(1), 16),
                 lambda: fa.cache_fork(i(2, 3), i(2), i(2), i(4), i(1), i(4), 16),
                 lambda: fa.cache_copy(c, i(2, 3))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ the tests' own implementation

def test_keep_closed_form():
    codes = np.zeros((3, 1, 16, 64), np.uint8)
    scales = np.array([[1.0], [4.0], [0.5]])
    table = np.array([[2, 1]])
    for at in range(20):   # the value of each token is its place
        p, r = table[0, at // 16], at % 16
        codes[p, 0, r] = U.encode(np.full(64, at / scales[p, 0]))
    # 10 tokens, then 10 at stake, of which 0, 5, 7 and 9 stay
    c, s, out = P.keep(codes, scales, table, [20], [0, 10], [[0b1010100001]], 16)
    value = [U.CODE_VALUES[c[table[0, i // 16], 0, i % 16, 0]] * s[table[0, i // 16], 0] for i in range(14)]
    assert out == [14] and s[2, 0] == 4.0 and s[1, 0] == 4.0
    want = [*range(11), 15, 17, 19]
    # (codes of a step of 4 have 3 bits below their leading one; all of these places fit but those that round)
    assert all(abs(v - w) <= 2.0 ** -4 * w for v, w in zip(value, want))


def test_release_and_fork_closed_forms():
    table = np.array([[5, 6, 7], [5, 8, -1]])
    free, nxt, sh = P.release(table, [40, 20], [16, 0], [1, 2, 3, 4], 4, 16, [0] * 5 + [1, 0, 0, 0])
    # request 0 gives up 6 and 7, request 1 its holding of 5, and 8
    assert free == [1, 8, 7, 6] and nxt == 1 and sh == [0] * 9
    rows, lens, copies, nxt, sh = P.fork(table, [40, 32], [0, 1, 0, 9], [3, 4], 0, [0] * 9, 16)
    assert rows.tolist() == [[5, 6, 3], [5, 8, -1], [5, 6, 4], [-1, -1, -1]]
    assert lens == [40, 32, 40, 0] and copies == [(7, 3, 8), (-1, -1, 0), (7, 4, 8), (-1, -1, 0)]
    assert nxt == 2 and sh == [0, 0, 0, 0, 0, 3, 2, 0, 1]
