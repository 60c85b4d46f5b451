"""fa_draft.h: exported symbols, every refusal of bad arguments before a GPU is
touched, and the tests' own implementation against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import cache_util as U
import draft_util as D
from attention_forward_flashattention_gb300 import build as fabuild
from attention_forward_flashattention_gb300 import cache as fc
from attention_forward_flashattention_gb300 import draft as fd

GOOD = 0x100000  # aligned stand-in addresses: never dereferenced by the checks


def addr(i):
    return GOOD + 0x10000 * i


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


def test_header_and_exports(lib):
    names = fa.header_functions(fd.HEADER)
    assert names == ["fa_cache_tree", "fa_fwd_cache_tree"]
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


TREE = dict(parents=addr(0), cu=addr(1), lens=addr(2), masks=addr(3), positions=addr(4), B=3, T=20, words=1)


def tree_rc(**kw):
    return fa.fa_cache_tree(*{**TREE, **kw}.values())


@pytest.mark.parametrize("kw", [*({n: 0} for n in ("parents", "cu", "lens", "masks", "positions")),
                                dict(parents=addr(0) + 2), dict(masks=addr(3) + 4), dict(B=0), dict(T=-1),
                                dict(words=0), dict(words=-1), dict(masks=addr(0)),
                                dict(positions=addr(2)), dict(positions=addr(3))])
def test_tree_refuses(kw):
    assert tree_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(words=17), dict(B=(1 << 20) + 1), dict(T=1 << 28, words=16)])
def test_tree_unsupported(kw):
    assert tree_rc(**kw) == fa.FA_ERR_UNSUPPORTED


CONTIG = (8, 128, 256)


def cache(**kw):
    d = dict(k=addr(20), v=addr(21), k_scales=addr(22), v_scales=addr(23), num_blocks=9, block=32,
             Hkv=2, d=128, block_stride=2 * 32 * 128, head_stride=32 * 128, token_stride=128)
    d.update(kw)
    return fc.FaCache(*d.values())


def attn_rc(c=None, q=addr(0), table=addr(1), width=4, kv=addr(2), cu=addr(3), masks=addr(7), words=1,
            o=addr(4), lse=addr(5), B=3, T=7, H=4, strides=(CONTIG, CONTIG), scale=0.1,
            dtype=fa.FA_DTYPE_FP16, ws=addr(6), size=1 << 40):
    return fa.fa_fwd_cache_tree(q, cache() if c is None else c, table, width, kv, cu, masks, words, o, lse,
                                B, T, H, strides, scale, dtype, ws, size)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(table=0), dict(kv=0), dict(o=0), dict(lse=0), dict(ws=0), dict(strides=None),
    dict(masks=0), dict(masks=addr(7) + 4), dict(words=0), dict(words=-3), dict(cu=addr(3) + 1),
    dict(B=0), dict(T=-1), dict(H=3), dict(width=0), dict(cu=None, T=7), dict(dtype=2),
    dict(scale=0.0), dict(scale=float("nan")), dict(c=cache(k=0)), dict(strides=(CONTIG, (8, 130, 256)))])
def test_attention_refuses(kw):
    assert attn_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(words=17), dict(T=1 << 28, words=8, H=2), dict(c=cache(d=96)),
                                dict(width=1 << 26)])
def test_attention_unsupported(kw):
    assert attn_rc(**kw) == fa.FA_ERR_UNSUPPORTED


def test_no_device_is_an_error_not_a_fallback():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (tree_rc(), tree_rc(T=0), attn_rc(), attn_rc(cu=None, T=6)):
        assert rc in (fa.FA_ERR_CUDA, fa.FA_ERR_ARCH)


def test_binding_refuses_cpu_tensors():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_tree(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32))
    c = fa.cache_empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.attention_forward_cache_tree(torch.zeros(3, 2, 64).half(), c, torch.zeros(3, 1, **i32),
                                        torch.ones(3, **i32), torch.ones(3, 1, dtype=torch.int64))


# ------------------------------------------------------------ the tests' own implementation

def test_masks_closed_form():
    # request 0: two roots, the first with children 2 and 3, 3 with child 4; request 1: a chain; a spare row
    masks, pos = D.masks_of([-1, -1, 0, 0, 3, 0, 0, 5], [0, 5, 7], [10, 0], 1)
    assert [m[0] for m in masks[:5]] == [1, 2, 5, 9, 25] and [m[0] for m in masks[5:7]] == [1, 3]
    assert pos[:7] == [10, 10, 11, 11, 12, 0, 1] and masks[7] is None and pos[7] is None
    assert D.signed([[1 << 63, 3]]).tolist() == [[-2 ** 63, 3]]


def test_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(1)
    k, v = (rng.integers(0, 0x70, (3, 2, 16, 64), dtype=np.uint8) for _ in range(2))
    ks, vs = (np.exp2(rng.integers(-9, -3, (3, 2)).astype(float)) for _ in range(2))
    q = rng.standard_normal((5, 4, 64))
    table = np.array([[2, 0], [1, 7]])
    masks, _ = D.masks_of([-1, 0, 1, -1, 0], [0, 3, 5], [20, 10], 1)
    a = D.attend(q, k, v, ks, vs, table, [23, 12], [0, 3, 5], masks, 16, 0.1, 2.0 ** -10)
    b = U.attend_columns(q, k, v, ks, vs, table, [23, 12], [0, 3, 5], 16, 0.1, True, 2.0 ** -10)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12, atol=0)
