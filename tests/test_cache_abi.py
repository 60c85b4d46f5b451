"""The block cache's C ABI (include/fa_cache.h): exported symbols, and every
refusal of bad arguments before a GPU is touched; the 64-bit implementations
that the GPU tests compare with, against closed forms."""
import ctypes

import numpy as np
import pytest

import attention_forward_flashattention_gb300 as fa
import cache_util as U
from attention_forward_flashattention_gb300 import build as fabuild
from attention_forward_flashattention_gb300 import cache as fc

GOOD = 0x100000  # aligned stand-in addresses: never dereferenced by the checks


def addr(i):
    return GOOD + 0x10000 * i


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def test_header_and_exports(lib):
    names = fa.header_functions(fc.HEADER)
    assert names == ["fa_cache_plan", "fa_cache_append", "fa_fwd_cache",
                     "fa_fwd_cache_workspace_size"]
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
    assert [f[0] for f in fc.FaCache._fields_] == [
        "k", "v", "k_scales", "v_scales", "num_blocks", "block", "Hkv", "d", "block_stride",
        "head_stride", "token_stride"]


PLAN = dict(lens=addr(0), new_lens=addr(1), block_table=addr(2), table_width=8,
            free_blocks=addr(3), n_free=10, free_pos=addr(4), slots=addr(5), T=20, cu_new=addr(6),
            kv_lens=addr(7), free_next=addr(8), B=3, block=16)


def plan_rc(**kw):
    return fa.fa_cache_plan(*{**PLAN, **kw}.values())


@pytest.mark.parametrize("kw", [
    *({n: 0} for n in ("lens", "new_lens", "block_table", "free_blocks", "free_pos", "slots",
                       "cu_new", "kv_lens", "free_next")),
    dict(lens=addr(0) + 2), dict(slots=addr(5) + 1), dict(B=0), dict(B=-1), dict(T=-1),
    dict(table_width=0), dict(n_free=-1),
    # written arrays that are read too, or twice
    dict(kv_lens=addr(0)), dict(free_next=addr(4)), dict(slots=addr(3)), dict(cu_new=addr(7))])
def test_plan_refuses(kw):
    assert plan_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(block=8), dict(block=48), dict(block=256),
                                dict(B=(1 << 20) + 1), dict(T=(1 << 30) + 1)])
def test_plan_unsupported(kw):
    assert plan_rc(**kw) == fa.FA_ERR_UNSUPPORTED


def cache(**kw):
    d = dict(k=addr(20), v=addr(21), k_scales=addr(22), v_scales=addr(23), num_blocks=9, block=32,
             Hkv=2, d=128, block_stride=2 * 32 * 128, head_stride=32 * 128, token_stride=128)
    d.update(kw)
    return fc.FaCache(*d.values())


BAD_CACHE = [dict(k=0), dict(v=0), dict(k_scales=0), dict(v_scales=0), dict(k=addr(20) + 8),
             dict(v_scales=addr(23) + 2), dict(num_blocks=0), dict(Hkv=0),
             dict(block_stride=0), dict(head_stride=-4096), dict(token_stride=136),
             dict(token_stride=112)]
ODD_CACHE = [dict(d=96), dict(d=32), dict(block=8), dict(block=100), dict(block=256),
             dict(num_blocks=1 << 27), dict(block_stride=1 << 38), dict(Hkv=40000)]

CONTIG = (8, 128, 256)


def append_rc(c=None, k=addr(0), v=addr(1), strides=(CONTIG, CONTIG), slots=addr(2), T=5,
              dtype=fa.FA_DTYPE_BF16):
    return fa.fa_cache_append(k, v, strides, slots, T, cache() if c is None else c, dtype)


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_bad_cache_refused(kw):
    assert append_rc(cache(**kw)) == fa.FA_ERR_INVALID_ARG
    assert attn_rc(cache(**kw), H=4 if kw.get("Hkv") != 0 else 1) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", ODD_CACHE)
def test_unsupported_cache(kw):
    assert append_rc(cache(**kw)) == fa.FA_ERR_UNSUPPORTED
    assert attn_rc(cache(**kw), H=40000 if "Hkv" in kw else 4, T=6) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(k=0), dict(v=0), dict(slots=0), dict(strides=None),
                                dict(T=-1), dict(k=addr(0) + 2), dict(slots=addr(2) + 2),
                                dict(dtype=2), dict(strides=((8, 128, 12), CONTIG)),
                                dict(strides=(CONTIG, (8, 0, 256)))])
def test_append_refuses(kw):
    assert append_rc(**kw) == fa.FA_ERR_INVALID_ARG


def test_append_unsupported():
    assert append_rc(strides=(CONTIG, (8, 128, 1 << 38))) == fa.FA_ERR_UNSUPPORTED
    assert append_rc(T=(1 << 30) + 1) == fa.FA_ERR_UNSUPPORTED


def attn_rc(c=None, q=addr(0), table=addr(1), width=4, kv=addr(2), cu=addr(3), o=addr(4),
            lse=addr(5), B=3, T=7, H=4, strides=(CONTIG, CONTIG), causal=True, scale=0.1,
            dtype=fa.FA_DTYPE_FP16, ws=addr(6), size=1 << 40):
    return fa.fa_fwd_cache(q, cache() if c is None else c, table, width, kv, cu, o, lse, B, T, H,
                           strides, causal, scale, dtype, ws, size)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(table=0), dict(kv=0), dict(o=0), dict(lse=0), dict(ws=0), dict(strides=None),
    dict(q=addr(0) + 8), dict(o=addr(4) + 8), dict(lse=addr(5) + 2), dict(ws=addr(6) + 8),
    dict(cu=addr(3) + 1), dict(B=0), dict(T=-1), dict(H=0), dict(H=3), dict(width=0),
    dict(cu=None, T=7), dict(dtype=-1), dict(strides=((8, 130, 256), CONTIG)),
    dict(strides=(CONTIG, (8, 128, -8))), dict(cu=None, T=6, strides=((4, 128, 256), CONTIG)),
    *(dict(scale=s) for s in (0.0, -1.0, float("nan"), float("inf")))])
def test_attention_refuses(kw):
    assert attn_rc(**kw) == fa.FA_ERR_INVALID_ARG


def test_attention_unsupported():
    assert attn_rc(T=1 << 30, H=4) == fa.FA_ERR_UNSUPPORTED
    assert attn_rc(strides=(CONTIG, (8, 1 << 38, 256))) == fa.FA_ERR_UNSUPPORTED


def test_null_cache_refused():
    assert fa.load_library().fa_cache_append(addr(0), addr(1), None, addr(2), 1, None, 0,
                                             None) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_fwd_cache(addr(0), None, addr(1), 1, addr(2), None, addr(4), addr(5), 1, 1, 1,
                           (CONTIG, CONTIG), True, 0.1, 0, addr(6), 1 << 40) \
        == fa.FA_ERR_INVALID_ARG


def test_workspace_size_refuses():
    n = ctypes.c_size_t(0)
    f = fa.load_library().fa_fwd_cache_workspace_size
    assert f(1, 1, 4, 3, 64, ctypes.byref(n)) == fa.FA_ERR_INVALID_ARG
    assert f(0, 1, 4, 4, 64, ctypes.byref(n)) == fa.FA_ERR_INVALID_ARG
    assert f(1, 1, 4, 4, 64, None) == fa.FA_ERR_INVALID_ARG
    assert f(1, 1, 4, 4, 80, ctypes.byref(n)) == fa.FA_ERR_UNSUPPORTED


def test_no_device_is_an_error_not_a_fallback():
    no_gpu()
    for rc in (plan_rc(), plan_rc(T=0, slots=0), plan_rc(n_free=0, free_blocks=0), append_rc(),
               attn_rc(), attn_rc(cu=None, T=6)):
        assert rc in (fa.FA_ERR_CUDA, fa.FA_ERR_ARCH)


def test_binding_refuses_cpu_tensors():
    import torch
    i32 = dict(dtype=torch.int32)
    c = fa.cache_empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        fa.cache_plan(torch.zeros(2, **i32), torch.ones(2, **i32), torch.zeros(2, 3, **i32),
                      torch.arange(4, **i32), torch.zeros(1, **i32), 2, 16)
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        fa.cache_append(x, x, torch.zeros(3, **i32), c)
    with pytest.raises(ValueError):
        fa.attention_forward_cache(x, c, torch.zeros(3, 1, **i32), torch.ones(3, **i32))


# ------------------------------------------------------------ the tests' own implementations

def test_plan_reference_closed_form():
    table = -np.ones((2, 4), dtype=np.int64)
    table[0, 0] = 5
    slots, cu, kv, tab, nxt = U.plan([10, 0], [8, 3], table, [7, 2, 9], 0, 12, 16)
    assert slots == [90, 91, 92, 93, 94, 95, 112, 113, 32, 33, 34, -1]
    assert (cu, kv, nxt) == ([0, 8, 11], [18, 3], 2)
    assert tab.tolist() == [[5, 7, -1, -1], [2, -1, -1, -1]]


def test_plan_reference_refusals():
    table = -np.ones((4, 2), dtype=np.int64)
    out = U.plan([0, 0, 0, 4], [40, 17, 1, 1], np.where(np.arange(4)[:, None] == 3, 1, table),
                 [0], 0, 100, 16)
    # too long for the table; two blocks of one; a block after that; no block needed
    assert out[2] == [0, 0, 0, 5] and out[4] == 0
    assert out[0][58] == 20 and all(s == -1 for s in out[0][:58])


def test_scales_and_codes_reference():
    assert U.need_scale(448.0) == 1.0 and U.need_scale(448.5) == 2.0 and U.need_scale(0) == 2.0 ** -40
    assert U.need_scale(3.5) == 2.0 ** -7 and U.pow2_above(0.5) == 0.5 and U.pow2_above(0.6) == 1.0
    x = np.array([[[1.0, -3.5, np.inf, np.nan] * 16]])
    codes, scales = U.append(x, [16], np.zeros((2, 1, 16, 64), np.uint8), np.ones((2, 1)), 16)
    assert scales[1, 0] == 2.0 ** -7
    assert (U.CODE_VALUES[codes[1, 0, 0, :2]] * scales[1, 0]).tolist() == [1.0, -3.5]
    assert (codes[1, 0, 0, 2:4] == 0x7F).all()
    # a larger token raises the scale and the older one is kept exactly
    codes, scales = U.append(np.full((1, 1, 64), 100.0), [17], codes, scales, 16)
    assert scales[1, 0] == 0.25 and U.CODE_VALUES[codes[1, 0, 0, 1]] * 0.25 == -3.5


def test_attention_reference_closed_form():
    # q = 0: the mean of the visible values
    k = np.zeros((2, 1, 16, 64), np.uint8)
    v = U.encode(np.arange(2 * 16 * 64).reshape(2, 1, 16, 64) % 7 - 3.0)
    one = np.ones((2, 1))
    out = U.attend(np.zeros((2, 1, 64)), k, v, one, one, np.array([[1, 0]]), [18], [0, 2], 16, 1.0,
                   True)
    rows = np.concatenate([U.CODE_VALUES[v[1, 0]], U.CODE_VALUES[v[0, 0, :2]]])
    assert np.allclose(out[0][0, 0], rows[:17].mean(0)) and np.allclose(out[0][1, 0], rows.mean(0))
    assert np.allclose(out[1], np.log([[17], [18]]))
