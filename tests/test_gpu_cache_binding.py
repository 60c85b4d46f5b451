"""Arguments that the block cache's torch calls have to refuse, and calls of nothing."""
import numpy as np
import pytest

import attention_forward_flashattention_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def ints(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def test_causal_without_a_truth_value_is_an_error():
    """The error that its truth test raises reaches the caller, and nothing is enqueued."""
    import torch

    class Odd:
        def __bool__(self):
            raise KeyError("no truth here")

    c = fa.cache_empty(4, 2, 16, 64, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    tab, lens = ints(np.zeros((3, 2))), ints([1, 1, 1])
    o, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device=DEV)
    ws = torch.empty(fa.fa_fwd_cache_workspace_size(3, 3, 4, 2, 64), dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError):
        fa.attention_forward_cache(q, c, tab, lens, causal=torch.tensor([True, False]))
    with pytest.raises(KeyError):
        fa.attention_forward_cache_into(q, c, tab, lens, o, lse, ws, causal=Odd())
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 7).all()
    fa.attention_forward_cache_into(q, c, tab, lens, o, lse, ws, causal=torch.tensor([True]))
    assert (o == 0).all()


def test_codes_of_another_8_bit_type_are_refused():
    """Codes are e4m3, as float8_e4m3fn or raw bytes: other 8-bit types would be read as it."""
    import torch
    c = fa.cache_empty(4, 2, 16, 64, device=DEV)
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    tab, lens = ints(np.zeros((3, 2))), ints([1, 1, 1])
    for t in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8, torch.bool):
        for bad in (c._replace(k=c.k.view(t)), c._replace(v=c.v.view(t))):
            with pytest.raises(ValueError):
                fa.cache_append(x, x, ints([0, 1, 2]), bad)
            with pytest.raises(ValueError):
                fa.attention_forward_cache(q, bad, tab, lens)
    fa.cache_append(x, x, ints([0, 1, 2]), c._replace(v=c.v.view(torch.uint8)))


def c_cache(cache):
    P, heads, bs, d = cache.k.shape
    return fa.FaCache(cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scales.data_ptr(),
                      cache.v_scales.data_ptr(), P, bs, heads, d, *cache.k.stride()[:3])


def test_a_call_of_no_rows():
    """T = 0 with the workspace that its size asks for succeeds and writes nothing; a
    workspace of no bytes is refused, as for any other call."""
    import torch
    c = fa.cache_empty(4, 2, 16, 64, device=DEV)
    tab, lens, cu = ints([[0, 1], [2, 3]]), ints([20, 30]), ints([0, 0, 0])
    q = torch.randn(2, 4, 64, device=DEV).half()
    o, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device=DEV)
    size = fa.fa_fwd_cache_workspace_size(2, 0, 4, 2, 64)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    strides = ((4 * 64, 64, 4 * 64),) * 2

    def call(cu_q, nbytes):
        return fa.fa_fwd_cache(q.data_ptr(), c_cache(c), tab.data_ptr(), 2, lens.data_ptr(), cu_q,
                               o.data_ptr(), lse.data_ptr(), 2, 0, 4, strides, True, 0.125,
                               fa.FA_DTYPE_FP16, ws.data_ptr(), nbytes)

    for cu_q in (None, cu.data_ptr()):
        assert call(cu_q, size) == fa.FA_OK
        assert call(cu_q, 0) == fa.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("short", ["rows", "blocks", "none"])
def test_a_large_plan_that_refuses(short):
    """A plan of many CTAs whose rows or free blocks run out on the way, with requests
    that are refused for their own numbers in between."""
    import cache_util as U
    rng = np.random.default_rng(7)
    B, bs, width = 700, 32, 40
    lens, new = rng.integers(0, 600, B), rng.integers(0, 60, B)
    lens[100], new[200], lens[300] = -1, -7, width * bs
    new[300] = 5
    T = int(np.maximum(new, 0).sum())
    T = T // 2 + 3 if short == "rows" else T + 9
    need = int((-(-(lens + np.maximum(new, 0)) // bs) - -(-lens // bs)).sum())
    free = rng.permutation(1 << 16)[:need // 2 if short == "blocks" else need + 4]
    table = rng.integers(0, 1 << 16, (B, width))
    tab = ints(table)
    got = fa.cache_plan(ints(lens), ints(new), tab, ints(free), ints([2]), T, bs)
    ref = U.plan(lens.tolist(), new.tolist(), table, free, 2, T, bs)
    assert [g.tolist() for g in got] == [ref[0], ref[1], ref[2], [ref[4]]]
    assert np.array_equal(tab.cpu().numpy(), ref[3])
    assert any(s == -1 for s in ref[0][:T - 9])
