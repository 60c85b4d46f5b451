"""Calls from host threads that have made no other CUDA call: such a thread has no
current context until something gives it one."""
import threading

import pytest

import attention_forward_flashattention_gb300 as fa
from attention_forward_flashattention_gb300 import cache as fc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def in_new_thread(call):
    out = []
    t = threading.Thread(target=lambda: out.append(call()))
    t.start()
    t.join()
    return out[0]


def test_first_call_of_a_thread():
    import torch
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (torch.randn(1, 2, 200, 64, device=DEV, generator=g).half() for _ in range(4))
    o, lse = fa.attention_forward(q, k, v)
    want = fa.attention_backward(q, k, v, o, lse, do)
    got = [torch.full_like(q, float("nan")) for _ in range(4)]
    lse2 = torch.zeros_like(lse)
    ws = torch.empty(fa.fa_bwd_workspace_size(1, 2, 200, 64), dtype=torch.uint8, device=DEV)
    p = [t.data_ptr() for t in (q, k, v, o, do, lse, *got, lse2, ws)]
    torch.cuda.synchronize()
    assert in_new_thread(lambda: fa.fa_fwd(*p[:3], p[9], p[10], 1, 2, 200, 64, False, 0.125, 0)) == fa.FA_OK
    assert in_new_thread(lambda: fa.fa_bwd(*p[:9], p[11], 1, 2, 200, 64, False, 0.125, 0)) == fa.FA_OK
    torch.cuda.synchronize()
    assert torch.equal(got[3], o) and torch.equal(lse2, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_first_cache_call_of_a_thread():
    import torch
    g = torch.Generator(device=DEV).manual_seed(2)
    cache = fa.cache_empty(4, 2, 16, 64, device=DEV)
    cache.k.view(torch.uint8).random_(0, 0x70, generator=g)
    cache.v.view(torch.uint8).random_(0, 0x70, generator=g)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    lens = torch.tensor([20, 32], dtype=torch.int32, device=DEV)
    for n in (1, 24):  # the kernel for few rows, and for many
        q = torch.randn(2, 2, n, 64, device=DEV, generator=g).half()
        want = fa.attention_forward_cache(q, cache, table, lens)
        o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        size = fa.fa_fwd_cache_workspace_size(2, 2 * n, 2, 2, 64)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        c = fc.FaCache(*(t.data_ptr() for t in cache), 4, 16, 2, 64, 2 * 16 * 64, 16 * 64, 64)
        st = (2 * n * 64, n * 64, 64)
        torch.cuda.synchronize()
        rc = in_new_thread(lambda: fa.fa_fwd_cache(
            q.data_ptr(), c, table.data_ptr(), 2, lens.data_ptr(), None, o.data_ptr(), lse.data_ptr(), 2,
            2 * n, 2, (st, st), True, 0.125, 0, ws.data_ptr(), size))
        assert rc == fa.FA_OK
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
