"""What autograd learns of tensors that calls write to: one that an operation has saved
counts as changed, as after torch's own in-place calls, so that its backward pass raises
and does not use what is there now."""
import pytest
import torch

import attention_forward_flashattention_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def heads(h=2):
    return torch.randn(1, h, 5, 64, device=DEV).half()


@pytest.fixture
def rope():
    return fa.rope_table(5, 64, device=DEV), torch.arange(5, **I32)


def test_inputs_saved_for_gradients_and_then_overwritten(rope):
    q, k = heads(), heads()
    w = torch.ones(64, device=DEV, requires_grad=True)
    out = fa.qk_norm_rope(q, k, *rope, w, None)
    fa.qk_norm_rope_forward_into(q, k, q, k, *rope)
    with pytest.raises(RuntimeError, match="inplace"):
        out[0].float().sum().backward()


def test_outputs_that_require_gradients_are_refused(rope):
    q, k = heads().requires_grad_(), heads()
    x, y = q * 1, k.clone()   # not a leaf
    before = x.detach().clone()
    for qo, ko in ((x, y), (y, x), (q, y)):
        with pytest.raises(ValueError):
            fa.qk_norm_rope_forward_into(q.detach(), k, qo, ko, *rope)
    assert torch.equal(x, before)
    want = fa.qk_norm_rope_forward(x, y, *rope)
    with torch.no_grad():
        fa.qk_norm_rope_forward_into(x, y, x, y, *rope)
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_inference_tensors_in_place(rope):
    with torch.inference_mode():
        q, k = heads(), heads()
        want = fa.qk_norm_rope_forward(q, k, *rope)
        fa.qk_norm_rope_forward_into(q, k, q, k, *rope)
    fa.qk_norm_rope_forward_into(*want, *want, *rope)   # outside of it, too
    assert torch.equal(want[0], fa.qk_norm_rope_forward(q, k, *rope)[0])


def changed(call, *tensors):
    """Whether the call leaves every one of the tensors with a new version, and whether without it they keep theirs."""
    before = [t._version for t in tensors]
    call()
    return all(t._version > v for t, v in zip(tensors, before))


def test_attention_into():
    q, k, v = heads(), heads(), heads()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 5, device=DEV)
    assert changed(lambda: fa.attention_forward_into(q, k, v, o, lse), o, lse)
    assert q._version == k._version == v._version == 0
    x = [torch.randn(1, 2, 5, 128, device=DEV).half() for _ in range(4)]
    assert changed(lambda: fa.attention_forward_pair_into(*x, lse), x[3], lse)
    host = [torch.randn(1, 2, 5, 64).half() for _ in range(4)]
    hl = torch.empty(1, 2, 5)
    ws = torch.empty(fa.fa_fwd_host_workspace_size(1, 2, 5, 64), dtype=torch.uint8, device=DEV)
    assert changed(lambda: fa.attention_forward_host_into(*host, hl, ws), host[3], hl)
    torch.cuda.synchronize()


def test_cache_calls():
    cache = fa.cache_empty(8, 2, 16, 64, device=DEV)
    table, lens = torch.full((2, 3), -1, **I32), torch.tensor([0, 0], **I32)
    new, free, pos = torch.tensor([5, 20], **I32), torch.arange(8, **I32), torch.zeros(1, **I32)
    plan = tuple(torch.zeros(n, **I32) for n in (25, 3, 2, 1))
    assert changed(lambda: fa.cache_plan_into(lens, new, table, free, pos, *plan, 16), table, *plan)
    slots, cu, kv, pos = plan
    k, v = torch.randn(25, 2, 64, device=DEV).half(), torch.randn(25, 2, 64, device=DEV).half()
    assert changed(lambda: fa.cache_append(k, v, slots, cache), *cache)
    q = torch.randn(25, 2, 64, device=DEV).half()
    o, lse = torch.empty_like(q), torch.empty(25, 2, device=DEV)
    ws = torch.empty(fa.fa_fwd_cache_workspace_size(2, 25, 2, 2, 64), dtype=torch.uint8, device=DEV)
    assert changed(lambda: fa.attention_forward_cache_into(q, cache, table, kv, o, lse, ws, cu), o, lse)
    masks, places = torch.zeros(25, 1, dtype=torch.int64, device=DEV), torch.zeros(25, **I32)
    parents = torch.full((25,), -1, **I32)
    assert changed(lambda: fa.cache_tree_into(parents, cu, lens, masks, places), masks, places)
    assert changed(lambda: fa.attention_forward_cache_tree_into(q, cache, table, kv, masks, o, lse, ws, cu), o, lse)
    after, shares = torch.zeros(2, **I32), torch.zeros(8, **I32)
    assert changed(lambda: fa.cache_keep(cache, table, kv, cu, masks[[0, 5]].contiguous(), out=after), after, *cache)
    nxt = torch.zeros(1, **I32)
    assert changed(lambda: fa.cache_release(table, kv, after, free, pos, 16, shares, out=nxt), free, shares, nxt)
    out = (torch.zeros(2, 3, **I32), torch.zeros(2, **I32), torch.zeros(2, 3, **I32), torch.zeros(1, **I32))
    src = torch.zeros(2, **I32)
    assert changed(lambda: fa.cache_fork(table, after, src, free, nxt, shares, 16, out=out), shares, *out)
    assert changed(lambda: fa.cache_copy(cache, out[2]), *cache)
    read = (q, k, v, parents, src, new)
    assert all(t._version == 0 for t in read)
