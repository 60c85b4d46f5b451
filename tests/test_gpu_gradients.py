"""Gradients as autograd hands them over, to the norm and rotation and to the attention:
parts of larger tensors at any address, of batches without tokens, with weights
that need none."""
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
from attention_forward_flashattention_gb300 import rope as fr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def heads(n=5, h=2):
    return torch.randn(1, h, n, 64, device=DEV).half().requires_grad_()


@pytest.mark.parametrize("odd", [1, 3, 8])
def test_gradients_that_are_parts_of_a_larger_tensor(odd):
    """The gradient of torch.cat's result reaches its inputs as views, behind `odd` elements."""
    x, y, z = heads(), heads(), torch.randn(odd, device=DEV).half().requires_grad_()
    table, pos = fa.rope_table(5, 64, device=DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    q, k = fa.qk_norm_rope(x, y, table, pos)
    all_ = torch.cat([z, q.flatten(), k.flatten()])
    g = torch.randn_like(all_)
    all_.backward(g)
    want = fa.qk_norm_rope_backward(g[odd:odd + q.numel()].clone().view_as(q), g[odd + q.numel():].clone().view_as(k),
                                    x.detach(), y.detach(), table, pos)
    assert torch.equal(x.grad, want[0]) and torch.equal(y.grad, want[1])


@pytest.mark.parametrize("odd", [1, 3, 8])
def test_attention_gradient_that_is_a_part_of_a_larger_tensor(odd):
    q, k, v, z = heads(), heads(), heads(), torch.randn(odd, device=DEV).half().requires_grad_()
    o = fa.attention(q, k, v)
    all_ = torch.cat([z, o.flatten()])
    g = torch.randn_like(all_)
    all_.backward(g)
    with torch.no_grad():
        o, lse = fa.attention_forward(q, k, v)
        want = fa.attention_backward(q, k, v, o, lse, g[odd:].clone().view_as(o))
    assert all(torch.equal(a.grad, b) for a, b in zip((q, k, v), want))


@pytest.mark.parametrize("shape", [(2, 4, 0, 64), (0, 4, 5, 64), (0, 4, 0, 64), (0, 4, 64)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_batches_without_tokens(shape, dt):
    """Empty gradients, and weights whose gradient is 0: from sums, whose gradients are broadcast, too."""
    kshape = (*shape[:1], 2, *shape[2:])
    q, k = (torch.zeros(s, device=DEV, dtype=dt, requires_grad=True) for s in (shape, kshape))
    w = [torch.ones(64, device=DEV, requires_grad=True) for _ in range(2)]
    table = fa.rope_table(5, 64, device=DEV)
    pos = torch.zeros(shape[2] if len(shape) == 4 else shape[0], dtype=torch.int32, device=DEV)
    for broadcast in (False, True):
        a, b = fa.qk_norm_rope(q, k, table, pos, *w)
        assert a.shape == q.shape and b.shape == k.shape
        if broadcast:
            got = torch.autograd.grad(a.sum() + b.sum(), (q, k, *w))
        else:
            got = torch.autograd.grad((a, b), (q, k, *w), (torch.zeros_like(a), torch.zeros_like(b)))
        assert got[0].shape == q.shape and got[1].shape == k.shape
        assert all(x.shape == (64,) and bool((x == 0).all()) for x in got[2:])


@pytest.mark.parametrize("of_q,of_k", [(False, False), (True, False), (False, True), (True, True)])
def test_weights_that_need_no_gradient(of_q, of_k, monkeypatch):
    """Their sums are not formed, and everything else has the same bits."""
    x, y = heads(700, 8), heads(700, 4)
    w = [(1 + 0.1 * torch.randn(64, device=DEV)).requires_grad_(need) for need in (of_q, of_k)]
    table, pos = fa.rope_table(700, 64, device=DEV), torch.arange(700, dtype=torch.int32, device=DEV)
    plain = fa.qk_norm_rope_backward
    made = []
    monkeypatch.setattr(fr, "qk_norm_rope_backward", lambda *a, **kw: made.append(plain(*a, **kw)) or made[-1])
    q, k = fa.qk_norm_rope(x, y, table, pos, *w)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    torch.autograd.backward((q, k), (dq, dk))
    with torch.no_grad():
        want = plain(dq, dk, x, y, table, pos, *w)
    assert torch.equal(x.grad, want[0]) and torch.equal(y.grad, want[1])
    for i, need in enumerate((of_q, of_k)):
        assert (made[0][2 + i] is not None) == need
        assert torch.equal(w[i].grad, want[2 + i]) if need else w[i].grad is None
    none = plain(dq, dk, x.detach(), y.detach(), table, pos, *w, weight_grads=(False, False))
    assert none[2] is None and none[3] is None and torch.equal(none[0], want[0])
