"""Norm and rotation of heads on the GPU against the 64-bit implementation of
rope_util, element by element: types, head layouts, strides, tokens from one
on, table rows, weights, values that are not finite; its gradients; streams,
graphs and the attention behind it."""
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import rope_util as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def make(B, N, heads, d, dt, layout, g):
    """[B, heads, N, d] views of unit d stride: heads or tokens outermost, or padded rows of more heads."""
    if layout == "heads":
        x = torch.randn(B, heads, N, d, generator=g).to(DEV, dt)
    elif layout == "tokens":
        x = torch.randn(B, N, heads, d, generator=g).to(DEV, dt).transpose(1, 2)
    else:
        x = torch.randn(B, N, heads + 3, d + 8, generator=g).to(DEV, dt)[:, :, 1:1 + heads, :d].transpose(1, 2)
    return x


def weights(kind, d, dt, g):
    if kind is None:
        return None
    return (1 + 0.3 * torch.randn(d, generator=g)).to(DEV, torch.float32 if kind == "fp32" else dt)


def ref(x):
    return x.detach().cpu().double()


def wref(w, d):
    return torch.ones(d, dtype=torch.float64) if w is None else ref(w)


def within(got, want, tol, what):
    bad = (got.cpu().double() - want).abs() - tol
    assert bool((bad <= 0).all()), f"{what}: {bad.max().item():.3e} over, {int((bad > 0).sum())} elements"


def check(q, k, table, pos, qw, kw, eps, pairs, dq=None, dk=None):
    """Forward, and backward where dq and dk are given, against 64 bits."""
    d = q.shape[-1]
    up = (lambda t: t) if q.dim() == 4 else (lambda t: t.transpose(0, 1)[None])
    cs = R.angles(table.cpu(), pos.cpu())
    if pos.dim() == 2:
        cs = tuple(t[:, None] for t in cs)
    half = HALF[q.dtype]
    out = fa.qk_norm_rope_forward(q, k, table, pos, qw, kw, eps=eps, interleaved=pairs)
    for name, x, w, y in (("q", q, qw, out[0]), ("k", k, kw, out[1])):
        assert y.shape == x.shape and y.is_contiguous() and y.dtype == x.dtype
        a = (up(ref(x)), wref(w, d), cs, eps, pairs)
        within(up(y), R.forward(*a), R.forward_tolerance(*a, half), name)
    if dq is None:
        return out
    g = fa.qk_norm_rope_backward(dq, dk, q, k, table, pos, qw, kw, eps=eps, interleaved=pairs)
    for name, x, dy, w, dx, dw in (("dq", q, dq, qw, g[0], g[2]), ("dk", k, dk, kw, g[1], g[3])):
        a = (up(ref(x)), up(ref(dy)), wref(w, d), cs, eps, pairs)
        want, tol = R.backward(*a), R.backward_tolerance(*a, half)
        assert dx.is_contiguous() and dx.dtype == x.dtype
        within(up(dx), want[0], tol[0], name)
        assert (dw is None) == (w is None)
        if w is not None:
            assert dw.dtype == torch.float32
            within(dw, want[1], tol[1], name + "_weight")
    return out, g


CASES = [
    # B, N, H, Hkv, r, pairs, weights, layout
    (1, 1, 1, 1, None, False, "same", "heads"),
    (1, 1, 32, 8, None, True, "same", "tokens"),
    (2, 1, 3, 1, 16, False, None, "padded"),
    (1, 7, 16, 16, None, False, "fp32", "tokens"),
    (3, 33, 5, 1, 8, True, "fp32", "heads"),
    (2, 129, 8, 4, 32, False, "same", "padded"),
    (1, 1000, 12, 3, 24, False, "same", "tokens"),
    (2, 257, 9, 9, 56, True, "same", "heads"),
    (1, 2500, 32, 4, None, False, "fp32", "heads"),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_against_64_bits(case, d, dt):
    B, N, H, Hkv, r, pairs, wk, layout = case
    g = torch.Generator().manual_seed(B * 1000 + N + d)
    q, dq = (make(B, N, H, d, dt, layout, g) for _ in range(2))
    k, dk = (make(B, N, Hkv, d, dt, layout, g) for _ in range(2))
    table = fa.rope_table(5000, r or d, device=DEV)
    pos = torch.randint(0, 5000, (N,), generator=g, dtype=torch.int32).to(DEV)
    check(q, k, table, pos, weights(wk, d, dt, g), weights(wk, d, dt, g), 1e-6, pairs, dq, dk)


@pytest.mark.parametrize("kind", ["each", "shared rows", "gaps"])
def test_positions_of_batches(kind):
    g = torch.Generator().manual_seed(5)
    q, dq = (make(3, 20, 4, 64, torch.bfloat16, "heads", g) for _ in range(2))
    k, dk = (make(3, 20, 2, 64, torch.bfloat16, "heads", g) for _ in range(2))
    pos = torch.randint(0, 90, (3, 20), generator=g, dtype=torch.int32).to(DEV)
    if kind == "shared rows":
        pos = pos[:1].expand(3, 20)
    elif kind == "gaps":
        pos = torch.randint(0, 90, (3, 31), generator=g, dtype=torch.int32).to(DEV)[:, :20]
    w = weights("fp32", 64, None, g)
    check(q, k, fa.rope_table(90, 64, device=DEV), pos, w, None, 1e-5, False, dq, dk)


def test_positions_out_of_range_are_taken_as_within():
    g = torch.Generator().manual_seed(6)
    q, k = make(1, 6, 2, 128, torch.float16, "heads", g), make(1, 6, 2, 128, torch.float16, "heads", g)
    pos = torch.tensor([-1, 0, 9, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    check(q, k, fa.rope_table(10, 128, device=DEV), pos, None, None, 1e-6, False, q.clone(), k.clone())


@pytest.mark.parametrize("T", [1, 5, 64])
def test_rows_of_tokens(T):
    """[T, H, d] parts of a fused projection's rows, as a serving step has them."""
    g = torch.Generator().manual_seed(T)
    whole = torch.randn(T, 8 + 2 + 2, 128, generator=g).to(DEV, torch.bfloat16)
    q, k = whole[:, :8], whole[:, 8:10]
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32).to(DEV)
    w = weights("same", 128, torch.bfloat16, g)
    check(q, k, fa.rope_table(300, 128, device=DEV), pos, w, w, 1e-6, False, q.clone(), k.clone())


def test_sizes_that_rows_may_have():
    """Rows of zeros, tiny and large values: eps alone, and none of it."""
    g = torch.Generator().manual_seed(8)
    x = make(1, 5, 3, 64, torch.bfloat16, "heads", g)
    x[0, :, 0] = 0
    x[0, :, 1] *= 2.0 ** -60
    x[0, :, 2] *= 2.0 ** 58
    x[0, :, 3, 1:] = 0
    dy = make(1, 5, 3, 64, torch.bfloat16, "heads", g)
    # (gradients of the tiny and zero rows are large: 1 / sqrt(eps))
    check(x, x.clone(), fa.rope_table(5, 64, device=DEV), torch.arange(5, dtype=torch.int32, device=DEV),
          None, None, 1e-6, True, dy, dy.clone())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_rows_that_are_not_finite_reach_no_other(bad):
    g = torch.Generator().manual_seed(9)
    q, k = (make(1, 9, 4, 128, torch.float16, "heads", g) for _ in range(2))
    table, pos = fa.rope_table(9, 128, device=DEV), torch.arange(9, dtype=torch.int32, device=DEV)
    dq, dk = q.flip(2).contiguous(), k.flip(2).contiguous()
    clean = fa.qk_norm_rope_forward(q, k, table, pos)
    clean_g = fa.qk_norm_rope_backward(dq, dk, q, k, table, pos)
    q[0, 2, 4, 77] = bad
    got = fa.qk_norm_rope_forward(q, k, table, pos)
    got_g = fa.qk_norm_rope_backward(dq, dk, q, k, table, pos)
    keep = torch.ones(1, 4, 9, dtype=torch.bool, device=DEV)
    keep[0, 2, 4] = False
    for a, b in ((got, clean), (got_g, clean_g)):
        assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1], b[1])
    y = got[0][0, 2, 4]
    assert bool(torch.isnan(y).any()) and bool((torch.isnan(y) | (y == 0)).all())


@pytest.mark.parametrize("layout", ["heads", "tokens", "padded"])
def test_in_place(layout):
    g = torch.Generator().manual_seed(10)
    q, k = make(2, 50, 8, 128, torch.bfloat16, layout, g), make(2, 50, 2, 128, torch.bfloat16, layout, g)
    table, pos = fa.rope_table(50, 128, device=DEV), torch.arange(50, dtype=torch.int32, device=DEV)
    w = weights("same", 128, torch.bfloat16, g)
    want = fa.qk_norm_rope_forward(q, k, table, pos, w, w)
    fa.qk_norm_rope_forward_into(q, k, q, k, table, pos, w, w)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_output_views_and_what_lies_around_them():
    g = torch.Generator().manual_seed(11)
    q, k = make(1, 30, 4, 64, torch.float16, "heads", g), make(1, 30, 2, 64, torch.float16, "heads", g)
    table, pos = fa.rope_table(30, 64, device=DEV), torch.arange(30, dtype=torch.int32, device=DEV)
    want = fa.qk_norm_rope_forward(q, k, table, pos)
    room = torch.full((1, 32, 8, 72), 7.0, dtype=torch.float16, device=DEV)
    qo, ko = room[:, 1:31, 1:5, :64].transpose(1, 2), room[:, 1:31, 5:7, :64].transpose(1, 2)
    fa.qk_norm_rope_forward_into(q, k, qo, ko, table, pos)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    qo.fill_(7.0)
    ko.fill_(7.0)
    assert bool((room == 7.0).all())


def test_rows_behind_four_gigabytes():
    """Distances between rows that do not fit into 32 bits, of inputs and of outputs."""
    g = torch.Generator().manual_seed(16)
    room = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device=DEV)
    far = [room[i * 2048:].as_strided((3, h, 128), (2 ** 30, 128, 1)) for i, h in enumerate((4, 2, 4, 2))]
    near = [torch.randn(3, h, 128, generator=g).to(DEV, torch.bfloat16) for h in (4, 2)]
    for a, b in zip(far, near):
        a.copy_(b)
    table, pos = fa.rope_table(9, 128, device=DEV), torch.tensor([2, 8, 0], dtype=torch.int32, device=DEV)
    want = fa.qk_norm_rope_forward(*near, table, pos)
    fa.qk_norm_rope_forward_into(far[0], far[1], far[2], far[3], table, pos)
    assert torch.equal(far[2], want[0]) and torch.equal(far[3], want[1])
    dwant = fa.qk_norm_rope_backward(*want, *near, table, pos)
    got = fa.qk_norm_rope_backward(far[2], far[3], far[0], far[1], table, pos)
    assert torch.equal(got[0], dwant[0]) and torch.equal(got[1], dwant[1])


def test_no_tokens():
    q, k = (torch.zeros(2, h, 0, 64, dtype=torch.float16, device=DEV) for h in (4, 2))
    table, pos = fa.rope_table(3, 64, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    out = fa.qk_norm_rope_forward(q, k, table, pos, w, w)
    assert out[0].shape == q.shape and out[1].shape == k.shape
    g = fa.qk_norm_rope_backward(q, k, q, k, table, pos, w, w)
    assert bool((g[2] == 0).all()) and bool((g[3] == 0).all())


def test_same_call_same_bits():
    g = torch.Generator().manual_seed(12)
    q, dq = (make(2, 700, 16, 64, torch.float16, "tokens", g) for _ in range(2))
    k, dk = (make(2, 700, 4, 64, torch.float16, "tokens", g) for _ in range(2))
    table, pos = fa.rope_table(700, 64, device=DEV), torch.arange(700, dtype=torch.int32, device=DEV)
    w = weights("fp32", 64, None, g)
    first = fa.qk_norm_rope_backward(dq, dk, q, k, table, pos, w, w)
    for _ in range(3):
        again = fa.qk_norm_rope_backward(dq, dk, q, k, table, pos, w, w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_binding_refuses():
    q = torch.zeros(2, 4, 5, 64, dtype=torch.float16, device=DEV)
    k = torch.zeros(2, 2, 5, 64, dtype=torch.float16, device=DEV)
    t, p = fa.rope_table(9, 64, device=DEV), torch.zeros(5, dtype=torch.int32, device=DEV)
    w = torch.ones(64, dtype=torch.float16, device=DEV)
    call = fa.qk_norm_rope_forward
    call(q, k, t, p, w, w)
    for bad in ((q.float(), k, t, p), (q, k.bfloat16(), t, p), (q, k[:1], t, p), (q, k[:, :, :4], t, p),
                (q, k, t.half(), p), (q, k, t.t(), p), (q, k, t, p.long()), (q, k, t, p[:4]),
                (q, k, t, p.cpu()), (q, k, t, p, w[:32]), (q, k, t, p, w.double()),
                (q, k, t, p, w, w.float()), (q, k, t, p, w.cpu()), (q.transpose(2, 3), k, t, p),
                (q[0, 0], k[0, 0], t, p), (q, k.cpu(), t, p)):
        with pytest.raises((ValueError, TypeError)):
            call(*bad)
    for kw in (dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(fa.FaError):
            call(q, k, t, p, **kw)
    with pytest.raises(fa.FaError):
        call(q, k, fa.rope_table(9, 128, device=DEV), p)
    with pytest.raises(fa.FaError):  # a broadcast gradient has no strides of its own
        fa.qk_norm_rope_backward(q[:, :1].expand_as(q), k, q, k, t, p)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward_into(q, k, q.float(), k, t, p)


def test_streams():
    g = torch.Generator().manual_seed(13)
    table, pos = fa.rope_table(64, 128, device=DEV), torch.arange(64, dtype=torch.int32, device=DEV)
    work = [tuple(make(1, 64, h, 128, torch.bfloat16, "tokens", g) for h in (8, 2, 8, 2)) for _ in range(4)]
    w = weights("same", 128, torch.bfloat16, g)

    def both(x, s=None):
        q, k, dq, dk = x
        return (fa.qk_norm_rope_forward(q, k, table, pos, w, w, stream=s)
                + fa.qk_norm_rope_backward(dq, dk, q, k, table, pos, w, w, stream=s))
    want = [both(x) for x in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [both(x, s) for x, s in zip(work, streams)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_graph():
    g = torch.Generator().manual_seed(14)
    q, dq = (make(2, 40, 8, 64, torch.float16, "heads", g) for _ in range(2))
    k, dk = (make(2, 40, 4, 64, torch.float16, "heads", g) for _ in range(2))
    table, pos = fa.rope_table(64, 64, device=DEV), torch.arange(40, dtype=torch.int32, device=DEV)
    w = weights("fp32", 64, None, g)

    def step():
        return (fa.qk_norm_rope_forward(q, k, table, pos, w, w)
                + fa.qk_norm_rope_backward(dq, dk, q, k, table, pos, w, w))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        fresh = torch.Generator().manual_seed(seed)
        for t in (q, k, dq, dk):
            t.copy_(torch.randn(t.shape, generator=fresh))
        pos.add_(3)
        want = step()
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("wk", ["same", "fp32", None])
def test_autograd_and_attention(wk):
    """qk_norm_rope then attention, as a training step has them: the gradients are
    those of the direct calls, bit for bit."""
    g = torch.Generator().manual_seed(15)
    dt = torch.bfloat16
    x = [make(2, 130, 4, 64, dt, "tokens", g).requires_grad_() for _ in range(3)]
    w = [weights(wk, 64, dt, g) for _ in range(2)]
    leaves = x + [t.requires_grad_() for t in w if t is not None]
    table, pos = fa.rope_table(130, 64, device=DEV), torch.arange(130, dtype=torch.int32, device=DEV)
    q, k = fa.qk_norm_rope(x[0], x[1], table, pos, *w, eps=1e-5, interleaved=True)
    o = fa.attention(q, k, x[2].contiguous(), causal=True)
    do = torch.randn(o.shape, generator=g).to(DEV, dt)
    got = torch.autograd.grad(o, leaves, do)
    with torch.no_grad():
        q2, k2 = fa.qk_norm_rope_forward(x[0], x[1], table, pos, *w, eps=1e-5, interleaved=True)
        v = x[2].contiguous()
        o2, lse = fa.attention_forward(q2, k2, v, causal=True)
        dq, dk, dv = fa.attention_backward(q2, k2, v, o2, lse, do, causal=True)
        want = fa.qk_norm_rope_backward(dq, dk, x[0], x[1], table, pos, *w, eps=1e-5, interleaved=True)
    assert torch.equal(o, o2)
    for a, b in zip(got, (want[0], want[1], dv, *(t for t in want[2:] if t is not None))):
        assert torch.equal(a, b.to(a.dtype))


def test_autograd_takes_broadcast_gradients():
    x = torch.randn(1, 2, 5, 64, device=DEV).half().requires_grad_()
    y = torch.randn(1, 2, 5, 64, device=DEV).half().requires_grad_()
    table, pos = fa.rope_table(5, 64, device=DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    q, k = fa.qk_norm_rope(x, y, table, pos)
    (q.sum() + 2 * k.sum()).backward()
    one = torch.ones_like(q)
    want = fa.qk_norm_rope_backward(one, 2 * one, x.detach(), y.detach(), table, pos)
    assert torch.equal(x.grad, want[0]) and torch.equal(y.grad, want[1])
