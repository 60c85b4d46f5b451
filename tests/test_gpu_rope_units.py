"""Norm and rotation of so many tokens that a lane group takes eight heads, in two
batches: numbers of heads that leave the second batch whole, half full and empty,
against 64 bits element by element (formed on the GPU, by rope_util)."""
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


def tokens_for_eight(d):
    """Tokens from which on a unit keeps eight heads: 2048 / (d / 8) units to an SM, two of a token."""
    return 1024 * 8 // d * torch.cuda.get_device_properties(0).multi_processor_count + 137


def within(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert bool((bad <= 0).all()), f"{what}: {bad.max().item():.3e} over, {int((bad > 0).sum())} elements"


@pytest.mark.parametrize("d,dt", [(64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("H,Hkv", [(8, 1), (12, 5), (13, 8), (4, 16)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_eight_heads_of_a_unit(layout, pairs, H, Hkv, d, dt):
    g = torch.Generator(device=DEV).manual_seed(H * 100 + Hkv + d)
    N, r, eps = tokens_for_eight(d), d // 2 if pairs else d, 1e-6

    def rows(heads):
        if layout == "heads":
            return torch.randn(1, heads, N, d, device=DEV, generator=g).to(dt)
        return torch.randn(1, N, heads, d, device=DEV, generator=g).to(dt).transpose(1, 2)
    x, dy = [rows(H), rows(Hkv)], [rows(H), rows(Hkv)]
    w = [1 + 0.3 * torch.randn(d, device=DEV, generator=g) for _ in range(2)]
    table = fa.rope_table(N, r, device=DEV)
    pos = torch.randint(0, N, (N,), device=DEV, generator=g, dtype=torch.int32)
    cs = R.angles(table, pos)
    out = fa.qk_norm_rope_forward(*x, table, pos, *w, eps=eps, interleaved=pairs)
    grads = fa.qk_norm_rope_backward(*dy, *x, table, pos, *w, eps=eps, interleaved=pairs)
    for i, name in enumerate("qk"):
        a = (x[i].double(), w[i].double(), cs, eps, pairs)
        within(out[i], R.forward(*a), R.forward_tolerance(*a, HALF[dt]), name)
        a = (x[i].double(), dy[i].double(), *a[1:])
        dx, dw = R.backward(*a)
        tol_x, tol_w = R.backward_tolerance(*a, HALF[dt])
        within(grads[i], dx, tol_x, "d" + name)
        within(grads[2 + i], dw, tol_w, name + "_weight")
    # in place, and the same bits again
    again = fa.qk_norm_rope_backward(*dy, *x, table, pos, *w, eps=eps, interleaved=pairs)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    fa.qk_norm_rope_forward_into(*x, *x, table, pos, *w, eps=eps, interleaved=pairs)
    assert all(torch.equal(a, b) for a, b in zip(x, out))
