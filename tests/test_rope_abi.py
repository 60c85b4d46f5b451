"""fa_rope.h: exported symbols, every refusal of bad arguments before a GPU is
touched, and the tests' own 64-bit implementation against closed forms and differences."""
import ctypes
import math

import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import rope_util as R
from attention_forward_flashattention_gb300 import build as fabuild
from attention_forward_flashattention_gb300 import rope as fr

GOOD = 0x100000  # aligned stand-in addresses: never dereferenced by the checks


def addr(i):
    return GOOD + 0x10000 * i


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


def test_header_and_exports(lib):
    names = fa.header_functions(fr.HEADER)
    assert names == ["fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size"]
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


def rope(**kw):
    r = dict(table=addr(30), positions=addr(31), positions_b=0, q_weight=addr(32), k_weight=addr(33),
             weights_fp32=0, n_positions=100, rotary_dim=128, interleaved=0, eps=1e-6)
    r.update(kw)
    return fr.FaRope(*r.values())


ST = (8192, 128, 512)


def fwd_rc(r=None, q=addr(0), k=addr(1), qo=addr(2), ko=addr(3), B=2, H=4, Hkv=2, N=5, d=128, st=(ST,) * 4,
           dtype=fa.FA_DTYPE_BF16):
    return fa.fa_qk_norm_rope(q, k, qo, ko, B, H, Hkv, N, d, st, rope() if r is None else r, dtype)


def bwd_rc(r=None, dqo=addr(0), dko=addr(1), q=addr(2), k=addr(3), dq=addr(4), dk=addr(5), dqw=addr(6),
           dkw=addr(7), B=2, H=4, Hkv=2, N=5, d=128, st=(ST,) * 6, dtype=fa.FA_DTYPE_BF16, ws=addr(8),
           size=1 << 40):
    return fa.fa_qk_norm_rope_bwd(dqo, dko, q, k, dq, dk, dqw, dkw, B, H, Hkv, N, d, st,
                                  rope() if r is None else r, dtype, ws, size)


SHARED = [dict(q=0), dict(k=addr(1) + 8), dict(B=0), dict(H=0), dict(Hkv=-1), dict(N=-1), dict(dtype=2)]


@pytest.mark.parametrize("kw", SHARED + [dict(qo=0), dict(ko=addr(3) + 2), dict(st=None),
                                         dict(st=(ST, ST, ST, (8192, 12, 512))),
                                         dict(st=(ST, (0, 128, 512), ST, ST))])
def test_forward_refuses(kw):
    assert fwd_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SHARED + [dict(dqo=0), dict(dk=0), dict(dqw=addr(6) + 2), dict(ws=0),
                                         dict(ws=addr(8) + 4), dict(st=None), dict(dkw=addr(6)),
                                         dict(st=(ST,) * 5 + ((8192, -128, 512),))])
def test_backward_refuses(kw):
    assert bwd_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(table=0), dict(positions=0), dict(table=addr(30) + 8),
                                dict(positions=addr(31) + 2), dict(q_weight=addr(32) + 4),
                                dict(positions_b=-1), dict(n_positions=0), dict(rotary_dim=0),
                                dict(rotary_dim=136), dict(rotary_dim=20), dict(eps=0.0),
                                dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan)])
def test_rope_refused(kw):
    assert fwd_rc(rope(**kw)) == fa.FA_ERR_INVALID_ARG
    assert bwd_rc(rope(**kw)) == fa.FA_ERR_INVALID_ARG
    assert fa.load_library().fa_qk_norm_rope(addr(0), addr(1), addr(2), addr(3), 1, 1, 1, 1, 128, None, None,
                                             0, None) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(d=96), dict(d=256), dict(N=1 << 29), dict(H=2147483647, Hkv=2147483647),
                                dict(B=2147483647, N=2147483647)])
def test_unsupported(kw):
    r = rope(rotary_dim=64)
    assert fwd_rc(r, **kw) == fa.FA_ERR_UNSUPPORTED
    assert bwd_rc(r, **kw) == fa.FA_ERR_UNSUPPORTED
    assert fwd_rc(st=(ST, ST, (1 << 38, 128, 512), ST)) == fa.FA_ERR_UNSUPPORTED


def test_no_device_is_an_error_not_a_fallback():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (fwd_rc(), fwd_rc(N=0), bwd_rc(), bwd_rc(dqw=0, dkw=0, ws=0, size=0)):
        assert rc in (fa.FA_ERR_CUDA, fa.FA_ERR_ARCH)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(x, x, torch.zeros(4, 64), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.rope_table(4, 64, freq=[1.0] * 31, device="cpu")


# ------------------------------------------------------------ the table, and the tests' own implementation

def test_table():
    t = fa.rope_table(131072, 64, device="cpu")
    assert t.shape == (131072, 64) and t.dtype == torch.float32
    for p, i in ((0, 0), (1, 3), (131071, 0), (99999, 31)):
        a = p * 10000.0 ** (-2 * i / 64)
        assert abs(t[p, i].item() - math.cos(a)) <= 2.0 ** -24
        assert abs(t[p, 32 + i].item() - math.sin(a)) <= 2.0 ** -24
    f = fa.rope_table(5, 8, freq=[1.0, 0.5, 0.25, 0.0], device="cpu")
    assert f[4, 7].item() == 0.0 and abs(f[4, 5].item() - math.sin(2.0)) <= 2.0 ** -24


@pytest.mark.parametrize("pairs", [False, True])
def test_reference_closed_form(pairs):
    # a quarter turn: (a, b) becomes (-b, a)
    x = torch.arange(1, 17, dtype=torch.float64).view(1, 1, 1, 16)
    cs = (torch.zeros(1, 1, 1, 4, dtype=torch.float64), torch.ones(1, 1, 1, 4, dtype=torch.float64))
    rms = math.sqrt((x * x).mean().item())
    y = R.forward(x, torch.full((16,), 2.0, dtype=torch.float64), cs, 0.0, pairs)[0, 0, 0] * rms / 2
    want = [-2, 1, -4, 3, -6, 5, -8, 7] if pairs else [-5, -6, -7, -8, 1, 2, 3, 4]
    assert torch.allclose(y, torch.tensor(want + list(range(9, 17)), dtype=torch.float64))


@pytest.mark.parametrize("pairs", [False, True])
def test_reference_gradient_is_the_differences(pairs):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(2, 3, 4, 16, dtype=torch.float64, generator=g) for _ in range(2))
    w = torch.randn(16, dtype=torch.float64, generator=g)
    cs = R.angles(fa.rope_table(50, 8, device="cpu"), torch.tensor([3, 49, 0, 17]))
    dx, dw = R.backward(x, dy, w, cs, 1e-5, pairs)
    f = lambda x, w: (R.forward(x, w, cs, 1e-5, pairs) * dy).sum()  # noqa: E731
    h = 1e-6
    for i in range(0, x.numel(), 7):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = h
        e = e.view_as(x)
        assert abs(((f(x + e, w) - f(x - e, w)) / (2 * h) - dx.flatten()[i]).item()) < 1e-8
    for i in range(16):
        e = torch.zeros(16, dtype=torch.float64)
        e[i] = h
        assert abs(((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]).item()) < 1e-8


# ------------------------------------------------------------ outputs at their inputs' addresses

TOK = (128, 4096, 128 * 64)   # the same memory, other places of the rows


@pytest.mark.parametrize("kw", [dict(qo=addr(3)), dict(qo=addr(1)), dict(ko=addr(0)), dict(q=addr(1), qo=addr(1)),
                                dict(qo=addr(0), st=(ST, ST, TOK, ST)), dict(ko=addr(1), st=(ST, ST, ST, TOK)),
                                dict(qo=addr(0), st=(ST, ST, (8192, 128, 520), ST))])
def test_forward_refuses_outputs_over_other_rows(kw):
    assert fwd_rc(**kw) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dq=addr(5)), dict(dq=addr(1)), dict(dk=addr(0)), dict(dq=addr(3)),
                                dict(dk=addr(2)), dict(dq=addr(0), st=(ST,) * 4 + (TOK, ST)),
                                dict(dk=addr(1), st=(ST,) * 5 + (TOK,)), dict(dq=addr(2), st=(ST,) * 4 + (TOK, ST))])
def test_backward_refuses_outputs_over_other_rows(kw):
    assert bwd_rc(**kw) == fa.FA_ERR_INVALID_ARG


def test_in_place_is_not_refused():
    """Accepted as far as the device is asked for (no GPU) or, without tokens, altogether; strides
    of axes of length one do not count."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_CUDA, fa.FA_ERR_ARCH)
    assert fwd_rc(qo=addr(0), ko=addr(1)) in none
    assert fwd_rc(qo=addr(0), ko=addr(1), st=(ST, ST, (64, 128, 512), (64, 128, 512)), B=1) in none
    assert fwd_rc(qo=addr(0), ko=addr(1), st=(ST, ST, (64, 8, 8), (64, 8, 8)), B=1, H=1, Hkv=1, N=1) in none
    assert fwd_rc(qo=addr(3), N=0) in none
    assert bwd_rc(dq=addr(0), dk=addr(1)) in none
