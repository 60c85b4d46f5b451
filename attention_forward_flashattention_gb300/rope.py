"""The pass before attention (``include/fa_rope.h``): an RMS norm of every head
of q and k with learned weights, and the rotation by the tokens' positions.

    rope = fa.rope_table(4096, 128)                                  # once
    q, k = fa.qk_norm_rope(q, k, rope, positions, q_weight, k_weight)   # differentiable
    o = fa.attention(q, k, v, causal=True)

q is [B, H, N, d] and k [B, Hkv, N, d] with positions [N] or [B, N], or as a
serving step has them [T, H, d], [T, Hkv, d] and [T]: any strides that are
multiples of 8 with unit stride along d, so parts of a fused projection's rows
serve as they are. Like the rest of the binding this only marshals arguments.
"""
from __future__ import annotations

import ctypes
import os

from . import FA_OK, FaError, FaStrides, _build, _gradient, cache, load_library

HEADER = os.path.join(_build.INCLUDE, "fa_rope.h")


class FaRope(ctypes.Structure):
    """fa_rope: table, positions, weights and options of a call."""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("positions_b", ctypes.c_longlong), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("weights_fp32", ctypes.c_int),
                ("n_positions", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("eps", ctypes.c_float)]


def bind(lib) -> None:
    """Argument types of the entry points."""
    vp, i = ctypes.c_void_p, ctypes.c_int
    strides, rope = ctypes.POINTER(FaStrides), ctypes.POINTER(FaRope)
    lib.fa_qk_norm_rope.argtypes = [vp, vp, vp, vp, i, i, i, i, i, strides, rope, i, vp]
    lib.fa_qk_norm_rope.restype = i
    lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 8 + [i] * 5 + [strides, rope, i, vp, ctypes.c_size_t, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i, ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = i


# ------------------------------------------------------------ raw C ABI

def fa_qk_norm_rope(q: int, k: int, q_out: int, k_out: int, B: int, H: int, Hkv: int, N: int, d: int,
                    strides, rope: FaRope, dtype: int, stream: int = 0) -> int:
    """Same arguments as the C function; strides: 4 (b, h, n) element-stride triples."""
    return load_library().fa_qk_norm_rope(q, k, q_out, k_out, B, H, Hkv, N, d, _strides(strides, 4),
                                          None if rope is None else ctypes.byref(rope), int(dtype),
                                          stream)


def fa_qk_norm_rope_bwd(dq_out: int, dk_out: int, q: int, k: int, dq: int, dk: int, dq_weight: int,
                        dk_weight: int, B: int, H: int, Hkv: int, N: int, d: int, strides,
                        rope: FaRope, dtype: int, workspace: int, workspace_size: int,
                        stream: int = 0) -> int:
    """Same arguments as the C function; strides: 6 (b, h, n) element-stride triples."""
    return load_library().fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, B, H,
                                              Hkv, N, d, _strides(strides, 6),
                                              None if rope is None else ctypes.byref(rope), int(dtype),
                                              workspace, int(workspace_size), stream)


def fa_qk_norm_rope_bwd_workspace_size(d: int) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().fa_qk_norm_rope_bwd_workspace_size(d, ctypes.byref(n))
    if rc != FA_OK:
        raise FaError(rc, "fa_qk_norm_rope_bwd_workspace_size")
    return int(n.value)


def _strides(strides, n: int):
    if strides is None:
        return None
    if len(strides) != n:
        raise ValueError(f"{n} stride triples")
    return (FaStrides * n)(*[FaStrides(*map(int, s)) for s in strides])


# ------------------------------------------------------------ torch helpers

def rope_table(n_positions: int, rotary_dim: int, base: float = 10000.0, freq=None, device=None):
    """The float32 table [n_positions, rotary_dim] of positions 0 .. n_positions - 1:
    cosines, then sines, of position * base ** (-2 i / rotary_dim), or of position *
    freq[i] with freq a sequence of rotary_dim / 2 numbers. The angles are formed in
    64 bits, so that far positions lose nothing, and the results rounded once."""
    import torch
    device = torch.device("cuda") if device is None else torch.device(device)
    half = rotary_dim // 2
    if freq is None:
        f = base ** (-torch.arange(half, dtype=torch.float64, device=device) * 2 / rotary_dim)
    else:
        f = torch.as_tensor(freq, dtype=torch.float64, device=device)
        if tuple(f.shape) != (half,):
            raise ValueError("freq must hold rotary_dim / 2 numbers")
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def qk_norm_rope_forward(q, k, rope, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                         interleaved: bool = False, stream=None):
    """(q, k) normalised and rotated, as new contiguous tensors. rope: float32
    [positions, rotary_dim] (rope_table); positions: int32, taken as within the
    table; weights: [d] tensors, both float32 or both of q's dtype, None for ones."""
    r = (cache._native or cache._module()).qk_norm_rope(q, k, rope, positions, q_weight, k_weight, eps,
                                                        interleaved, None, stream)
    if type(r) is int:
        raise FaError(r, "fa_qk_norm_rope")
    return r


def qk_norm_rope_forward_into(q, k, q_out, k_out, rope, positions, q_weight=None, k_weight=None,
                              eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """qk_norm_rope_forward into q_out and k_out: q and k themselves (views of the
    same strides), or tensors that share no memory with them. Not differentiable:
    tensors that require gradients are refused unless gradients are off, and what
    autograd has saved of the overwritten ones counts as changed, as after torch's
    in-place calls."""
    r = cache._module().qk_norm_rope(q, k, rope, positions, q_weight, k_weight, eps, interleaved,
                                     (q_out, k_out), stream)
    if type(r) is int:
        raise FaError(r, "fa_qk_norm_rope")


def qk_norm_rope_backward(dq_out, dk_out, q, k, rope, positions, q_weight=None, k_weight=None,
                          eps: float = 1e-6, interleaved: bool = False, stream=None,
                          weight_grads=(True, True)):
    """Gradients (dq, dk, dq_weight, dk_weight) at the forward's inputs q and k for
    the gradients dq_out and dk_out of its results: dq and dk contiguous, those of the
    weights float32 (None for a weight that is None, or whose entry in weight_grads is
    False: without either there is no sum over the rows and no second launch)."""
    r = cache._module().qk_norm_rope_bwd(dq_out, dk_out, q, k, rope, positions, q_weight, k_weight, eps,
                                         interleaved, stream, *weight_grads)
    if type(r) is int:
        raise FaError(r, "fa_qk_norm_rope_bwd")
    return r


_autograd_fn = None


def _function():
    """The torch.autograd.Function behind `qk_norm_rope` (built on first use)."""
    global _autograd_fn
    if _autograd_fn is None:
        import torch

        class _QkNormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, rope, positions, q_weight, k_weight, eps, interleaved):
                ctx.save_for_backward(q, k, rope, positions, q_weight, k_weight)
                ctx.eps, ctx.interleaved = eps, interleaved
                return qk_norm_rope_forward(q, k, rope, positions, q_weight, k_weight, eps, interleaved)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dq, dk):
                q, k, rope, positions, qw, kw = ctx.saved_tensors
                g = qk_norm_rope_backward(_gradient(dq), _gradient(dk), q, k, rope, positions, qw, kw,
                                          ctx.eps, ctx.interleaved,
                                          weight_grads=ctx.needs_input_grad[4:6])
                dw = [None if x is None else x.to(w.dtype) for x, w in zip(g[2:], (qw, kw))]
                return g[0], g[1], None, None, dw[0], dw[1], None, None

        _autograd_fn = _QkNormRope
    return _autograd_fn


def qk_norm_rope(q, k, rope, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False):
    """qk_norm_rope_forward, differentiable (once) in q, k and the weights: autograd runs
    fa_qk_norm_rope_bwd on the saved inputs."""
    return _function().apply(q, k, rope, positions, q_weight, k_weight, float(eps), bool(interleaved))
