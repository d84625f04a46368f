"""Orthogonalised updates by Newton-Schulz products, as an inner step of
meta-learning or test-time training takes them.

``orthogonalize`` moves the singular values of a matrix towards one and leaves its
singular vectors: an update of the same size in every direction.  Every
product runs in the library's tensor-core kernel (``fbob_orth_forward``), and
so does its derivative (``fbob_orth_backward``), through which an outer gradient
passes to what the update was computed from.
"""
from __future__ import annotations

import functools
import math
import operator

import torch

from . import _binding as _b

#: a x + b x^3 + c x^5: lifts small singular values by 3.4 a step and holds the
#: others between 0.68 and 1.21
QUINTIC = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=64)
def _coefficients(steps, polynomials):
    """The steps' a, b, c as a C array (kept alive by the cache's callers)."""
    if len(polynomials) == 1:
        polynomials = polynomials * steps
    if len(polynomials) != steps:
        raise ValueError(f"{len(polynomials)} polynomials for {steps} steps")
    flat = [float(x) for abc in polynomials for x in abc]
    if len(flat) != 3 * steps or not all(math.isfinite(x) for x in flat):
        raise ValueError("a polynomial is three finite numbers a, b, c of a x + b x^3 + c x^5")
    return (_b.ctypes.c_float * len(flat))(*flat)


def _problem(g, steps, polynomials, eps, keep):
    coefficients = _coefficients(steps, polynomials)
    m, n = g.shape[-2:]
    o = _b.Orth(math.prod(g.shape[:-2]), m, n, _b.DTYPES[g.dtype], steps, int(keep), eps,
                _b.ctypes.addressof(coefficients))
    return o, coefficients


def _workspace(op, o, device):
    size = _b.lib().fbob_orth_workspace_size(op, _b.ctypes.byref(o))
    if size == 0:
        raise _b.FbobError(2, "fbob_orth_workspace_size")
    return torch.empty(size, dtype=torch.uint8, device=device)


def _forward(g, how, keep):
    o, coefficients = _problem(g, *how, keep)
    y = torch.empty(g.shape, dtype=g.dtype, device=g.device)
    ws = _workspace(_b.OP_FORWARD, o, g.device)
    _b.call_on(g.device, "fbob_orth_forward", _b.lib().fbob_orth_forward, _b.ctypes.byref(o),
               g.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel())
    return y, ws


class _Orthogonalize(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, how):
        y, kept = _forward(g, how, True)
        ctx.save_for_backward(g, kept)
        ctx.how = how
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        g, kept = ctx.saved_tensors
        _b.refuse_dual("orthogonalize's derivative", dy)
        dy = dy.contiguous()
        o, coefficients = _problem(g, *ctx.how, True)
        dg = torch.empty(g.shape, dtype=g.dtype, device=g.device)
        ws = _workspace(_b.OP_BACKWARD, o, g.device)
        _b.call_on(g.device, "fbob_orth_backward", _b.lib().fbob_orth_backward, _b.ctypes.byref(o),
                   g.data_ptr(), dy.data_ptr(), dg.data_ptr(), kept.data_ptr(), kept.numel(),
                   ws.data_ptr(), ws.numel())
        return dg, None


def orthogonalize(g: torch.Tensor, steps: int = 5, coefficients=QUINTIC,
                  eps: float = 1e-7) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of a matrix [m, n], or of each of a stack
    [..., m, n]: X = g / (|g| + eps) with |g| its Frobenius norm, then ``steps``
    times X <- a X + b (X X^T) X + c (X X^T)^2 X.

    g: bf16 or fp32 CUDA tensor, not empty (copied first if not contiguous).
    coefficients: (a, b, c), or one such triple for each step; singular values
    that start in [0, 1] must stay below 64 under them.  steps from 1 to 16.
    eps >= 0.  The shorter side is taken as the rows of X.

    Returns a contiguous tensor of g's shape and dtype.  Differentiable once in g, in
    reverse mode.  bf16: products of fp16 operands with fp32 sums, about as far from
    the exact result as its own rounding; fp32: operands of 22 bits.
    """
    if not g.is_cuda:
        raise _b.FbobError(1, "orthogonalize: g must be a CUDA tensor")
    if g.dim() < 2:
        raise ValueError("g must be a matrix or a stack of matrices")
    if g.dtype not in _b.DTYPES:
        raise TypeError(f"unsupported dtype {g.dtype}; use bfloat16 or float32")
    steps = operator.index(steps)
    if not 1 <= steps <= 16:
        raise ValueError(f"steps must be from 1 to 16, got {steps}")
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be at least 0 and finite, got {eps}")
    if coefficients is not QUINTIC:
        coefficients = tuple(coefficients)
    polynomials = coefficients if isinstance(coefficients[0], (tuple, list)) else (coefficients,)
    how = (steps, tuple(tuple(p) for p in polynomials), float(eps))
    _coefficients(*how[:2])
    g = g.contiguous()
    if (torch.is_grad_enabled() and g.requires_grad) or _b.dual(g):
        return _Orthogonalize.apply(g, how)
    return _forward(g, how, False)[0]
