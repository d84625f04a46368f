"""Orthogonalised updates by Newton-Schulz products, as an inner step of
meta-learning or test-time training takes them.

``orthogonalize`` moves the singular values of a matrix towards one and leaves its
singular vectors: an update of the same size in every direction.  Every
product runs in the library's tensor-core kernel (``fbob_orth_forward``), and
so does its derivative (``fbob_orth_backward``), through which an outer gradient
passes to what the update was computed from.
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator

import torch

from . import _binding as _b

#: a x + b x^3 + c x^5: lifts small singular values by 3.4 a step and holds the
#: others between 0.68 and 1.21
QUINTIC = (3.4445, -4.7750, 2.0315)


# limits of a call, as the library has them
_MOST_MATRICES, _MOST_ROWS, _MOST_COLUMNS, _MOST_ELEMENTS = 65535, 1 << 16, 1 << 22, 1 << 36


def _numbers(coefficients):
    """One triple or several as tuples of Python's floats, which calls can be told apart by:
    a tensor could be another number the next time."""
    if type(coefficients) is tuple and all(type(x) is float for x in coefficients):
        return (coefficients,)
    if torch.is_tensor(coefficients) or hasattr(coefficients, "tolist"):
        if torch.is_tensor(coefficients) and (coefficients.requires_grad or _b.dual(coefficients)):
            raise ValueError("coefficients are not differentiated: pass them detached")
        coefficients = coefficients.tolist()
    if not isinstance(coefficients, (tuple, list)) or not coefficients:
        raise ValueError("coefficients are (a, b, c), or one such triple for each step")
    if not isinstance(coefficients[0], (tuple, list)) and getattr(coefficients[0], "ndim", 0) == 0:
        coefficients = (coefficients,)
    for x in (x for abc in coefficients for x in abc):
        if torch.is_tensor(x) and (x.requires_grad or _b.dual(x)):
            raise ValueError("coefficients are not differentiated: pass them detached")
    return tuple(tuple(float(x) for x in abc) for abc in coefficients)


def _coefficients(steps, polynomials):
    """The steps' a, b, c as a C array."""
    if len(polynomials) == 1:
        polynomials = polynomials * steps
    if len(polynomials) != steps:
        raise ValueError(f"{len(polynomials)} polynomials for {steps} steps")
    flat = [float(x) for abc in polynomials for x in abc]
    if any(len(abc) != 3 for abc in polynomials) or not all(math.isfinite(x) for x in flat):
        raise ValueError("a polynomial is three finite numbers a, b, c of a x + b x^3 + c x^5")
    return (ctypes.c_float * len(flat))(*flat)


@functools.lru_cache(maxsize=256)
def _problem(shape, dtype, steps, polynomials, eps, keep):
    """The C description of a call on tensors of ``shape``, and its workspaces' bytes
    (forward, backward)."""
    coefficients = _coefficients(steps, polynomials)
    sizes = math.prod(shape[:-2]), shape[-2], shape[-1]
    L, short, long = sizes[0], min(sizes[1:]), max(sizes[1:])
    if L > _MOST_MATRICES or short > _MOST_ROWS or long > _MOST_COLUMNS or L * short * long > _MOST_ELEMENTS:
        raise _b.FbobError(2, f"orthogonalize: {L} matrices of {sizes[1]} x {sizes[2]}; at most "
                              f"{_MOST_MATRICES} of {_MOST_ROWS} by {_MOST_COLUMNS} (either way round), "
                              f"{_MOST_ELEMENTS} elements in all")
    o = _b.Orth(*sizes, _b.DTYPES[dtype], steps, int(keep), eps,
                ctypes.addressof(coefficients))
    o.held = coefficients  # lives as long as its address is used
    ref = ctypes.byref(o)
    sizes = tuple(_b.lib().fbob_orth_workspace_size(op, ref) for op in (_b.OP_FORWARD, _b.OP_BACKWARD))
    if 0 in sizes:
        raise _b.FbobError(2, "orthogonalize: more tiles than a call counts, a polynomial under which singular "
                              "values of [0, 1] reach 64 or small ones fall below 1/256, or eps beyond fp32")
    return ref, sizes


def _forward(g, how, keep):
    ref, sizes = _problem(g.shape, g.dtype, *how, keep)
    dev = g.device
    y = torch.empty(g.shape, dtype=g.dtype, device=dev)
    ws = torch.empty(sizes[0], dtype=torch.uint8, device=dev)
    _b.call_on(dev, "fbob_orth_forward", _b.lib().fbob_orth_forward, ref, g.data_ptr(), y.data_ptr(),
               ws.data_ptr(), sizes[0])
    return y, ws


def _backward(g, kept, dy, how):
    ref, sizes = _problem(g.shape, g.dtype, *how, True)
    dev = g.device
    dy = dy.contiguous()
    dg = torch.empty(g.shape, dtype=g.dtype, device=dev)
    ws = torch.empty(sizes[1], dtype=torch.uint8, device=dev)
    _b.call_on(dev, "fbob_orth_backward", _b.lib().fbob_orth_backward, ref, g.data_ptr(), dy.data_ptr(),
               dg.data_ptr(), kept.data_ptr(), sizes[0], ws.data_ptr(), sizes[1])
    return dg


class _Orthogonalize(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, how):
        y, kept = _forward(g, how, True)
        ctx.save_for_backward(g, kept)
        ctx.how = how
        return y

    @staticmethod
    def backward(ctx, dy):
        g, kept = ctx.saved_tensors
        if torch.is_grad_enabled() or _b.dual(dy):
            return _OrthogonalizeBackward.apply(g, dy, kept, ctx.how), None
        return _backward(g, kept, dy, ctx.how), None


class _OrthogonalizeBackward(torch.autograd.Function):
    """(g, dY) -> dG, of which no further derivative is known."""

    @staticmethod
    def forward(ctx, g, dy, kept, how):
        return _backward(g, kept, dy, how)

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError("orthogonalize has no second derivative")


def orthogonalize(g: torch.Tensor, steps: int = 5, coefficients=QUINTIC,
                  eps: float = 1e-7) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of a matrix [m, n], or of each of a stack
    [..., m, n]: X = g / (|g| + eps) with |g| its Frobenius norm, then ``steps``
    times X <- a X + b (X X^T) X + c (X X^T)^2 X.

    g: bf16 or fp32 CUDA tensor, not empty (copied first if not contiguous): up to 65535
    matrices, the shorter side up to 65536, the longer up to 2^22, 2^36 elements in all.
    coefficients: (a, b, c), or one such triple for each step, numbers, which are not
    differentiated (a tensor on the GPU is waited for); singular values
    that start in [0, 1] must stay below 64 under them, and small ones must not fall
    far: the product of those |a| that are below 1 is at least 1/256.  steps from 1 to 16.
    eps >= 0.  The shorter side is taken as the rows of X.  Norms, of g and of what comes
    from above in the backward, may be from 1e-34 to 1e38, or 0.

    Returns a contiguous tensor of g's shape and dtype.  Differentiable once in g, in
    reverse mode.  bf16: products of fp16 operands with fp32 sums.  With five steps the
    result is 1.7e-3 to 1.9e-3 of its norm off and its own rounding 1.7e-3 of that; the
    gradient 1.8e-3 to 2.6e-3 off for white noise from above, 2.4e-3 to 4.0e-3 for what lies
    among g's strong directions.  More steps enlarge what the iterates were rounded by: with
    eight, 2.7e-3 to 2.9e-3 and 0.7e-2 to 1.4e-2.  fp32: operands of 22 bits, of the largest
    entries (of others down to 2^-36 of the bound on singular values).
    """
    if not g.is_cuda:
        raise _b.FbobError(1, "orthogonalize: g must be a CUDA tensor")
    if g.dim() < 2:
        raise ValueError("g must be a matrix or a stack of matrices")
    if g.dtype not in _b.DTYPES:
        raise TypeError(f"unsupported dtype {g.dtype}; use bfloat16 or float32")
    if 0 in g.shape:
        raise _b.FbobError(1, "orthogonalize: g must not be empty")
    steps = operator.index(steps)
    if not 1 <= steps <= 16:
        raise ValueError(f"steps must be from 1 to 16, got {steps}")
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be at least 0 and finite, got {eps}")
    how = (steps, _numbers(coefficients), float(eps))
    g = g.contiguous()
    if (torch.is_grad_enabled() and g.requires_grad) or _b.dual(g):
        return _Orthogonalize.apply(g, how)
    return _forward(g, how, False)[0]
