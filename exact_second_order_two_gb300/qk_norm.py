"""Norms of queries and keys for each head, with their rotary positions in the
same pass.

``qk_norm_rotary`` takes the queries and keys of a layer, straight from their
projection, to what ``attention`` reads: every row of a head is divided by its
root mean square, weighted, turned by its position and written dense in the
wanted dtype, in one kernel for both (``fbob_qk_norm_forward``).  Its first
derivative (``fbob_qk_norm_backward``) and its second (``fbob_qk_norm_bob``),
which a MAML step takes, are one pass over the rows each, and a small sum.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _binding as _b
from .rotary import _angles

# fbob_qk_norm_t: eight ints, eps, magnitude, the stride of the positions' batches
# and the first position; fbob_norm_side_t: heads, eight pointers, five strides
_pack = struct.Struct("@8i2f2q").pack
_pack_side = struct.Struct("@i8P15q").pack
_NONE = (0, 0, 0)
_FP32_END = 3.4e38  # eps and magnitude are passed in fp32


def _strides(t):
    return _NONE if t is None else t.stride()[:3]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t):
    """t with feature stride 1, as the calls read it."""
    return t if t is None or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _like(x):
    """A dense tensor for x's gradient, laid out as the projection that x shows
    heads of: [B, N, H, d] where its heads lie within its positions."""
    B, H, N, d = x.shape
    if x.stride(2) > x.stride(1):
        return torch.empty_strided(x.shape, (N * H * d, d, H * d, 1), dtype=x.dtype, device=x.device)
    return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _side(x, w, y, dy=None, a=None, c=None, dw=None, ddy=None):
    if dy is None:  # forward
        return _pack_side(x.shape[1], x.data_ptr(), 0 if w is None else w.data_ptr(), 0, 0, 0, y.data_ptr(),
                          0, 0, *x.stride()[:3], *_NONE, *_NONE, *y.stride()[:3], *_NONE)
    at = [0 if t is None else t.data_ptr() for t in (x, w, dy, a, c, y, dw, ddy)]
    return _pack_side(x.shape[1], *at, *x.stride()[:3], *_strides(dy), *_strides(a), *y.stride()[:3],
                      *_strides(ddy))


def _forward(q, k, wq, wk, inv_freq, positions, problem, dtype):
    dev = q.device
    yq = torch.empty(q.shape, dtype=dtype, device=dev)
    yk = torch.empty(k.shape, dtype=dtype, device=dev)
    _b.call_on(dev, "fbob_qk_norm_forward", _b.lib().fbob_qk_norm_forward, problem, _side(q, wq, yq),
               _side(k, wk, yk), _ptr(inv_freq), _ptr(positions))
    return yq, yk


@functools.lru_cache(maxsize=64)
def _workspace_size(problem):
    return _b.lib().fbob_qk_norm_workspace_size(problem)


def _derivative(name, problem, sides, inv_freq, positions, sums, device):
    """A backward call on one or two sides; sums: whether it writes a weight's
    gradient."""
    n = _workspace_size(problem) if sums else 0
    ws = torch.empty(n, dtype=torch.uint8, device=device) if sums else None
    _b.call_on(device, name, getattr(_b.lib(), name), problem, sides[0],
               sides[1] if len(sides) > 1 else None, _ptr(inv_freq), _ptr(positions), _ptr(ws), n)


def _backward(xs, ws, dys, inv_freq, positions, problem, wanted):
    """(dq, dk, dwq, dwk); None for a tensor whose dy is None, and for the
    weights that are not ``wanted``."""
    out, sides, sums = [None] * 4, [], False
    for i, (x, w, dy) in enumerate(zip(xs, ws, dys)):
        if dy is None:
            continue
        dy = _rows(dy)
        out[i] = _like(x)
        if w is not None and wanted[i]:
            out[2 + i] = torch.empty(w.shape, dtype=w.dtype, device=w.device)
            sums = True
        sides.append(_side(x, w, out[i], dy, dw=out[2 + i]))
    if sides:
        _derivative("fbob_qk_norm_backward", problem, sides, inv_freq, positions, sums, xs[0].device)
    return tuple(out)


class _QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, inv_freq, positions, problem, dtype):
        ctx.save_for_backward(q, k, wq, wk, inv_freq, positions)
        ctx.problem = problem
        ctx.set_materialize_grads(False)
        return _forward(q, k, wq, wk, inv_freq, positions, problem, dtype)

    @staticmethod
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, inv_freq, positions = ctx.saved_tensors
        wanted = ctx.needs_input_grad[2:4]
        if torch.is_grad_enabled() or _b.dual(dyq, dyk):
            grads = _QkNormBackward.apply(q, k, wq, wk, dyq, dyk, inv_freq, positions, ctx.problem,
                                          wanted)
        else:
            grads = _backward((q, k), (wq, wk), (dyq, dyk), inv_freq, positions, ctx.problem, wanted)
        return *grads, None, None, None, None


class _QkNormBackward(torch.autograd.Function):
    """(q, k, wq, wk, dyq, dyk) -> (dq, dk, dwq, dwk)."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, dyq, dyk, inv_freq, positions, problem, wanted):
        ctx.save_for_backward(q, k, wq, wk, dyq, dyk, inv_freq, positions)
        ctx.problem = problem
        ctx.set_materialize_grads(False)
        return _backward((q, k), (wq, wk), (dyq, dyk), inv_freq, positions, problem, wanted)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, aq, ak, cq, ck):
        q, k, wq, wk, dyq, dyk, inv_freq, positions = ctx.saved_tensors
        _b.refuse_dual("qk_norm_rotary's second derivative", aq, ak, cq, ck)
        out, sides, sums = [None] * 6, [], False
        for i, (x, w, dy, a, c) in enumerate(((q, wq, dyq, aq, cq), (k, wk, dyk, ak, ck))):
            if dy is None or (a is None and c is None):
                continue
            dy, a = _rows(dy), _rows(a)
            c = None if c is None else c.contiguous()
            out[i], out[4 + i] = _like(x), torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
            if w is not None and ctx.needs_input_grad[2 + i]:
                out[2 + i] = torch.empty(w.shape, dtype=w.dtype, device=w.device)
                sums = True
            sides.append(_side(x, w, out[i], dy, a, c, out[2 + i], out[4 + i]))
        if sides:
            _derivative("fbob_qk_norm_bob", ctx.problem, sides, inv_freq, positions, sums, q.device)
        return *out, None, None, None, None


def _weight(name, w, d, device):
    """A weight's dtype, checked."""
    if w.device != device or w.dim() != 1 or w.shape[0] != d:
        raise ValueError(f"{name} must be [{d}] on {device}")
    if w.dtype not in _b.DTYPES:
        raise TypeError(f"unsupported {name} dtype {w.dtype}; use bfloat16 or float32")
    return w.dtype


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None = None,
                   k_weight: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None,
                   positions=None, *, eps: float = 1e-6, interleaved: bool = False,
                   magnitude: float = 1.0, dtype: torch.dtype | None = None
                   ) -> tuple[torch.Tensor, torch.Tensor]:
    """Queries and keys divided by the root mean square of each row of d
    features, weighted, and turned by position:
    rotary(x (mean(x^2) + eps)^(-1/2) weight).

    q [B, H, N, d], k [B, Hk, N, d]: bf16 or fp32 CUDA tensors of one dtype,
    feature stride 1, any other strides (another feature stride is copied
    first), d up to 256.  Weights: [d], bf16 or fp32, or None for ones; both of
    one dtype.  inv_freq, positions, interleaved and magnitude as for ``rotary``;
    without inv_freq nothing is turned.  eps >= 0.

    Returns dense tensors of ``dtype`` (default q.dtype).  Differentiable twice in
    q, k and the weights, in reverse mode (forward-mode derivatives raise
    NotImplementedError).  Gradients of the weights are sums over all rows in fp32, in a
    fixed order.  Arithmetic is fp32, rounded once.
    """
    for name, t in (("q", q), ("k", k)):
        if not t.is_cuda:
            raise _b.FbobError(1, f"qk_norm_rotary: {name} must be a CUDA tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, heads, N, d]")
    shape, device, in_dtype = q.shape, q.device, q.dtype
    if dtype is None:
        dtype = in_dtype
    if in_dtype not in _b.DTYPES or dtype not in _b.DTYPES:
        raise TypeError(f"unsupported dtypes {in_dtype}, {dtype}; use bfloat16 or float32")
    if k.dtype != in_dtype or k.device != device:
        raise ValueError(f"k must match q: {in_dtype} on {device}")
    B, _, N, d = shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError(f"k must be [{B}, heads, {N}, {d}] to go with q")
    if max(*shape, k.shape[1]) >= 1 << 31:
        raise _b.FbobError(2, "qk_norm_rotary")
    weight_dtype = torch.float32
    if q_weight is not None:
        weight_dtype = _weight("q_weight", q_weight, d, device)
    if k_weight is not None:
        if _weight("k_weight", k_weight, d, device) != weight_dtype and q_weight is not None:
            raise ValueError("the weights must have one dtype")
        weight_dtype = k_weight.dtype
    if not 0 <= eps < _FP32_END:
        raise ValueError(f"eps must be at least 0 and finite, got {eps}")
    if not abs(magnitude) < _FP32_END:
        raise ValueError(f"magnitude must be finite, got {magnitude}")
    offset, turned = 0, 0
    if inv_freq is not None:
        inv_freq, positions, offset = _angles(inv_freq, positions, q)
        turned = 2 * inv_freq.shape[0]
    elif positions is not None:
        raise ValueError("positions need inv_freq")
    problem = _pack(B, N, d, turned, bool(interleaved), _b.DTYPES[in_dtype], _b.DTYPES[dtype],
                    _b.DTYPES[weight_dtype], eps, magnitude,
                    0 if positions is None else positions.stride(0), offset)
    tensors = (_rows(q), _rows(k), _rows(q_weight), _rows(k_weight))
    seen = torch.is_grad_enabled() and (
        q.requires_grad or k.requires_grad or (q_weight is not None and q_weight.requires_grad)
        or (k_weight is not None and k_weight.requires_grad))
    if seen or _b.dual(*tensors):
        return _QkNorm.apply(*tensors, inv_freq, positions, problem, dtype)
    return _forward(*tensors, inv_freq, positions, problem, dtype)
