"""Rotary positions for the queries and keys of an attention layer.

``rotary`` turns the feature pairs of every row by its position times the
pairs' frequencies (``fbob_rotary``), reading strided projections in place
and writing the dense [B, H, N, d] tensor in the dtype that ``attention``
takes.  The map is linear in its input, so its derivative of every order runs
the same kernel: a MAML step differentiates through it twice.

``rotary_frequencies`` computes the frequencies, also scaled for contexts
longer than those a model was trained on.
"""
from __future__ import annotations

import math
import operator
import struct

import torch

from . import _binding as _b


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None,
                       factor: float = 1.0, trained_length: int | None = None,
                       few_turns: float = 1.0, many_turns: float = 32.0,
                       device="cuda") -> tuple[torch.Tensor, float]:
    """Frequencies base^(-2i / rotary_dim), i < rotary_dim / 2, in radians per
    position, and the magnitude to give ``rotary`` with them.

    scaling stretches the context by ``factor`` >= 1:
      None      no scaling
      "linear"  positions interpolated: every frequency divided by factor
      "ntk"     the base raised to base * factor^(r / (r - 2)), which divides
                the lowest frequency by factor and leaves the highest
      "yarn"    by how often a pair turns within ``trained_length`` positions:
                with at most ``few_turns`` its frequency is divided by factor,
                with at least ``many_turns`` it stays, linear in between; the
                magnitude is 0.1 ln(factor) + 1
    Returns (float64 tensor [rotary_dim / 2] on ``device``, magnitude).
    """
    r = operator.index(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError(f"rotary_dim must be even and at least 2, got {rotary_dim}")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError(f"base must be positive and finite, got {base}")
    if not (factor >= 1 and math.isfinite(factor)):
        raise ValueError(f"factor must be at least 1 and finite, got {factor}")
    i = torch.arange(r // 2, dtype=torch.float64)
    magnitude = 1.0
    if scaling == "ntk":
        if r == 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (r / (r - 2))
    freq = float(base) ** (-2.0 * i / r)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if trained_length is None or trained_length < 1:
            raise ValueError("yarn scaling needs trained_length >= 1")
        if not few_turns < many_turns:
            raise ValueError("few_turns must be below many_turns")
        turns = trained_length * freq / (2 * math.pi)
        keep = ((turns - few_turns) / (many_turns - few_turns)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")
    return freq.to(device), magnitude


# fbob_rotary_t: nine ints, the magnitude, the strides of x and y, the stride of
# the positions' batches and the first position
_pack = struct.Struct("@9if8q").pack


def _turn(x, inv_freq, positions, how, strides):
    """One fbob_rotary call into a new tensor (dense, or with ``strides``);
    how: offset, interleaved, magnitude, output dtype, inverse."""
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        x = x.contiguous()
    shape = x.shape
    offset, interleaved, magnitude, dtype, inverse = how
    if strides is None:
        y = torch.empty(shape, dtype=dtype, device=x.device)
    else:
        y = torch.empty_strided(shape, strides, dtype=dtype, device=x.device)
    r = _pack(*shape, 2 * inv_freq.shape[0], interleaved, inverse, _b.DTYPES[x.dtype],
              _b.DTYPES[dtype], magnitude, *x.stride()[:3], *y.stride()[:3],
              0 if positions is None else positions.stride(0), offset)
    _b.call_on(x.device, "fbob_rotary", _b.lib().fbob_rotary, r, x.data_ptr(), inv_freq.data_ptr(),
               None if positions is None else positions.data_ptr(), y.data_ptr())
    return y


class _Rotary(torch.autograd.Function):
    """x -> rotary(x); its backward is itself with the angle negated."""

    @staticmethod
    def forward(ctx, x, inv_freq, positions, how, strides):
        ctx.save_for_backward(inv_freq, positions)
        ctx.how = (*how[:3], x.dtype, not how[4])
        # the gradient takes the layout of a dense projection, read as [B, H, N, d]
        # or as [B, N, H, d], and is dense otherwise
        ctx.strides = None if x.is_contiguous() or not x.transpose(1, 2).is_contiguous() \
            else x.stride()
        return _turn(x, inv_freq, positions, how, strides)

    @staticmethod
    def backward(ctx, dy):
        inv_freq, positions = ctx.saved_tensors
        turn = _Rotary.apply if torch.is_grad_enabled() or _b.dual(dy) else _turn
        return turn(dy, inv_freq, positions, ctx.how, ctx.strides), None, None, None, None


def rotary(x: torch.Tensor, inv_freq: torch.Tensor, positions=None, *, interleaved: bool = False,
           magnitude: float = 1.0, dtype: torch.dtype | None = None) -> torch.Tensor:
    """Turn the first 2 * len(inv_freq) features of x [B, H, N, d] by position.

    Pair i is features (2i, 2i + 1) when ``interleaved``, else (i, i + r/2)
    with r = 2 * len(inv_freq); at position p it turns by p * inv_freq[i] and
    is scaled by ``magnitude``.  Later features are copied.

    x: bf16 or fp32 CUDA tensor, feature stride 1, any other strides (another
    feature stride is copied first).  inv_freq: float64 CUDA tensor of
    frequencies (``rotary_frequencies``), not differentiated.  positions:
    None (0 .. N-1), an int (that position on), or an int64 CUDA tensor
    [N] or [B, N].  Returns a dense [B, H, N, d] tensor of ``dtype`` (default
    x.dtype), differentiable in x to any order in reverse mode; forward-mode
    derivatives raise NotImplementedError.
    """
    if not x.is_cuda:
        raise _b.FbobError(1, "rotary: x must be a CUDA tensor")
    if x.dim() != 4:
        raise ValueError("x must be [B, H, N, d]")
    dtype = x.dtype if dtype is None else dtype
    if x.dtype not in _b.DTYPES or dtype not in _b.DTYPES:
        raise TypeError(f"unsupported dtypes {x.dtype}, {dtype}; use bfloat16 or float32")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.device != x.device:
        raise ValueError(f"inv_freq must be a float64 vector on {x.device}")
    if inv_freq.requires_grad or _b.dual(inv_freq):
        raise ValueError("inv_freq is not differentiated: pass it detached")
    if 2 * inv_freq.numel() > x.shape[-1]:
        raise ValueError(f"inv_freq turns {2 * inv_freq.numel()} features of {x.shape[-1]}")
    if not inv_freq.is_contiguous():
        inv_freq = inv_freq.contiguous()
    offset = 0
    if positions is not None and not torch.is_tensor(positions):
        offset, positions = operator.index(positions), None
        if not -(1 << 62) <= offset < 1 << 62:
            raise ValueError(f"position {offset} is out of range")
    if positions is not None:
        B, N = x.shape[0], x.shape[2]
        if positions.dtype != torch.int64 or positions.device != x.device or \
                tuple(positions.shape) not in ((N,), (B, N)):
            raise ValueError(f"positions must be int64 [{N}] or [{B}, {N}] on {x.device}")
        if positions.dim() == 1:
            positions = positions.expand(B, N)
        if positions.stride(1) != 1 and N > 1:
            positions = positions.contiguous()
    # without autograd's node where no derivative can follow
    seen = (x.requires_grad and torch.is_grad_enabled()) or _b.dual(x)
    turn = _Rotary.apply if seen else _turn
    how = (offset, bool(interleaved), float(magnitude), dtype, False)
    return turn(x, inv_freq, positions, how, None)
