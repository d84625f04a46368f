"""Differential attention: the weighted difference of two softmax maps over
the same values, O = softmax(c Q1 K1^T) V - lam softmax(c Q2 K2^T) V, with a
learned lam.

``diff_forward`` and ``diff_backward`` are the library's two calls
(``fbob_diff_forward``, ``fbob_diff_backward``); ``diff_attention`` is the
twice-differentiable function on top of them, next to ``attention``.

The second derivative needs no kernel of its own.  The first backward is that
of plain attention for each map, with upstream gradient dO for the first and
-lam dO for the second, and dlam_i = -dO_i . O2_i.  So its backward is the
library's backward-over-backward (``fbob_bob``) of each map, with the chain
rule through -lam dO, plus, for the cotangent g of dlam, a first backward of
the second map with upstream -g dO.  The maps' queries and keys are padded
with zero features (or the values with zero columns) where their widths
differ, which changes no score and no product.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding as _b

LAM_ONE, LAM_HEAD, LAM_ROW = 0, 1, 2


def _shape(q, k, v, lam, causal, scale) -> _b.DiffShape:
    """Checks the inputs against one another and describes the problem."""
    if not q.is_cuda:
        raise _b.FbobError(1, "diff_attention: tensors must be CUDA tensors")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4:
            raise ValueError(f"{name} must have four dimensions")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, expected {q.device}")
        if t.dtype != q.dtype:
            raise ValueError(f"{name} must match q: {q.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dtype not in _b.DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}; use bfloat16 or float32")
    B, H2, N, d = q.shape
    Hk, dv = v.shape[1], v.shape[3]
    if H2 % 2:
        raise ValueError("q must hold two query heads per head: [B, 2H, N, d]")
    H = H2 // 2
    if tuple(k.shape) != (B, 2 * Hk, N, d):
        raise ValueError(f"k must be [{B}, 2 * {Hk}, {N}, {d}] to go with q and v")
    if v.shape[0] != B or v.shape[2] != N:
        raise ValueError(f"v must be [{B}, heads, {N}, width] to go with q")
    if Hk == 0 or H % Hk:
        raise ValueError(f"{H} query heads cannot share {Hk} key heads evenly")
    if not torch.is_tensor(lam):
        raise TypeError(f"lam must be a tensor, got {type(lam).__name__}")
    if lam.device != q.device:
        raise ValueError(f"lam is on {lam.device}, expected {q.device}")
    if lam.dtype not in _b.DTYPES:
        raise TypeError(f"unsupported lam dtype {lam.dtype}; use bfloat16 or float32")
    if lam.dim() == 0:
        kind = LAM_ONE
    elif tuple(lam.shape) == (H,):
        kind = LAM_HEAD
    elif tuple(lam.shape) == (B, H, N):
        kind = LAM_ROW
    else:
        raise ValueError(f"lam must have no dimensions, [{H}] or [{B}, {H}, {N}]")
    if not lam.is_contiguous():
        raise ValueError("lam must be contiguous")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return _b.DiffShape(B, H, Hk, N, d, dv, _b.DTYPES[q.dtype], int(bool(causal)), kind,
                        _b.DTYPES[lam.dtype], float(scale))


def _match(name, t, shape, dtype, device):
    if t is None or tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {device}")


def _rest_shape(shp):
    return (shp.B, shp.H, shp.N, 3 if shp.dtype == _b.DTYPES[torch.bfloat16] else 1, shp.dv)


def _workspace(op, shp, device, given=None):
    """The caller's workspace, checked (its size is the library's to check), or
    a new one."""
    if given is not None:
        if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
            raise ValueError(f"workspace must be contiguous uint8 on {device}")
        return given
    n = _b.lib().fbob_diff_workspace_size(op, ctypes.byref(shp))
    if n == 0:
        raise _b.FbobError(2, "fbob_diff_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def diff_forward(q, k, v, lam, causal: bool = False, scale: float | None = None,
                 need_rest: bool = True, workspace=None):
    """Differential attention forward: returns (O, rest, LSE).  rest is what
    else ``diff_backward`` reads, or None where ``need_rest`` is false:
    [B, H, N, 1, dv] with O2 = softmax(c Q2 K2^T) V for fp32, [B, H, N, 3, dv]
    with O2 and what its and O's rounding left off for bf16.  LSE [B, 2H, N] holds
    the rows' log-sum-exp of both maps.

    q: [B, 2H, N, d], the two queries of head h as heads 2h and 2h + 1;
    k: [B, 2Hk, N, d] likewise; v: [B, Hk, N, dv], with H a multiple of Hk
    (query head h reads key head h // (H / Hk)); bf16 or fp32, contiguous and at
    16-byte boundaries, d and dv up to 128 (bf16 multiples of 8 run on the tensor
    cores).
    lam: no dimensions, [H] or [B, H, N], bf16 or fp32.  scale, above 0 and up to 2e38,
    defaults to 1/sqrt(d); with ``causal`` key j is visible to query i iff j <= i.  A key
    whose score is -inf has no weight; but as in the dense product, an infinite
    or NaN value reaches rows that give it none (0 times it is NaN): v and
    upstream gradients are to be finite in padded rows too.

    workspace: uint8 tensor of ``fbob_diff_workspace_size`` bytes for one call
    at a time, whose ``status`` can be read afterwards; by default a new one.
    """
    return _forward(_shape(q, k, v, lam, causal, scale), q, k, v, lam, need_rest, workspace)


def _forward(shp, q, k, v, lam, need_rest, workspace=None):
    dev = q.device
    o = torch.empty((shp.B, shp.H, shp.N, shp.dv), dtype=q.dtype, device=dev)
    rest = torch.empty(_rest_shape(shp), dtype=q.dtype, device=dev) if need_rest else None
    lse = torch.empty((shp.B, 2 * shp.H, shp.N), dtype=torch.float32, device=dev)
    ws = _workspace(_b.OP_FORWARD, shp, dev, workspace)
    _b.call_on(dev, "fbob_diff_forward", _b.lib().fbob_diff_forward, ctypes.byref(shp),
               q.data_ptr(), k.data_ptr(), v.data_ptr(), lam.data_ptr(), o.data_ptr(),
               None if rest is None else rest.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    return o, rest, lse


def diff_backward(q, k, v, lam, o, rest, lse, do, causal: bool = False,
                  scale: float | None = None, workspace=None):
    """First backward for upstream gradient ``do`` and the forward's results:
    returns (dQ, dK, dV, dlam), of the inputs' shapes and dtypes.  As in the dense
    products, an infinite or NaN query or key reaches the gradients of rows that
    give it no weight."""
    shp = _shape(q, k, v, lam, causal, scale)
    rows = (shp.B, shp.H, shp.N, shp.dv)
    for name, t, shape in (("o", o, rows), ("rest", rest, _rest_shape(shp)), ("do", do, rows)):
        _match(name, t, shape, q.dtype, q.device)
    _match("lse", lse, (shp.B, 2 * shp.H, shp.N), torch.float32, q.device)
    return _backward(shp, q, k, v, lam, o, rest, lse, do, workspace)


def _backward(shp, q, k, v, lam, o, rest, lse, do, workspace=None):
    dev = q.device
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dv, dlam = torch.empty_like(v), torch.empty_like(lam)
    ws = _workspace(_b.OP_BACKWARD, shp, dev, workspace)
    _b.call_on(dev, "fbob_diff_backward", _b.lib().fbob_diff_backward, ctypes.byref(shp),
               q.data_ptr(), k.data_ptr(), v.data_ptr(), lam.data_ptr(), o.data_ptr(),
               rest.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(),
               dv.data_ptr(), dlam.data_ptr(), ws.data_ptr(), ws.numel())
    return dq, dk, dv, dlam


def _contig(t: torch.Tensor) -> torch.Tensor:
    return t if t.is_contiguous() else t.contiguous()


def _rows(lam, B, H, N):
    """lam, or its cotangent, as fp32 [B, H, N, 1]."""
    f = lam.float()
    f = f[:, None] if f.dim() == 1 else f
    return f.expand(B, H, N).unsqueeze(-1)


class _DiffBackward(torch.autograd.Function):
    """(q, k, v, lam, dO) -> (dQ, dK, dV, dlam); its backward runs fbob_bob
    on each map."""

    @staticmethod
    def forward(ctx, q, k, v, lam, do, o, rest, lse, shp):
        do = _b.dense(do)
        grads = _backward(shp, q, k, v, lam, o, rest, lse, do)
        ctx.save_for_backward(q, k, v, lam, do, o, rest, lse)
        ctx.causal, ctx.scale = bool(shp.causal), shp.scale
        ctx.set_materialize_grads(False)
        return grads

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk, gv, glam):
        q, k, v, lam, do, o, rest, lse = ctx.saved_tensors
        o2 = rest[..., 0, :].contiguous()
        none = (None,) * 4
        if gq is None and gk is None and gv is None and glam is None:
            return (None,) * 5 + none
        _b.refuse_dual("diff_attention's second derivative", gq, gk, gv, glam)
        B, H2, N, d = q.shape
        H, Hk, dv = H2 // 2, v.shape[1], v.shape[3]
        G, wide = H // Hk, max(d, dv)
        dtype = q.dtype

        def fit(t, per_head):
            """[B, heads, N, w] with every query head its own, zero-padded."""
            if t is None:
                return None
            if per_head != H:
                t = t.repeat_interleave(G, 1)
            if t.shape[-1] < wide:
                t = torch.nn.functional.pad(t, (0, wide - t.shape[-1]))
            return _b.dense(t)

        # What fbob_bob and fbob_backward read is in the tensors' type, as the
        # forward of plain attention leaves it: O of either map is rounded for
        # them.  The products formed here take O2 with what its rounding left
        # off.  The results are linear in the upstream gradient, so one factor
        # per head is multiplied in behind them, in fp32; one per query goes into
        # the upstream gradient, which rounds it (2 heads x 800 tokens, d = 64,
        # dv = 128, bf16: gradients of q, k and v 0.0029 to 0.0031 of their norm
        # off, with a factor per head 0.0027 to 0.0029).
        w = _rows(lam, B, H, N)
        per_query = lam.dim() == 3
        vv, gvv = fit(v, Hk), fit(gv, Hk)
        dof, o2f = do.float(), rest[..., 0, :].float()
        if rest.shape[3] == 3:
            o2f = o2f + rest[..., 1, :].float()
        o1 = o.float() + w * o2f
        if rest.shape[3] == 3:
            o1 += rest[..., 2, :].float()
        o1 = o1.to(dtype)

        def upstream(f):
            """dO to give to the library for f dO, and how to read its results."""
            if per_query:
                return fit((f * dof).to(dtype), H), torch.Tensor.float
            return fit(do, H), lambda t: f * t.float()

        gdo = torch.zeros(do.shape, dtype=torch.float32, device=do.device)
        grad_lam = torch.zeros((B, H, N), dtype=torch.float32, device=do.device)
        gradq, gradk, gradv = [], [], torch.zeros((B, H, N, wide), dtype=torch.float32,
                                                  device=do.device)
        for m in (0, 1):
            qm, km = fit(q[:, m::2], H), fit(k[:, m::2], Hk)
            om = fit(o2 if m else o1, H)
            lm = _b.dense(lse[:, m::2])  # at B = H = 1 contiguous as it is, at any address
            up, read = upstream(-w) if m else (fit(do, H), torch.Tensor.float)
            gqm = None if gq is None else fit(gq[:, m::2], H)
            gkm = None if gk is None else fit(gk[:, m::2], Hk)
            a = _b.bob(qm, km, vv, om, lm, up, gqm, gkm, gvv, ctx.causal, ctx.scale)
            rq, rk = read(a[0]), read(a[1])
            gradv += read(a[2])
            gup = a[3][..., :dv].float()  # does not depend on the upstream gradient
            if m == 0:
                gdo += gup
            else:
                gdo -= w * gup
                grad_lam -= (dof * gup).sum(-1)
                if glam is not None:
                    g = _rows(glam, B, H, N)
                    up, read = upstream(-g)
                    b = _b.backward(qm, km, vv, om, lm, up, ctx.causal, ctx.scale)
                    rq += read(b[0])
                    rk += read(b[1])
                    gradv += read(b[2])
                    gdo -= g * o2f
            gradq.append(rq[..., :d])
            gradk.append(rk[..., :d].unflatten(1, (Hk, G)).sum(2))
        gradv = gradv[..., :dv].unflatten(1, (Hk, G)).sum(2).to(dtype)
        gradq = torch.stack(gradq, 2).flatten(1, 2).to(dtype)
        gradk = torch.stack(gradk, 2).flatten(1, 2).to(dtype)
        if lam.dim() == 0:
            grad_lam = grad_lam.sum()
        elif lam.dim() == 1:
            grad_lam = grad_lam.sum((0, 2))
        return (gradq, gradk, gradv, grad_lam.to(lam.dtype), gdo.to(dtype)) + none


class _DiffAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, shp):
        o, rest, lse = _forward(shp, q, k, v, lam, True)
        ctx.save_for_backward(q, k, v, lam, o, rest, lse)
        ctx.shp = shp
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, lam, o, rest, lse = ctx.saved_tensors
        # o, rest and lse enter as values: the second derivative's paths through
        # them are part of what fbob_bob returns
        if torch.is_grad_enabled() or _b.dual(do):
            grads = _DiffBackward.apply(q, k, v, lam, do, o.detach(), rest, lse, ctx.shp)
        else:
            grads = _backward(ctx.shp, q, k, v, lam, o, rest, lse, _b.dense(do))
        return *grads, None


def diff_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                   causal: bool = False, scale: float | None = None) -> torch.Tensor:
    """Differential attention whose first and second derivatives run in the
    library: per head, softmax(scale Q1 K1^T) V - lam softmax(scale Q2 K2^T) V,
    masked to j <= i when causal.

    q [B, 2H, N, d], k [B, 2Hk, N, d], v [B, Hk, N, dv] and lam as for
    ``diff_forward`` (inputs that are not contiguous, or not at a 16-byte
    boundary, are copied first).  Returns
    [B, H, N, dv].  Differentiable twice in q, k, v and lam, in reverse mode
    (forward-mode derivatives raise NotImplementedError); scale is not
    differentiated.  Backward passes can be captured into a CUDA graph together
    with their forward, from leaves that no live eager graph was built from
    (autograd would tie the capture to that graph's stream).
    """
    if not torch.is_tensor(lam):
        raise TypeError(f"lam must be a tensor, got {type(lam).__name__}")
    q, k, v, lam = _b.dense(q), _b.dense(k), _b.dense(v), _contig(lam)
    shp = _shape(q, k, v, lam, causal, scale)
    if (torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                     or lam.requires_grad)) or _b.dual(q, k, v, lam):
        return _DiffAttention.apply(q, k, v, lam, shp)
    # no backward can follow: rest is not written
    return _forward(shp, q, k, v, lam, False)[0]
