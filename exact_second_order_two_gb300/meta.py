"""A synthetic second-order workload: one MAML / test-time-training step of a
single attention layer, on random weights.

Test-time training and meta-learning are among the uses of exact
differentiation through the backward pass that FlashBoB names ("FlashBoB:
I/O-Efficient Exact Backward-over-Backward for Softmax Attention",
Abstract).  The layer here is

    y = attention(x Wq, x Wk, x Wv) Wo        (heads split from the width)

The inner step adapts the weights on a support batch:

    W' = W - lr * grad_W L_support(W)         (create_graph=True)

The outer (meta) loss L_query(W') is then differentiated back to W through
that inner gradient.  The attention part of this second derivative is
exactly the library's backward-over-backward: fbob_forward, fbob_backward and
fbob_bob, run through ``attention``.  No N x N tensor is formed at any point.

``DiffAttentionLayer`` is the same with differential attention, whose map
weights lam are learned with the projections; and either layer can turn its
queries and keys by position (``rope``), which ``rotary`` does on the way from
the projection's layout to the heads', in the dtype that attention takes.

Only the projections and the losses (plain torch matmuls and reductions)
run outside the library.  They are the workload around the hot path, not part
of it.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from .autograd import attention
from .diff_attention import diff_attention
from .rotary import rotary


@dataclass
class AttentionLayer:
    """Weights of one multi-head attention layer: width = heads * head_dim.
    rope: (inv_freq, magnitude) of ``rotary_frequencies``, or None for a layer
    without positions."""
    wq: torch.Tensor
    wk: torch.Tensor
    wv: torch.Tensor
    wo: torch.Tensor
    heads: int
    rope: tuple | None = None

    def params(self):
        return [self.wq, self.wk, self.wv, self.wo]

    def forward(self, params, x, causal, compute_dtype, attn=None, turn=None):
        return layer_forward(params, x, self.heads, causal, compute_dtype, attn or attention,
                             self.rope, turn or rotary)

    @staticmethod
    def random(width: int, heads: int, device, dtype=torch.float32, seed: int = 0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        std = width ** -0.5
        ws = [(torch.randn(width, width, generator=g) * std).to(device, dtype)
              for _ in range(4)]
        for w in ws:
            w.requires_grad_(True)
        return AttentionLayer(*ws, heads=heads)


@dataclass
class DiffAttentionLayer:
    """Weights of one differential attention layer: ``heads`` heads with two
    queries of ``head_dim`` features each, ``key_heads`` (a divisor of heads)
    with two keys of head_dim and a value of ``value_dim`` features, and one
    learned weight of the second map per head.  rope as in AttentionLayer."""
    wq: torch.Tensor    # [width, 2 heads head_dim]
    wk: torch.Tensor    # [width, 2 key_heads head_dim]
    wv: torch.Tensor    # [width, key_heads value_dim]
    wo: torch.Tensor    # [heads value_dim, width]
    lam: torch.Tensor   # [heads]
    heads: int
    key_heads: int
    rope: tuple | None = None

    def params(self):
        return [self.wq, self.wk, self.wv, self.wo, self.lam]

    @staticmethod
    def random(width: int, heads: int, key_heads: int, head_dim: int, value_dim: int, device,
               dtype=torch.float32, seed: int = 0, rope: tuple | None = None):
        g = torch.Generator(device="cpu").manual_seed(seed)
        shapes = [(width, 2 * heads * head_dim), (width, 2 * key_heads * head_dim),
                  (width, key_heads * value_dim), (heads * value_dim, width)]
        ws = [(torch.randn(s, generator=g) * s[0] ** -0.5).to(device, dtype) for s in shapes]
        ws.append((0.2 + 0.6 * torch.rand(heads, generator=g)).to(device, dtype))
        for w in ws:
            w.requires_grad_(True)
        return DiffAttentionLayer(*ws, heads=heads, key_heads=key_heads, rope=rope)

    def forward(self, params, x, causal, compute_dtype, attn=None, turn=None):
        wq, wk, wv, wo, lam = params
        B, N, _ = x.shape
        q = _heads(x @ wq, 2 * self.heads, compute_dtype, self.rope, turn or rotary)
        k = _heads(x @ wk, 2 * self.key_heads, compute_dtype, self.rope, turn or rotary)
        v = _heads(x @ wv, self.key_heads, compute_dtype)
        o = (attn or diff_attention)(q, k, v, lam, causal=causal)
        return o.to(x.dtype).transpose(1, 2).reshape(B, N, -1) @ wo


def _heads(t, heads, compute_dtype, rope=None, turn=rotary):
    """A projection's [B, N, heads * d] as the [B, heads, N, d] that attention
    reads, turned by position where there is a rope."""
    t = t.view(t.shape[0], t.shape[1], heads, -1).transpose(1, 2)
    if rope is not None:
        return turn(t, rope[0], magnitude=rope[1], dtype=compute_dtype)
    return t.contiguous().to(compute_dtype)


def layer_forward(params, x: torch.Tensor, heads: int, causal: bool = True,
                  compute_dtype=torch.bfloat16, attn=attention, rope=None,
                  turn=rotary) -> torch.Tensor:
    """x: [B, N, width] -> [B, N, width].  Attention runs in `compute_dtype`
    with [B, H, N, d] inputs; the projections run in the weights' dtype."""
    wq, wk, wv, wo = params
    B, N, W = x.shape
    q = _heads(x @ wq, heads, compute_dtype, rope, turn)
    k = _heads(x @ wk, heads, compute_dtype, rope, turn)
    v = _heads(x @ wv, heads, compute_dtype)
    o = attn(q, k, v, causal=causal)
    o = o.to(x.dtype).transpose(1, 2).reshape(B, N, W)
    return o @ wo


def mse(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    return ((a - b) ** 2).mean()


def maml_step(layer, support, query, inner_lr: float = 0.1, causal: bool = True,
              compute_dtype=torch.bfloat16, attn=None, turn=None):
    """One meta-learning step of an AttentionLayer or DiffAttentionLayer.

    support, query: (x, y) pairs of [B, N, width] tensors.  attn and turn
    replace the layer's attention and rotary positions (for a reference).
    Returns (outer_loss, meta_grads): the query loss after one inner SGD step
    on the support loss, and its exact gradient with respect to the
    original weights (second order through the inner gradient).
    """
    params = layer.params()
    xs, ys = support
    xq, yq = query
    inner = mse(layer.forward(params, xs, causal, compute_dtype, attn, turn), ys)
    grads = torch.autograd.grad(inner, params, create_graph=True)
    adapted = [w - inner_lr * g for w, g in zip(params, grads)]
    outer = mse(layer.forward(adapted, xq, causal, compute_dtype, attn, turn), yq)
    meta_grads = torch.autograd.grad(outer, params)
    return outer.detach(), meta_grads
