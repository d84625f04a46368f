"""Rotary positions and differential attention together, as a layer uses
them: a MAML step (first and second derivatives through projection, positions,
attention and learned map weights) against the same step written densely in
64 bits on the CPU."""
import math

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300.meta import AttentionLayer, DiffAttentionLayer, maml_step

LR = 5.0  # as large as makes the second-order term a good part of the meta-gradient


def dense_attention(q, k, v, causal=True):
    dt = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    s = q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])
    n = q.shape[-2]
    if causal:
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -math.inf)
    return (torch.softmax(s, -1) @ v).to(dt)


def dense_diff(q, k, v, lam, causal=True):
    G = q.shape[1] // k.shape[1]
    v = v.repeat_interleave(G, 1)
    k1, k2 = (k[:, m::2].repeat_interleave(G, 1) for m in (0, 1))
    a = dense_attention(q[:, 0::2], k1, v, causal).double()
    b = dense_attention(q[:, 1::2], k2, v, causal).double()
    return (a - lam.double()[:, None, None] * b).to(q.dtype)


def dense_turn(x, inv_freq, positions=None, interleaved=False, magnitude=1.0, dtype=None):
    r, n = 2 * inv_freq.numel(), x.shape[2]
    angle = torch.arange(n, dtype=torch.float64)[:, None] * inv_freq.double()
    cos, sin = magnitude * angle.cos(), magnitude * angle.sin()
    a, b, rest = x[..., : r // 2].double(), x[..., r // 2: r].double(), x[..., r:].double()
    return torch.cat((a * cos - b * sin, a * sin + b * cos, rest), -1).to(dtype)


def task(B, N, width, seed):
    g = torch.Generator().manual_seed(seed)
    xs, ys, xq, yq = (torch.randn(B, N, width, generator=g) for _ in range(4))
    return (xs, 0.5 * ys), (xq, 0.5 * yq)


def layer_of(kind, device, rope):
    if kind == "attention":
        layer = AttentionLayer.random(128, 2, device, seed=1)
        layer.rope = rope
        return layer
    return DiffAttentionLayer.random(128, 2, 1, 64, 128, device, seed=1, rope=rope)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("kind", ["attention", "differential"])
@pytest.mark.parametrize("compute,tol", [(torch.float32, 1e-3), (torch.bfloat16, 5e-2)],
                         ids=["fp32_cuda_cores", "bf16_tensor_cores"])
def test_maml_step_with_positions(kind, compute, tol):
    """Tolerances as for the plain layer's step: 1e-3 and 5e-2 of each
    gradient's largest value."""
    rope = fbob.rotary_frequencies(32, 10000.0, "yarn", 4.0, trained_length=64)
    layer = layer_of(kind, "cuda", rope)
    support, query = task(2, 96, 128, 2)
    gpu = tuple(tuple(t.cuda() for t in p) for p in (support, query))
    loss, grads = maml_step(layer, *gpu, inner_lr=LR, compute_dtype=compute)
    ref = layer_of(kind, "cpu", (rope[0].cpu(), rope[1]))
    for name in ("wq", "wk", "wv", "wo") + (("lam",) if kind == "differential" else ()):
        setattr(ref, name, getattr(ref, name).detach().double().requires_grad_(True))
    cpu = tuple(tuple(t.double() for t in p) for p in (support, query))
    want_loss, want = maml_step(
        ref, *cpu, inner_lr=LR, compute_dtype=torch.float64 if compute == torch.float32 else compute,
        attn=dense_attention if kind == "attention" else dense_diff, turn=dense_turn)
    assert abs(loss.item() - want_loss.item()) <= tol * abs(want_loss.item())
    for i, (a, b) in enumerate(zip(grads, want)):
        err = (a.double().cpu() - b).abs().max() / b.abs().max()
        assert err <= tol, (i, err.item())


def test_layers_reject_cpu_inputs():
    rope = fbob.rotary_frequencies(8, device="cpu")
    layer = DiffAttentionLayer.random(16, 2, 1, 8, 8, "cpu", rope=rope)
    with pytest.raises(fbob.FbobError):
        maml_step(layer, *task(1, 4, 16, 0))
    layer.rope = None
    with pytest.raises(fbob.FbobError):
        maml_step(layer, *task(1, 4, 16, 0))
