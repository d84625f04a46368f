"""The size of orthogonalised inner updates of layers that are not square."""
import pytest
import torch

from exact_second_order_two_gb300.meta import AttentionLayer, DiffAttentionLayer, maml_step, orthogonal_updates
from test_layer_operators import dense_diff, task
from test_meta_operators import dense_orthogonal


def orthogonal(g):
    """The nearest matrix with singular values 1."""
    u, _, v = torch.linalg.svd(g, full_matrices=False)
    return u @ v


@pytest.mark.parametrize("inputs,outputs", [(8, 32), (32, 8), (8, 8), (1, 7), (7, 1)])
def test_outputs_move_alike(inputs, outputs):
    """The largest root mean square of an update's outputs, for inputs of root mean square 1: 1 for
    square layers and those with more outputs, as much as singular values of 1 give for others."""
    w = torch.randn(inputs, outputs, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    (u,) = orthogonal_updates([w], orthogonal, inputs_first=True)
    most = torch.linalg.matrix_norm(u, 2) * (inputs / outputs) ** 0.5
    assert abs(most - max(1.0, (inputs / outputs) ** 0.5)) < 1e-12
    (t,) = orthogonal_updates([w.T.contiguous()], orthogonal)  # [outputs, inputs]
    assert (t.T - u).abs().max() < 1e-12


def test_inner_steps_take_weights_as_the_layers_hold_them():
    """The step of a differential layer with 4 times as many query features as key features, by
    hand: weights are [inputs, outputs]."""
    layer = DiffAttentionLayer.random(16, 4, 1, 8, 8, "cpu", dtype=torch.float64, seed=2)
    support, query = (tuple(t.double() for t in p) for p in task(1, 12, 16, 3))
    how = dict(compute_dtype=torch.float64, attn=dense_diff)
    loss, _ = maml_step(layer, support, query, inner_lr=0.05, inner="orthogonal", orthogonal=dense_orthogonal, **how)
    params = layer.params()

    def error(ps, pair):
        return ((layer.forward(ps, pair[0], True, torch.float64, dense_diff) - pair[1]) ** 2).mean()

    grads = torch.autograd.grad(error(params, support), params)
    moved = []
    for w, g in zip(params, grads):
        if g.dim() == 2:
            g = dense_orthogonal(g) * max(1.0, w.shape[1] / w.shape[0]) ** 0.5
        moved.append(w - 0.05 * g)
    assert {tuple(w.shape) for w in params} == {(16, 64), (16, 16), (16, 8), (32, 16), (4,)}
    want = error(moved, query)
    assert abs(loss - want) <= 1e-12 * abs(want)


def dense_on_gpu(G):
    return dense_orthogonal(G.double()).to(G.dtype)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("kind", ["attention", "differential"])
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2.0 ** -8), (torch.bfloat16, 2.0 ** -5)], ids=["fp32", "bf16"])
def test_meta_gradients_through_bf16_attention(kind, dtype, tol):
    """Weights of both types, bf16 attention, and the inner updates by the library against the
    same step with updates in 64 bits: all else is equal, so that every gradient is
    held.  bf16: the update is u = 2^-8 off at most in each entry and its gradient 4 u of its norm;
    attention rounds its inputs and its outputs in both passes, of which those that come out on
    another side of a step are u off each: 8 u.  fp32: the update is 2^-16 off, and few
    of those roundings change: u."""
    if kind == "attention":
        layer = AttentionLayer.random(128, 2, "cuda", dtype=dtype, seed=1, qk_norm=True)
    else:
        layer = DiffAttentionLayer.random(128, 2, 1, 64, 128, "cuda", dtype=dtype, seed=1, qk_norm=True)
    support, query = (tuple(t.cuda().to(dtype) for t in p) for p in task(2, 96, 128, 2))
    out = [maml_step(layer, support, query, inner_lr=0.02, inner="orthogonal", orthogonal=o)
           for o in (None, dense_on_gpu)]
    assert abs(out[0][0].item() - out[1][0].item()) <= tol * abs(out[1][0].item())
    for i, (a, b) in enumerate(zip(out[0][1], out[1][1])):
        assert a.dtype == dtype and torch.isfinite(a).all()
        assert (a.double() - b.double()).norm() <= tol * b.double().norm(), i
