"""Normalised queries and keys and orthogonalised updates together, as a
meta-learned layer uses them: a MAML step (first and second derivatives through
projection, norms, positions, attention and the orthogonalised inner update) against
the same step written densely in 64 bits on the CPU."""
import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300.meta import AttentionLayer, DiffAttentionLayer, maml_step, orthogonal_updates
from test_layer_operators import dense_attention, dense_diff, dense_turn, task

NAMES = ("wq", "wk", "wv", "wo")


def dense_norm(q, k, wq, wk, inv_freq=None, positions=None, *, eps=1e-6, interleaved=False,
               magnitude=1.0, dtype=None):
    out = []
    for x, w in ((q, wq), (k, wk)):
        x = x.double()
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
        out.append(y.to(dtype) if inv_freq is None else dense_turn(y, inv_freq, magnitude=magnitude,
                                                                    dtype=dtype))
    return tuple(out)


def dense_orthogonal(G):
    X = G / (torch.linalg.matrix_norm(G, keepdim=True) + 1e-7)
    X = X.mT if G.shape[-2] > G.shape[-1] else X
    for _ in range(5):
        A = X @ X.mT
        X = 3.4445 * X + (-4.7750 * A + 2.0315 * (A @ A)) @ X
    return X.mT if G.shape[-2] > G.shape[-1] else X


def layer_of(kind, device, rope):
    if kind == "attention":
        layer = AttentionLayer.random(128, 2, device, seed=1, qk_norm=True)
        layer.rope = rope
        return layer
    return DiffAttentionLayer.random(128, 2, 1, 64, 128, device, seed=1, rope=rope, qk_norm=True)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("kind", ["attention", "differential"])
@pytest.mark.parametrize("inner,lr", [("sgd", 5.0), ("orthogonal", 0.02)])
@pytest.mark.parametrize("with_rope", [True, False])
@pytest.mark.parametrize("compute,tol", [(torch.float32, 1e-3), (torch.bfloat16, 5e-2)],
                         ids=["fp32_cuda_cores", "bf16_tensor_cores"])
def test_maml_step(kind, inner, lr, with_rope, compute, tol):
    """Tolerances as for the plain layer's step: 1e-3 and 5e-2 of each
    gradient's norm.  The orthogonalised update divides by the inner gradient's
    norm, which multiplies the error of every singular value by up to 3.9 (the
    polynomial's steepest) a step where these gradients are weak; with bf16 attention, whose
    gradients are 2^-8 off, the step is compared for its loss alone."""
    rope = fbob.rotary_frequencies(32, 10000.0, "yarn", 4.0, trained_length=64) if with_rope else None
    layer = layer_of(kind, "cuda", rope)
    support, query = task(2, 96, 128, 2)
    gpu = tuple(tuple(t.cuda() for t in p) for p in (support, query))
    loss, grads = maml_step(layer, *gpu, inner_lr=lr, compute_dtype=compute, inner=inner)
    ref = layer_of(kind, "cpu", rope and (rope[0].cpu(), rope[1]))
    for name in NAMES + (("lam",) if kind == "differential" else ()):
        setattr(ref, name, getattr(ref, name).detach().double().requires_grad_(True))
    ref.qk_norm = tuple(w.detach().double().requires_grad_(True) for w in ref.qk_norm)
    cpu = tuple(tuple(t.double() for t in p) for p in (support, query))
    want_loss, want = maml_step(
        ref, *cpu, inner_lr=lr, compute_dtype=torch.float64 if compute == torch.float32 else compute,
        attn=dense_attention if kind == "attention" else dense_diff, turn=dense_turn, norm=dense_norm,
        inner=inner, orthogonal=dense_orthogonal)
    assert abs(loss.item() - want_loss.item()) <= tol * abs(want_loss.item())
    assert len(grads) == len(want) == (7 if kind == "differential" else 6)
    if inner == "orthogonal" and compute == torch.bfloat16:
        return
    for i, (a, b) in enumerate(zip(grads, want)):
        err = (a.double().cpu() - b).norm() / b.norm()
        assert err <= tol, (i, err.item())


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_updates_of_one_shape_go_through_one_call():
    g = torch.Generator("cuda").manual_seed(0)
    grads = [torch.randn(s, generator=g, device="cuda") for s in ((64, 32), (32, 64), (64, 32), (5,), ())]
    calls = []

    def spy(x):
        calls.append(tuple(x.shape))
        return fbob.orthogonalize(x)

    out = orthogonal_updates(grads, spy)
    assert sorted(calls) == [(1, 32, 64), (2, 64, 32)]
    for i in (0, 2):
        assert torch.equal(out[i], 2 ** 0.5 * fbob.orthogonalize(torch.stack((grads[0], grads[2])))[i // 2])
    assert torch.equal(out[1], fbob.orthogonalize(grads[1][None])[0])
    assert out[3] is grads[3] and out[4] is grads[4]


def test_updates_keep_their_dtypes():
    """Matrices of one shape and different dtypes do not go through one call."""
    grads = [torch.ones(4, 3, dtype=t) for t in (torch.float32, torch.bfloat16, torch.float32)]
    calls = []

    def spy(x):
        calls.append((x.dtype, x.shape[0]))
        return x

    out = orthogonal_updates(grads, spy)
    assert [t.dtype for t in out] == [t.dtype for t in grads]
    assert sorted(calls, key=str) == [(torch.bfloat16, 1), (torch.float32, 2)]


def test_refusals():
    layer = AttentionLayer.random(16, 2, "cpu", qk_norm=True)
    assert len(layer.params()) == 6
    with pytest.raises(ValueError):
        maml_step(layer, *task(1, 4, 16, 0), inner="adam")
    with pytest.raises(fbob.FbobError):
        maml_step(layer, *task(1, 4, 16, 0))
