"""Gradients of bf16 orthogonalisation for what a loss sends back: directions among the
matrix's strong ones, where an error in the weak ones has nothing to hide behind."""
import pytest
import torch

import exact_second_order_two_gb300 as fbob
from test_orthogonalize import ONE, exact, gradient

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def strong(shape, rank, seed=0):
    """G of ``rank`` strong directions and noise of 0.3, and dY = U C V^T among those."""
    g = torch.Generator("cuda").manual_seed(seed)
    m, n = shape
    U, V = (torch.randn(k, rank, generator=g, device="cuda") for k in (m, n))
    G = 1e-3 * (U @ V.T / rank ** 0.5 + 0.3 * torch.randn(m, n, generator=g, device="cuda"))
    C = torch.randn(rank, rank, generator=g, device="cuda")
    return G.bfloat16(), (torch.linalg.qr(U)[0] @ C @ torch.linalg.qr(V)[0].T).bfloat16()


LARGE = [((512, 512), 16), ((512, 512), 64), ((1024, 1024), 16), ((1024, 1024), 128), ((700, 1500), 16),
         ((1500, 700), 16)]
SMALL = [((128, 128), 16), ((128, 192), 16), ((128, 193), 16), ((128, 250), 16), ((250, 128), 16), ((100, 180), 16),
         ((120, 256), 20), ((64, 64), 8)]


@pytest.mark.parametrize("shape,rank,steps", [(*c, 5) for c in LARGE + SMALL] + [(*c, 8) for c in LARGE], ids=str)
def test_directions_among_the_strong_ones(shape, rank, steps):
    """dG against 64 bits, in units of bf16's half step u = 2^-8.  The result's rounding is at
    most one.  H, S and T are rounded to 11 bits (2^-12.8 of their norm, as an rms) where later
    steps multiply an error by 4 at most: two steps, three values, 6^(1/2) 4 2^-12.8 = u / 3.
    The iterates that the products of the forward read are of 11 bits as well: an rms of 2^-12.8
    for each of X, A and B of a step, enlarged by the polynomial's slope (3.9 at most) once
    on the way to the gradient: (3 steps)^(1/2) 3.9 2^-12.8 = 0.55 u for five steps, and the
    strong part, to which all is held, shrinks by up to 0.72 a step (the slope at 1) behind the
    fifth: 0.7 u / 0.72^3 = 1.9 u for eight.  2 u and 4 u hold both, with the rounding.  (Eight
    steps of small matrices, where a rank of 16 leaves too few entries to average over and the
    forward's roundings are most of the error, are not held to it.)"""
    G, dY = strong(shape, rank)
    G.requires_grad_()
    (dG,) = torch.autograd.grad(fbob.orthogonalize(G, steps), G, dY)
    want = exact(G, dY, [ONE] * steps)[1]
    err = ((dG.double() - want).norm() / want.norm()).item() * 2 ** 8
    assert err <= (2 if steps == 5 else 4), err


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 16])
@pytest.mark.parametrize("shape", [(100, 120), (128, 250), (300, 500), (2, 260, 140)], ids=str)
def test_every_number_of_steps(shape, steps):
    """Steps with one and with two terms in every place of the chain, under a polynomial with slopes
    between -0.8 and 1.9 (1.875 x - 1.25 x^3 + 0.375 x^5, that flattens at 1) and one that
    enlarges by 3.4: against fp32's gradient of the same call, which has two terms throughout."""
    flat = (1.875, -1.25, 0.375)
    for poly in ([flat] * steps, ([ONE] * steps)[:3] + [flat] * (steps - 3)):
        g = torch.Generator("cuda").manual_seed(1)
        G, dY = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
        out = []
        for t in (G, G.float()):
            leaf = t.clone().requires_grad_()
            out.append(torch.autograd.grad(fbob.orthogonalize(leaf, steps, poly), leaf, dY.to(t.dtype))[0].double())
        # of white noise: six values of 11 bits a step (X, A, B, H, S, T; 2^-12.8 as an rms),
        # 96^(1/2) 2^-12.8 = 0.35 u for 16 steps, enlarged by 4 at most where they have one
        # term, and the result's rounding, an rms of 0.43 u
        assert (out[0] - out[1]).norm() <= 2 * 2.0 ** -8 * out[1].norm()


@pytest.mark.parametrize("shape", [(16, 16, 24), (16, 17, 25), (16, 24, 16), (16, 24, 36), (16, 64, 96), (8, 128, 200)],
                         ids=str)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_small_matrices(shape, seed):
    """Value and gradient of small stacks for white noise from above, in units of u = 2^-8 (an rms:
    the results' rounding is 0.43).  What has one term adds 2^-12.8 = 0.036 u each: A in five
    steps, enlarged by the slope of 3.9 at most, 5^(1/2) 0.036 3.9 = 0.31, which with the
    rounding is 0.53 for the value, held to 0.55; the first terms of X, A and B that the backward
    reads, enlarged by 3.4, 15^(1/2) 0.036 3.4 = 0.47: 0.71 for the gradient, held to 0.75."""
    G, dY = gradient(shape, torch.bfloat16, seed=seed)
    G.requires_grad_()
    Y = fbob.orthogonalize(G)
    (dG,) = torch.autograd.grad(Y, G, dY)
    for got, want, most in zip((Y.detach(), dG), exact(G, dY, [ONE] * 5), (0.55, 0.75)):
        err = ((got.double() - want).norm() / want.norm()).item() * 2 ** 8
        assert err <= most, err


def test_against_fp32():
    """The same matrix and gradient as fp32 tensors: 22-bit operands, 2^-16 of the result."""
    G, dY = (t.float() for t in strong((512, 512), 16))
    G.requires_grad_()
    (dG,) = torch.autograd.grad(fbob.orthogonalize(G), G, dY)
    want = exact(G, dY, [ONE] * 5)[1]
    assert (dG.double() - want).norm() <= 2.0 ** -16 * want.norm()
