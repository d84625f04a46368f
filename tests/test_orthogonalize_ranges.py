"""Orthogonalisation of matrices whose norm is small beside eps, against the
definition in 64 bits: what eps takes off the norm is no loss of digits."""
import pytest
import torch

import exact_second_order_two_gb300 as fbob
from test_orthogonalize import CUBIC, DT, MIXED, ONE, check, exact, gradient, model

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def both(G, dY, polynomials, eps=1e-7):
    leaf = G.clone().requires_grad_()
    Y = fbob.orthogonalize(leaf, len(polynomials), polynomials, eps=eps)
    return Y.detach(), torch.autograd.grad(Y, leaf, dY)[0]


def held(G, dY, polynomials, eps=1e-7):
    """Value and gradient within the documented roundings (``check``: relative to the norm
    of what the definition gives, whatever its size)."""
    Y, dG = both(G, dY, polynomials, eps)
    (X, want), (mY, mG) = exact(G, dY, polynomials, eps), model(G, dY, polynomials, eps)
    check(Y, X, mY, G.dtype)
    check(dG, want, mG, G.dtype)


@pytest.mark.parametrize("shape", [(60, 80), (300, 400), (403, 301), (128, 250)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("std", [1e-9, 1e-11, 1e-13, 1e-15, 1e-17])
def test_eps_outweighs_the_norm(shape, dtype, std):
    """Norms of about 1e-7 to 1e-15 beside an eps of 1e-7: X starts as small and grows by a
    every step."""
    held(*gradient(shape, DT[dtype], std=std), [ONE] * 5)


@pytest.mark.parametrize("polynomials", [MIXED, CUBIC, ((0.5, 2.0, -1.0),) * 4, ((1.1, -0.1, 0.0),) * 16],
                         ids=["mixed", "cubic", "falls", "long"])
@pytest.mark.parametrize("shape", [(60, 80), (300, 200)], ids=str)
@pytest.mark.parametrize("eps", [1e-6, 1e-2, 1.0])
def test_other_polynomials_beside_eps(polynomials, shape, eps):
    """Steps that enlarge, keep or reduce what is small, in fp32."""
    held(*gradient(shape, torch.float32, std=1e-6), list(polynomials), eps)


def test_polynomials_under_which_what_is_small_falls_far_are_refused():
    G = torch.ones(4, 5, device="cuda")
    fbob.orthogonalize(G, 2, (0.0625, 0.5, 0.0))
    for steps, a in ((1, 0.0), (1, 0.0039), (5, 0.25), (16, -0.7)):
        with pytest.raises(fbob.FbobError):
            fbob.orthogonalize(G, steps, (a, 0.5, 0.0))


@pytest.mark.parametrize("shape", [(60, 80), (150, 300)], ids=str)
def test_each_matrix_of_a_stack_has_a_scale_of_its_own(shape):
    G, dY = gradient((5, *shape), torch.float32, std=1.0)
    G *= 10.0 ** torch.tensor([-17.0, 0.0, -11.0, -8.0, 3.0], device="cuda")[:, None, None]
    Y, dG = both(G, dY, [ONE] * 5)
    for i in range(5):
        y, d = both(G[i], dY[i], [ONE] * 5)
        assert torch.equal(y, Y[i]) and torch.equal(d, dG[i])
        held(G[i], dY[i], [ONE] * 5)


@pytest.mark.parametrize("shape", [(60, 80), (300, 400)], ids=str)
def test_small_beside_eps_it_is_linear(shape):
    """Y = a^5 G / eps for G far below eps, to the rounding of fp32's 22-bit operands: x^3 is
    below 2^-60 of x."""
    G, dY = gradient(shape, torch.float32, std=1e-17)
    Y, dG = both(G, dY, [ONE] * 5)
    by = 3.4445 ** 5 / 1e-7
    for got, want in ((Y, by * G.double()), (dG, by * dY.double())):
        assert (got.double() - want).norm() <= 2.0 ** -18 * want.norm()
