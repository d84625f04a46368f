"""Orthogonalisation of matrices whose norm is small beside eps, or whose squares are
past fp32's range, against the definition in 64 bits and against themselves times
powers of two."""
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


def same(got, want, power):
    """got is want 2^power: the same bits, but for results about the subnormal ones.  There
    both terms of dG = by_h H - by_g G, or their sum, are rounded to the subnormals' step
    (2^-126 eps; fp32's for the terms): up to half a step for each of the two roundings here and
    of the one there.  Above 2^-124 a half of that step is below half of the result's own."""
    want = want * 2.0 ** power
    step = 2.0 ** -126 * torch.finfo(got.dtype).eps
    off = torch.where(want.abs() >= 2.0 ** -124, 0.0, 1.5 * step).double()
    return bool(torch.isfinite(want).all() and ((got.double() - want.double()).abs() <= off).all())


@pytest.mark.parametrize("shape", [(60, 80), (300, 400), (403, 301), (3, 40, 50), (2048, 2048)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("power", [-90, -80, -66, 66, 80, 105])
def test_a_power_of_two_leaves_the_bits(shape, dtype, power):
    """Without eps the result does not know G's size, and the gradient goes with its
    reciprocal: bits are the same, for entries whose squares are past fp32's range on both sides."""
    G, dY = gradient(shape, DT[dtype], std=1.0)
    Y, dG = both(G, dY, [ONE] * 5, eps=0.0)
    y, dg = both(G * 2.0 ** power, dY, [ONE] * 5, eps=0.0)
    assert same(y, Y, 0) and same(dg, dG, -power)


@pytest.mark.parametrize("shape", [(60, 80), (300, 400), (403, 301), (2048, 2048)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("power", [-90, -80, -66, 66, 80, 105])
def test_a_power_of_two_in_the_gradient_leaves_the_bits(shape, dtype, power):
    G, dY = gradient(shape, DT[dtype], std=1.0)
    want = both(G, dY, [ONE] * 5)[1]
    assert same(both(G, dY * 2.0 ** power, [ONE] * 5)[1], want, power)


def test_one_entry_of_any_size_among_zeros():
    """x / |x| for the smallest and largest entries, in an edge of one matrix of a stack.  One
    singular value of 1 takes the polynomial's own values.  X, A and B are rounded once a step
    (2^-11 for bf16, 2^-22 for fp32), which the step multiplies by at most 8 all three together
    (|b x| + 2 |c x| and what X gives A, for x <= 1.2), and the slopes behind it, of 1.3 at most, by
    3: five steps, 120 roundings; the result's own is 2^-8 and 2^-24."""
    for dtype, tol in ((torch.bfloat16, 120 * 2.0 ** -11 + 2.0 ** -8), (torch.float32, 120 * 2.0 ** -22)):
        for shape in ((2, 30, 40), (2, 200, 300), (2, 1500, 1600)):
            for x in (1e-34, 1e-20, 1e18, 1e37):
                G = torch.zeros(shape, dtype=dtype, device="cuda")
                G[0, 0, 0] = 1.0
                G[1, -1, -1] = x
                Y = fbob.orthogonalize(G, eps=0.0)
                want = 1.0
                for _ in range(5):
                    want = 3.4445 * want - 4.775 * want ** 3 + 2.0315 * want ** 5
                assert abs(Y[1, -1, -1].item() - want) <= tol * abs(want), (dtype, shape, x)
                Y[0, 0, 0] = Y[1, -1, -1] = 0
                assert not Y.any()


def test_norms_past_fp32_of_entries_within():
    """Entries of 1e38 in rows, norms of up to 3e38."""
    for dtype in DT.values():
        G = torch.zeros(200, 300, dtype=dtype, device="cuda")
        G[torch.arange(8), torch.arange(8)] = 1e38
        Y = fbob.orthogonalize(G)
        X, own = exact(G.float() * 2.0 ** -100, None, [ONE] * 5, eps=0.0)[0], model(G * 2.0 ** -100, None, [ONE] * 5)[0]
        check(Y, X, own, dtype)


@pytest.mark.parametrize("shape", [(60, 80), (300, 400), (1500, 1600)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_power_of_two_about_the_ends_of_squares(shape, dtype):
    """Norms whose squares, or sums of them in parts, or parts of them, are past fp32's range:
    every size of G and of dY from 2^40 to 2^70, and from 2^-40 to 2^-70."""
    G, dY = gradient(shape, DT[dtype], std=1.0)
    Y, dG = both(G, dY, [ONE] * 5, eps=0.0)
    for power in (*range(40, 71), *range(-70, -39)):
        y, dg = both(G * 2.0 ** power, dY * 2.0 ** power, [ONE] * 5, eps=0.0)
        assert torch.equal(y, Y) and torch.equal(dg, dG), power
