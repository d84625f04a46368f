"""Polynomials of orthogonalisation in every form that a program may hold them in."""
import importlib

import numpy as np
import pytest
import torch

import exact_second_order_two_gb300 as fbob

numbers = importlib.import_module("exact_second_order_two_gb300.orthogonalize")._numbers
ONE, TWO = (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)


def forms(*polynomials):
    """The same numbers as tuples, lists, tensors and arrays, whole and number by number."""
    some = [polynomials, [list(p) for p in polynomials], torch.tensor(polynomials), np.array(polynomials),
            tuple(tuple(torch.tensor(x) for x in p) for p in polynomials),
            [torch.tensor(p) for p in polynomials], [np.array(p) for p in polynomials],
            tuple(tuple(np.float32(x) for x in p) for p in polynomials)]
    if len(polynomials) == 1:
        some += [s[0] for s in some]
    return some


@pytest.mark.parametrize("polynomials", [(ONE,), (ONE, TWO, TWO)], ids=["one", "three"])
def test_forms(polynomials):
    for form in forms(*polynomials):
        got = numbers(form)
        assert got == polynomials, form
        assert all(type(x) is float for p in got for x in p)


def test_tensors_are_read_at_each_call():
    """Coefficients that change in place, as learned ones do, are other coefficients."""
    abc = [torch.tensor(x) for x in ONE]
    before = numbers(abc)
    abc[0].fill_(2.0)
    assert before == (ONE,) and numbers(abc) == ((2.0, -0.5, 0.0),)
    whole = torch.tensor(ONE)
    whole[0] = 2.0
    assert numbers(whole) == ((2.0, -0.5, 0.0),)


def test_gradients_are_not_dropped_in_silence():
    leaf = torch.tensor(ONE, requires_grad=True)
    for bad in (leaf, list(leaf), tuple(leaf.unbind()), [leaf, leaf], 2 * leaf):
        with pytest.raises(ValueError):
            numbers(bad)
    assert numbers(leaf.detach()) == (ONE,)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_a_polynomial_changed_in_place():
    G = torch.randn(30, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    for device in ("cpu", "cuda"):
        abc = tuple(torch.tensor(x, device=device) for x in ONE)
        whole = torch.tensor(ONE, device=device)
        for a in (1.5, 1.25, 1.0):
            abc[0].fill_(a)
            whole[0] = a
            want = fbob.orthogonalize(G, 3, (a, -0.5, 0.0))
            assert torch.equal(fbob.orthogonalize(G, 3, abc), want)
            assert torch.equal(fbob.orthogonalize(G, 3, whole), want)
        with pytest.raises(ValueError):
            fbob.orthogonalize(G, 3, whole.requires_grad_())
