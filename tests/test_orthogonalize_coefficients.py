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


@pytest.mark.parametrize("bad", [(), [], ((),), ((), ()), [[]], None, 1.5, torch.zeros(0), torch.zeros(0, 3), np.zeros((0, 3)),
                                 (1.0, 2.0), (1.0, 2.0, 3.0, 4.0), ((1.0, 2.0), (1.0, 2.0, 3.0, 4.0)),
                                 torch.ones(4), torch.ones(2, 4), (1.0, float("nan"), 0.0), "abc", torch.ones(1, 1, 3)],
                         ids=repr)
def test_what_is_no_polynomial(bad):
    """Refused by name, before any tensor is looked at."""
    module = importlib.import_module("exact_second_order_two_gb300.orthogonalize")
    with pytest.raises((ValueError, TypeError)):
        module._coefficients(2, numbers(bad))


def test_a_call_with_no_polynomial(monkeypatch):
    """The public call says what it wants (its tensor stands for one on a GPU)."""
    class Gpu(torch.Tensor):
        is_cuda = True
    g = torch.zeros(3, 4).as_subclass(Gpu)
    for bad in ((), [], torch.zeros(0)):
        with pytest.raises(ValueError):
            fbob.orthogonalize(g, 2, bad)


@pytest.mark.parametrize("shape", [(65536, 2, 3), (65537, 65537), (4, (1 << 22) + 1), ((1 << 22) + 1, 4),
                                   (60000, 2048, 2048)], ids=str)
def test_limits_are_named(shape):
    problem = importlib.import_module("exact_second_order_two_gb300.orthogonalize")._problem
    with pytest.raises(fbob.FbobError, match="at most 65535 of 65536 by 4194304"):
        problem(shape, torch.bfloat16, 5, (ONE,), 1e-7, False)


def test_polynomials_that_are_refused_are_named():
    problem = importlib.import_module("exact_second_order_two_gb300.orthogonalize")._problem
    for poly in ((4.0, 0.0, 0.0), (0.1, 0.5, 0.0)):
        with pytest.raises(fbob.FbobError, match="polynomial"):
            problem((4, 5), torch.bfloat16, 5, (poly,), 1e-7, False)
