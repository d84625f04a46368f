"""The two descriptions of the norms' C structures: packed by the calls, and by name in
the binding."""
import importlib

from exact_second_order_two_gb300 import _binding as B

Q = importlib.import_module("exact_second_order_two_gb300.qk_norm")


def fields(s):
    out = []
    for name, _ in s._fields_:
        v = getattr(s, name)
        out += list(v) if hasattr(v, "__len__") else [v or 0]
    return out


def test_a_problem():
    values = [2, 5, 64, 32, 1, 0, 1, 0, 0.5, 1.25, -(1 << 40), 1 << 41]
    assert fields(B.QkNorm.from_buffer_copy(Q._pack(*values))) == values
    assert fields(B.QkNorm(*values)) == values


def test_a_side():
    values = [7, *(1 << 40 | i for i in range(8)), *((-1) ** i * (1 << 41 | i) for i in range(15))]
    packed = Q._pack_side(*values)
    assert fields(B.NormSide.from_buffer_copy(packed)) == values
