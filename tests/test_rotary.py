"""Rotary positions against the definition in 64 bits, written with complex
numbers: values, gradients, layouts, positions, and what the call refuses."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B


TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")


def angles(positions, inv_freq):
    """positions x inv_freq less whole turns, to 64 bits: exact in rational
    numbers where a 64-bit product would lose the fraction of a turn."""
    if int(positions.abs().max()) < 1 << 20:  # off by at most 2^20 2^-53 radians per unit of f
        return positions.double()[..., None] * inv_freq
    turns = [Fraction(f) / TWO_PI for f in inv_freq.tolist()]
    rows = [[float((p * t) % 1 * TWO_PI) for t in turns] for p in positions.flatten().tolist()]
    return torch.tensor(rows, dtype=torch.float64, device=positions.device).view(
        *positions.shape, -1)


def reference(x, inv_freq, positions, interleaved, magnitude, inverse=False):
    """x turned, in 64 bits; positions [B, N]."""
    x, r = x.detach().double(), 2 * inv_freq.numel()
    angle = angles(positions, inv_freq)[:, None]
    factor = magnitude * torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    head, tail = x[..., :r], x[..., r:]
    if interleaved:
        z = torch.complex(head[..., 0::2], head[..., 1::2]) * factor
        return torch.cat((torch.stack((z.real, z.imag), -1).flatten(-2), tail), -1)
    z = torch.complex(head[..., : r // 2], head[..., r // 2:]) * factor
    return torch.cat((z.real, z.imag, tail), -1)


def assert_turned(y, x, inv_freq, positions, interleaved, magnitude, inverse=False):
    """Elementwise bound, in units of u = 2^-24 and of m(|a| + |b|): the angle
    in half turns rounds to 24 bits (pi u) and to 2^-33 turns (0.05 u), sine
    and cosine are within 2 ulp (4 u), their product with m rounds (1 u), two
    products and a sum round (3 u): below 12 u.  The stored value adds half a
    step of its type."""
    want = reference(x, inv_freq, positions, interleaved, magnitude, inverse)
    mag = reference(x, inv_freq, positions, interleaved, magnitude, inverse) * 0
    r = 2 * inv_freq.numel()
    ax = x.detach().double().abs()
    if interleaved:
        s = (ax[..., 0:r:2] + ax[..., 1:r:2]).repeat_interleave(2, -1)
    else:
        s = (ax[..., : r // 2] + ax[..., r // 2: r]).repeat(1, 1, 1, 2)
    mag[..., :r] = 12 * 2.0 ** -24 * abs(magnitude) * s
    step = torch.finfo(y.dtype).eps / 2
    bound = mag + step * (want.abs() + mag)
    err = (y.detach().double() - want).abs()
    assert (err <= bound).all(), (err / bound.clamp_min(1e-300)).max().item()


CASES = [
    # B, H, N, d, turned, in, out, layout, interleaved
    (1, 1, 1, 2, 2, "fp32", "fp32", "bhnd", False),
    (2, 3, 5, 64, 64, "bf16", "bf16", "bhnd", False),
    (2, 3, 5, 64, 64, "bf16", "bf16", "bhnd", True),
    (1, 17, 33, 128, 64, "bf16", "bf16", "bnhd", True),
    (3, 5, 7, 128, 128, "fp32", "bf16", "bnhd", False),
    (2, 2, 65, 96, 32, "fp32", "fp32", "bnhd", True),
    (1, 4, 9, 40, 40, "bf16", "fp32", "bhnd", False),
    (2, 2, 3, 13, 6, "fp32", "bf16", "bhnd", True),     # odd width: single features
    (2, 2, 3, 13, 6, "bf16", "bf16", "bnhd", False),
    (1, 2, 4, 16, 0, "bf16", "fp32", "bhnd", False),    # nothing turned: a copy
    (1, 40, 300, 64, 64, "bf16", "bf16", "bhnd", False),  # a partial group of heads
]
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(case, seed=0):
    b, h, n, d, r, tin, tout, layout, il = case
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (b, n, h, d) if layout == "bnhd" else (b, h, n, d)
    x = torch.randn(shape, generator=g, device="cuda").to(DT[tin])
    x = x.transpose(1, 2) if layout == "bnhd" else x
    f = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64, device="cuda") * 2 / max(r, 1))
    return x, f, DT[tout], il


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
class TestValues:
    @pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
    @pytest.mark.parametrize("far", [False, True])
    def test_forward_and_gradient(self, case, far):
        x, f, out, il = make(case)
        b, n = x.shape[0], x.shape[2]
        if far:  # up to 2^40, where a 32-bit angle would be noise
            pos = at = torch.randint(0, 1 << 40, (b, n), device="cuda")
        else:
            pos, at = None, torch.arange(n, device="cuda").expand(b, n)
        if far:  # multiples of 2^-12 turns up to rounding, zeros among them
            f = torch.round(f / (2 * math.pi) * 2.0 ** 12) / 2.0 ** 12 * (2 * math.pi)
        x.requires_grad_()
        y = fbob.rotary(x, f, pos, interleaved=il, magnitude=1.25, dtype=out)
        assert y.is_contiguous() and y.dtype == out and y.shape == x.shape
        assert_turned(y, x, f, at, il, 1.25)
        dy = torch.randn_like(y)
        (dx,) = torch.autograd.grad(y, x, dy)
        assert dx.dtype == x.dtype
        assert dx.stride() == x.stride() or 1 in x.shape
        assert_turned(dx, dy, f, at, il, 1.25, inverse=True)

    def test_positions_forms_agree(self):
        x, f, out, il = make(CASES[1])
        n = x.shape[2]
        a = fbob.rotary(x, f, 1000)
        p = torch.arange(1000, 1000 + n, device="cuda")
        assert torch.equal(a, fbob.rotary(x, f, p))
        assert torch.equal(a, fbob.rotary(x, f, p.expand(2, n)))
        strided = torch.stack((p, p), 1)[:, 0].expand(2, n)  # position stride 2
        assert torch.equal(a, fbob.rotary(x, f, strided))
        assert torch.equal(fbob.rotary(x, f), fbob.rotary(x, f, 0))
        b = fbob.rotary(x, f, -n)  # negative positions
        assert_turned(b, x, f, torch.arange(-n, 0, device="cuda").expand(2, n), False, 1.0)

    def test_broken_strides_and_offsets(self):
        """Rows, heads and addresses off the 16-byte steps, a broadcast head, a
        feature stride other than 1: the same values as from a copy."""
        f = make(CASES[1])[1]
        flat = torch.randn(2 * 5 * 3 * 70 + 1, device="cuda").bfloat16()
        for x in (flat[1:].view(2, 5, 3, 70)[..., :64],           # odd address, row stride 70
                  flat[:-1].view(2, 5, 3, 70)[..., 3:67],
                  flat[:2 * 3 * 64].view(2, 1, 3, 64).expand(2, 4, 3, 64),
                  flat[:2 * 5 * 64 * 3].view(2, 5, 64, 3).transpose(2, 3)):
            assert torch.equal(fbob.rotary(x, f), fbob.rotary(x.contiguous(), f))
            y = x.detach().requires_grad_()
            (g,) = torch.autograd.grad(fbob.rotary(y, f), y, torch.ones_like(y))
            assert_turned(g, torch.ones_like(y), f,
                          torch.arange(x.shape[2], device="cuda").expand(2, -1), False, 1.0, True)

    def test_every_order_of_derivative(self):
        """The gradient is linear in dy: its own gradient turns forward again,
        and finite differences of the forward agree (fp32, exact steps)."""
        x, f, out, il = make(CASES[5])
        n = x.shape[2]
        at = torch.arange(n, device="cuda").expand(2, n)
        x.requires_grad_()
        dy = torch.randn_like(x).requires_grad_()
        (dx,) = torch.autograd.grad(fbob.rotary(x, f, interleaved=True), x, dy, create_graph=True)
        g = torch.randn_like(x)
        (back,) = torch.autograd.grad(dx, dy, g, create_graph=True)
        assert_turned(back, g, f, at, True, 1.0)
        t = torch.randn_like(x)
        moved = fbob.rotary(x + t, f, interleaved=True).double() - fbob.rotary(x, f, interleaved=True).double()
        a, b = (moved * dy).sum(), (t.double() * dx).sum()
        # fp32 rounding of x + t and of both results, each below 2^-22 of |x| + |t|
        assert abs(a - b) <= 2.0 ** -20 * ((x.abs() + t.abs()) * dy.abs()).double().sum()

    def test_graph_capture_and_other_stream(self):
        x, f, out, il = make(CASES[1])
        want = fbob.rotary(x, f)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = fbob.rotary(x, f)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        static = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = fbob.rotary(static, f)
        other = torch.randn_like(x)
        static.copy_(other)
        graph.replay()
        assert torch.equal(y, fbob.rotary(other, f))

    def test_nothing_is_written_outside(self):
        """The C call into the middle of a guarded buffer, with row strides of
        its own: elements between the rows and around stay as they were."""
        x, f, out, il = make(CASES[1])
        buf = torch.full((2 * 3 * 5 * 72 + 128,), 7.0, device="cuda", dtype=torch.bfloat16)
        y = buf[64:64 + 2 * 3 * 5 * 72].view(2, 3, 5, 72)[..., :64]
        r = B.Rotary(2, 3, 5, 64, 64, 0, 0, 0, 0, 1.0, (ctypes.c_longlong * 3)(*x.stride()[:3]),
                     (ctypes.c_longlong * 3)(*y.stride()[:3]), 0, 0)
        assert B.lib().fbob_rotary(ctypes.byref(r), x.data_ptr(), f.data_ptr(), None, y.data_ptr(),
                                   B._stream(x.device)) == 0
        assert torch.equal(y, fbob.rotary(x, f))
        y.fill_(7.0)
        assert (buf == 7.0).all()

    def test_refusals(self):
        x, f, out, il = make(CASES[1])
        for bad in (lambda: fbob.rotary(x[0], f), lambda: fbob.rotary(x, f.float()),
                    lambda: fbob.rotary(x[..., :32], f), lambda: fbob.rotary(x, f[None]),
                    lambda: fbob.rotary(x, f, torch.zeros(5, device="cuda")),
                    lambda: fbob.rotary(x, f, torch.zeros(6, dtype=torch.int64, device="cuda")),
                    lambda: fbob.rotary(x, f, torch.zeros(5, dtype=torch.int64)),
                    lambda: fbob.rotary(x, f.clone().requires_grad_()),
                    lambda: fbob.rotary(x, f, 1 << 62)):
            with pytest.raises(ValueError):
                bad()
        with pytest.raises(TypeError):
            fbob.rotary(x.half(), f)
        with pytest.raises(TypeError):
            fbob.rotary(x, f, dtype=torch.float16)
        with pytest.raises(fbob.FbobError):
            fbob.rotary(x.cpu(), f)
        with pytest.raises(fbob.FbobError):
            fbob.rotary(x[:0], f)


def test_c_call_refuses_bad_arguments():
    lib = B.lib()
    good = ctypes.c_void_p(1 << 20)

    def call(x=good, f=good, p=None, y=good, **kw):
        a = dict(B=1, H=2, N=3, d=64, rotary_dim=64, interleaved=0, inverse=0, in_dtype=0,
                 out_dtype=0, magnitude=1.0)
        a.update(kw)
        r = B.Rotary(**a)
        return lib.fbob_rotary(ctypes.byref(r), x, f, p, y, None)

    assert lib.fbob_rotary(None, good, good, None, good, None) == 1
    for kw in (dict(B=0), dict(H=0), dict(N=-1), dict(d=0), dict(rotary_dim=3),
               dict(rotary_dim=66), dict(rotary_dim=-2), dict(interleaved=2), dict(inverse=-1),
               dict(magnitude=float("nan"))):
        assert call(**kw) == 1, kw
    for kw in (dict(in_dtype=2), dict(out_dtype=-1), dict(d=1026), dict(H=65536),
               dict(B=1 << 20, N=1 << 20)):
        assert call(**kw) == 2, kw
    odd = ctypes.c_void_p((1 << 20) + 1)
    assert call(x=None) == 1 and call(y=None) == 1 and call(f=None) == 1
    assert call(x=odd) == 1 and call(y=odd) == 1
    assert call(f=ctypes.c_void_p((1 << 20) + 4)) == 1 and call(p=ctypes.c_void_p((1 << 20) + 4)) == 1


def test_frequencies():
    f, m = fbob.rotary_frequencies(8, 100.0, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64
    torch.testing.assert_close(f, torch.tensor([100.0 ** (-i / 4) for i in range(4)],
                                               dtype=torch.float64), rtol=1e-15, atol=0)
    lin, m = fbob.rotary_frequencies(8, 100.0, "linear", 4.0, device="cpu")
    assert m == 1.0 and torch.equal(lin, f / 4)
    ntk, m = fbob.rotary_frequencies(8, 100.0, "ntk", 4.0, device="cpu")
    assert m == 1.0 and ntk[0] == 1.0
    assert abs(ntk[-1] * 4 / f[-1] - 1) < 1e-14  # the lowest frequency, divided by the factor
    # 2 pi, 1 and 0.01 turns in a trained length of 6.28..: kept, blended, divided
    yarn, m = fbob.rotary_frequencies(64, 10000.0, "yarn", 8.0, trained_length=4096, device="cpu")
    plain, _ = fbob.rotary_frequencies(64, 10000.0, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], plain[turns >= 32])
    torch.testing.assert_close(yarn[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((yarn < plain) & (yarn > plain / 8))[mid].all()
    assert (yarn[1:] < yarn[:-1]).all()
    assert m == 0.1 * math.log(8.0) + 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(base=0.0),
                                dict(base=float("inf")), dict(factor=0.5),
                                dict(scaling="cubic"), dict(scaling="yarn"),
                                dict(scaling="ntk", rotary_dim=2),
                                dict(scaling="yarn", trained_length=10, few_turns=3.0, many_turns=3.0)])
def test_frequencies_refusals(kw):
    a = dict(rotary_dim=8, device="cpu")
    a.update(kw)
    with pytest.raises(ValueError):
        fbob.rotary_frequencies(**a)
