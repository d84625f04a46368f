"""Newton-Schulz orthogonalisation and its gradient against the definition in 64
bits (torch's autograd), at the sizes, shapes and values where it can go wrong,
and what the call refuses."""
import ctypes
import importlib
import math

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ONE = (3.4445, -4.7750, 2.0315)
MIXED = (ONE,) * 3 + ((1.875, -1.25, 0.375),) * 2
CUBIC = ((1.5, -0.5, 0.0),) * 3


def exact(G, dY, polynomials, eps=1e-7):
    """(X, dG) of one stack in 64 bits."""
    G = G.detach().double().requires_grad_()
    X = G / (torch.linalg.matrix_norm(G, keepdim=True) + eps)
    tall = G.shape[-2] > G.shape[-1]
    X = X.mT if tall else X
    for a, b, c in polynomials:
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X.mT if tall else X
    (dG,) = torch.autograd.grad(X, G, dY.double()) if dY is not None else (None,)
    return X.detach(), dG


def rounded(x, terms):
    """x to one or two fp16 terms, at a power of two that keeps small entries normal."""
    s = 2.0 ** math.floor(math.log2(2.0 ** 12 / max(float(x.abs().max()), 1e-30)))
    hi = (x * s).half().double()
    return (hi + ((x * s - hi).half().double() if terms == 2 else 0)) / s


def model(G, dY, polynomials, eps=1e-7):
    """(X, dG) with the roundings that the operator documents and exact sums: operands
    in fp16 terms, one for bf16 tensors (and X in two where it is added and the steps from
    it on enlarge a rounding by more than 16), two for fp32."""
    bf16 = G.dtype == torch.bfloat16
    one = 1 if bf16 else 2
    g = G.detach().double()
    tall = g.shape[-2] > g.shape[-1]
    g = g.mT if tall else g
    norm = torch.linalg.matrix_norm(g, keepdim=True)
    X, kept = g / (norm + eps), []
    for i, (a, b, c) in enumerate(polynomials):
        grow = math.prod(max(1.0, abs(p[0])) for p in polynomials[i:])
        X = rounded(X, 2 if grow > 16 else one)
        Xm = rounded(X, one)
        A = rounded(Xm @ Xm.mT, one)
        P = rounded(b * A + c * (A @ A), one)
        kept.append((Xm, A, P))
        X = a * X + P @ Xm
    Y = (X.mT if tall else X).to(G.dtype)
    if dY is None:
        return Y, None
    H = dY.double()
    H = H.mT if tall else H
    for (a, b, c), (X, A, P) in zip(reversed(polynomials), reversed(kept)):
        H = rounded(H, one)
        S = H @ X.mT
        S = rounded(S + S.mT, one)
        T = A @ S
        T = rounded(b * S + c * (T + T.mT), one)
        H = a * H + P @ H + T @ X
    s = 1 / (norm + eps)
    H = s * (H - g * ((H * g).sum((-1, -2), keepdim=True) * s / norm))
    return Y, (H.mT if tall else H).to(G.dtype)


def check(got, want, modelled, dtype):
    """In the Frobenius norm of the whole stack: twice the documented roundings' own error
    (the same number of roundings at other places: over 1000 entries and more their norms
    agree to a tenth), the result's rounding, and what fp32 sums of up to 2048 products of 16
    lose (2^-24 each) through 15 products: 2^-16 at worst."""
    err, own, size = ((t.double()).norm() for t in (got.double() - want, modelled.double() - want, want))
    limit = 2 * own + (torch.finfo(dtype).eps / 2 + 2.0 ** -16) * size
    assert torch.isfinite(got).all() and err <= limit, ((err / size).item(), (limit / size).item())


def gradient(shape, dtype, seed=0, std=1e-3):
    """A few strong directions and noise."""
    g = torch.Generator("cuda").manual_seed(seed)
    *L, m, n = shape
    r = max(1, min(m, n) // 8)
    x = torch.randn(*L, m, r, generator=g, device="cuda") @ torch.randn(*L, r, n, generator=g, device="cuda")
    x = x / r ** 0.5 + 0.3 * torch.randn(*L, m, n, generator=g, device="cuda")
    dY = 0.1 * torch.randn(*L, m, n, generator=g, device="cuda")
    return (std * x).to(dtype), dY.to(dtype)


SHAPES = [(1, 1), (40, 1, 37), (40, 37, 1), (300, 2, 5), (16, 64, 64), (65, 63), (2, 3, 30, 100), (128, 128),
          (129, 257), (2, 333, 127), (130, 1000), (1000, 130), (256, 256), (300, 300), (515, 519),
          (700, 100), (3, 384, 1152), (1024, 640),
          (128, 256), (129, 90), (200, 3, 17), (128, 200), (256, 64), (5, 129, 128), (257, 128)]


class TestValues:
    pytestmark = gpu

    @pytest.mark.parametrize("shape", SHAPES, ids=str)
    @pytest.mark.parametrize("dtype", ["bf16", "fp32"])
    @pytest.mark.parametrize("polynomials", ["one", "mixed"])
    def test_value_and_gradient(self, shape, dtype, polynomials):
        poly = [ONE] * 5 if polynomials == "one" else list(MIXED)
        G, dY = gradient(shape, DT[dtype])
        G.requires_grad_()
        Y = fbob.orthogonalize(G, 5, ONE if polynomials == "one" else MIXED)
        (dG,) = torch.autograd.grad(Y, G, dY)
        assert Y.dtype == dG.dtype == G.dtype and Y.is_contiguous() and dG.is_contiguous()
        alone = fbob.orthogonalize(G.detach(), 5, ONE if polynomials == "one" else MIXED)
        assert torch.equal(alone, Y)
        (X, want), (mY, mG) = exact(G, dY, poly), model(G, dY, poly)
        check(Y, X, mY, G.dtype)
        if min(shape[-2:]) == 1:
            # one singular value, which the norm fixes: dG is what is left of terms
            # that cancel along G, to be held against those
            scale = (torch.linalg.matrix_norm(dY.double()) / torch.linalg.matrix_norm(G.double()) * 500).max()
            assert (dG.double() - want).abs().max() <= torch.finfo(G.dtype).eps * scale
        else:
            check(dG, want, mG, G.dtype)

    @pytest.mark.parametrize("steps", [1, 2, 3, 7, 16])
    def test_steps(self, steps):
        poly = [(1.5, -0.5, 0.0)] * steps
        for dtype in DT.values():
            G, dY = gradient((100, 150), dtype)
            G.requires_grad_()
            Y = fbob.orthogonalize(G, steps, (1.5, -0.5, 0.0))
            (dG,) = torch.autograd.grad(Y, G, dY)
            (X, want), (mY, mG) = exact(G, dY, poly), model(G, dY, poly)
            check(Y, X, mY, dtype)
            check(dG, want, mG, dtype)

    @pytest.mark.parametrize("std", [1e-12, 1e-4, 1.0, 1e8])
    def test_sizes_of_values(self, std):
        """What is divided out leaves no trace, down to eps beside the norm, and the
        upstream gradient's own size does not matter either."""
        G, dY = gradient((96, 200), torch.float32, std=std)
        dY = dY * std
        G.requires_grad_()
        Y = fbob.orthogonalize(G)
        (dG,) = torch.autograd.grad(Y, G, dY)
        (X, want), (mY, mG) = exact(G, dY, [ONE] * 5), model(G, dY, [ONE] * 5)
        check(Y, X, mY, G.dtype)
        check(dG, want, mG, G.dtype)

    def test_matrices_of_a_stack_do_not_meet(self):
        """Zeros stay zeros, an infinity or a NaN spoils its own matrix, and the others
        are what they are alone, in value and gradient."""
        G, dY = gradient((5, 70, 90), torch.float32)
        G[1] = 0
        G[2, 3, 4] = float("nan")
        G[3, 5, 6] = float("inf")
        leaf = G.clone().requires_grad_()
        Y = fbob.orthogonalize(leaf)
        (dG,) = torch.autograd.grad(Y, leaf, dY)
        assert (Y[1] == 0).all() and torch.isfinite(dG[1]).all()
        assert Y[2].isnan().any() and Y[3].isnan().any()
        for i in (0, 4):
            one = G[i].clone().requires_grad_()
            y = fbob.orthogonalize(one)
            assert torch.equal(y, Y[i])
            assert torch.equal(torch.autograd.grad(y, one, dY[i])[0], dG[i])
        # the gradient at zero: that of a^5 x / eps
        want = dY[1].double() * 3.4445 ** 5 / 1e-7
        assert (dG[1].double() - want).abs().max() <= 1e-5 * want.abs().max()

    def test_zero_upstream_gradient(self):
        G, dY = gradient((40, 50), torch.float32)
        G.requires_grad_()
        (dG,) = torch.autograd.grad(fbob.orthogonalize(G), G, torch.zeros_like(dY))
        assert (dG == 0).all()

    @pytest.mark.parametrize("shape", [(60, 80), (150, 300)], ids=str)
    @pytest.mark.parametrize("dtype", ["bf16", "fp32"])
    @pytest.mark.parametrize("power", [-62, -57, -50, 40, 55])
    def test_gradients_of_any_size(self, shape, dtype, power):
        """The gradient is linear in what comes from above, and a power of two in it only
        moves exponents: the result's bits are the same, times it."""
        G, dY = gradient(shape, DT[dtype])
        G.requires_grad_()
        Y = fbob.orthogonalize(G)
        (want,) = torch.autograd.grad(Y, G, dY, retain_graph=True)
        (got,) = torch.autograd.grad(Y, G, dY * 2.0 ** power)
        assert torch.equal(got, want * 2.0 ** power)

    @pytest.mark.parametrize("shape", [(60, 80), (150, 300)], ids=str)
    def test_a_small_gradient_of_one_entry(self, shape):
        """The same where a step enlarges fifty times what lies in one entry."""
        G, dY = gradient(shape, torch.float32)
        G.requires_grad_()
        dY.zero_()[3, 5] = 1.0
        Y = fbob.orthogonalize(G, 5, CUBIC + ((50.0, 0.0, 0.0), (1.0, 0.0, 0.0)))
        (want,) = torch.autograd.grad(Y, G, dY, retain_graph=True)
        (got,) = torch.autograd.grad(Y, G, dY * 2.0 ** -62)
        assert torch.isfinite(want).all() and torch.equal(got, want * 2.0 ** -62)

    @pytest.mark.parametrize("shape", [(60, 80), (150, 300)], ids=str)
    def test_zeros_with_little_or_no_eps(self, shape):
        """A zero matrix stays zero for any eps above 0; without it, it is 0 / 0."""
        G = torch.zeros(shape, device="cuda")
        for eps in (1e-38, 1e-30, 1e-7):
            assert (fbob.orthogonalize(G, eps=eps) == 0).all()
        assert fbob.orthogonalize(G, eps=0.0).isnan().all()

    def test_views(self):
        """Transposed, strided, offset and expanded inputs and upstream gradients."""
        G, dY = gradient((70, 90), torch.bfloat16)
        want = fbob.orthogonalize(G)
        tall = fbob.orthogonalize(G.T.contiguous())
        check(tall.T, exact(G, None, [ONE] * 5)[0], model(G, None, [ONE] * 5)[0], G.dtype)
        assert torch.equal(fbob.orthogonalize(G.T), tall)  # (its norm is summed in another order)
        assert torch.equal(fbob.orthogonalize(G.T.contiguous().T), want)
        flat = torch.cat((G.new_zeros(1), G.flatten()))[1:].view(70, 90)  # off the 16-byte steps
        assert torch.equal(fbob.orthogonalize(flat), want)
        assert torch.equal(fbob.orthogonalize(G.expand(3, 70, 90)), want.expand(3, 70, 90))
        leaf = G.clone().requires_grad_()
        (a,) = torch.autograd.grad(fbob.orthogonalize(leaf), leaf, dY.T.contiguous().T)
        (b,) = torch.autograd.grad(fbob.orthogonalize(leaf), leaf, dY)
        assert torch.equal(a, b)
        (c,) = torch.autograd.grad(fbob.orthogonalize(leaf).sum(), leaf)  # expanded ones
        (d,) = torch.autograd.grad(fbob.orthogonalize(leaf), leaf, torch.ones_like(dY))
        assert torch.equal(c, d)

    def test_against_differences(self):
        """The gradient against the forward's differences along one direction, fp32: steps of
        2^-7 of G give a third-order term below 2^-14 times the third derivative's size
        (below 2^4 of the first's, at these singular values), the forward's error of 2^-16
        over the step 2^-9."""
        G, dY = gradient((48, 80), torch.float32, std=1.0)
        t = torch.randn(G.shape, generator=torch.Generator("cuda").manual_seed(9), device="cuda")
        t = t * (torch.linalg.matrix_norm(G) / torch.linalg.matrix_norm(t))
        G.requires_grad_()
        (dG,) = torch.autograd.grad(fbob.orthogonalize(G, 2), G, dY)
        h = 2.0 ** -7
        with torch.no_grad():
            d = (fbob.orthogonalize(G + h * t, 2).double() - fbob.orthogonalize(G - h * t, 2).double()) / (2 * h)
        a, b = (d * dY).sum(), (dG.double() * t).sum()
        scale = torch.linalg.matrix_norm(d) * torch.linalg.matrix_norm(dY.double())
        assert abs(a - b) <= 2.0 ** -9 * scale

    def test_same_bits_again_on_other_streams_and_in_graphs(self):
        G, dY = gradient((2, 200, 300), torch.bfloat16)

        def step(x):
            y = fbob.orthogonalize(x)
            return y, torch.autograd.grad(y, x, dY)[0]

        want = step(G.clone().requires_grad_())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step(G.clone().requires_grad_())
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        leaves = [torch.zeros_like(G).requires_grad_() for _ in range(2)]
        graphs, outs = [], []
        for leaf in leaves:  # two graphs, replayed in turn
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(step(leaf))
        other = gradient((2, 200, 300), torch.bfloat16, seed=3)[0]
        with torch.no_grad():
            leaves[0].copy_(G)
            leaves[1].copy_(other)
        for g in graphs:
            g.replay()
        expect = step(other.clone().requires_grad_())
        assert all(torch.equal(a, b) for a, b in zip(outs[0], want))
        assert all(torch.equal(a, b) for a, b in zip(outs[1], expect))

    def test_calls_at_once_on_two_streams(self):
        """Chains whose blocks wait for one another's tiles, two of them at a time and
        each too large for the GPU beside the other."""
        inputs = [gradient((2, 1100, 1500), d, seed=i) for i, d in enumerate(DT.values())]

        def step(x, dY):
            leaf = x.clone().requires_grad_()
            y = fbob.orthogonalize(leaf)
            return y, torch.autograd.grad(y, leaf, dY)[0]

        want = [step(*i) for i in inputs]
        streams = [torch.cuda.Stream() for _ in inputs]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = []
        for _ in range(5):
            for s, i in zip(streams, inputs):
                with torch.cuda.stream(s):
                    got.append(step(*i))
        torch.cuda.synchronize()
        for k, pair in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(pair, want[k % 2]))

    @pytest.mark.parametrize("shape", [(2, 700, 900), (8, 100, 128)], ids=str)
    @pytest.mark.parametrize("dtype", ["bf16", "fp32"])
    def test_waits_that_run_out_end_the_call(self, shape, dtype):
        """With a limit of 1 ns the first wait that is not over runs out: the call ends, its
        status word says so, and the next call with the default limit is right.  (A small
        matrix's waits can be over before the timer moves.)"""
        G, dY = gradient(shape, DT[dtype])
        coef = (ctypes.c_float * 15)(*(ONE * 5))
        o = B.Orth(*shape, B.DTYPES[DT[dtype]], 5, 1, 1e-7, ctypes.addressof(coef))
        lib, r = B.lib(), ctypes.byref(o)
        sizes = [lib.fbob_orth_workspace_size(op, r) for op in (0, 1)]
        kept, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)
        y, dG = torch.empty_like(G), torch.empty_like(G)
        stream = B._stream(G.device)
        p = lambda t: t.data_ptr()  # noqa: E731

        def forward():
            assert lib.fbob_orth_forward(r, p(G), p(y), p(kept), sizes[0], stream) == 0
            return fbob.status(kept)

        def backward():
            assert lib.fbob_orth_backward(r, p(G), p(dY), p(dG), p(kept), sizes[0], p(ws), sizes[1], stream) == 0
            return fbob.status(ws)

        assert forward() == 0 and backward() == 0
        want = y.clone(), dG.clone()
        for call in (backward, forward):
            old = fbob.set_wait_limit(1)
            try:
                st = call()
            finally:
                fbob.set_wait_limit(old)
            assert st == 5 or (st == 0 and shape[1] <= 128)
        assert forward() == 0 and backward() == 0
        assert torch.equal(y, want[0]) and torch.equal(dG, want[1])

    def test_past_31_bits_of_elements_in_a_stack(self):
        """The last matrices of 2.2e9 elements are what they are alone."""
        G = torch.zeros(530, 1024, 4096, dtype=torch.bfloat16, device="cuda")
        some, dY = gradient((2, 1024, 4096), torch.bfloat16)
        G[0], G[-1] = some[0], some[1]
        Y = fbob.orthogonalize(G)
        for i, k in ((0, 0), (-1, 1)):
            assert torch.equal(Y[i], fbob.orthogonalize(some[k]))
        assert (Y[1:-1:50] == 0).all()

    @pytest.mark.parametrize("tall", [False, True])
    def test_past_32_bits_of_elements_in_a_matrix(self, tall):
        """A block in the last corner of 4.3e9 elements of zeros: the block's own result,
        which sums the same products, among zeros."""
        p, q = 8192, (1 << 19) + 128
        block, _ = gradient((300, 200), torch.bfloat16)
        shape = (q, p) if tall else (p, q)
        G = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        G[-300:, -200:] = block
        Y = fbob.orthogonalize(G)
        want, own = exact(block, None, [ONE] * 5)[0], model(block, None, [ONE] * 5)[0]
        check(Y[-300:, -200:], want, own, torch.bfloat16)
        Y[-300:, -200:] = 0
        assert not Y.any()

    def test_many_and_long_matrices(self):
        """As many matrices, and as long a side, as one launch's grids come to."""
        for dtype in DT.values():
            G, _ = gradient((65535, 2, 3), dtype)
            Y = fbob.orthogonalize(G)
            check(Y, exact(G, None, [ONE] * 5)[0], model(G, None, [ONE] * 5)[0], dtype)
            for shape in ((1, 1 << 22), (1 << 22, 2)):
                G, dY = gradient(shape, dtype)
                G.requires_grad_()
                Y = fbob.orthogonalize(G)
                (dG,) = torch.autograd.grad(Y, G, dY)
                (X, want), (mY, mG) = exact(G, dY, [ONE] * 5), model(G, dY, [ONE] * 5)
                check(Y, X, mY, dtype)
                check(dG, want, mG, dtype)

    def test_nothing_is_written_outside(self):
        """Outputs and workspaces of the C calls between guards, at sizes off every tile."""
        for dtype in DT.values():
            G, dY = gradient((2, 67, 131), dtype)
            coef = (ctypes.c_float * 15)(*(ONE * 5))
            o = B.Orth(2, 67, 131, B.DTYPES[dtype], 5, 1, 1e-7, ctypes.addressof(coef))
            lib = B.lib()

            def guarded(n, value, dt):
                buf = torch.full((n + 2 * 256,), value, dtype=dt, device="cuda")
                return buf, buf[256:256 + n]

            sizes = [lib.fbob_orth_workspace_size(op, ctypes.byref(o)) for op in (0, 1)]
            bufs = [guarded(n, 0x5A, torch.uint8) for n in sizes]
            outs = [guarded(G.numel(), 7.0, dtype) for _ in range(2)]
            s = B._stream(G.device)
            p = lambda t: t.data_ptr()  # noqa: E731
            assert lib.fbob_orth_forward(ctypes.byref(o), p(G), p(outs[0][1]), p(bufs[0][1]), sizes[0], s) == 0
            assert lib.fbob_orth_backward(ctypes.byref(o), p(G), p(dY), p(outs[1][1]), p(bufs[0][1]), sizes[0],
                                          p(bufs[1][1]), sizes[1], s) == 0
            assert fbob.status(bufs[0][1]) == 0 and fbob.status(bufs[1][1]) == 0
            leaf = G.clone().requires_grad_()
            y = fbob.orthogonalize(leaf)
            assert torch.equal(outs[0][1].view_as(G), y)
            assert torch.equal(outs[1][1].view_as(G), torch.autograd.grad(y, leaf, dY)[0])
            for buf, view in bufs + outs:
                fill = 0x5A if buf.dtype == torch.uint8 else 7.0
                view.fill_(fill)
                assert (buf == fill).all()

    def test_refusals(self):
        G = torch.zeros(4, 5, device="cuda")
        for bad in (lambda: fbob.orthogonalize(G[0]), lambda: fbob.orthogonalize(G, 0),
                    lambda: fbob.orthogonalize(G, 17), lambda: fbob.orthogonalize(G, eps=-1.0),
                    lambda: fbob.orthogonalize(G, eps=float("nan")),
                    lambda: fbob.orthogonalize(G, 5, (ONE,) * 4),
                    lambda: fbob.orthogonalize(G, 5, (1.0, 2.0)),
                    lambda: fbob.orthogonalize(G, 5, (1.0, 2.0, float("inf")))):
            with pytest.raises(ValueError):
                bad()
        for bad in (lambda: fbob.orthogonalize(G.half()), lambda: fbob.orthogonalize(G, 2.5)):
            with pytest.raises(TypeError):
                bad()
        for bad in (lambda: fbob.orthogonalize(G.cpu()), lambda: fbob.orthogonalize(G[:0]),
                    lambda: fbob.orthogonalize(G, 5, (4.0, 0.0, 0.0))):  # runs away
            with pytest.raises(fbob.FbobError):
                bad()

    def test_second_and_forward_mode_derivatives_are_refused(self):
        G, dY = gradient((20, 30), torch.float32)
        G.requires_grad_()
        (dG,) = torch.autograd.grad(fbob.orthogonalize(G), G, dY, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(dG, G, torch.ones_like(dG))
        with torch.autograd.forward_ad.dual_level():
            t = torch.autograd.forward_ad.make_dual(G.detach(), torch.ones_like(G))
            with pytest.raises((NotImplementedError, RuntimeError)):
                fbob.orthogonalize(t)


def test_c_call_refuses_bad_arguments():
    lib = B.lib()
    good = 1 << 20
    coef = (ctypes.c_float * 48)(*(ONE * 16))
    wild = (ctypes.c_float * 48)(*((9.0, 9.0, 9.0) * 16))

    def problem(**kw):
        a = dict(L=1, m=8, n=9, dtype=1, steps=5, keep=1, eps=1e-7, coefficients=ctypes.addressof(coef))
        a.update(kw)
        return B.Orth(**a)

    def calls(o, g=good, y=good, ws=good, n=1 << 30):
        r = ctypes.byref(o)
        return (lib.fbob_orth_forward(r, g, y, ws, n, None),
                lib.fbob_orth_backward(r, g, good, y, good, 1 << 30, ws, n, None))

    for kw in (dict(L=0), dict(m=0), dict(n=-1), dict(steps=0), dict(keep=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(coefficients=None),
               dict(coefficients=ctypes.addressof(wild))):
        assert calls(problem(**kw)) == (1, 1), kw
        assert lib.fbob_orth_workspace_size(0, ctypes.byref(problem(**kw))) == 0
    for kw in (dict(dtype=2), dict(steps=17), dict(L=65536), dict(m=65537, n=65537), dict(n=(1 << 22) + 1),
               dict(L=60000, m=2048, n=2048)):
        assert calls(problem(**kw)) == (2, 2), kw
    o = problem()
    assert calls(o, g=None) == (1, 1) and calls(o, y=None) == (1, 1) and calls(o, ws=None) == (1, 1)
    assert calls(o, g=good + 2) == (1, 1) and calls(o, ws=good + 16) == (1, 1)
    assert calls(o, n=100) == (3, 3)
    assert calls(problem(keep=0))[1] == 1  # nothing was kept
    assert lib.fbob_orth_workspace_size(2, ctypes.byref(o)) == 0
    assert lib.fbob_orth_workspace_size(0, None) == 0
    r = ctypes.byref(o)
    assert lib.fbob_orth_backward(r, good, good, good, good, 100, good, 1 << 30, None) == 3
    assert lib.fbob_orth_backward(r, good, None, good, good, 1 << 30, good, 1 << 30, None) == 1
    # without a backward two buffers in turn; with one, all steps
    assert lib.fbob_orth_workspace_size(0, r) > lib.fbob_orth_workspace_size(0, ctypes.byref(problem(keep=0)))


@pytest.mark.parametrize("shape", [((1 << 32) + 5, 4, 4), (1 << 16, 1 << 16, 4, 4), (4, (1 << 32) + 4),
                                   ((1 << 32) + 4, 4), (4, 1 << 31)], ids=str)
def test_sizes_past_32_bits_are_refused(shape):
    """None is taken for what its lowest 32 bits say."""
    problem = importlib.import_module("exact_second_order_two_gb300.orthogonalize")._problem
    with pytest.raises(fbob.FbobError):
        problem(shape, torch.bfloat16, 5, (ONE,), 1e-7, False)


def test_cpu_tensors_are_refused():
    with pytest.raises(fbob.FbobError):
        fbob.orthogonalize(torch.zeros(3, 4))
