"""Norms of queries and keys with rotary positions against the definition in
64 bits (torch's autograd, once and twice): values, gradients, second derivatives,
layouts, positions, and what the call refuses."""
import ctypes

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def turned(x, inv_freq, at, interleaved, magnitude, absolute=False):
    """x [B, H, N, d] with its pairs turned, in 64 bits; ``absolute``: the sum of
    the pair's magnitudes in both places, which bounds either result."""
    r = 2 * inv_freq.numel()
    head, tail = x[..., :r], x[..., r:]
    pairs = head.unflatten(-1, (r // 2, 2)) if interleaved else head.unflatten(-1, (2, r // 2)).mT
    a, b = pairs[..., 0], pairs[..., 1]
    if absolute:
        u = v = abs(magnitude) * (a.abs() + b.abs())
    else:
        angle = at.double()[:, None, :, None] * inv_freq
        cos, sin = magnitude * angle.cos(), magnitude * angle.sin()
        u, v = a * cos - b * sin, a * sin + b * cos
    both = torch.stack((u, v), -1)
    both = both.flatten(-2) if interleaved else both.mT.flatten(-2)
    return torch.cat((both, tail.abs() if absolute else tail), -1)


def reference(x, w, dy, a, c, inv_freq, at, il, m, eps):
    """(y, dx, dw, gx, gw, gdy) by autograd in 64 bits, and what bounds the
    rounding of each: its sums with every term in magnitude."""
    x = x.detach().double().requires_grad_()
    d = x.shape[-1]
    ones = torch.ones(d, dtype=torch.float64, device=x.device)
    w = (ones if w is None else w.detach().double()).clone().requires_grad_()
    dy = dy.detach().double().requires_grad_()
    a, c = a.double(), c.double()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    y = turned(w * n, inv_freq, at, il, m)
    dx, dw = torch.autograd.grad(y, (x, w), dy, create_graph=True)
    gx, gw, gdy = torch.autograd.grad((dx, dw), (x, w, dy), (a, c))

    def big(t):
        return turned(t, inv_freq, at, il, m, absolute=True)

    with torch.no_grad():
        mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
        rs = 1 / torch.sqrt(mean(x.square()) + eps)
        W, A, C, Nn = w.abs(), a.abs(), c.abs(), n.abs()
        G = big(dy)
        H = W * G
        an, hn = mean(A * Nn), mean(H * Nn)
        t = rs * (A + Nn * an)
        u = C * G + rs * (an * H + hn * A)
        rows = (0, 1, 2)
        bound = (big(W * Nn), rs * (H + Nn * hn), (G * Nn).sum(rows),
                 rs * (u + Nn * mean(u * Nn) + Nn * mean(H * t)), (G * t).sum(rows),
                 big(W * t + C * Nn))
    return [t.detach() for t in (y, dx, dw, gx, gw, gdy)], bound


# Roundings, in units of u = 2^-24 of those bounds.  A turn is good to 12 (angle 4,
# sine and cosine 4, products and sum 4).  A sum over d <= 256 features has chains of 16
# products a lane and 5 exchanges: 22; 1/sqrt halves that and adds 4 of its own (2 ulp) and 1 for
# eps: r is good to 16.  y: r, two products and a turn, 32.  dx: h 13, <h, x> 35, r^3
# 48, four more products and sums: below 110.  gx: products of two such sums and r^3: below 220.
# Sums over rows: what is summed (60, second 120), and a chain of additions: a
# lane's rows, at most rows / 64 in these cases, and 100 across lanes, blocks and parts.
UNITS = (32, 110, 160, 220, 220, 160)


def check(got, want, bound, rows):
    for i, (g, w, b) in enumerate(zip(got, want, bound)):
        if g is None:
            continue
        units = UNITS[i] + (rows / 64 if i in (2, 4) else 0)
        step = torch.finfo(g.dtype).eps / 2
        limit = units * U * b * (1 + step) + step * w.abs()
        err = (g.detach().double() - w).abs()
        assert g.shape == w.shape and (err <= limit).all(), \
            (i, (err / limit.clamp_min(1e-300)).max().item())


CASES = [
    # B, H, Hk, N, d, turned, in, out, weights, layout, interleaved
    (1, 1, 1, 1, 2, 2, "fp32", "fp32", "fp32", "bhnd", False),
    (8, 16, 4, 1, 128, 128, "bf16", "bf16", "fp32", "fused", False),     # a token
    (2, 3, 1, 5, 64, 64, "bf16", "bf16", "bf16", "bhnd", False),
    (2, 3, 3, 5, 64, 64, "bf16", "fp32", "fp32", "bnhd", True),
    (3, 5, 2, 37, 128, 64, "fp32", "bf16", "fp32", "fused", True),
    (2, 2, 1, 65, 96, 32, "fp32", "fp32", "bf16", "bnhd", True),          # 6 of 8 lanes
    (1, 4, 2, 9, 40, 40, "bf16", "fp32", "fp32", "bhnd", False),          # runs of 4
    (2, 2, 3, 3, 13, 6, "fp32", "bf16", "fp32", "bhnd", True),            # odd width
    (2, 2, 1, 3, 37, 36, "bf16", "bf16", "fp32", "fused", False),
    (1, 2, 2, 4, 16, 0, "bf16", "bf16", "fp32", "bhnd", False),           # nothing turned
    (1, 2, 1, 7, 256, 256, "fp32", "fp32", "fp32", "bhnd", False),        # the widest
    (1, 2, 1, 7, 255, 254, "fp32", "fp32", "fp32", "bhnd", False),
    (1, 3, 1, 6, 1, 0, "fp32", "fp32", "fp32", "bhnd", False),
    (1, 2, 1, 4, 64, 64, "bf16", "bf16", None, "bhnd", False),            # no weights
    (2, 40, 8, 1200, 64, 64, "bf16", "bf16", "fp32", "fused", False),     # blocks that stay
    (2, 8, 8, 1500, 128, 128, "fp32", "bf16", "fp32", "bnhd", True),
]


def make(case, seed=0):
    b, h, hk, n, d, r, tin, tout, tw, layout, il = case
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if layout == "fused":
        base = rand(b, n, h + 2 * hk, d).to(DT[tin]).transpose(1, 2)
        xs = [base[:, :h], base[:, h:h + hk]]
    elif layout == "bnhd":
        xs = [rand(b, n, i, d).to(DT[tin]).transpose(1, 2) for i in (h, hk)]
    else:
        xs = [rand(b, i, n, d).to(DT[tin]) for i in (h, hk)]
    ws = [None if tw is None else (1 + 0.3 * rand(d)).to(DT[tw]) for _ in xs]
    f = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64, device="cuda") * 2 / max(r, 1))
    dys = [rand(*x.shape).to(DT[tout]) for x in xs]
    cots = [rand(*x.shape).to(DT[tin]) for x in xs]
    cws = [rand(d) if w is None else rand(d).to(w.dtype) for w in ws]
    return xs, ws, f, dys, cots, cws


class TestValues:
    pytestmark = gpu

    @pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
    @pytest.mark.parametrize("far", [False, True])
    def test_value_and_both_derivatives(self, case, far):
        xs, ws, f, dys, cots, cws = make(case)
        b, h, hk, n, d, r, tin, tout, tw, layout, il = case
        if far:  # a place of its own for each sequence; f in few bits, so that 64 bits hold the angle
            at = torch.randint(0, 1 << 20, (b, n), device="cuda")
            pos = at
        else:
            at, pos = torch.arange(n, device="cuda").expand(b, n), None
        m, eps = 1.25, 1e-3
        leaves = [x.requires_grad_() for x in xs] + [w.requires_grad_() for w in ws if w is not None]
        y = fbob.qk_norm_rotary(*xs, *ws, f, pos, eps=eps, interleaved=il, magnitude=m, dtype=DT[tout])
        dys = [t.requires_grad_() for t in dys]
        first = torch.autograd.grad(y, leaves, dys, create_graph=True)
        second = torch.autograd.grad(first, leaves + dys, cots + (cws if tw else []))
        plain = torch.autograd.grad(fbob.qk_norm_rotary(
            *xs, *ws, f, pos, eps=eps, interleaved=il, magnitude=m, dtype=DT[tout]), leaves, dys)
        assert all(torch.equal(s, t) for s, t in zip(first, plain))
        for i in (0, 1):
            c = cws[i] if tw else torch.zeros(d, device="cuda")
            want, bound = reference(xs[i], ws[i], dys[i], cots[i], c, f, at, il, m, eps)
            got = (y[i], first[i], first[2 + i] if tw else None, second[i],
                   second[2 + i] if tw else None, second[-2 + i])
            assert y[i].is_contiguous() and y[i].dtype == DT[tout]
            assert first[i].dtype == xs[i].dtype and second[i].dtype == xs[i].dtype
            check(got, want, bound, xs[i][..., 0].numel())

    def test_against_differences(self):
        """The gradient against the forward's own differences, in fp32, along one
        direction: steps h = 2^-6 of the values, whose third-order term is at most
        15 h^2 / 6 < 2^-10.6 of them (the third derivative of x / |x| along a t as long as
        x), and rounding below 2^-13 of the sums."""
        xs, ws, f, dys, cots, cws = make(CASES[11])
        leaves = xs + ws
        for t in leaves:
            t.requires_grad_()
        call = lambda v: fbob.qk_norm_rotary(*v, f, eps=1e-3)  # noqa: E731
        grads = torch.autograd.grad(call(leaves), leaves, dys)
        g = torch.Generator("cuda").manual_seed(5)
        t = [torch.randn(v.shape, generator=g, device="cuda") for v in leaves]
        h = 2.0 ** -6
        with torch.no_grad():
            up, down = (call([v + s * h * e for v, e in zip(leaves, t)]) for s in (1, -1))
        moved = sum(((a.double() - b.double()) * dy).sum() for a, b, dy in zip(up, down, dys)) / (2 * h)
        along = sum((a.double() * b).sum() for a, b in zip(grads, t))
        scale = sum((a.double() * b).abs().sum() for a, b in zip(grads, t))
        scale += sum((a * dy).abs().double().sum() for a, dy in zip(up, dys))
        assert abs(moved - along) <= 2.0 ** -10 * scale

    def test_parts_of_the_derivatives(self):
        """Upstream gradients and cotangents that are missing: what is left is what
        zeros give."""
        xs, ws, f, dys, cots, cws = make(CASES[4])
        for t in xs + ws + dys:
            t.requires_grad_()
        y = fbob.qk_norm_rotary(*xs, *ws, f, dtype=torch.bfloat16)
        all_ = torch.autograd.grad(y, xs + ws, dys, retain_graph=True)
        for i in (0, 1):
            part = torch.autograd.grad(y[i], [xs[i], ws[i]], dys[i], retain_graph=True)
            assert torch.equal(part[0], all_[i]) and torch.equal(part[1], all_[2 + i])
        (only,) = torch.autograd.grad(y, xs[0], dys, retain_graph=True)
        assert torch.equal(only, all_[0])
        first = torch.autograd.grad(y, xs + ws, dys, create_graph=True)
        zero = [torch.zeros_like(t) for t in first]
        for k, cot in enumerate(cots + cws):
            given = list(zero)
            given[k] = cot
            want = torch.autograd.grad(first, xs + ws + dys, given, retain_graph=True)
            got = torch.autograd.grad(first[k], xs + ws + dys, cot, retain_graph=True, allow_unused=True)
            for a, b in zip(got, want):
                assert (b == 0).all() if a is None else torch.equal(a, b)

    def test_broken_strides_and_offsets(self):
        """Addresses and strides off the 16-byte steps, a broadcast head, a feature
        stride other than 1, strided weights: the values of a copy, up to
        the order of the sums."""
        f = 100.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        w = torch.rand(128, device="cuda")[::2] + 0.5
        flat = torch.randn(2 * 5 * 3 * 70 + 1, device="cuda").bfloat16()
        for x in (flat[1:].view(2, 5, 3, 70)[..., :64], flat[:-1].view(2, 5, 3, 70)[..., 3:67],
                  flat[:2 * 3 * 64].view(2, 1, 3, 64).expand(2, 4, 3, 64),
                  flat[:2 * 5 * 64 * 3].view(2, 5, 64, 3).transpose(2, 3)):
            at = torch.arange(x.shape[2], device="cuda").expand(2, -1)
            leaf = x.detach().requires_grad_()
            y = fbob.qk_norm_rotary(leaf, leaf[:, :1], w, w, f)[0]
            dy = torch.ones_like(y)[..., :1].expand_as(y)  # feature stride 0
            (dx,) = torch.autograd.grad(y, leaf, dy)
            z = torch.zeros_like(x)
            want, bound = reference(x, w, dy, z, z[0, 0, 0], f, at, False, 1.0, 1e-6)
            check((y, dx, None, None, None, None), want, bound, 1)

    def test_graph_capture_and_other_stream(self):
        xs, ws, f, dys, cots, cws = make(CASES[4])
        leaves = [t.detach().requires_grad_() for t in xs + ws]

        def step(leaves):
            y = fbob.qk_norm_rotary(*leaves, f)
            return y + torch.autograd.grad(y, leaves, [t.float() for t in dys])

        want = [t.detach() for t in step([t.detach().requires_grad_() for t in xs + ws])]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step([t.detach().requires_grad_() for t in xs + ws])
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(leaves)
        other = [torch.randn_like(t) for t in leaves]
        with torch.no_grad():
            for t, o in zip(leaves, other):
                t.copy_(o)
        graph.replay()
        want = step([t.detach().requires_grad_() for t in other])
        assert all(torch.equal(a, b) for a, b in zip(out, want))

    def test_rows_of_zeros_infinities_and_nan(self):
        """A row of zeros stays zero; a row with an infinity or a NaN spoils itself and
        the weights' gradient, no other row."""
        x = torch.randn(1, 2, 6, 64, device="cuda")
        x[0, 0, 1] = 0
        x[0, 0, 2, 5], x[0, 1, 3, 7] = float("inf"), float("nan")
        w = torch.rand(64, device="cuda") + 0.5
        leaf = x.clone().requires_grad_()
        wl = w.clone().requires_grad_()
        y, _ = fbob.qk_norm_rotary(leaf, leaf[:, :1].detach(), wl, w)
        dx, dw = torch.autograd.grad(y, (leaf, wl), torch.ones_like(y))
        bad = torch.zeros(1, 2, 6, dtype=torch.bool, device="cuda")
        bad[0, 0, 2] = bad[0, 1, 3] = True
        assert (y[0, 0, 1] == 0).all()
        for t in (y, dx):
            assert torch.isfinite(t[~bad]).all() and t[bad].isnan().any(-1).all()
        assert dw.isnan().any()

    @pytest.mark.parametrize("d", [37, 64])
    def test_without_eps_lanes_without_a_row_add_nothing(self, d):
        """eps = 0, and fewer rows than a block's lanes hold: gradients are those with an
        eps far below the rows' squares."""
        g = torch.Generator("cuda").manual_seed(5)
        leaves = [torch.randn(s, generator=g, device="cuda").requires_grad_()
                  for s in ((1, 2, 3, d), (1, 1, 3, d), (d,), (d,))]
        got = []
        for eps in (0.0, 1e-30):
            y = fbob.qk_norm_rotary(*leaves, eps=eps)
            first = torch.autograd.grad(y, leaves, [torch.ones_like(t) for t in y], create_graph=True)
            got.append([*first, *torch.autograd.grad(first, leaves, [torch.ones_like(t) for t in first])])
        for a, b in zip(*got):
            assert torch.isfinite(a).all() and torch.equal(a, b)

    def test_past_32_bit_offsets(self):
        """Two batches 2^32 + 64 elements apart."""
        buf = torch.empty((1 << 32) + 64 + 4 * 64 * 3, dtype=torch.bfloat16, device="cuda")
        x = buf.as_strided((2, 4, 3, 64), ((1 << 32) + 64, 192, 64, 1))
        x.copy_(torch.randn(2, 4, 3, 64, device="cuda"))
        f = 100.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        w = torch.rand(64, device="cuda")
        y, yk = fbob.qk_norm_rotary(x, x, w, w, f)
        want, _ = fbob.qk_norm_rotary(x.contiguous(), x[:, :1].contiguous(), w, w, f)
        assert torch.equal(y, want) and torch.equal(yk, want)

    def test_nothing_is_written_outside(self):
        xs, ws, f, dys, cots, cws = make(CASES[2])
        q = xs[0].contiguous()
        buf = torch.full((2 * 3 * 5 * 72 + 128,), 7.0, device="cuda", dtype=torch.bfloat16)
        y = buf[64:64 + 2 * 3 * 5 * 72].view(2, 3, 5, 72)[..., :64]
        s = B.QkNorm(2, 5, 64, 64, 0, 0, 0, 0, 1e-6, 1.0, 0, 0)
        three = ctypes.c_longlong * 3
        side = B.NormSide(H=3, x=q.data_ptr(), weight=ws[0].data_ptr(), y=y.data_ptr(),
                          x_strides=three(*q.stride()[:3]), y_strides=three(*y.stride()[:3]))
        assert B.lib().fbob_qk_norm_forward(ctypes.byref(s), ctypes.byref(side), None, f.data_ptr(),
                                            None, B._stream(q.device)) == 0
        assert torch.equal(y, fbob.qk_norm_rotary(q, q, ws[0], ws[0], f)[0])
        y.fill_(7.0)
        assert (buf == 7.0).all()

    def test_changed_positions_are_noticed(self):
        xs, ws, f, dys, cots, cws = make(CASES[4])
        pos = torch.arange(37, device="cuda")
        leaf = xs[0].detach().requires_grad_()
        y, _ = fbob.qk_norm_rotary(leaf, xs[1], *ws, f, pos)
        pos.add_(1)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y, leaf, torch.ones_like(y))

    def test_refusals(self):
        (q, k), (wq, wk), f, *_ = make(CASES[2])
        for bad in (lambda: fbob.qk_norm_rotary(q[0], k), lambda: fbob.qk_norm_rotary(q, k[0]),
                    lambda: fbob.qk_norm_rotary(q, k.float()),
                    lambda: fbob.qk_norm_rotary(q, k[:, :, 1:]),
                    lambda: fbob.qk_norm_rotary(q, k[..., :32]),
                    lambda: fbob.qk_norm_rotary(q, k, wq[:32], wk),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk.float()),
                    lambda: fbob.qk_norm_rotary(q, k, wq.cpu(), wk),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, f.float()),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, None, 3),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, f, torch.zeros(6, dtype=torch.int64,
                                                                             device="cuda")),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, f, eps=-1.0),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, f, eps=float("nan")),
                    lambda: fbob.qk_norm_rotary(q, k, wq, wk, f, magnitude=float("inf"))):
            with pytest.raises(ValueError):
                bad()
        for bad in (lambda: fbob.qk_norm_rotary(q.half(), k.half()),
                    lambda: fbob.qk_norm_rotary(q, k, wq.half(), None),
                    lambda: fbob.qk_norm_rotary(q, k, dtype=torch.float16)):
            with pytest.raises(TypeError):
                bad()
        for bad in (lambda: fbob.qk_norm_rotary(q.cpu(), k), lambda: fbob.qk_norm_rotary(q[:0], k[:0]),
                    lambda: fbob.qk_norm_rotary(*(torch.zeros(1, 1, 1, 257, device="cuda"),) * 2)):
            with pytest.raises(fbob.FbobError):
                bad()

    def test_numbers_past_their_c_types_are_refused(self):
        (q, k), (wq, wk), f, *_ = make(CASES[2])
        for how in (dict(eps=1e39), dict(magnitude=1e39), dict(magnitude=-1e39)):
            with pytest.raises(ValueError):
                fbob.qk_norm_rotary(q, k, wq, wk, f, **how)
        one = torch.zeros(1, 1, 1, 1, device="cuda")
        long, many = one.expand(1, 1, 1 << 31, 1), one.expand(1, 1 << 31, 1, 1)
        for q, k in ((long, long), (many, one), (one, many), (many.transpose(0, 1),) * 2):
            with pytest.raises(fbob.FbobError):
                fbob.qk_norm_rotary(q, k)

    def test_third_and_forward_mode_derivatives_are_refused(self):
        (q, k), (wq, wk), f, (dy, _), *_ = make(CASES[2])
        q.requires_grad_()
        (first,) = torch.autograd.grad(fbob.qk_norm_rotary(q, k, wq, wk, f)[0], q, dy, create_graph=True)
        (second,) = torch.autograd.grad(first, q, torch.ones_like(q), create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(second, q, torch.ones_like(q))
        with torch.autograd.forward_ad.dual_level():
            t = torch.autograd.forward_ad.make_dual(q.detach(), torch.ones_like(q))
            with pytest.raises((NotImplementedError, RuntimeError)):
                fbob.qk_norm_rotary(t, k, wq, wk, f)


def test_c_call_refuses_bad_arguments():
    lib = B.lib()
    good = 1 << 20

    def call(op="forward", side=None, k=None, f=good, p=None, ws=good, n=1 << 22, **kw):
        a = dict(B=1, N=3, d=64, rotary_dim=64, interleaved=0, in_dtype=0, out_dtype=0,
                 weight_dtype=1, eps=1e-6, magnitude=1.0)
        a.update(kw)
        one = dict(H=2, x=good, weight=good, dy=good, y=good, dweight=good, ddy=good)
        sides = [None if t is None else B.NormSide(**{**one, **t}) for t in (side or {}, k)]
        args = [ctypes.byref(B.QkNorm(**a))] + [None if t is None else ctypes.byref(t) for t in sides]
        tail = [] if op == "forward" else [ws, n]
        return getattr(lib, "fbob_qk_norm_" + op)(*args, f, p, *tail, None)

    for op in ("forward", "backward", "bob"):
        for kw in (dict(B=0), dict(N=-1), dict(d=0), dict(rotary_dim=3), dict(rotary_dim=66),
                   dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(magnitude=float("nan")), dict(side=dict(H=0)), dict(side=dict(x=None)),
                   dict(side=dict(y=None)), dict(side=dict(x=good + 1)), dict(side=dict(y=good + 1)),
                   dict(side=dict(weight=good + 2)), dict(k=dict(x=None)), dict(f=None),
                   dict(f=good + 4), dict(p=good + 4)):
            assert call(op, **kw) == 1, (op, kw)
        for kw in (dict(in_dtype=2), dict(out_dtype=-1), dict(weight_dtype=7), dict(d=257, rotary_dim=0),
                   dict(side=dict(H=65536)), dict(side=dict(H=40000), k=dict(H=40000)),
                   dict(B=1 << 20, N=1 << 20)):
            assert call(op, **kw) == 2, (op, kw)
    for op in ("backward", "bob"):
        assert call(op, side=dict(dy=None)) == 1 and call(op, side=dict(dy=good + 1)) == 1
        assert call(op, side=dict(dweight=good + 2)) == 1
        assert call(op, ws=None) == 1 and call(op, ws=good + 8) == 1
        assert call(op, n=100) == 3
    assert call("bob", side=dict(ddy=None)) == 1 and call("bob", side=dict(a=good + 1)) == 1
    assert call("bob", side=dict(c=good + 2)) == 1
    assert lib.fbob_qk_norm_workspace_size(None) == 0
    assert lib.fbob_qk_norm_forward(None, None, None, None, None, None) == 1
