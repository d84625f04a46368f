"""Differential attention against its formulas in 64 bits: forward, first and
second derivatives, layouts, masks and refusals.

The bounds are elementwise and follow the roundings, each by at most half a
step h of the tensors' type (2^-8 for bf16; for fp32 tensors nothing is held
in fewer bits).  Probabilities, W = P1 - lam P2 and dS are operands of bf16
products, O2 is stored and read back for D (O with what its rounding left
off, in two bf16 numbers: h^2), results round once:
  |dO_err|  <= h (P1 |V| + lam P2 |V|) + h |O|
  |dV_err|  <= h |W|^T |dO| + h |dV|
  |dS_err|  <= h |dS| + P |D_err|, |D2_err| <= h |dO|.|O2|,
               |D1_err| <= h |dO|.(lam |O2| + h |O|)
  |dQ_err|  <= c |dS_err| |K| + h |dQ|, dK likewise
plus 32-bit arithmetic: sums of n terms are off by at most n u times the sum of
their magnitudes (u = 2^-24), scores by (d + 4) u c |q|.|k| and the exponential
by 4 u, which every term with a P or a dP carries.
"""
import ctypes
import math

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B

U = 2.0 ** -24


def oracle(q, k, v, lam, do, causal, scale):
    """Values and error bounds, all float64, on the inputs' device."""
    h = 0.0 if q.dtype == torch.float32 else torch.finfo(q.dtype).eps / 2
    step = torch.finfo(q.dtype).eps / 2
    lam_step = torch.finfo(lam.dtype).eps / 2
    q, k, v, do = (t.detach().double() for t in (q, k, v, do))
    Bt, H2, N, d = q.shape
    H, Hk, dv = H2 // 2, v.shape[1], v.shape[3]
    G = H // Hk
    shape = lam.shape
    w = lam.detach().double()
    w = (w[:, None] if w.dim() == 1 else w).expand(Bt, H, N)[..., None]
    kk = k.view(Bt, Hk, 2, N, d).repeat_interleave(G, 1)
    qq = q.view(Bt, H, 2, N, d)
    vv = v.repeat_interleave(G, 1)
    hidden = torch.ones(N, N, dtype=torch.bool, device=q.device).triu(1) if causal else None

    S = scale * qq @ kk.transpose(-1, -2)
    if causal:
        S = S.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(S, -1)
    P = torch.exp(S - lse[..., None])
    O12 = P @ vv[:, :, None]
    O1, O2 = O12[:, :, 0], O12[:, :, 1]
    O = O1 - w * O2
    dP = do @ vv.transpose(-1, -2)
    D = (do[:, :, None] * O12).sum(-1, keepdim=True)
    W = P[:, :, 0] - w * P[:, :, 1]
    coef = torch.stack((torch.ones_like(w), -w), 2)
    dS = coef * P * (dP[:, :, None] - D)
    dQ = scale * dS @ kk
    dK = (scale * dS.transpose(-1, -2) @ qq).view(Bt, Hk, G, 2, N, d).sum(2)
    dV = (W.transpose(-1, -2) @ do).view(Bt, Hk, G, N, dv).sum(2)
    dl = -D[:, :, 1, :, 0]

    def to_lam(x):
        return x.sum() if len(shape) == 0 else x.sum((0, 2)) if len(shape) == 1 else x

    # magnitudes for the 32-bit terms
    smax = (scale * qq.abs() @ kk.abs().transpose(-1, -2)).amax()
    r = (2 * (d + 4) * smax + 8 + N + dv) * U * 2   # relative error of P, and of sums over keys
    aw, av, ado = w.abs(), vv.abs(), do.abs()
    aP = P
    PV = aP @ av[:, :, None]
    mix = PV[:, :, 0] + aw * PV[:, :, 1]
    eO2 = (h + r) * PV[:, :, 1] + step * O2.abs()
    eO = (h + r) * mix
    eO = eO + step * (O.abs() + eO)
    keep = step * step if h else step  # bf16 keeps what the roundings of O and O2 left off
    eD2 = (ado * (keep * O2.abs() + (h + r) * PV[:, :, 1])).sum(-1, keepdim=True) \
        + dv * U * (ado * O2.abs()).sum(-1, keepdim=True)
    eD1 = (ado * (step * step * O.abs() + keep * aw * O2.abs() + (h + r) * (mix + aw * PV[:, :, 1]))).sum(
        -1, keepdim=True) + dv * U * (ado * (O.abs() + aw * O2.abs())).sum(-1, keepdim=True)
    adP = ado @ av.transpose(-1, -2)
    eD = torch.stack((eD1, eD2), 2)
    edS = h * dS.abs() + coef.abs() * aP * (eD + r * (adP[:, :, None] + D.abs()) +
                                            dv * U * adP[:, :, None])
    m = (r + h * 0)
    eQ = scale * (edS @ kk.abs() + m * (dS.abs() @ kk.abs()))
    eQ = eQ + step * (dQ.abs() + eQ)
    eK = scale * (edS.transpose(-1, -2) @ qq.abs() + G * m * (dS.abs().transpose(-1, -2) @ qq.abs()))
    eK = eK.view(Bt, Hk, G, 2, N, d).sum(2)
    eK = eK + step * (dK.abs() + eK)
    aW = aP[:, :, 0] + aw * aP[:, :, 1]
    eV = ((h * W.abs() + 2 * G * r * aW).transpose(-1, -2) @ ado).view(Bt, Hk, G, N, dv).sum(2)
    eV = eV + step * (dV.abs() + eV)
    el = eD2[..., 0] + (U * Bt * H * N * D[:, :, 1, :, 0].abs() if len(shape) < 3 else 0)
    el = to_lam(el)
    el = el + lam_step * (to_lam(dl).abs() + el)
    vals = dict(o=O, o2=O2, lse=lse.view(Bt, H2, N), dq=dQ.view(Bt, H2, N, d),
                dk=dK.reshape(Bt, 2 * Hk, N, d), dv=dV, dlam=to_lam(dl))
    elog = (r + (d + 4) * smax * U + 4 * U * (1 + lse.abs())).view(Bt, H2, N)
    errs = dict(o=eO, o2=eO2 + step * eO2, lse=elog, dq=eQ.view(Bt, H2, N, d),
                dk=eK.reshape(Bt, 2 * Hk, N, d), dv=eV, dlam=el)
    return vals, errs


def inputs(Bt, H, Hk, N, d, dv, dtype, lam, seed=0, device="cuda", spread=1.0):
    g = torch.Generator(device).manual_seed(seed)

    def r(*s, std=1.0):
        return (torch.randn(s, generator=g, device=device) * std).to(dtype)

    shape = {"one": (), "head": (H,), "row": (Bt, H, N)}[lam[0]]
    w = (torch.rand(shape, generator=g, device=device) * 1.5 - 0.3).to(lam[1])
    return (r(Bt, 2 * H, N, d, std=spread), r(Bt, 2 * Hk, N, d, std=spread), r(Bt, Hk, N, dv), w,
            r(Bt, H, N, dv, std=0.3))


def check(got, vals, errs, names):
    for name in names:
        e = (got[name].detach().double() - vals[name]).abs()
        bad = e > errs[name]
        assert not bad.any(), (name, (e / errs[name].clamp_min(1e-300)).max().item(),
                               int(bad.sum()))


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    # B, H, Hk, N, d, dv, dtype, causal, lam
    (1, 1, 1, 1, 64, 128, BF, True, ("one", BF)),
    (1, 2, 2, 2, 64, 64, BF, False, ("head", BF)),
    (2, 2, 1, 37, 64, 128, BF, True, ("head", F32)),
    (1, 2, 2, 127, 64, 128, BF, True, ("row", BF)),
    (1, 1, 1, 128, 64, 64, BF, True, ("one", F32)),
    (2, 4, 2, 129, 64, 128, BF, False, ("head", BF)),
    (1, 4, 1, 300, 64, 64, BF, True, ("row", F32)),
    (3, 3, 3, 257, 64, 128, BF, False, ("one", BF)),
    (1, 2, 1, 641, 64, 128, BF, True, ("head", BF)),
    # dK and dV in parts: over the heads of a group, and over the queries, with
    # parts that a causal mask leaves empty
    (1, 8, 2, 1000, 64, 64, BF, False, ("one", BF)),
    (1, 1, 1, 2050, 64, 128, BF, True, ("head", F32)),
    (1, 2, 1, 1500, 128, 128, BF, True, ("head", BF)),
    (1, 2, 2, 70, 40, 80, BF, True, ("head", BF)),
    (1, 1, 1, 1, 128, 128, BF, True, ("one", BF)),
    (1, 1, 1, 65, 128, 128, BF, False, ("row", BF)),
    (2, 4, 2, 129, 128, 64, BF, True, ("head", BF)),
    (1, 4, 1, 300, 128, 128, BF, False, ("head", F32)),
    (1, 2, 2, 641, 128, 128, BF, True, ("row", BF)),
    (1, 2, 1, 640, 128, 64, BF, False, ("one", F32)),
    (1, 2, 2, 90, 96, 128, BF, True, ("head", BF)),
    # rows narrower than the kernels' widths, on one and on both sides, cut and whole
    (2, 2, 1, 300, 40, 40, BF, True, ("row", BF)),
    (1, 4, 2, 200, 24, 128, BF, False, ("head", F32)),
    (1, 2, 2, 257, 8, 8, BF, True, ("one", BF)),
    (1, 8, 2, 500, 128, 72, BF, True, ("head", BF)),
    (1, 1, 1, 130, 104, 120, BF, False, ("row", F32)),
    (1, 4, 1, 420, 80, 56, BF, True, ("head", BF)),
    # and sizes that run on CUDA cores
    (1, 2, 1, 90, 60, 100, BF, True, ("head", BF)),
    (1, 2, 2, 33, 7, 33, BF, False, ("one", F32)),
    (1, 1, 1, 1, 64, 64, F32, True, ("one", F32)),
    (2, 2, 1, 65, 64, 128, F32, True, ("head", F32)),
    (1, 2, 2, 200, 32, 64, F32, False, ("row", F32)),
    (1, 2, 1, 63, 1, 3, F32, True, ("head", F32)),
    (1, 1, 1, 130, 128, 128, F32, True, ("one", BF)),
    (1, 2, 2, 77, 70, 50, F32, False, ("head", F32)),
    # dK and dV in parts, some of them empty
    (1, 4, 1, 300, 40, 72, F32, True, ("one", F32)),
    (1, 1, 1, 700, 16, 20, F32, True, ("head", F32)),
    (2, 2, 1, 260, 10, 3, BF, False, ("head", BF)),
]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
class TestOnGpu:
    @pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
    def test_forward_and_backward(self, case):
        Bt, H, Hk, N, d, dv, dtype, causal, lam = case
        q, k, v, w, do = inputs(Bt, H, Hk, N, d, dv, dtype, lam)
        scale = 0.7 / math.sqrt(d)
        vals, errs = oracle(q, k, v, w, do, causal, scale)
        o, rest, lse = fbob.diff_forward(q, k, v, w, causal, scale)
        check(dict(o=o, o2=rest[..., 0, :], lse=lse), vals, errs, ("o", "o2", "lse"))
        grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, causal, scale)
        check(dict(zip(("dq", "dk", "dv", "dlam"), grads)), vals, errs, ("dq", "dk", "dv", "dlam"))
        # through autograd, from strided views of the same values
        leaf = [t.clone().requires_grad_() for t in (q, k, v, w)]
        qs = leaf[0].transpose(1, 2).contiguous().transpose(1, 2)
        out = fbob.diff_attention(qs, *leaf[1:], causal=causal, scale=scale)
        assert torch.equal(out, o)
        again = torch.autograd.grad(out, leaf, do)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
        with torch.no_grad():
            assert torch.equal(fbob.diff_attention(*leaf, causal=causal, scale=scale), o)

    def test_cuda_core_family_on_the_tensor_core_sizes(self):
        q, k, v, w, do = inputs(1, 2, 1, 150, 64, 128, BF, ("head", BF), seed=3)
        vals, errs = oracle(q, k, v, w, do, True, 0.125)
        old = fbob.force_path(fbob.PATH_SIMT)
        try:
            o, rest, lse = fbob.diff_forward(q, k, v, w, True)
            grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True)
        finally:
            fbob.force_path(old)
        check(dict(zip(("o", "o2", "lse", "dq", "dk", "dv", "dlam"), (o, rest[..., 0, :], lse, *grads))), vals,
              errs, ("o", "o2", "lse", "dq", "dk", "dv", "dlam"))

    @pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
    def test_peaked_rows(self, dtype, d):
        """Scores of tens: probabilities near 0 and 1, maxima that move late."""
        q, k, v, w, do = inputs(1, 2, 2, 300, d, 128, dtype, ("head", dtype), seed=4, spread=4.0)
        k = k * torch.linspace(0.1, 1.0, 300, device="cuda").to(dtype)[:, None]
        vals, errs = oracle(q, k, v, w, do, True, 0.125)
        o, rest, lse = fbob.diff_forward(q, k, v, w, True, 0.125)
        check(dict(o=o, o2=rest[..., 0, :], lse=lse), vals, errs, ("o", "o2", "lse"))
        grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, 0.125)
        check(dict(zip(("dq", "dk", "dv", "dlam"), grads)), vals, errs, ("dq", "dk", "dv", "dlam"))

    @pytest.mark.parametrize("dtype", [BF, F32])
    def test_equal_maps_cancel(self, dtype):
        """Q1 = Q2, K1 = K2 and lam = 1: O = 0 up to rounding, dV = 0."""
        q, k, v, w, do = inputs(1, 2, 2, 200, 64, 128, dtype, ("head", dtype), seed=5)
        q[:, 1::2], k[:, 1::2] = q[:, 0::2], k[:, 0::2]
        w.fill_(1.0)
        vals, errs = oracle(q, k, v, w, do, True, 0.125)
        o, rest, lse = fbob.diff_forward(q, k, v, w, True, 0.125)
        check(dict(o=o), vals, errs, ("o",))
        grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, 0.125)
        check(dict(zip(("dq", "dk", "dv", "dlam"), grads)), vals, errs, ("dq", "dk", "dv", "dlam"))

    @pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 128), (BF, 128, 128), (F32, 64, 64)])
    def test_same_bits_every_time_and_on_two_streams(self, dtype, d, dv):
        q, k, v, w, do = inputs(2, 4, 1, 500, d, dv, dtype, ("head", dtype), seed=6)

        def both():
            o, rest, lse = fbob.diff_forward(q, k, v, w, True)
            return (o, rest, lse) + fbob.diff_backward(q, k, v, w, o, rest, lse, do, True)

        first = both()
        streams = [torch.cuda.Stream() for _ in range(2)]
        results = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                results.append(both())
        torch.cuda.synchronize()
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(first, r))

    @pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 128), (BF, 64, 64), (BF, 128, 128), (BF, 128, 64),
                                            (BF, 40, 72), (BF, 104, 24), (BF, 20, 12), (F32, 64, 64)])
    def test_outputs_fully_written_and_guards_intact(self, dtype, d, dv):
        """NaN-filled outputs and workspace with guards behind them, through the
        C calls: everything inside is written, nothing outside."""
        q, k, v, w, do = inputs(1, 8, 1, 200, d, dv, dtype, ("head", dtype), seed=7)
        from exact_second_order_two_gb300.diff_attention import _shape

        shp = _shape(q, k, v, w, True, None)
        lib, st = B.lib(), B._stream(q.device)

        def guarded(shape, dt):
            n = math.prod(shape)
            buf = torch.full((n + 4096,), float("nan"), dtype=dt, device="cuda")
            return buf, buf[:n].view(shape)

        def workspace(op):
            n = lib.fbob_diff_workspace_size(op, ctypes.byref(shp))
            buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
            return buf, n

        o = guarded((1, 8, 200, dv), dtype)
        rest = guarded((1, 8, 200, 3 if dtype == BF else 1, dv), dtype)
        lse = guarded((1, 16, 200), F32)
        fws, fn = workspace(0)
        args = [t.data_ptr() for t in (q, k, v, w)]
        assert lib.fbob_diff_forward(ctypes.byref(shp), *args, o[1].data_ptr(), rest[1].data_ptr(),
                                     lse[1].data_ptr(), fws.data_ptr(), fn, st) == 0
        grads = [guarded(t.shape, t.dtype) for t in (q, k, v, w)]
        bws, bn = workspace(1)
        assert lib.fbob_diff_backward(ctypes.byref(shp), *args, o[1].data_ptr(), rest[1].data_ptr(),
                                      lse[1].data_ptr(), do.data_ptr(),
                                      *(g[1].data_ptr() for g in grads), bws.data_ptr(), bn, st) == 0
        torch.cuda.synchronize()
        for buf, view in [o, rest, lse] + grads:
            assert torch.isfinite(view.float()).all()
            assert torch.isnan(buf[view.numel():].float()).all()
        assert (fws[fn:] == 0xFF).all() and (bws[bn:] == 0xFF).all()
        assert fbob.status(fws) == 0 and fbob.status(bws) == 0
        vals, errs = oracle(q, k, v, w, do, True, d**-0.5)
        check(dict(zip(("dq", "dk", "dv", "dlam"), (g[1] for g in grads))), vals, errs,
              ("dq", "dk", "dv", "dlam"))
        # a workspace one byte short is refused
        assert lib.fbob_diff_backward(ctypes.byref(shp), *args, o[1].data_ptr(), rest[1].data_ptr(),
                                      lse[1].data_ptr(), do.data_ptr(),
                                      *(g[1].data_ptr() for g in grads), bws.data_ptr(), bn - 1,
                                      st) == 3

    @pytest.mark.parametrize("lam", ["one", "head", "row"])
    @pytest.mark.parametrize("d,dv,Hk", [(64, 128, 2), (64, 64, 1), (24, 16, 2)])
    def test_second_derivative(self, lam, d, dv, Hk):
        """fp32: the derivative of <gQ,dQ> + <gK,dK> + <gV,dV> + <g,dlam> in
        q, k, v, lam and dO against torch's double backward in 64 bits (CPU).
        The library's backward-over-backward is held to 1e-4 of each result's
        largest value in fp32; these sums have three such terms."""
        N = 50
        q, k, v, w, do = inputs(1, 2, Hk, N, d, dv, F32, (lam, F32), seed=8)
        cots = [0.5 * torch.randn_like(t) for t in (q, k, v, w)]

        def second(args, attn):
            leaves = [t.clone().requires_grad_() for t in args]
            out = attn(*leaves[:4])
            first = torch.autograd.grad(out, leaves[:4], leaves[4], create_graph=True)
            loss = sum((c.to(g) * g).sum() for c, g in zip(cots, first))
            return torch.autograd.grad(loss, leaves)

        def dense(q, k, v, w):
            G = 2 // Hk
            kk, vv = k.view(1, Hk, 2, N, d).repeat_interleave(G, 1), v.repeat_interleave(G, 1)
            s = q.view(1, 2, 2, N, d) @ kk.transpose(-1, -2) / math.sqrt(d)
            s = s.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -math.inf)
            o = torch.softmax(s, -1) @ vv[:, :, None]
            ww = (w[:, None] if w.dim() == 1 else w).expand(1, 2, N)[..., None]
            return o[:, :, 0] - ww * o[:, :, 1]

        got = second((q, k, v, w, do), lambda *a: fbob.diff_attention(*a, causal=True))
        want = second([t.double().cpu() for t in (q, k, v, w, do)], dense)
        for name, a, b in zip(("q", "k", "v", "lam", "do"), got, want):
            err = (a.double().cpu() - b).abs().max() / b.abs().max()
            assert err <= 3e-4, (name, err.item())

    def test_second_derivative_of_one_gradient(self):
        """A loss that reads dlam alone, and one that reads dK alone, in bf16.
        The library's backward-over-backward is held to 2e-2 of each result's
        largest value in bf16, and q, k, v and dO sum up to two of its
        results.  lam's gradient is a sum of its own, -sum dO . U over rows and
        features with U the gradient in the second map's upstream, where terms
        cancel: it is off by at most sum |dO| times U's error of 2e-2 max |U|."""
        q, k, v, w, do = inputs(1, 2, 2, 160, 64, 128, BF, ("head", BF), seed=9)
        for pick in (3, 1):
            def second(args, attn):
                leaves = [t.clone().requires_grad_() for t in args]
                first = torch.autograd.grad(attn(*leaves[:4]), leaves[:4], leaves[4], create_graph=True)
                g = first[pick]
                c = torch.linspace(-1, 1, g.numel(), device=g.device).to(g).view(g.shape)
                return torch.autograd.grad((c * g).sum(), leaves, allow_unused=True,
                                           materialize_grads=True)

            def dense(q, k, v, w):
                s = q.view(1, 2, 2, 160, 64) @ k.view(1, 2, 2, 160, 64).transpose(-1, -2) / 8
                o = torch.softmax(s, -1) @ v[:, :, None]
                return o[:, :, 0] - w[:, None, None] * o[:, :, 1]

            def map2(q, k, v, w):
                s = q.view(1, 2, 2, 160, 64) @ k.view(1, 2, 2, 160, 64).transpose(-1, -2) / 8
                return torch.softmax(s[:, :, 1], -1) @ v + 0 * w[:, None, None]

            x = [t.double().cpu() for t in (q, k, v, w, do)]
            up = second(x[:4] + [-x[3][:, None, None] * x[4]], map2)[4] if pick == 1 else None
            got = second((q, k, v, w, do), lambda *a: fbob.diff_attention(*a))
            want = second([t.double().cpu() for t in (q, k, v, w, do)], dense)
            for name, a, b in zip(("q", "k", "v", "lam", "do"), got, want):
                if b.abs().max() == 0:
                    assert (a == 0).all(), name
                    continue
                err = (a.double().cpu() - b).abs()
                if name == "lam":
                    bound = 2e-2 * up.abs().max() * x[4].abs().sum((0, 2, 3)) + 2.0 ** -8 * b.abs()
                    assert (err <= bound).all(), (pick, name, (err / bound).max().item())
                    continue
                err = err.max() / b.abs().max()
                assert err <= 4e-2, (pick, name, err.item())

    def test_gradient_against_differences(self):
        """Directional differences of the fp32 forward: with step t the
        difference quotient is off by the third derivative times t^2 and by
        rounding over t, both below 1e-3 of the slope's scale here."""
        q, k, v, w, do = inputs(1, 2, 1, 40, 16, 24, F32, ("head", F32), seed=10)
        leaves = [t.clone().requires_grad_() for t in (q, k, v, w)]
        grads = torch.autograd.grad(fbob.diff_attention(*leaves, causal=True), leaves, do)
        g = torch.Generator("cuda").manual_seed(1)
        t = 2.0 ** -6
        for i in range(4):
            step = torch.randn(leaves[i].shape, generator=g, device="cuda")
            step = step / step.norm()

            def at(s):
                a = [x.detach() for x in leaves]
                a[i] = a[i] + s * step
                return (fbob.diff_attention(*a, causal=True).double() * do.double()).sum()

            slope = (grads[i].double() * step.double()).sum()
            quotient = (at(t) - at(-t)) / (2 * t)
            assert abs(slope - quotient) <= 1e-3 * grads[i].norm().item()

    def test_graph_capture(self):
        """Forward and backward captured once, replayed on new inputs."""
        q, k, v, w, do = inputs(1, 2, 2, 200, 64, 128, BF, ("head", BF), seed=11)

        def both(q, k, v, w, do):
            o, rest, lse = fbob.diff_forward(q, k, v, w, True)
            return (o,) + fbob.diff_backward(q, k, v, w, o, rest, lse, do, True)

        static = [t.clone() for t in (q, k, v, w, do)]
        both(*static)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both(*static)
        for seed in (12, 13):
            new = inputs(1, 2, 2, 200, 64, 128, BF, ("head", BF), seed=seed)
            for s, t in zip(static, new):
                s.copy_(t)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(got, both(*new)))

    @pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 64)])
    def test_captured_training_step(self, dtype, d):
        """Forward and gradients through autograd, captured twice from fresh
        leaves and replayed in turn: each graph has its own workspaces."""
        graphs = []
        stream = torch.cuda.Stream()
        for seed in (15, 16):
            q, k, v, w, do = inputs(1, 2, 1, 150, d, 64, dtype, ("head", dtype), seed=seed)
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                leaves = [t.clone().requires_grad_() for t in (q, k, v, w)]
                torch.autograd.grad(fbob.diff_attention(*leaves, causal=True), leaves, do)
            torch.cuda.current_stream().wait_stream(stream)
            torch.cuda.synchronize()
            leaves = [t.clone().requires_grad_() for t in (q, k, v, w)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                out = fbob.diff_attention(*leaves, causal=True)
                got = (out.detach(),) + torch.autograd.grad(out, leaves, do)
            del out
            graphs.append((graph, leaves, do, got))
        for _ in range(2):
            for graph, *_ in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for _, leaves, do, got in graphs:
            q, k, v, w = (t.detach() for t in leaves)
            o, rest, lse = fbob.diff_forward(q, k, v, w, True)
            want = (o,) + fbob.diff_backward(q, k, v, w, o, rest, lse, do, True)
            assert all(torch.equal(a, b) for a, b in zip(got, want))

    @pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 128), (BF, 128, 64), (F32, 64, 64), (BF, 40, 24)])
    def test_keys_whose_scores_are_minus_infinity(self, dtype, d, dv):
        """Keys with an infinite feature, the first 300 of 350: whole tiles of
        -inf before the first key that counts give what the other keys give."""
        q, k, v, w, do = inputs(1, 2, 2, 350, d, dv, dtype, ("head", dtype), seed=17)
        q[..., 0] = 0.5
        k[..., 0] = 0.25
        k[:, :, :300, 0] = -math.inf
        o, rest, lse = fbob.diff_forward(q, k, v, w)
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
        # the same values densely, in 64 bits, over the last 50 keys; a key's
        # weight is off by a rounding of P (bf16) and by those of its score
        S = q.double().view(1, 2, 2, 350, d) @ k[:, :, 300:].double().view(1, 2, 2, 50, d).transpose(-1, -2)
        P = torch.softmax(S / math.sqrt(d), -1)
        ww = w.double()[:, None, None]
        O12 = P @ v[:, :, None, 300:].double()
        PV = P @ v[:, :, None, 300:].double().abs()
        eps = torch.finfo(dtype).eps / 2
        smax = (q.double().abs().amax() * k[:, :, 300:].double().abs().sum(-1).amax() / math.sqrt(d)).item()
        r = (2 * (d + 4) * smax + 8 + 350 + dv) * U * 2  # as in the oracle
        mix = PV[:, :, 0] + ww.abs() * PV[:, :, 1]
        want = O12[:, :, 0] - ww * O12[:, :, 1]
        err = ((0 if dtype == F32 else eps) + r) * mix
        err = err + eps * (want.abs() + err)
        assert ((o.double() - want).abs() <= err).all()

    def test_third_derivative_is_refused(self):
        q, k, v, w, do = inputs(1, 1, 1, 8, 16, 16, F32, ("one", F32))
        q.requires_grad_()
        first, = torch.autograd.grad(fbob.diff_attention(q, k, v, w), q, do, create_graph=True)
        second, = torch.autograd.grad(first.square().sum(), q, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(second.sum(), q)

    @pytest.mark.parametrize("d,dv", [(64, 128), (64, 64), (128, 128)])
    def test_kernels_stop_cleanly_when_their_waits_run_out(self, d, dv):
        """A 1 ns wait limit: each call reports the timeout in its workspace's
        status word, and the next call with the default limit is as before."""
        from exact_second_order_two_gb300.diff_attention import _shape, _workspace

        q, k, v, w, do = inputs(1, 2, 1, 2048, d, dv, BF, ("head", BF), seed=14)
        shp = _shape(q, k, v, w, True, None)
        fws, bws = (_workspace(op, shp, q.device) for op in (0, 1))
        o, rest, lse = fbob.diff_forward(q, k, v, w, True, workspace=fws)
        calls = ((fws, lambda: fbob.diff_forward(q, k, v, w, True, workspace=fws)),
                 (bws, lambda: fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, workspace=bws)))
        for ws, call in calls:
            want = call()
            assert fbob.status(ws) == 0
            old = fbob.set_wait_limit(1)
            try:
                call()
                st = fbob.status(ws)
            finally:
                fbob.set_wait_limit(old)
            assert st == 5  # FBOB_ERR_TIMEOUT
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
            assert fbob.status(ws) == 0

    def test_refusals(self):
        q, k, v, w, do = inputs(1, 2, 2, 8, 64, 64, BF, ("head", BF))
        for bad in (lambda: fbob.diff_attention(q[:, :3], k, v, w),
                    lambda: fbob.diff_attention(q, k[:, :2], v, w),
                    lambda: fbob.diff_attention(q, k[:, :, :4], v, w),
                    lambda: fbob.diff_attention(q, k, v[:, :, :4], w),
                    lambda: fbob.diff_attention(q, k[..., :32], v, w),
                    lambda: fbob.diff_attention(q, k.float(), v, w),
                    lambda: fbob.diff_attention(q, k, v, w[:1]),
                    lambda: fbob.diff_attention(q, k, v, w.cpu()),
                    lambda: fbob.diff_attention(q[0], k, v, w),
                    lambda: fbob.diff_forward(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, w)):
            with pytest.raises(ValueError):
                bad()
        with pytest.raises(TypeError):
            fbob.diff_attention(q.half(), k.half(), v.half(), w)
        with pytest.raises(TypeError):
            fbob.diff_attention(q, k, v, w.double())
        with pytest.raises(TypeError):
            fbob.diff_attention(q, k, v, 0.5)
        for ws in (torch.empty(1 << 20, dtype=torch.uint8),
                   torch.empty(1 << 20, dtype=torch.int8, device="cuda"),
                   torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                fbob.diff_forward(q, k, v, w, workspace=ws)
        with pytest.raises(fbob.FbobError):
            fbob.diff_forward(q, k, v, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            with pytest.raises(fbob.FbobError):
                fbob.diff_attention(q, k, v, w, scale=scale)
        with pytest.raises(fbob.FbobError):
            wide = torch.zeros(1, 4, 8, 256, dtype=BF, device="cuda")
            fbob.diff_attention(wide, wide, v, w)
        o, rest, lse = fbob.diff_forward(q, k, v, w)
        with pytest.raises(ValueError):
            fbob.diff_backward(q, k, v, w, o, rest, lse, do.float())
        with pytest.raises(ValueError):
            fbob.diff_backward(q, k, v, w, o, rest, lse[:, :2], do)
        with pytest.raises(ValueError):  # of a forward that no backward was to follow
            fbob.diff_backward(q, k, v, w, o, fbob.diff_forward(q, k, v, w, need_rest=False)[1], lse, do)


def test_rejects_cpu_tensors():
    q, k, v, w, do = inputs(1, 1, 1, 4, 8, 8, F32, ("head", F32), device="cpu")
    with pytest.raises(fbob.FbobError):
        fbob.diff_attention(q, k, v, w)


def shape(**kw):
    a = dict(B=1, H=4, Hk=2, N=100, d=64, dv=128, dtype=0, causal=1, lam_kind=1, lam_dtype=0,
             scale=0.125)
    a.update(kw)
    return B.DiffShape(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(H=3), 1), (dict(Hk=0), 1), (dict(N=0), 1), (dict(d=0), 1),
    (dict(dv=0), 1), (dict(causal=2), 1), (dict(lam_kind=3), 1), (dict(lam_kind=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(dtype=2), 2), (dict(lam_dtype=2), 2), (dict(d=129), 2),
    (dict(dv=129), 2), (dict(B=32768, H=2), 2), (dict(N=(1 << 30) + 1, B=1, H=2), 2)])
def test_c_calls_refuse_bad_shapes(kw, code):
    lib, s = B.lib(), shape(**kw)
    good = ctypes.c_void_p(1 << 20)
    for op in (0, 1):
        assert lib.fbob_diff_workspace_size(op, ctypes.byref(s)) == 0
        assert lib.fbob_diff_path(op, ctypes.byref(s)) == -1
    assert lib.fbob_diff_forward(ctypes.byref(s), *[good] * 7, good, 1 << 40, None) == code
    assert lib.fbob_diff_backward(ctypes.byref(s), *[good] * 12, good, 1 << 40, None) == code


def test_c_calls_refuse_bad_pointers_and_workspaces():
    lib, s = B.lib(), shape()
    good, off = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
    odd = ctypes.c_void_p((1 << 20) + 1)
    n = lib.fbob_diff_workspace_size(0, ctypes.byref(s))
    # q, k, v, lam, o, rest, lse; rest may be null, lam needs its own alignment only
    for i in range(7):
        for bad in (None, off, odd):
            args = [good] * 7
            args[i] = bad
            fine = (i == 5 and bad is None) or (i == 3 and bad is off)
            rc = lib.fbob_diff_forward(ctypes.byref(s), *args, good, n - 1, None)
            assert rc == (3 if fine or (i == 3 and bad is odd) else 1), (i, bad)
    assert lib.fbob_diff_forward(ctypes.byref(s), *[good] * 7, None, n, None) == 1
    assert lib.fbob_diff_forward(None, *[good] * 7, good, n, None) == 1
    n = lib.fbob_diff_workspace_size(1, ctypes.byref(s))
    assert n >= 256 + 2 * 4 * 100 * 4
    for i in range(12):
        args = [good] * 12
        args[i] = None
        assert lib.fbob_diff_backward(ctypes.byref(s), *args, good, n - 1, None) == 1
    assert lib.fbob_diff_backward(ctypes.byref(s), *[good] * 12, good, n - 1, None) == 3
    assert lib.fbob_diff_workspace_size(2, ctypes.byref(s)) == 0  # no backward-over-backward call


def test_kernel_family_choice():
    lib = B.lib()
    for op in (0, 1):
        def path(**kw):
            return lib.fbob_diff_path(op, ctypes.byref(shape(**kw)))
        for kw in (dict(), dict(dv=64), dict(d=128), dict(d=128, dv=64), dict(d=96), dict(d=8, dv=40)):
            assert path(**kw) == fbob.PATH_TCGEN05, kw
        for kw in (dict(dtype=1), dict(d=60), dict(dv=97), dict(d=1, dv=4)):
            assert path(**kw) == fbob.PATH_SIMT, kw
        old = fbob.force_path(fbob.PATH_SIMT)
        try:
            assert path() == fbob.PATH_SIMT
            fbob.force_path(fbob.PATH_TCGEN05)
            assert path() == fbob.PATH_TCGEN05 and path(dtype=1) == -1
        finally:
            fbob.force_path(old)


def test_oracle_matches_autograd():
    """The formulas of ``oracle`` against torch's autograd in 64 bits, with a
    mistake planted in each to see that the comparison bites."""
    q, k, v, w, do = (t.double() for t in inputs(1, 2, 1, 9, 4, 6, F32, ("head", F32), device="cpu"))
    leaves = [t.clone().requires_grad_() for t in (q, k, v, w)]
    qq, kk = leaves[0].view(1, 2, 2, 9, 4), leaves[1].view(1, 1, 2, 9, 4)
    s = (0.3 * qq @ kk.transpose(-1, -2)).masked_fill(torch.ones(9, 9, dtype=torch.bool).triu(1), -math.inf)
    both = torch.softmax(s, -1) @ leaves[2][:, :, None]
    o = both[:, :, 0] - leaves[3][:, None, None] * both[:, :, 1]
    grads = torch.autograd.grad(o, leaves, do)
    vals, _ = oracle(q.float(), k.float(), v.float(), w.float(), do.float(), True, 0.3)
    for name, g in zip(("o", "dq", "dk", "dv", "dlam"), (o, *grads)):
        torch.testing.assert_close(vals[name], g.detach(), rtol=1e-12, atol=1e-13)
        assert not torch.allclose(vals[name] * 1.001, g.detach(), rtol=1e-6, atol=1e-9)
