"""Calls of the layer operators (rotary positions, differential attention) that
their documentation allows, at the edges: tensors at any address, one batch and
one head, forward-mode derivatives, second derivatives that round no more than
they have to, and sizes whose offsets pass 32 bits."""
import math

import pytest
import torch

import exact_second_order_two_gb300 as fbob
import test_diff_attention as diff

BF, F32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")


def shifted(t):
    """t at an address one element behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.detach().flatten()
    out = flat[1:].view(t.shape)
    assert out.is_contiguous() and out.data_ptr() % 16
    return out


def dense_diff(q, k, v, w, causal):
    """Differential attention in elementary operations, differentiable."""
    B, H2, N, d = q.shape
    H, Hk = H2 // 2, v.shape[1]
    kk = k.view(B, Hk, 2, N, d).repeat_interleave(H // Hk, 1)
    s = q.view(B, H, 2, N, d) @ kk.transpose(-1, -2) / math.sqrt(d)
    if causal:
        s = s.masked_fill(torch.ones(N, N, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    o = torch.softmax(s, -1) @ v.repeat_interleave(H // Hk, 1)[:, :, None]
    ww = (w[:, None] if w.dim() == 1 else w).expand(B, H, N)[..., None]
    return o[:, :, 0] - ww * o[:, :, 1]


def dense_attention(q, k, v, causal):
    s = q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])
    if causal:
        n = q.shape[2]
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    return torch.softmax(s, -1) @ v


def second(args, cots, attn):
    """The gradient of <cots, first gradients> in every argument; args end with
    the upstream gradient, and a None in cots leaves a gradient out."""
    leaves = [t.clone().requires_grad_() for t in args]
    first = torch.autograd.grad(attn(*leaves[:-1]), leaves[:-1], leaves[-1], create_graph=True)
    loss = sum((c * g).sum() for c, g in zip(cots, first) if c is not None)
    return torch.autograd.grad(loss, leaves, allow_unused=True, materialize_grads=True)


# ---- tensors at any address ---------------------------------------------------
@gpu
@needs_gpu
@pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 128), (BF, 40, 20), (F32, 64, 64), (F32, 10, 3)])
def test_diff_attention_of_unaligned_tensors(dtype, d, dv):
    """Inputs sliced from a flat buffer, and an upstream gradient that is a slice
    of the gradient of a concatenation: the same bits as from aligned copies."""
    ins = diff.inputs(1, 2, 1, 70, d, dv, dtype, ("head", dtype), seed=20)
    q, k, v, w, do = ins
    leaves = [t.clone().requires_grad_() for t in (q, k, v, w)]
    out = fbob.diff_attention(*leaves, causal=True)
    want = torch.autograd.grad(out, leaves, do)
    moved = [shifted(t).requires_grad_() for t in (q, k, v, w)]
    got = fbob.diff_attention(*moved, causal=True)
    assert torch.equal(got, out)
    with torch.no_grad():
        assert torch.equal(fbob.diff_attention(*moved, causal=True), out)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(got, moved, shifted(do)), want))
    # what autograd hands back behind a cat along batch or heads
    scalar = torch.zeros(1, dtype=dtype, device="cuda", requires_grad=True)
    out = fbob.diff_attention(*leaves, causal=True)
    joined = torch.cat((scalar, out.flatten()))
    again = torch.autograd.grad(joined, leaves, torch.cat((torch.ones_like(scalar), do.flatten())))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


@gpu
@needs_gpu
@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 10)])
def test_attention_of_unaligned_tensors(dtype, d):
    """Plain attention likewise, through its second derivative."""
    g = torch.Generator("cuda").manual_seed(21)
    q, k, v, do, gq, gk, gv = (torch.randn(1, 2, 70, d, generator=g, device="cuda").to(dtype)
                               for _ in range(7))

    def grads(args, up, cots):
        leaves = [t.requires_grad_() for t in args]
        up = up.requires_grad_()
        out = fbob.attention(*leaves, causal=True)
        first = torch.autograd.grad(out, leaves, up, create_graph=True)
        return (out, *first, *torch.autograd.grad(first, leaves + [up], cots))

    want = grads([t.clone() for t in (q, k, v)], do.clone(), [gq, gk, gv])
    got = grads([shifted(t) for t in (q, k, v)], shifted(do), [shifted(t) for t in (gq, gk, gv)])
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):  # (sums of bf16 dQ and gradQ have no fixed order)
        torch.testing.assert_close(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3)


# ---- one batch, one head ------------------------------------------------------
@gpu
@needs_gpu
@pytest.mark.parametrize("dtype,N,d,dv,tol", [
    (F32, 7, 16, 24, 3e-4), (F32, 13, 10, 3, 3e-4), (F32, 50, 64, 64, 3e-4),
    (BF, 50, 64, 64, 4e-2), (BF, 131, 20, 12, 4e-2)])
@pytest.mark.parametrize("lam", ["one", "row"])
def test_second_derivative_of_one_head(dtype, N, d, dv, tol, lam):
    """B = H = 1, where a map's slice of the log-sum-exps is contiguous as it
    is, at any offset.  Cotangents come as slices of a flat buffer.  Bounds as
    for more heads: 3e-4 and 4e-2 of each result's largest value; lam's
    gradient in bf16 is a sum that cancels, held by the sum of magnitudes."""
    args = diff.inputs(1, 1, 1, N, d, dv, dtype, (lam, dtype), seed=22)
    g = torch.Generator("cuda").manual_seed(23)
    cots = [0.5 * torch.randn(t.shape, generator=g, device="cuda").to(dtype) for t in args[:4]]
    got = second([shifted(t) for t in args], [shifted(c) for c in cots],
                 lambda *a: fbob.diff_attention(*a, causal=True))
    want = second([t.double() for t in args], [c.double() for c in cots],
                  lambda *a: dense_diff(*a, True))
    for name, a, b in zip(("q", "k", "v", "lam", "do"), got, want):
        err, top = (a.double() - b).abs().max(), b.abs().max()
        if name == "lam":
            # -sum dO . U, U the gradient in the second map's upstream
            x = [t.double() for t in args]
            lo, up = [c.double() for c in cots], -(x[3][:, None] if x[3].dim() == 1 else x[3])
            up = up.expand(1, 1, N)[..., None] * x[4]
            lo[0], lo[1] = lo[0][:, 1:], lo[1][:, 1:]
            U = second([x[0][:, 1:], x[1][:, 1:], x[2], up], lo[:3], lambda *a: dense_attention(*a, True))[3]
            mag = x[4].abs().sum(-1)
            mag = mag.sum() if lam == "one" else mag.max()
            assert err <= tol * U.abs().max() * mag + 2.0 ** -8 * top, (name, err.item())
        else:
            assert err <= tol * top, (name, err.item(), top.item())


# ---- forward-mode derivatives ---------------------------------------------------
@gpu
@needs_gpu
class TestForwardMode:
    """Neither operator has a forward-mode derivative: it is refused, and a
    tangent never dropped."""

    def test_rotary(self):
        x = torch.randn(1, 2, 5, 64, device="cuda")
        f, _ = fbob.rotary_frequencies(64)
        t = torch.randn_like(x)
        with torch.autograd.forward_ad.dual_level():
            dual = torch.autograd.forward_ad.make_dual(x, t)
            with pytest.raises(NotImplementedError):
                fbob.rotary(dual, f)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                fbob.rotary(dual, f)
            with pytest.raises(ValueError):  # frequencies are not differentiated
                fbob.rotary(x, torch.autograd.forward_ad.make_dual(f, torch.ones_like(f)))
            y = fbob.rotary(x, f)  # no tangent, none lost
            assert torch.autograd.forward_ad.unpack_dual(y).tangent is None
            # forward over reverse
            leaf = x.clone().requires_grad_()
            y = fbob.rotary(leaf, f)
            up = torch.autograd.forward_ad.make_dual(torch.ones_like(y), t)
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(y, leaf, up)
        with pytest.raises((NotImplementedError, RuntimeError)):
            torch.func.jvp(lambda a: fbob.rotary(a, f), (x,), (t,))

    @pytest.mark.parametrize("which", range(4))
    def test_diff_attention(self, which):
        args = list(diff.inputs(1, 2, 1, 9, 16, 24, F32, ("head", F32), seed=24))
        do = args.pop()
        t = torch.ones_like(args[which])
        with torch.autograd.forward_ad.dual_level():
            dual = list(args)
            dual[which] = torch.autograd.forward_ad.make_dual(args[which], t)
            with pytest.raises(NotImplementedError):
                fbob.diff_attention(*dual)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                fbob.diff_attention(*dual)
            leaves = [a.clone().requires_grad_() for a in args]
            out = fbob.diff_attention(*leaves)
            up = torch.autograd.forward_ad.make_dual(do, torch.ones_like(do))
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(out, leaves, up)
        with pytest.raises((NotImplementedError, RuntimeError)):
            torch.func.jvp(lambda a: fbob.diff_attention(*args[:which], a, *args[which + 1:]),
                           (args[which],), (t,))

    @pytest.mark.parametrize("op", ["attention", "differential"])
    def test_second_derivative(self, op):
        """A tangent on the cotangent of a first gradient."""
        q, k, v, w, do = diff.inputs(1, 1, 1, 9, 16, 16, F32, ("head", F32), seed=25)
        args = (q, k, v, w) if op == "differential" else (q[:, :1].clone(), k[:, :1].clone(), v)
        fn = fbob.diff_attention if op == "differential" else fbob.attention
        leaves = [a.clone().requires_grad_() for a in args]
        first = torch.autograd.grad(fn(*leaves), leaves, do, create_graph=True)
        with torch.autograd.forward_ad.dual_level():
            c = torch.autograd.forward_ad.make_dual(torch.ones_like(first[0]), torch.ones_like(first[0]))
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(first[0], leaves, c, allow_unused=True)


# ---- roundings of the second derivative -----------------------------------------
@gpu
@needs_gpu
@pytest.mark.parametrize("kind", ["one", "head"])
@pytest.mark.parametrize("d,dv", [(20, 12), (40, 80)])
def test_second_derivative_scales_with_lam(kind, d, dv):
    """The second map's part of a second derivative in q is lam times that at
    lam = 1, rounded once: 0.75 R, with R in bf16 already."""
    q, k, v, w, do = diff.inputs(1, 2, 2, 150, d, dv, BF, (kind, BF), seed=26)
    c = torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(27), device="cuda").to(BF)

    def grad_q2(value):
        return second((q, k, v, torch.full_like(w, value), do), (c, None, None, None),
                      lambda *a: fbob.diff_attention(*a, causal=True))[0][:, 1::2]

    assert torch.equal(grad_q2(0.75), (0.75 * grad_q2(1.0).float()).to(BF))


@gpu
@needs_gpu
def test_second_derivative_in_the_upstream_gradient_rounds_once():
    """A loss of dlam alone, sum g dlam: its gradient in dO is -g O2.  On CUDA
    cores O2 is as good as fp32 before it is rounded, and what the rounding left
    off is kept, so -g O2 is off by half a step of bf16 (2^-8), by the square of
    one, and by sums of 32 bits: N + d + 20 steps of 2^-24 of P |V|."""
    N, d, dv = 90, 20, 12
    q, k, v, w, do = diff.inputs(1, 2, 2, N, d, dv, BF, ("row", F32), seed=28)
    g = torch.Generator("cuda").manual_seed(29)
    c = torch.randn(w.shape, generator=g, device="cuda")
    got = second((q, k, v, w, do), (None, None, None, c), lambda *a: fbob.diff_attention(*a))[4]
    s = q[:, 1::2].double() @ k[:, 1::2].double().transpose(-1, -2) / math.sqrt(d)
    P = torch.softmax(s, -1)
    want = -c.double()[..., None] * (P @ v.double())
    mag = c.double().abs()[..., None] * (P @ v.double().abs())
    smax = (q.double().abs() @ k.double().abs().transpose(-1, -2)).max().item() / math.sqrt(d)
    small = 2.0 ** -24 * (N + 2 * (d + 4) * smax + 20) + 2.0 ** -16
    bound = 2.0 ** -8 * (want.abs() + small * mag) + small * mag
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()


# ---- positions -------------------------------------------------------------------
@gpu
@needs_gpu
def test_rotary_refuses_a_fractional_position():
    x = torch.randn(1, 2, 5, 64, device="cuda")
    f, _ = fbob.rotary_frequencies(64)
    for bad in (2.5, 2.0, "2"):
        with pytest.raises(TypeError):
            fbob.rotary(x, f, bad)


def test_frequencies_refuse_a_fractional_width():
    with pytest.raises(TypeError):
        fbob.rotary_frequencies(64.5, device="cpu")


# ---- scale -----------------------------------------------------------------------
def test_scale_up_to_its_limit():
    """scale log2 e, which the kernels multiply with, is to be finite."""
    import ctypes

    lib = fbob.lib()
    for scale, ok in ((2.0e38, True), (2.4e38, False), (3.0e38, False), (1e-30, True)):
        assert (lib.fbob_diff_workspace_size(0, ctypes.byref(diff.shape(scale=scale))) > 0) == ok


@gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [2.0e38, 1e-30])
def test_extreme_scales_of_zero_scores(dtype, scale):
    """Queries of zeros: every score is 0 at any scale, and a row the mean of
    the values it sees, up to roundings (half a step of the type, and for P)."""
    q, k, v, w, do = diff.inputs(1, 2, 1, 130, 64, 64, dtype, ("head", dtype), seed=33)
    got = fbob.diff_attention(torch.zeros_like(q), k, v, w, causal=True, scale=scale)
    n = torch.arange(1, 131, device="cuda")[:, None]
    mean, mag = v.double().cumsum(2) / n, v.double().abs().cumsum(2) / n
    ww = w.double()[:, None, None]
    h = torch.finfo(dtype).eps / 2 if dtype == BF else 0
    err = (h + 200 * 2.0 ** -24) * (1 + ww.abs()) * mag
    want = (1 - ww) * mean
    err = err + torch.finfo(dtype).eps / 2 * (want.abs() + err)
    assert ((got.double() - want).abs() <= err).all()


@gpu
@needs_gpu
@pytest.mark.parametrize("d", [64, 96, 128])
def test_every_head_where_loads_are_waited_for(d):
    """2000 heads of keys of their own, as many bytes as the memory can bring:
    tiles land later than the warps want them.  Every element of both maps'
    products against plain attention over the same map, whose kernels round
    alike: each is off by h P|V| (P a bf16 operand, h = 2^-8), by half a step of
    its result, and by 32-bit sums; P|V| comes from plain attention over |V|,
    itself within 2 h of it."""
    H, N, h = 2000, 1024, 2.0 ** -8
    g = torch.Generator("cuda").manual_seed(35)
    q, k = (torch.randn(1, 2 * H, N, d, generator=g, device="cuda", dtype=BF) for _ in range(2))
    v = torch.randn(1, H, N, d, generator=g, device="cuda", dtype=BF)
    w = torch.rand(H, generator=g, device="cuda")
    scale = d ** -0.5
    o, rest, lse = fbob.diff_forward(q, k, v, w, True, scale)
    o2 = rest[..., 0, :]
    got = (o.float() + w[:, None, None] * (o2.float() + rest[..., 1, :].float()) + rest[..., 2, :].float(), o2)
    del rest, o
    wide = 64 if d == 64 else 128
    pad = lambda t: torch.nn.functional.pad(t, (0, wide - d)).contiguous()
    small = 2.0 ** -24 * (N + 20 * d)
    for m in (0, 1):
        qm, km = pad(q[:, m::2]), pad(k[:, m::2])
        want, want_lse = fbob.forward(qm, km, pad(v), True, scale)
        mag, _ = fbob.forward(qm, km, pad(v.abs()), True, scale)
        err = 2 * (h + small) * (1 + 2 * h) * mag[..., :d].float() + 2 * h * want[..., :d].float().abs() + 1e-6
        off = (got[m].float() - want[..., :d].float()).abs()
        assert (off <= err).all(), (m, int((off > err).sum()), (off / err).max().item())
        assert ((lse[:, m::2] - want_lse).abs() <= 2.0 ** -24 * 40 * (d + 8)).all()
    del got, q, k, v
    torch.cuda.empty_cache()


@gpu
@needs_gpu
@pytest.mark.parametrize("d,dv", [(64, 128), (128, 128)])
def test_every_gradient_where_loads_are_waited_for(d, dv):
    """608 heads of keys of their own, forward and backward, every element against
    the definition in 64 bits, 38 heads at a time."""
    import test_diff_finite as finite

    H, N, step, scale = 608, 1024, 38, d ** -0.5
    q, k, v, w, do = diff.inputs(1, H, H, N, d, dv, BF, ("row", F32), seed=36)
    o, rest, lse = fbob.diff_forward(q, k, v, w, True, scale)
    grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, scale)
    for h in range(0, H, step):
        maps, some = slice(2 * h, 2 * (h + step)), slice(h, h + step)
        part = tuple(t.contiguous() for t in (q[:, maps], k[:, maps], v[:, some], w[:, some], do[:, some]))
        vals, errs = diff.oracle(*part, True, scale)
        got = (o[:, some], rest[:, some, :, 0], lse[:, maps], grads[0][:, maps], grads[1][:, maps],
               grads[2][:, some], grads[3][:, some])
        finite.hold(dict(zip(finite.NAMES, got)), vals, errs, finite.underflow(*part, scale))
    del vals, errs
    torch.cuda.empty_cache()
# ---- offsets past 32 bits --------------------------------------------------------
def needs_memory(gb):
    return pytest.mark.skipif(
        torch.cuda.is_available() and torch.cuda.get_device_properties(0).total_memory < gb * 2 ** 30,
        reason=f"needs {gb} GB of device memory")


@gpu
@needs_gpu
@needs_memory(60)
def test_rotary_of_more_than_2_to_the_32_elements():
    """8 heads of 2^22 + 3 tokens, as [B, N, H, d] and dense: the last rows, of
    values and gradients, are those of a call on the last rows alone."""
    n, tail = (1 << 22) + 3, 5
    f, _ = fbob.rotary_frequencies(128)
    for layout in ("bnhd", "bhnd"):
        shape = (1, n, 8, 128) if layout == "bnhd" else (1, 8, n, 128)
        x = torch.randn(shape, device="cuda", dtype=BF)
        x = (x.transpose(1, 2) if layout == "bnhd" else x).requires_grad_()
        y = fbob.rotary(x, f)
        end = x.detach()[:, :, -tail:].clone().requires_grad_()
        want = fbob.rotary(end, f, n - tail)
        assert torch.equal(y[:, :, -tail:], want)
        assert torch.equal(torch.autograd.grad(y, x, y.detach())[0][:, :, -tail:],
                           torch.autograd.grad(want, end, want.detach())[0])
        del x, y
    torch.cuda.empty_cache()


@gpu
@needs_gpu
@needs_memory(160)
@pytest.mark.parametrize("dtype,H,N", [(BF, 16400, 1024), (F32, 32767, 520)])
def test_diff_attention_of_more_than_2_to_the_32_elements(dtype, H, N):
    """Queries and keys of 2^32 elements and more: the first, a middle and the
    last head against the definition in 64 bits."""
    import test_diff_finite as finite

    g = torch.Generator("cuda").manual_seed(34)
    q, k = (torch.randn(1, 2 * H, N, 128, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    v, do = (torch.randn(1, H, N, 128, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    w = torch.rand(1, H, N, generator=g, device="cuda").to(dtype)
    assert q.numel() > 1 << 32
    scale = 128 ** -0.5
    o, rest, lse = fbob.diff_forward(q, k, v, w, True, scale)
    grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, scale)
    for h in (0, H // 2, H - 1):
        maps, one = slice(2 * h, 2 * h + 2), slice(h, h + 1)
        part = (q[:, maps], k[:, maps], v[:, one], w[:, one], do[:, one])
        vals, errs = diff.oracle(*part, True, scale)
        got = (o[:, one], rest[:, one, :, 0], lse[:, maps], grads[0][:, maps], grads[1][:, maps],
               grads[2][:, one], grads[3][:, one])
        finite.hold(dict(zip(finite.NAMES, got)), vals, errs, finite.underflow(*part, scale))
    del q, k, v, do, w, o, rest, lse, grads, part, got
    torch.cuda.empty_cache()
