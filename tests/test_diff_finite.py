"""Differential attention where a softmax would give NaN if it gave one: peaked
rows, maps that cancel, and the CUDA-core kernels at the tensor cores' sizes,
by a comparison that a NaN fails."""
import math

import pytest
import torch

import exact_second_order_two_gb300 as fbob
import test_diff_attention as diff

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("o", "o2", "lse", "dq", "dk", "dv", "dlam")


def hold(got, vals, errs, under=0.0):
    for name, t in got.items():
        e, bound = (t.detach().double() - vals[name]).abs(), errs[name] + under
        assert (e <= bound).all(), (name, int((~(e <= bound)).sum()), e.numel())


def underflow(q, k, v, w, do, scale):
    """What the oracle's relative bounds leave out: a weight below 2^-126, the
    smallest normal number of fp32 and bf16, may come out as zero.  A result sums
    at most N of them for each query head, each times at most c (|dP| + |D|) |q|
    or |k| (dS is P (dP - D), |D| <= max |dP|), |v| or |dO|, and rounds to a step
    of 2^-133 at most there."""
    dp = (do.abs().amax() * v.abs().amax() * v.shape[-1]).double().item()
    most = max(t.abs().amax().double().item() for t in (q, k, v, do))
    lam = 1 + w.abs().amax().double().item()
    return 2.0 ** -126 * q.shape[2] * q.shape[1] * lam * (1 + 2 * scale * dp) * most + 2.0 ** -133


def run(args, scale):
    q, k, v, w, do = args
    vals, errs = diff.oracle(*args, True, scale)
    o, rest, lse = fbob.diff_forward(q, k, v, w, True, scale)
    grads = fbob.diff_backward(q, k, v, w, o, rest, lse, do, True, scale)
    hold(dict(zip(NAMES, (o, rest[..., 0, :], lse, *grads))), vals, errs, underflow(*args, scale))


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
class TestOnGpu:
    @pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 128), (BF, 128, 128), (BF, 40, 72), (BF, 20, 12),
                                            (F32, 64, 64)])
    def test_peaked_rows(self, dtype, d, dv):
        q, k, v, w, do = diff.inputs(1, 2, 2, 300, d, dv, dtype, ("head", dtype), seed=30, spread=4.0)
        k = k * torch.linspace(0.1, 1.0, 300, device="cuda").to(dtype)[:, None]
        run((q, k, v, w, do), 0.125)

    @pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)])
    def test_equal_maps(self, dtype, d):
        q, k, v, w, do = diff.inputs(1, 2, 2, 200, d, 128, dtype, ("head", dtype), seed=31)
        q[:, 1::2], k[:, 1::2] = q[:, 0::2], k[:, 0::2]
        w.fill_(1.0)
        run((q, k, v, w, do), 0.125)

    @pytest.mark.parametrize("d,dv,causal_n", [(64, 128, 150), (128, 64, 97), (40, 72, 64)])
    def test_cuda_core_family(self, d, dv, causal_n):
        args = diff.inputs(1, 2, 1, causal_n, d, dv, BF, ("head", BF), seed=32)
        old = fbob.force_path(fbob.PATH_SIMT)
        try:
            run(args, 1.0 / math.sqrt(d))
        finally:
            fbob.force_path(old)


def test_a_planted_nan_fails_the_comparison():
    vals, errs = {"o": torch.zeros(3, dtype=torch.float64)}, {"o": torch.ones(3, dtype=torch.float64)}
    hold({"o": torch.zeros(3)}, vals, errs)
    with pytest.raises(AssertionError):
        hold({"o": torch.tensor([0.0, math.nan, 0.0])}, vals, errs)
    errs["o"][1] = math.nan
    with pytest.raises(AssertionError):
        hold({"o": torch.zeros(3)}, vals, errs)
