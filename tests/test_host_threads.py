"""Calls of one kernel at different sizes from several host threads: what one sets for
its launch takes nothing from another's."""
import importlib
import threading

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B
from exact_second_order_two_gb300 import qk_norm as Q

O = importlib.import_module("exact_second_order_two_gb300.orthogonalize")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def at_once(calls, times):
    """Calls over and over, each in a thread and on a stream of its own: how many failed."""
    failed, ready = [0] * len(calls), threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(i):
        with torch.no_grad(), torch.cuda.stream(streams[i]):
            ready.wait()
            for _ in range(times):
                try:
                    failed[i] += calls[i](streams[i].cuda_stream) != 0
                except fbob.FbobError:
                    failed[i] += 1

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def normal(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def orthogonal(shape, dtype):
    """The C calls forward and backward, prepared: little else is between two of them."""
    g, dy = normal(*shape, dtype=dtype), normal(*shape, dtype=dtype, seed=1)
    out = [torch.empty_like(g) for _ in range(2)]
    ref, sizes = O._problem(g.shape, dtype, 2, ((1.5, -0.5, 0.0),), 1e-7, True)
    kept, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)
    lib, p = B.lib(), lambda t: t.data_ptr()  # noqa: E731

    def call(stream):
        return (lib.fbob_orth_forward(ref, p(g), p(out[0]), p(kept), sizes[0], stream)
                or lib.fbob_orth_backward(ref, p(g), p(dy), p(out[1]), p(kept), sizes[0], p(ws), sizes[1], stream))

    return call, out


def second(d):
    """A second derivative of norms of d features."""
    x, dy, a = (normal(1, 2, 5, d, seed=i) for i in range(3))
    w, c = 1.0 + 0.1 * normal(d), normal(d, seed=4)
    inv_freq = torch.linspace(1.0, 0.1, d // 2, dtype=torch.float64, device="cuda")
    problem = Q._pack(1, 5, d, d, 0, 1, 1, 1, 1e-6, 1.0, 0, 0)
    out = [torch.empty_like(t) for t in (x, w, dy)]
    side = Q._side(x, w, out[0], dy, a, c, out[1], out[2])
    n = Q._workspace_size(problem)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    held = x, dy, a, w, c

    def call(stream, held=held):
        return B.lib().fbob_qk_norm_bob(problem, side, None, inv_freq.data_ptr(), None, ws.data_ptr(), n, stream)

    return call, out


def check(some):
    """Results beside others as they are alone."""
    stream = torch.cuda.current_stream().cuda_stream
    want = []
    for call, out in some:
        assert call(stream) == 0
        want.append([t.clone() for t in out])
    assert at_once([call for call, _ in some], 3000) == [0] * len(some)
    for (_, out), w in zip(some, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_orthogonalize(dtype):
    check([orthogonal((1, *s), dtype) for s in ((30, 40), (100, 128), (30, 50), (128, 250))])


def test_second_derivatives_of_norms():
    check([second(d) for d in (16, 256, 32, 128)])


def test_attention_on_cuda_cores():
    """Heads of different widths, plain and differential."""
    lam = torch.full((1,), 0.3, device="cuda")
    calls = []
    for d in (8, 128):
        q, k, v = (normal(1, 2, 40, d, seed=i) for i in range(3))
        calls += [lambda s, t=(q, k, v): fbob.attention(*t, causal=True) is None,
                  lambda s, t=(q, k, v[:, :1].contiguous()): fbob.diff_attention(*t, lam, causal=True) is None]
    assert at_once(calls, 1000) == [0] * 4
