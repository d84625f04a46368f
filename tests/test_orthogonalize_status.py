"""The status word of orthogonalisations: whatever a workspace held, and whichever block
reports."""
import ctypes

import pytest
import torch

import exact_second_order_two_gb300 as fbob
from exact_second_order_two_gb300 import _binding as B
from test_orthogonalize import ONE, gradient

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("shape", [(3000, 64, 64), (3000, 100, 128), (2, 300, 400)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_status(shape, dtype):
    """Set to something else before each call: 0 after it, or what the waits that ran out say.  (A
    small matrix's waits, of a microsecond each, are over within the first look at the barrier,
    which may itself last longer, before the limit counts.)"""
    G, dY = gradient(shape, dtype)
    coef = (ctypes.c_float * 15)(*(ONE * 5))
    o = B.Orth(*shape, B.DTYPES[dtype], 5, 1, 1e-7, ctypes.addressof(coef))
    lib, r, stream = B.lib(), ctypes.byref(o), B._stream(G.device)
    sizes = [lib.fbob_orth_workspace_size(op, r) for op in (0, 1)]
    kept, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)
    y, dG = torch.empty_like(G), torch.empty_like(G)
    p = lambda t: t.data_ptr()  # noqa: E731

    def forward():
        return lib.fbob_orth_forward(r, p(G), p(y), p(kept), sizes[0], stream), kept

    def backward():
        return lib.fbob_orth_backward(r, p(G), p(dY), p(dG), p(kept), sizes[0], p(ws), sizes[1], stream), ws

    small = shape[1] <= 128
    for limit, want in ((None, (0,)), (1, (0, 5) if small else (5,)), (None, (0,))):
        for call in (forward, backward):
            (kept if call is forward else ws)[:4] = torch.tensor([9, 9, 9, 9], dtype=torch.uint8)
            old = fbob.set_wait_limit(limit) if limit else None
            try:
                status, words = call()
                assert status == 0 and fbob.status(words) in want
            finally:
                if limit:
                    fbob.set_wait_limit(old)
            if limit:  # the backward reads what a whole forward kept
                assert forward()[0] == 0 and fbob.status(kept) == 0


@pytest.mark.parametrize("shape", [(16, 64, 64), (3, 100, 250), (2, 250, 100)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_captured_and_replayed(shape, dtype):
    """Two graphs of a call with its gradient, replayed in turn with inputs that change, beside
    calls of the same size outside: every result is that of a call by itself."""
    def step(x, d):
        y = fbob.orthogonalize(x)
        return y, torch.autograd.grad(y, x, d)[0]

    some = [gradient(shape, dtype, seed=i) for i in range(4)]
    want = [[t.detach().clone() for t in step(G.clone().requires_grad_(), dY)] for G, dY in some]
    leaves = [(torch.zeros_like(G).requires_grad_(), torch.zeros_like(dY)) for G, dY in some[:2]]
    graphs, outs = [], []
    for leaf in leaves:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*leaf))
    for first in (0, 2, 1):
        at = [first, (first + 1) % 4]
        with torch.no_grad():
            for (x, d), i in zip(leaves, at):
                x.copy_(some[i][0])
                d.copy_(some[i][1])
        for g in graphs:
            g.replay()
        alone = step(some[3][0].clone().requires_grad_(), some[3][1])
        assert all(torch.equal(a, b) for a, b in zip(alone, want[3]))
        for out, i in zip(outs, at):
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
