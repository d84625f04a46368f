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
