"""Norms of aligned heads of which a part is turned: runs of 8 and 4 features that tile both
parts, and parts that no run tiles, one feature at a time."""
import pytest
import torch

from test_qk_norm import TestValues as Values

CASES = [
    # B, H, Hk, N, d, turned, in, out, weights, layout, interleaved
    (2, 4, 2, 9, 40, 20, "bf16", "bf16", "fp32", "bhnd", False),   # 10 pairs: no run tiles them
    (2, 4, 2, 9, 40, 20, "fp32", "bf16", "fp32", "fused", True),
    (1, 8, 2, 33, 64, 12, "bf16", "fp32", "bf16", "bnhd", False),  # 6 pairs
    (1, 8, 2, 33, 128, 4, "fp32", "fp32", "fp32", "bhnd", True),   # 2 pairs
    (3, 2, 2, 17, 256, 12, "bf16", "bf16", "fp32", "fused", False),
    (2, 2, 1, 5, 64, 8, "bf16", "bf16", "fp32", "bhnd", False),    # runs of 4
    (2, 2, 1, 5, 80, 40, "fp32", "bf16", "fp32", "bnhd", True),
    (2, 2, 1, 5, 96, 48, "bf16", "bf16", "fp32", "fused", False),  # runs of 8
]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
@pytest.mark.parametrize("far", [False, True])
def test_value_and_both_derivatives(case, far):
    Values().test_value_and_both_derivatives(case, far)
