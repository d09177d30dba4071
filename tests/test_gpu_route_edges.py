"""Routing from logits at its edges, against its definition in fp64 (as in its own tests)."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_route_logits import both, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [-1e-6, -0.5, -5.0, -16.0, -17.5, -30.0, -59.0, -60.5, -87.0, -400.0])
@pytest.mark.parametrize("groups", [1, 4])
def test_renormalised_sigmoids_far_below_the_largest(top, groups):
    """A sigmoid that fp32 does not hold may still be a good part of the chosen ones' sum."""
    import torch
    x = make(70, 64, 3) * 0.01 - 2000.0
    below = torch.tensor([0.0, 1.0, 4.0, 20.0, 33.0, 50.0, 75.0, 84.0], device="cuda")
    for t in range(70):
        x[t, 3 * (t % 7):3 * (t % 7) + 8] = top - below * (1.0 + 0.001 * t)
    both(x, 8, score=mx.MX_SIGMOID, n_groups=groups, topk_groups=max(1, groups - 1))
