"""Refusals of the FP8 operators' torch binding (no GPU: raised before any call of the library)."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx


def pair(count, rows, cols):
    import torch
    return torch.zeros(count, rows, cols).to(torch.float8_e4m3fn), torch.zeros(count, -(-rows // 128), -(-cols // 128))


@pytest.mark.parametrize("n", [1, 2, 4])
def test_shared_expert_has_three_matrices(n):
    """Gate, up and down, or none: a missing or a fourth pair is refused, not left out."""
    routed = pair(2, 128, 256), pair(2, 128, 256), pair(2, 256, 128)
    shared = [pair(1, 64, 256), pair(1, 64, 256), pair(1, 256, 64), pair(1, 64, 256)]
    with pytest.raises(mx.MxError):
        mx.Fp8Layer(*routed, shared=shared[:n], top_k=2)
    assert mx.Fp8Layer(*routed, shared=shared[:3], top_k=2).c.shared_down.cols == 64
    for none in (None, []):
        assert not mx.Fp8Layer(*routed, shared=none, top_k=2).c.shared_gate.w
