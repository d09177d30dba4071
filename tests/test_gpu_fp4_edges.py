"""The 4-bit operators at their edges: a handle built on another stream than the current one.

Tolerances are those of the products' own tests."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_fp4 import check_product, operands, random_scales, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("as_handle", [False, True])
def test_weights_of_a_side_stream_while_the_current_one_is_busy(as_handle):
    """The current stream still writes a block that the host has freed; a handle of the same size built on another stream
    must not be given it."""
    import torch
    M, N, K = 40, 700, 2000
    q, s, tx, weight, X, W = operands(M, N, K, 16)
    scales = random_scales((1, N, K // 16), 16, 2)  # (as operands made them)
    ws = workspace(weight, M)
    n = weight.packed.numel()
    clean = weight.packed.clone()
    out = torch.empty(M, N, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    block.fill_(0x7F)
    at = block.data_ptr()
    del block
    other = mx.Fp4Weight(weight.w, scales.view(torch.float8_e4m3fn), weight.tensor_scale, cols=K,
                         stream=side.cuda_stream if as_handle else side)
    mx.fp4_matmul(q, s, other, out, ws, tensor_scale=tx, stream=side)
    assert other.packed.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(other.packed, clean)
    check_product(out, X, W[0], K)
