"""The 4-bit operators at their edges: a handle built on another stream than the current one, factors and scales of any
size.

Tolerances are those of the products' own tests."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_fp4 import check_product, matmul, operands, pack, random_scales, scale_rows, values, workspace

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


# one row by integers and by the tensor cores, more rows, clusters
@pytest.mark.parametrize("M,N,K", [(1, 300, 30), (1, 300, 500), (1, 4096, 7000), (20, 300, 30), (20, 300, 500), (20, 300, 6000), (300, 520, 300)])
@pytest.mark.parametrize("tx,tw", [(-120, 120), (120, -120), (-126, 126), (126, -126), (-100, 60), (118, -12), (-12, 118), (60, -126),
                                   (20, -126), (-126, 20)])
@pytest.mark.parametrize("top", [2.0 ** -9, 16.0, 448.0])
def test_factors_that_make_up_for_one_another(M, N, K, tx, tw, top):
    """Neither factor alone takes the sums out of fp32's range where the result is in it."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    xc = torch.randint(0, 16, (M, K), device="cuda", generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 16, (1, N, K), device="cuda", generator=g, dtype=torch.uint8)
    scales = [torch.full(shape, top, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
              for shape in ((M, -(-K // 16)), (1, N, -(-K // 16)))]
    t = [torch.full((1,), 2.0 ** e, device="cuda") * 1.37 for e in (tx, tw)]
    weight = mx.Fp4Weight(pack(wc), scales[1].view(torch.float8_e4m3fn), t[1], cols=K)
    X = values(xc, scales[0], 16, t[0].double())
    W = values(wc, scales[1], 16, t[1].double().view(1, 1, 1))
    mag = float((X.abs() @ W[0].abs().T).max())
    if not 2.0 ** -112 < mag < 2.0 ** 127:
        pytest.skip("the result itself leaves fp32's range")
    check_product(matmul(pack(xc), scale_rows(scales[0], K, 16), t[0], weight, torch.float32), X, W[0], K)


# (2^a and 2^b: scales of a block of the rows and of the matrix; x and w: one code of each there, the others are 0)
@pytest.mark.parametrize("M", [1, 2, 40])
@pytest.mark.parametrize("a,b,x,w", [(100, 100, 0, 2), (127, 127, 0, 7), (64, 64, 0, 0), (64, 64, 1, 1), (65, 64, 1, 1), (127, 1, 1, 1),
                                     (1, 127, 9, 1), (127, -120, 7, 7), (-120, 127, 7, 15), (-100, -100, 7, 7), (-127, 127, 1, 1),
                                     (-127, 120, 7, 7), (-70, -75, 2, 2)])
def test_e8m0_scales_whose_product_leaves_the_range(M, a, b, x, w):
    """A block's term counts as the definition has it, whatever its two scales are by themselves."""
    import torch
    K, N = 96, 130
    xc, wc = (torch.full(shape, 2, dtype=torch.uint8, device="cuda") for shape in ((M, K), (1, N, K)))
    xs, ws = (torch.full(shape, 127, dtype=torch.uint8, device="cuda") for shape in ((M, 3), (1, N, 3)))
    xc[:, 32:64], wc[..., 32:64] = 0, 0
    xc[:, 37], wc[..., 37] = x, w
    xs[:, 1], ws[..., 1] = 127 + a, 127 + b
    weight = mx.Fp4Weight(pack(wc), ws.view(torch.float8_e8m0fnu), cols=K)
    got = matmul(pack(xc), scale_rows(xs, K, 32), None, weight, torch.float32)
    check_product(got, values(xc, xs, 32), values(wc, ws, 32)[0], K)
