"""The 4-bit operators at their edges: a handle built on another stream than the current one, factors and scales of any
size, spare nibbles, long sums, and matrices of more pieces than a launch has threads.

Tolerances are those of the products' own tests."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_fp4 import (check_product, gen, matmul, operands, pack, plain_scales, random_scales, ref_quantize, scale_rows, unpack,
                                values, workspace)

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


@pytest.mark.parametrize("M,N,K", [(1, 300, 501), (1, 4096, 7001), (30, 300, 1999), (300, 300, 501), (20, 300, 6001)])
@pytest.mark.parametrize("block", [16, 32])
def test_the_spare_nibble_of_a_rows_last_byte_does_not_count(M, N, K, block):
    import torch
    q, s, tx, weight, X, W = operands(M, N, K, block)
    clean = matmul(q, s, tx, weight, torch.float32).clone()
    q[:, -1] |= torch.where(torch.arange(M, device="cuda") % 2 == 0, 0x70, 0xF0).to(torch.uint8)
    got = matmul(q, s, tx, weight, torch.float32)
    assert torch.equal(got, clean)
    check_product(got, X, W[0], K)


# one row by integers and by the tensor cores, whole, in four and eight, every token tile
@pytest.mark.parametrize("M,N,K", [(1, 700, 6144), (1, 2000, 32768), (20, 700, 32768), (20, 3000, 8192), (64, 700, 32768), (200, 130, 32768),
                                   (300, 2500, 8000), (1000, 4096, 1024)])
@pytest.mark.parametrize("block", [16, 32])
def test_sums_that_fp32_holds_are_exact(M, N, K, block):
    """Scales of 1: every product is a multiple of 1/4, and every partial sum has less than 24 bits."""
    import torch
    g = gen(M + N + K)
    xc = torch.randint(0, 16, (M, K), device="cuda", generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 16, (1, N, K), device="cuda", generator=g, dtype=torch.uint8)
    one = 0x38 if block == 16 else 127
    xs, ws = (torch.full(shape, one, dtype=torch.uint8, device="cuda") for shape in ((M, -(-K // block)), (1, N, -(-K // block))))
    weight = mx.Fp4Weight(pack(wc), ws.view(torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu), cols=K)
    got = matmul(pack(xc), scale_rows(xs, K, block), None, weight, torch.float32)
    X, W = values(xc, xs, block), values(wc, ws, block)[0]
    assert 36 * K < 2 ** 22  # of any order
    assert torch.equal(got.double(), X @ W.T)


# whole stages of 256 columns, whole and ragged pieces of sixteen
@pytest.mark.parametrize("rows,cols", [(8200, 2048), (20011, 704), (20011, 701), (70001, 31)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_more_than_one_pass(rows, cols, block, dtype):
    """Each thread goes on to further pieces, rows and columns on."""
    import torch
    x = torch.randn(rows, cols, device="cuda", generator=gen(cols)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x *= torch.exp2((torch.arange(rows, device="cuda") % 23 - 11).float())[:, None].to(x.dtype)
    t = torch.full((1,), 0.0371, device="cuda") if block == 16 else None
    q, s = mx.fp4_empty(rows, cols, block)
    q.fill_(0xCC)
    s.view(torch.uint8).fill_(0xEE)
    mx.fp4_quantize(x, q, s, tensor_scale=t)
    codes, scales = ref_quantize(x.double(), block, t.double() if block == 16 else None)
    assert torch.equal(unpack(q, cols).long(), codes)
    assert torch.equal(plain_scales(s, cols, block), scales)


@pytest.mark.parametrize("cols", [32768, 32750])
def test_quantise_rows_past_32_bits(cols):
    """More than 2^33 values and 2^32 bytes of codes."""
    import torch
    rows = 270000
    one = torch.randn(1000, cols, device="cuda", generator=gen(1)).bfloat16()
    x = one.repeat(270, 1)
    q, s = mx.fp4_empty(rows, cols, 32)
    mx.fp4_quantize(x, q, s)
    codes, scales = ref_quantize(one[:8].double(), 32, None)
    s = s.view(torch.uint8)
    assert torch.equal(unpack(q[:8], cols).long(), codes) and torch.equal(plain_scales(s[:, :8], cols, 32), scales)
    for k in (1, 131, 269):
        at = slice(1000 * k, 1000 * k + 1000)
        assert torch.equal(q[at], q[:1000]) and torch.equal(s[:, at], s[:, :1000])
