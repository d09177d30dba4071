"""Microscaled 4-bit operators on the GPU against plain fp64 implementations.

The quantiser is compared bit for bit: every step of its definition is a correctly rounded fp32 operation.  A product:
the tensor core multiplies e2m1 numbers and block scales exactly and adds them in fp32, and may truncate where fp32
rounds: at most 2 (K + 8) 2^-24 sum |terms| for K columns, the tensors' two factors and a split over eight CTAs
included.  A bf16 output adds half a step, 2^-8 of its value."""
from __future__ import annotations

import math

import pytest

import expert_ffn_gb300 as mx

pytestmark = pytest.mark.gpu

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TINY = 2.0 ** -126


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def up(n, m):
    return -(-n // m) * m


# ------------------------------------------------- the definitions, in fp64

def e4m3_bits(v):
    """Codes of fp64 values 0 <= v to the nearest e4m3 number, at most 448."""
    import torch
    v = v.clamp(max=448.0)  # (an fp32 product that overflowed is infinite)
    step = torch.exp2(torch.floor(torch.log2(v.clamp_min(2.0 ** -6))) - 3)
    r = (torch.round(v / step) * step).clamp(max=448.0)
    return r.float().to(torch.float8_e4m3fn)


def e2m1_codes(v):
    """Codes of fp64 values to the nearest e2m1 number, ties to even, at most 6; the sign kept."""
    import torch
    g = v.abs()
    step = torch.where(g < 2, 0.5, torch.where(g < 4, 1.0, 2.0))
    r = (torch.round(g / step) * step).clamp(max=6.0)
    code = torch.searchsorted(torch.tensor(GRID, dtype=torch.float64, device=v.device), r.contiguous())
    return code + 8 * torch.signbit(v)


def ref_quantize(x, block, t):
    """(codes, scale bytes) of fp64 rows that hold fp32 numbers."""
    import torch
    rows, cols = x.shape
    nb = -(-cols // block)
    codes = torch.zeros(rows, nb * block, dtype=torch.long, device=x.device)
    scales = torch.zeros(rows, nb, dtype=torch.uint8, device=x.device)
    f = lambda v: v.float().double()  # noqa: E731
    for b in range(nb):
        p = x[:, b * block:(b + 1) * block]
        bad = ~p.isfinite().all(1)
        p = torch.where(bad[:, None], torch.zeros_like(p), p)
        a = p.abs().amax(1)
        if block == 16:
            e = e4m3_bits(f(a * f(1.0 / f(6.0 * t))))
            s = f(e.double() * t)
            v = torch.where((s >= TINY)[:, None], f(p * f(1.0 / s.clamp_min(TINY))[:, None]), p * 0.0)
            byte = torch.where(bad, 0x7F, e.view(torch.uint8).long())
        else:
            k = torch.ceil(torch.log2(a.clamp_min(1e-300) / 6.0) - 1e-9).clamp(-127, 127)  # near the border: by the test
            k = torch.where(6.0 * torch.exp2(k) < a, k + 1, k)
            k = torch.where(6.0 * torch.exp2(k - 1) >= a, k - 1, k).clamp(-127, 127)
            v = p / torch.exp2(k)[:, None]
            byte = torch.where(bad, 0xFF, (k + 127).long())
        codes[:, b * block:b * block + p.shape[1]] = torch.where(bad[:, None], 0, e2m1_codes(v))
        scales[:, b] = byte.to(torch.uint8)
    return codes[:, :cols], scales


def scale_value(byte, block):
    import torch
    if block == 16:
        return byte.view(torch.float8_e4m3fn).double()
    return torch.where(byte == 255, math.nan, torch.exp2(byte.double() - 127))


def values(codes, scales, block, t=None):
    """codes [.., cols], scale bytes [.., blocks] to fp64."""
    import torch
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=codes.device)
    s = scale_value(scales, block).repeat_interleave(block, -1)[..., :codes.shape[-1]]
    v = grid[codes.long()] * s
    return v if t is None else v * t


# ----------------------------------------------------------------- buffers

def unpack(q, cols):
    """Codes of packed rows."""
    import torch
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., :cols]


def pack(codes, pitch=0):
    """Packed rows at multiples of 16 bytes (and `pitch` more)."""
    import torch
    cols = codes.shape[-1]
    c = torch.nn.functional.pad(codes.to(torch.uint8), (0, cols % 2))
    n = (cols + 1) // 2
    q = torch.full((*codes.shape[:-1], up(n, 16) + 16 * pitch), 0xAB, dtype=torch.uint8, device=codes.device)[..., :n]
    return q.copy_(c[..., 0::2] | c[..., 1::2] << 4)


def scale_rows(scales, cols, block):
    """[rows, blocks] bytes in the operators' layout, and back."""
    import torch
    per, stages = 256 // block, -(-cols // 256)
    s = torch.nn.functional.pad(scales, (0, stages * per - scales.shape[1])).view(scales.shape[0], stages, per)
    return s.permute(1, 0, 2).contiguous().view(torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu)


def plain_scales(s, cols, block):
    import torch
    return s.view(torch.uint8).permute(1, 0, 2).flatten(1)[:, :-(-cols // block)].contiguous()


def random_scales(shape, block, seed, spread=2):
    import torch
    g = gen(seed)
    if block == 16:
        return (torch.rand(shape, device="cuda", generator=g) * 400 + 1).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.randint(127 - spread, 128 + spread, shape, device="cuda", generator=g, dtype=torch.uint8)


def operands(M, N, K, block, E=1, factors=True, seed=0, pitch=0):
    """Random rows and matrices, as the operators take them and in fp64."""
    import torch
    g = gen(seed + M + N + K)
    xc = torch.randint(0, 16, (M, K), device="cuda", generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 16, (E, N, K), device="cuda", generator=g, dtype=torch.uint8)
    xs, ws = random_scales((M, -(-K // block)), block, seed + 1), random_scales((E, N, -(-K // block)), block, seed + 2)
    with_t = factors and block == 16
    tx = torch.full((1,), 0.013, device="cuda") if with_t else None
    tw = torch.rand(E, device="cuda", generator=g) + 0.5 if with_t else None
    kind = torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu
    q, w = pack(xc, pitch), torch.empty(E, N, up((K + 1) // 2, 16) + 16 * pitch, dtype=torch.uint8, device="cuda")
    w = w[..., :(K + 1) // 2].copy_(pack(wc))
    weight = mx.Fp4Weight(w, ws.view(kind), tw, cols=K)
    X = values(xc, xs, block, tx.double() if with_t else None)
    W = values(wc, ws, block, tw.double().view(-1, 1, 1) if with_t else None)
    return q, scale_rows(xs, K, block), tx, weight, X, W


def workspace(weight, rows):
    import torch
    n = mx.fp4_matmul_workspace_bytes(weight, rows)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mx.workspace_init(ws, n, stream=torch.cuda.current_stream())
    return ws


def check_product(out, X, W, K):
    import torch
    exact, mag = X @ W.T, X.abs() @ W.abs().T
    tol = 2 * (K + 8) * 2.0 ** -24 * mag
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * exact.abs()
    bad = ~((out.double() - exact).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((out.double() - exact).abs() / tol.clamp_min(1e-300)).nan_to_num(9e9).max()))


def matmul(q, s, tx, weight, dtype, pitch=0, shift=0):
    import torch
    M, N = q.shape[0], weight.rows
    ws = workspace(weight, M)
    flat = torch.full((M * (N + pitch) + shift,), -7.0, dtype=dtype, device="cuda")
    wide = flat[shift:].view(M, N + pitch)
    mx.fp4_matmul(q, s, weight, wide[:, :N], ws, tensor_scale=tx)
    mx.workspace_check(ws, torch.cuda.current_stream())
    assert (wide[:, N:] == -7.0).all() and (flat[:shift] == -7.0).all()
    return wide[:, :N]


# ------------------------------------------------------------------ quantise

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 15), (3, 16), (2, 17), (5, 31), (4, 33), (2, 255), (7, 256), (3, 257), (1, 2816),
                                       (40, 1037), (33, 2112), (700, 640), (2, 8200)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise(rows, cols, block, dtype):
    import torch
    x = torch.randn(rows, cols, device="cuda", generator=gen(cols)) * torch.exp(2 * torch.randn(rows, 1, device="cuda", generator=gen(1)))
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = torch.full((1,), 0.0371, device="cuda") if block == 16 else None
    q, s = mx.fp4_empty(rows, cols, block)
    whole = torch.as_strided(q, (rows, q.stride(0) if rows > 1 else q.shape[1]), (q.stride(0) if rows > 1 else q.shape[1], 1))
    whole.fill_(0xCC)
    s.view(torch.uint8).fill_(0xEE)
    mx.fp4_quantize(x, q, s, tensor_scale=t)
    codes, scales = ref_quantize(x.double(), block, t.double() if block == 16 else None)
    assert torch.equal(unpack(q, cols).long(), codes)
    assert torch.equal(plain_scales(s, cols, block), scales)
    if cols % 2:
        assert not (q[:, -1] >> 4).any()  # the spare nibble
    assert (whole[:, q.shape[1]:] == 0xCC).all()
    assert not s.view(torch.uint8).permute(1, 0, 2).flatten(1)[:, -(-cols // block):].any()  # behind the last block


@pytest.mark.parametrize("block", [16, 32])
def test_quantise_ties_borders_and_special_values(block):
    """Values on and beside every border, zeros of both signs, subnormals, the largest numbers, NaN and infinities."""
    import torch
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0, 5.5], device="cuda")
    rows = [mid, -mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1), mid * 2.0 ** -20, mid * 2.0 ** 100,
            mid * 2.0 ** -126, mid * 2.0 ** -149, torch.zeros(16, device="cuda"), -torch.zeros(16, device="cuda")]
    for top in (6.0, 6.0000004, 5.9999995, 1.5, 1.5000001, 3.4e38, 1.1754944e-38, 1e-45, 448.0 * 6, 500.0 * 6):
        rows.append(torch.where(torch.arange(16, device="cuda") == 3, top, mid * 0.0))
    for bad in (math.nan, math.inf, -math.inf):
        rows.append(torch.where(torch.arange(16, device="cuda") == 9, bad, mid))
    x = torch.stack(rows).repeat(1, 3)
    x[:, 16:32] = 1.0  # (a block of its own beside each)
    for t in ([1.0, 0.01, 2.0 ** -100, 3e30] if block == 16 else [None]):
        f = None if t is None else torch.full((1,), t, device="cuda")
        q, s = mx.fp4_empty(x.shape[0], 48, block)
        mx.fp4_quantize(x, q, s, tensor_scale=f)
        codes, scales = ref_quantize(x.double(), block, None if t is None else f.double())
        bad = codes != unpack(q, 48).long()
        assert not bad.any(), (t, bad.nonzero()[:5])
        assert torch.equal(plain_scales(s, 48, block), scales)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,shift", [(0, 1), (3, 0), (8, 4)])
def test_quantise_of_slices(dtype, pitch, shift):
    import torch
    rows, cols = 21, 1000
    flat = torch.randn((rows + 1) * (cols + pitch), device="cuda", generator=gen(3)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x = flat[shift:shift + rows * (cols + pitch)].view(rows, cols + pitch)[:, :cols]
    q = torch.full((rows, 501), 0xCC, dtype=torch.uint8, device="cuda")[:, :500]  # rows at odd addresses
    _, s = mx.fp4_empty(rows, cols, 32)
    mx.fp4_quantize(x, q, s)
    codes, scales = ref_quantize(x.double(), 32, None)
    assert torch.equal(unpack(q, cols).long(), codes) and torch.equal(plain_scales(s, cols, 32), scales)


def test_quantise_without_a_factor_is_one():
    import torch
    x = torch.randn(5, 100, device="cuda", generator=gen(4))
    a, b = mx.fp4_empty(5, 100, 16), mx.fp4_empty(5, 100, 16)
    mx.fp4_quantize(x, *a)
    mx.fp4_quantize(x, *b, tensor_scale=torch.ones(1, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.uint8), b[1].view(torch.uint8))


# ------------------------------------------------------------------- products

# one row by integers and by the tensor cores; every token tile; whole, and in four and eight
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 100, 31), (1, 704, 2816), (1, 2112, 2817), (1, 300, 6144), (1, 4096, 7000),
                                   (1, 129, 9000), (2, 5, 3), (3, 129, 64), (5, 128, 257), (8, 2112, 1000), (16, 64, 2048), (17, 700, 333),
                                   (32, 2816, 512), (33, 1000, 4096), (64, 300, 2000), (65, 1024, 1024), (100, 4096, 300), (128, 512, 777),
                                   (200, 5001, 1037), (224, 130, 256), (225, 2000, 255), (449, 1500, 640), (1000, 4096, 700),
                                   (20, 131, 8000), (40, 2047, 5000), (64, 700, 4500), (30, 3000, 4096)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_product(M, N, K, block, out):
    import torch
    q, s, tx, weight, X, W = operands(M, N, K, block, factors=M % 2 == 0 or M == 1)
    got = matmul(q, s, tx, weight, torch.bfloat16 if out == "bf16" else torch.float32)
    check_product(got, X, W[0], K)


@pytest.mark.parametrize("M", [1, 20, 70, 300])
@pytest.mark.parametrize("out,pitch,shift", [("bf16", 8, 0), ("bf16", 1, 0), ("bf16", 0, 1), ("f32", 3, 0), ("f32", 4, 1), ("bf16", 24, 8)])
def test_product_into_slices(M, out, pitch, shift):
    """Output rows at any address; operand rows further apart than they need be; nothing beside the output is written."""
    import torch
    q, s, tx, weight, X, W = operands(M, 264, 600, 16, pitch=2)
    got = matmul(q, s, tx, weight, torch.bfloat16 if out == "bf16" else torch.float32, pitch, shift)
    check_product(got, X, W[0], 600)


@pytest.mark.parametrize("M,N,K", [(1, 300, 500), (30, 300, 2000), (300, 300, 500)])
@pytest.mark.parametrize("block", [16, 32])
def test_what_lies_behind_the_columns_does_not_count(M, N, K, block):
    """Bytes behind a row's last are any; of an odd last column's byte the weights' spare nibble is zero."""
    import torch
    q, s, tx, weight, X, W = operands(M, N, K + 1, block)
    del X, W
    q, s, tx, weight, X, W = operands(M, N, K, block)
    torch.as_strided(q, (M, q.stride(0)), q.stride())[:, (K + 1) // 2:].fill_(0x77)
    w = weight.w
    torch.as_strided(w, (1, N, w.stride(1)), w.stride())[:, :, (K + 1) // 2:].fill_(0x77)
    check_product(matmul(q, s, tx, weight, torch.float32), X, W[0], K)


@pytest.mark.parametrize("M,N,K", [(1, 300, 2000), (40, 300, 2000), (300, 2048, 800)])
@pytest.mark.parametrize("block", [16, 32])
def test_nan_scales_stay_in_their_row_and_column(M, N, K, block):
    import torch
    q, s, tx, weight, X, W = operands(M, N, K, block)
    clean = matmul(q, s, tx, weight, torch.float32).clone()
    r = M // 2
    s.view(torch.uint8)[K // 512, r, 3] = 0x7F if block == 16 else 0xFF
    got = matmul(q, s, tx, weight, torch.float32)
    assert got[r].isnan().all()
    rest = torch.arange(M, device="cuda") != r
    assert torch.equal(got[rest], clean[rest])
    q, s, tx, weight, X, W = operands(M, N, K, block)
    scales = random_scales((1, N, -(-K // block)), block, 2)
    scales[0, 77, 5] = 0x7F if block == 16 else 0xFF
    weight = mx.Fp4Weight(weight.w, scales.view(torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu), weight.tensor_scale, cols=K)
    got = matmul(q, s, tx, weight, torch.float32)
    cols = torch.arange(N, device="cuda") != 77
    assert got[:, 77].isnan().all() and torch.equal(got[:, cols], clean[:, cols])


@pytest.mark.parametrize("M,N,K", [(40, 300, 2000), (40, 300, 4096), (40, 2001, 5000), (200, 300, 500), (600, 2048, 800)])
def test_a_row_does_not_depend_on_the_others(M, N, K):
    import torch
    q, s, tx, weight, X, W = operands(M, N, K, 16)
    a = matmul(q, s, tx, weight, torch.float32).clone()
    keep = torch.arange(M, device="cuda") % 3 == 0
    other = operands(M, N, K, 16, seed=9)
    q[~keep] = other[0][~keep]
    s.view(torch.uint8)[:, ~keep] = other[1].view(torch.uint8)[:, ~keep]
    b = matmul(q, s, tx, weight, torch.float32)
    assert torch.equal(a[keep], b[keep]) and not torch.equal(a, b)


def test_extreme_e8m0_scales():
    import torch
    for M in (1, 20):
        q, s, tx, weight, X, W = operands(M, 128, 256, 32)
        s.view(torch.uint8).fill_(127 + 90)
        ws = torch.full((1, 128, 8), 127 - 95, dtype=torch.uint8, device="cuda")
        weight = mx.Fp4Weight(weight.w, ws.view(torch.float8_e8m0fnu))
        got = matmul(q, s, None, weight, torch.float32)
        x = values(unpack(q, 256), torch.full((M, 8), 217, dtype=torch.uint8, device="cuda"), 32)
        check_product(got, x, values(unpack(weight.w, 256), ws, 32)[0], 256)


# -------------------------------------------------------------------- grouped

def grouped(q, s, tx, weight, offsets, dtype, ws=None, out=None):
    import torch
    M, N = q.shape[0], weight.rows
    ws = workspace(weight, M) if ws is None else ws
    out = torch.full((M, N), -7.0, dtype=dtype, device="cuda") if out is None else out
    mx.fp4_grouped_matmul(q, s, offsets, weight, out, ws, tensor_scale=tx)
    mx.workspace_check(ws, torch.cuda.current_stream())
    return out


def check_grouped(out, offsets, X, W, K):
    M = X.shape[0]
    at = [min(max(int(o), 0), M) for o in offsets.tolist()]
    seen = [False] * M
    for e in range(len(at) - 1):
        if at[e + 1] > at[e]:
            check_product(out[at[e]:at[e + 1]], X[at[e]:at[e + 1]], W[e], K)
            seen[at[e]:at[e + 1]] = [True] * (at[e + 1] - at[e])
    for r in (i for i, v in enumerate(seen) if not v):
        assert (out[r] == -7.0).all(), r


# average rows of a matrix: below one, a few, tens, hundreds; every token tile
@pytest.mark.parametrize("rows,E,N,K", [(1, 1, 5, 7), (5, 8, 128, 100), (40, 30, 300, 512), (100, 8, 260, 333), (300, 10, 704, 640),
                                        (500, 4, 129, 1000), (900, 3, 1000, 300), (2000, 60, 200, 256)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_grouped(rows, E, N, K, block, out):
    import torch
    q, s, tx, weight, X, W = operands(rows + 3, N, K, block, E=E)
    which = torch.randint(0, E, (rows,), device="cuda", generator=gen(rows))
    which = torch.where(torch.rand(rows, device="cuda", generator=gen(1)) < 0.3, 0, which)  # one has more
    counts = torch.bincount(which, minlength=E)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    got = grouped(q, s, tx, weight, offsets, torch.bfloat16 if out == "bf16" else torch.float32)
    check_grouped(got, offsets, X, W, K)


@pytest.mark.parametrize("offsets", [[0, 0, 0, 0, 0], [0, 50, 50, 50, 50], [0, 0, 0, 0, 50], [7, 9, 9, 30, 41], [0, 16, 32, 48, 50],
                                     [-5, 3, 20, 900, 1000], [10, 30, 20, 40, 35], [50, 50, 50, 50, 50], [49, 50, 51, 52, 53]])
def test_grouped_offsets(offsets):
    """Empty groups, rows in front of the first and behind the last, entries outside, decreasing pairs."""
    import torch
    q, s, tx, weight, X, W = operands(50, 200, 300, 16, E=4)
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = grouped(q, s, tx, weight, o, torch.float32)
    at = [min(max(v, 0), 50) for v in offsets]
    if offsets == [10, 30, 20, 40, 35]:  # rows 20 to 30 belong to two groups: either product
        check_product(out[10:20], X[10:20], W[0], 300)
        check_product(out[30:40], X[30:40], W[2], 300)
        assert (out[:10] == -7.0).all() and (out[40:] == -7.0).all()
    else:
        check_grouped(out, torch.tensor(at), X, W, 300)


def test_grouped_512_matrices():
    import torch
    E = 512
    q, s, tx, weight, X, W = operands(700, 40, 64, 32, E=E)
    counts = torch.bincount(torch.randint(0, E, (700,), device="cuda", generator=gen(5)), minlength=E)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    check_grouped(grouped(q, s, tx, weight, offsets, torch.float32), offsets, X, W, 64)


# ----------------------------------------------------- streams, graphs, sizes

@pytest.mark.parametrize("M,N,K", [(1, 704, 2816), (40, 704, 2816), (300, 704, 512)])
def test_quantise_and_product_captured_and_replayed(M, N, K):
    """One after another on a stream of their own, captured with two products that share a workspace."""
    import torch
    _, _, _, weight, _, W = operands(2, N, K, 16)
    x = torch.randn(M, K, device="cuda", generator=gen(1)).bfloat16()
    t = torch.full((1,), 0.002, device="cuda")
    q, sc = mx.fp4_empty(M, K, 16)
    out, out2 = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    ws = workspace(weight, M)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def run():
        mx.fp4_quantize(x, q, sc, tensor_scale=t)
        mx.fp4_matmul(q, sc, weight, out, ws, tensor_scale=t)
        mx.fp4_matmul(q, sc, weight, out2, ws, tensor_scale=t)

    with torch.cuda.stream(s):
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run()
    for seed in (2, 3):
        x.copy_(torch.randn(M, K, device="cuda", generator=gen(seed)))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        codes, scales = ref_quantize(x.double(), 16, t.double())
        check_product(out, values(codes, scales, 16, t.double()), W[0], K)
        assert torch.equal(out, out2)


def test_two_products_at_once():
    """Two streams, a workspace each."""
    import torch
    a = operands(300, 2048, 4096, 16)
    b = operands(20, 3000, 4096, 32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(300, 2048, device="cuda"), torch.empty(20, 3000, device="cuda")]
    wss = [workspace(p[3], p[0].shape[0]) for p in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, o, w, s in zip((a, b), outs, wss, streams):
            with torch.cuda.stream(s):
                mx.fp4_matmul(p[0], p[1], p[3], o, w, tensor_scale=p[2])
    torch.cuda.synchronize()
    for p, o in zip((a, b), outs):
        check_product(o, p[4], p[5][0], 4096)


def test_rows_past_32_bits():
    """More than 2^31 output elements and 2^32 bytes of codes."""
    import torch
    M, N, K = 270000, 8192, 32768
    _, _, _, weight, _, W = operands(2, N, K, 32)
    one = torch.randint(0, 256, (1000, K // 2), device="cuda", generator=gen(1), dtype=torch.uint8)
    q = one.repeat(270, 1)
    s1 = random_scales((1000, K // 32), 32, 3)
    s = scale_rows(s1.repeat(270, 1), K, 32)
    out = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    ws = workspace(weight, M)
    mx.fp4_matmul(q, s, weight, out, ws)
    mx.workspace_check(ws, torch.cuda.current_stream())
    X = values(unpack(one, K), s1, 32)
    check_product(out[-8:], X[-8:], W[0], K)
    assert torch.equal(out[-1000:], out[:1000]) and torch.equal(out[100000:101000], out[:1000])
