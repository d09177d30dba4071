"""FP8 block-scaled operators at the ends of their number ranges: magnitudes, non-finite weights, signs of zero,
borders of e4m3, and what a token's result may depend on.  Tolerances and definitions are those of test_gpu_fp8."""
from __future__ import annotations

import math

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_fp8 import (check_layer, gen, make_layer, make_rows, make_weight, nb, ref_expert, ref_quantize, routing,
                                rows_value, weight_value, workspace)

pytestmark = pytest.mark.gpu


# ------------------------------------------------- magnitudes of a layer's results

def scaled_layer(power, D=320, I=160, E=6, K=3, act=mx.MX_SILU, dtype="bf16", seed=210):
    """A layer whose down scales, and so its results, are 2^power times the usual ones."""
    layer, ws, _ = make_layer(E, D, I, 0, seed, K, act, dtype)
    ws[2][1].mul_(2.0 ** power)
    return layer, ws


@pytest.mark.parametrize("T", [1, 40, 90])
@pytest.mark.parametrize("power", [-100, 60, 114, 118])
def test_moe_results_of_any_magnitude(T, power):
    """Results near either end of the type's range keep their precision, whatever the number of tokens."""
    import torch
    layer, ws = scaled_layer(power)
    x = torch.randn(T, 320, device="cuda", generator=gen(211)).bfloat16()
    idx, wts = routing(T, 6, 3, 212)
    out = torch.empty_like(x)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    assert out.isfinite().all()
    check_layer(out, x, idx, wts, ws, None, mx.MX_SILU, 0.5, None, 3)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("T", [1, 40, 90])
def test_moe_non_finite_output_column_keeps_to_itself(T, value):
    """An output column that is NaN or infinite leaves its neighbours as they are, also when they are large."""
    import torch
    layer, ws = scaled_layer(40)
    x = torch.randn(T, 320, device="cuda", generator=gen(213)).bfloat16()
    idx, wts = routing(T, 6, 3, 214)
    out = torch.empty_like(x)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    w = ws[2][0].view(torch.uint8)
    if math.isnan(value):
        w[:, 70] = 0x7F  # e4m3's NaN in a row of every down matrix
        mx.fp8_moe_forward(x, idx, wts, layer, out, work)
        hit = slice(70, 71)
        assert out[:, hit].isnan().all()
    else:
        ws[2][1][:, 1] = math.inf  # scales of a block of rows: 128 columns of the results
        mx.fp8_moe_forward(x, idx, wts, layer, out, work)
        hit = slice(128, 256)
        assert not out[:, hit].isfinite().any()
    w[:, 70] = 0
    ws[2][1][:, 1] = 0.0
    out[:, hit] = 0.0
    clean = torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, clean, work)
    clean[:, hit] = 0.0
    if not math.isnan(value):
        clean[:, 70] = out[:, 70]  # (this row was set to zero for the second call alone)
    else:
        clean[:, 128:256] = out[:, 128:256]
    assert torch.equal(out, clean)


# -------------------------------------------------------- what a token depends on

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,I,S", [(2, 384, 160, 128), (8, 384, 160, 128), (20, 384, 160, 128), (40, 384, 160, 128),
                                     (64, 384, 160, 128), (90, 384, 160, 128), (64, 384, 64, 0), (20, 40000, 64, 0)])
def test_moe_non_finite_weights_reach_their_tokens_alone(T, D, I, S, dtype):
    """A NaN code, an infinite and a NaN scale of one expert's down matrix, a NaN code of its gate matrix: the tokens
    that chose the expert have it, the others keep their bits."""
    import torch
    E, K = 6, 3
    layer, ws, _ = make_layer(E, D, I, S, 220, K, mx.MX_SILU, dtype)
    x = torch.randn(T, D, device="cuda", generator=gen(221)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    # token t: experts t, t + 1, t + 2 (modulo 6), so that each expert is some tokens' and not others'
    idx = ((torch.arange(T, device="cuda")[:, None] + torch.arange(K, device="cuda")) % E).to(torch.int32)
    wts = torch.rand(T, K, device="cuda", generator=gen(222)) + 0.1
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    clean, out = torch.empty_like(x), torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, clean, work)
    assert clean.isfinite().all()

    def run(e, tensor, at, value, columns):
        old = tensor[at].clone()
        tensor[at] = value
        mx.fp8_moe_forward(x, idx, wts, layer, out, work)
        mx.workspace_check(work, torch.cuda.current_stream())
        tensor[at] = old
        chose = (idx == e).any(1)
        assert torch.equal(out[~chose], clean[~chose])
        assert not out[chose][:, columns].isfinite().any()
        rest = torch.ones(D, dtype=torch.bool, device="cuda")
        rest[columns] = False
        if columns != slice(None):
            assert torch.equal(out[chose][:, rest], clean[chose][:, rest])

    down = ws[2][0].view(torch.uint8)
    run(2, down, (2, 100, 7), 0x7F, slice(100, 101))
    run(5, down, (5, D - 1, I - 1), 0xFF, slice(D - 1, D))
    run(3, ws[2][1], (3, 1, 0), math.inf, slice(128, 256))
    run(1, ws[2][1], (1, 2, nb(I) - 1), math.nan, slice(256, 384))
    run(4, ws[0][0].view(torch.uint8), (4, 11, 300), 0x7F, slice(None))
    run(0, ws[1][1], (0, 0, 2), math.nan, slice(None))


@pytest.mark.parametrize("T,E,K,D,I,S", [
    (2, 16, 4, 2816, 384, 256), (5, 40, 2, 1040, 640, 0), (31, 32, 4, 2816, 704, 300), (20, 12, 3, 4096, 1024, 128),
    (60, 24, 2, 2816, 256, 64), (64, 9, 3, 640, 130, 130), (90, 16, 4, 640, 384, 128)])
def test_moe_bits_do_not_depend_on_the_other_tokens(T, E, K, D, I, S):
    """A token has the same bits whatever the other tokens hold and whichever experts they choose."""
    import torch
    layer, _, _ = make_layer(E, D, I, S, 230, K, mx.MX_SILU, "f32")
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    x, (idx, wts) = torch.randn(T, D, device="cuda", generator=gen(231)), routing(T, E, K, 232)
    first, out = torch.empty_like(x), torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, first, work)
    same = [0, T - 1] if T > 2 else [1]
    for i in range(4):
        y, (oidx, owts) = torch.randn(T, D, device="cuda", generator=gen(240 + i)), routing(T, E, K, 250 + i, skew=float(i))
        if i == 3:
            oidx.fill_(-1)  # (the others with no expert at all)
        for t in same:
            y[t], oidx[t], owts[t] = x[t], idx[t], wts[t]
        mx.fp8_moe_forward(y, oidx, owts, layer, out, work)
        mx.workspace_check(work, torch.cuda.current_stream())
        assert torch.equal(out[same], first[same])


def test_moe_thousands_of_hidden_blocks():
    """More hidden blocks to a CTA of down than its list has room for."""
    import torch
    T, E, K, D, I, S = 9, 2, 1, 128, 530000, 128
    layer, ws, sh = make_layer(E, D, I, S, 233, K, mx.MX_SILU, "f32")
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    x, (idx, wts) = torch.randn(T, D, device="cuda", generator=gen(234)), routing(T, E, K, 235)
    idx[0], idx[1] = 0, 1
    first, out = torch.empty_like(x), torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, first, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_layer(first, x, idx, wts, ws, sh, mx.MX_SILU, 0.5, None, K)
    idx[2:] = 1 - idx[2:]
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    assert torch.equal(out[:2], first[:2])


# ------------------------------------------------------------------ signs of zero

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch", [256, 259])
def test_quantize_keeps_the_sign_of_zero(dtype, pow2, pitch):
    """Byte for byte e4m3(x / s): a negative zero, and a negative value that rounds to zero, is 0x80 in a block of any
    magnitude, of zeros as well."""
    import torch
    x = torch.randn(40, pitch, device="cuda", generator=gen(260))[:, :256]
    x[:, ::3] = 0.0
    x[:, 1::3] *= torch.where(torch.rand(40, 85, device="cuda", generator=gen(261)) < 0.5, 1e-7, 1.0)
    x[:, 2::5] = -0.0
    x[5, :128] = -0.0
    x[6, :128], x[6, :64] = 0.0, -0.0
    x[7] *= 2.0 ** -128
    x[8] *= 2.0 ** -90
    x[9] *= 2.0 ** 110
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    q = torch.empty(40, 256, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(40, 2, device="cuda")
    mx.fp8_quantize(x, q, s, pow2=pow2)
    rq, rs = ref_quantize(x.double(), pow2)
    want = rq.float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(s.double(), rs)
    assert (want == 0x80).any() and (want == 0).any()
    assert torch.equal(q.view(torch.uint8), want)


# --------------------------------------------- hidden values on a border of e4m3

TIES = {17: 16, 19: 20, 21: 20, 23: 24, 25: 24, 27: 28, 29: 28, 31: 32}  # between two e4m3 numbers: the even one


@pytest.mark.parametrize("act", [mx.MX_SILU, mx.MX_GELU_TANH])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 40, 90])
@pytest.mark.parametrize("sigma", [262085 / 65536, 262080 / 65536])
def test_moe_hidden_values_are_quantised_by_division(T, dtype, act, sigma):
    """Hidden values that are exactly sigma times a number halfway between two e4m3 numbers, in a block whose scale is
    exactly sigma: their quotients lie on the border and go to the even number.  (The product with the rounded 1 /
    sigma lands beside it: above for the first sigma, below for the second, or the other way round.)"""
    import torch
    f8 = torch.float8_e4m3fn
    D = I = 128
    gate, up, down = (torch.zeros(1, 128, 128, device="cuda") for _ in range(3))
    up[0, :, 2] = 1.0
    gate[0, 0, 1] = 28.0  # 448: the block's largest
    want = torch.zeros(128, device="cuda")
    want[0] = 448.0
    for j, (tie, even) in enumerate(TIES.items()):
        gate[0, j + 1, 1], gate[0, j + 1, 2], want[j + 1] = 1.0, tie - 16.0, even
    down[0].fill_diagonal_(1.0)
    one = torch.ones(1, 1, 1, device="cuda")
    layer = mx.Fp8Layer((gate.to(f8), one * sigma), (up.to(f8), one), (down.to(f8), one), top_k=1,
                        act_dtype=mx.MX_BF16 if dtype == "bf16" else mx.MX_F32, activation=act)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.zeros(T, D, device="cuda", dtype=dt)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, 16.0, 1.0  # (quantised by the scale 1: themselves)
    out = torch.empty_like(x)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    mx.fp8_moe_forward(x, torch.zeros(T, 1, device="cuda", dtype=torch.int32), torch.ones(T, 1, device="cuda"), layer, out, work)
    assert torch.equal(out, (want * sigma).to(dt).expand(T, D))


@pytest.mark.parametrize("T", [1, 5, 40, 90])
@pytest.mark.parametrize("power", [-92, 105])
def test_moe_hidden_values_of_any_magnitude(T, power):
    """Hidden values beyond the range in which their quotients come from a reciprocal as they are."""
    import torch
    D, I, E, K = 320, 200, 6, 3
    layer, ws, _ = make_layer(E, D, I, 0, 265, K, mx.MX_GELU_TANH, "f32")
    ws[1][1].mul_(2.0 ** power)
    ws[2][1].mul_(2.0 ** -power)
    x = torch.randn(T, D, device="cuda", generator=gen(266))
    idx, wts = routing(T, E, K, 267)
    out = torch.empty_like(x)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_layer(out, x, idx, wts, ws, None, mx.MX_GELU_TANH, 0.5, None, K)


# ----------------------------------------------------- precision of fp32 products

@pytest.mark.parametrize("m,n,k", [(1, 2112, 2816), (8, 1000, 4096), (40, 1024, 2816), (64, 704, 4096), (500, 1024, 2816),
                                   (600, 2600, 1037)])
@pytest.mark.parametrize("grouped", [False, True])
def test_fp32_products_keep_fp32(m, n, k, grouped):
    """In the 2-norm.  Were each of a block's 128 sums truncated (a step of 2^-23) in the direction of the running sum,
    which grows like the square root of the terms, the block would be off by 2^-23 sum_i sqrt(i) / sqrt(128) = 2^-23 85
    = 2^-16.6 of its deviation; blocks add as independent, and their B sums in fp32 are off by half a step of at most the
    whole each, B 2^-24 <= 2^-18.9 for B <= 33.  Together below 2^-16 of the results' norm, a hundredth of what sums in
    bf16 (2^-8, or 2^-9.6 in the norm) would leave."""
    import torch
    q, s = make_rows(m, k, 270)
    w, ws = make_weight(1, n, k, 271)
    out = torch.empty(m, n, device="cuda")
    if grouped:
        offsets = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        mx.fp8_grouped_matmul(q, s, offsets, mx.Fp8Weight(w, ws), out, workspace(256))
    else:
        mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), out, workspace(256))
    exact = rows_value(q, s) @ weight_value(w[0], ws[0]).T
    assert (out.double() - exact).norm() <= 2.0 ** -16 * exact.norm()


# --------------------------------------------------------------------- one token

def test_moe_one_token_in_place_and_captured():
    """out may be x or the residual itself; a captured and replayed call follows its buffers' values."""
    import torch
    E, K, D, I, S = 16, 4, 1040, 256, 200
    layer, ws, sh = make_layer(E, D, I, S, 280, K, mx.MX_GELU_TANH, "bf16")
    x = torch.randn(1, D, device="cuda", generator=gen(281)).bfloat16()
    residual = torch.randn(1, D, device="cuda", generator=gen(282)).bfloat16()
    idx, wts = routing(1, E, K, 283)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, 1))
    out = torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, out, work, residual=residual)
    check_layer(out, x, idx, wts, ws, sh, mx.MX_GELU_TANH, 0.5, residual, K)
    for target in ("x", "residual"):
        a = {"x": x.clone(), "residual": residual.clone()}
        mx.fp8_moe_forward(a["x"], idx, wts, layer, a[target], work, residual=a["residual"])
        assert torch.equal(a[target], out)
    side, buf = torch.cuda.Stream(), torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mx.fp8_moe_forward(x, idx, wts, layer, buf, work, residual=residual)
            mx.fp8_moe_forward(buf, idx, wts, layer, buf, work, residual=buf)
    torch.cuda.synchronize()
    for seed in (284, 285):
        x.copy_(torch.randn(1, D, device="cuda", generator=gen(seed)))
        i2, w2 = routing(1, E, K, seed)
        idx.copy_(i2)
        wts.copy_(w2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        one, two = torch.empty_like(x), torch.empty_like(x)
        mx.fp8_moe_forward(x, idx, wts, layer, one, work, residual=residual)
        mx.fp8_moe_forward(one, idx, wts, layer, two, work, residual=one)
        assert torch.equal(buf, two)


@pytest.mark.parametrize("D,blocks,two", [(2816, 65, True), (4096, 72, True), (5120, 40, True), (5120, 80, False),
                                          (8192, 24, True), (8192, 56, False), (16384, 16, True), (16384, 56, False),
                                          (32768, 16, True), (32768, 40, False), (33024, 8, False)])
def test_moe_one_token_takes_two_launches_while_its_blocks_run_at_once(D, blocks, two):
    """The two launches leave the workspace's quantised token alone, the three write it.  Right either way."""
    import torch
    K = 4 if blocks % 4 == 0 else 5
    layer, ws, _ = make_layer(5, D, 128 * blocks // K, 0, 290, K, mx.MX_SILU, "bf16")
    x = torch.randn(1, D, device="cuda", generator=gen(291)).bfloat16()
    idx, wts = routing(1, 5, K, 292)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, 1))
    work[256:256 + D] = 0x7F
    out = torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    assert (work[256:256 + D] == 0x7F).all().item() == two
    check_layer(out, x, idx, wts, ws, None, mx.MX_SILU, 0.5, None, K)


# ------------------------------------------------------ rows held between launches

@pytest.mark.parametrize("T,E,K,D,I,S", [(403, 78, 1, 6, 1, 0), (323, 22, 5, 21, 1, 0), (361, 3, 1, 6, 5, 5),
                                         (490, 2, 2, 2, 129, 28), (200, 8, 4, 130, 40, 64)])
def test_moe_rows_of_many_bf16_tokens_keep_eleven_bits(T, E, K, D, I, S):
    """Above 64 tokens with bf16 activations an expert's row is rounded to 11 bits, half a step of 2^-11 of it, before
    the weighted sum: where rows cancel one another or the residual, that is what is left of the result."""
    import torch
    layer, ws, sh = make_layer(E, D, I, S, 300, K, mx.MX_SILU, "bf16")
    x = torch.randn(T, D, device="cuda", generator=gen(301)).bfloat16()
    residual = torch.randn(T, D, device="cuda", generator=gen(302)).bfloat16()
    idx, wts = routing(T, E, K, 303)
    out = torch.empty_like(x)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    mx.fp8_moe_forward(x, idx, wts, layer, out, work, residual=residual)
    xv = rows_value(*ref_quantize(x.double()))
    y, tol, mag = (torch.zeros_like(xv) for _ in range(3))
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            p, b = ref_expert(xv[t], *((w[0][e], w[1][e]) for w in ws), mx.MX_SILU)
            wt = wts[t, k].double()[:, None]
            y.index_add_(0, t, p * wt)
            tol.index_add_(0, t, b * wt.abs())
            mag.index_add_(0, t, (p * wt).abs())
    if sh:
        p, b = ref_expert(xv, *((w[0][0], w[1][0]) for w in sh), mx.MX_SILU)
        y, tol, mag = y + p, tol + b, mag + p.abs()
    exact = 0.5 * y + residual.double()
    # as check_layer, with 2^-11 of each row (and of its own error)
    tol = 0.5 * (tol * (1 + 2.0 ** -11) + (2.0 ** -11 + (K + 4) * 2.0 ** -23) * mag)
    tol = tol + 2.0 ** -22 * exact.abs() + 2.0 ** -23 * residual.double().abs() + 2.0 ** -8 * exact.abs()
    assert ((out.double() - exact).abs() <= tol).all()
