"""Routing, the RMS norm and the experts' products one after another, as a decoder's block calls them.

Each stage is compared with its definition on what the stage before it left, so each has its own tolerance: routing and
quantised values exactly, products as in their own tests."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_fp4 import check_product, operands, random_scales, ref_quantize, pack, values
from tests.test_gpu_route_logits import check as check_route
from tests.test_gpu_rmsnorm import check as check_norm, reference as norm_reference

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def fp8_weight(n, rows, cols, seed):
    import torch
    g = gen(seed)
    w = (torch.randn(n, rows, cols, device="cuda", generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand(n, -(-rows // 128), -(-cols // 128), device="cuda", generator=g) + 0.5) / (100 * cols ** 0.5)
    return w, s


def ws_of(n):
    import torch
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mx.workspace_init(ws, n, stream=torch.cuda.current_stream())
    return ws


@pytest.mark.parametrize("T", [1, 30, 200])
@pytest.mark.parametrize("captured", [False, True])
def test_norm_router_and_fp8_layer(T, captured):
    """x + residual, normed into bf16 and e4m3 rows; logits by an FP8 product of those; routing in groups; the FP8 layer."""
    import torch
    D, I, E, K = 512, 256, 32, 4
    x, res = (torch.randn(T, D, device="cuda", generator=gen(i)).bfloat16() for i in (1, 2))
    w = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen(3))).bfloat16()
    head = mx.Fp8Weight(*(t[0] for t in fp8_weight(1, E, D, 4)))
    layer = mx.Fp8Layer(fp8_weight(E, I, D, 5), fp8_weight(E, I, D, 6), fp8_weight(E, D, I, 7), top_k=K, activation=mx.MX_SILU)
    router = mx.Router(E, K, score=mx.MX_SIGMOID, bias=0.1 * torch.randn(E, device="cuda", generator=gen(8)), n_groups=4,
                       topk_groups=2, group_best=2, scale=2.5)
    h, q = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, D, device="cuda").to(torch.float8_e4m3fn)
    s = torch.empty(D // 128, T, device="cuda").t()
    logits = torch.empty(T, E, device="cuda")
    idx, tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    out, total = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), res.clone()
    work = [ws_of(mx.fp8_matmul_workspace_bytes(head, T)), ws_of(mx.fp8_moe_workspace_bytes(layer, T))]

    def run():
        mx.fp8_rmsnorm(x, w, residual=total, residual_out=total, out=h, q=q, scales=s)
        mx.fp8_matmul(q, s, head, logits, work[0])
        mx.route_logits(logits, router, idx, tw)
        mx.fp8_moe_forward(h, idx, tw, layer, out, work[1], residual=total)

    run()
    if captured:
        total.copy_(res)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        total.copy_(res)
        for t in (h, logits, out):
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    check_norm({"sum": total, "out": h, "q": q, "scales": s}, norm_reference(x, w, res, 1e-6, 0.0, torch.bfloat16, False))
    check_route(logits, K, (idx, tw), score=mx.MX_SIGMOID, bias=router.bias, n_groups=4, topk_groups=2, group_best=2, scale=2.5)
    again = torch.empty_like(out)
    mx.fp8_moe_forward(h, idx, tw, layer, again, work[1], residual=total)
    assert torch.equal(out, again) and out.isfinite().all()


@pytest.mark.parametrize("T", [1, 9, 150])
@pytest.mark.parametrize("block", [16, 32])
def test_router_and_grouped_4_bit_products(T, block):
    """Slots grouped by expert, their rows quantised, gate and up by grouped products, and back to their tokens."""
    import torch
    D, I, E, K = 512, 200, 12, 3
    x = torch.randn(T, D, device="cuda", generator=gen(1)).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen(2))
    router = mx.Router(E, K)
    idx, tw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    counts, offsets, perm = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, T * K))
    mx.route_logits(logits, router, idx, tw, counts, offsets, perm, ws=ws_of(mx.route_logits_workspace_bytes(router, T)))
    check_route(logits, K, (idx, tw, counts, offsets, perm))
    rows = x[torch.div(perm, K, rounding_mode="floor").long()]
    n = T * K
    t = torch.full((1,), 5.0 / (6 * 448), device="cuda") if block == 16 else None
    q, s = mx.fp4_empty(n, D, block)
    mx.fp4_quantize(rows, q, s, tensor_scale=t)
    _, _, _, weight, _, W = operands(2, I, D, block, E=E)
    out = torch.empty(n, I, device="cuda")
    ws = ws_of(mx.fp4_matmul_workspace_bytes(weight, n))
    mx.fp4_grouped_matmul(q, s, offsets, weight, out, ws, tensor_scale=t)
    mx.workspace_check(ws, torch.cuda.current_stream())
    codes, scales = ref_quantize(rows.double(), block, t.double() if block == 16 else None)
    X = values(codes, scales, block, t.double() if block == 16 else None)
    at = offsets.tolist()
    assert at[0] == 0 and at[-1] == n
    for e in range(E):
        if at[e + 1] > at[e]:
            check_product(out[at[e]:at[e + 1]], X[at[e]:at[e + 1]], W[e], D)
    back = torch.empty_like(out)
    back[perm.long()] = out
    for k in range(T * K):  # slot k is its token's row by its expert's matrix
        e = int(idx.flatten()[k])
        pos = int((perm == k).nonzero()[0])
        assert at[e] <= pos < at[e + 1] and torch.equal(back[k], out[pos])


def test_a_layer_of_4_bit_experts():
    """gate, up and down of one expert's rows with the hidden rows quantised again, against the same steps in fp64."""
    import torch
    M, D, I = 70, 512, 384
    x = torch.randn(M, D, device="cuda", generator=gen(1)).bfloat16()
    q, s = mx.fp4_empty(M, D, 32)
    mx.fp4_quantize(x, q, s)
    mats = []
    for n, k, seed in ((I, D, 2), (I, D, 3), (D, I, 4)):
        c = torch.randint(0, 16, (n, k), device="cuda", generator=gen(seed), dtype=torch.uint8)
        sc = random_scales((n, k // 32), 32, seed) - 6
        mats.append((mx.Fp4Weight(pack(c), sc.view(torch.float8_e8m0fnu)), values(c, sc, 32)))
    g, u = torch.empty(M, I, device="cuda"), torch.empty(M, I, device="cuda")
    ws = ws_of(mx.fp4_matmul_workspace_bytes(mats[0][0], M))
    mx.fp4_matmul(q, s, mats[0][0], g, ws)
    mx.fp4_matmul(q, s, mats[1][0], u, ws)
    h = torch.nn.functional.silu(g) * u
    hq, hs = mx.fp4_empty(M, I, 32)
    mx.fp4_quantize(h, hq, hs)
    out = torch.empty(M, D, device="cuda", dtype=torch.bfloat16)
    mx.fp4_matmul(hq, hs, mats[2][0], out, ws)
    codes, scales = ref_quantize(x.double(), 32, None)
    X = values(codes, scales, 32)
    check_product(g, X, mats[0][1], D)
    check_product(u, X, mats[1][1], D)
    codes, scales = ref_quantize(h.double(), 32, None)
    check_product(out, values(codes, scales, 32), mats[2][1], I)
