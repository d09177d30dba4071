"""Routing from logits on the GPU against its definition in fp64.

Indices, counts, offsets and permutations have to be equal: the operator orders as exact arithmetic does.  Weights:
expf is off by 2 ulp at most (4 half steps of 2^-24), the argument l - m by a half step of itself, a sum of up to 512
terms by 21 half steps (16 in a lane, 5 between lanes), and the divisions and products by one each."""
from __future__ import annotations

import math

import pytest

import expert_ffn_gb300 as mx

pytestmark = pytest.mark.gpu

INF = math.inf


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def first(c, k):
    """The k highest, ties to the lower index."""
    import torch
    return torch.sort(c, dim=-1, descending=True, stable=True)[1][:, :k]


def reference(logits, top_k, score, bias, n_groups, keep, best, renorm, scale):
    """(indices, weights, how far the largest used logit is above the chosen ones) in fp64."""
    import torch
    l = logits.double()
    l = torch.where(l.isnan(), -INF, l)
    T, E = l.shape
    m = l.amax(1, keepdim=True)
    if score == mx.MX_SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        z = torch.exp(torch.where(l == m, torch.zeros_like(l), l - m))
        s = z / z.sum(1, keepdim=True)
    c = l if bias is None else s + bias.double()
    c = torch.where(c.isnan(), -INF, c)
    if keep < n_groups:
        by = (s if bias is None and best == 2 else c).view(T, n_groups, -1)
        g = by.amax(-1) if best == 1 else torch.sort(by, -1, descending=True)[0][..., :2].sum(-1)
        g = torch.where(g.isnan(), -INF, g)
        open_ = torch.zeros(T, n_groups, dtype=torch.bool, device=l.device).scatter_(1, first(g, keep), True)
        rank = torch.where(open_.repeat_interleave(E // n_groups, 1), c, -INF)
        # (an expert of a closed run never comes before one of -inf in an open run)
        order = torch.sort(torch.where(open_.repeat_interleave(E // n_groups, 1), 0, 1), dim=1, stable=True)[1]
        idx = torch.gather(order, 1, first(torch.gather(rank, 1, order), top_k))
    else:
        idx = first(c, top_k)
    x = torch.gather(l, 1, idx)
    if renorm:
        if score == mx.MX_SIGMOID:
            w = torch.gather(s, 1, idx)
        else:
            top = x.amax(1, keepdim=True)
            w = torch.exp(torch.where(x == top, torch.zeros_like(x), x - top))
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    else:
        w = torch.gather(s, 1, idx)
    far = torch.where(x == m, torch.zeros_like(x), (m - x).abs())
    return idx, w * scale, far


def call(logits, top_k, group=True, ws=None, stream=None, **kw):
    import torch
    T, E = logits.shape
    a = dict(score=mx.MX_SOFTMAX, bias=None, n_groups=1, topk_groups=1, group_best=1, renormalise=True, scale=1.0)
    a.update(kw)
    r = mx.Router(E, top_k, **a)
    idx = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), -7.0, device="cuda")
    if not group:
        mx.route_logits(logits, r, idx, w, stream=stream)
        return idx, w
    if ws is None:
        n = mx.route_logits_workspace_bytes(r, T)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        mx.workspace_init(ws, n, stream=torch.cuda.current_stream())
    out = [torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (E, E + 1, T * top_k)]
    mx.route_logits(logits, r, idx, w, *out, ws=ws, stream=stream)
    return (idx, w, *out)


def check(logits, top_k, got, **kw):
    import torch
    a = dict(score=mx.MX_SOFTMAX, bias=None, n_groups=1, topk_groups=1, group_best=1, renormalise=True, scale=1.0)
    a.update(kw)
    idx, w, far = reference(logits, top_k, a["score"], a["bias"], a["n_groups"], a["topk_groups"], a["group_best"],
                            a["renormalise"], a["scale"])
    assert torch.equal(got[0].long(), idx)
    tol = 2.0 ** -24 * (64 + far.clamp_max(1000)) * w.abs() + 1e-37
    assert ((got[1].double() - w).abs() <= tol).all(), float(((got[1].double() - w).abs() / tol).max())
    if len(got) > 2:
        T, E = logits.shape
        flat = idx.flatten()
        counts = torch.bincount(flat, minlength=E)
        assert torch.equal(got[2].long(), counts)
        assert torch.equal(got[3].long(), torch.nn.functional.pad(counts.cumsum(0), (1, 0)))
        assert torch.equal(got[4].long(), torch.argsort(flat, stable=True))


def both(logits, top_k, **kw):
    check(logits, top_k, call(logits, top_k, **kw), **kw)


def make(T, E, seed, dtype="f32", spread=1.5):
    import torch
    x = spread * torch.randn(T, E, device="cuda", generator=gen(seed))
    return x.bfloat16() if dtype == "bf16" else x


def bias_of(E, seed):
    import torch
    return 0.1 * torch.randn(E, device="cuda", generator=gen(seed + 100))


# every lane width (P = 1 .. 16), whole and ragged
@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (8, 8), (31, 4), (32, 8), (33, 8), (60, 6), (64, 32), (128, 8), (160, 8),
                                 (250, 3), (256, 8), (256, 32), (300, 8), (512, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score,biased", [(mx.MX_SOFTMAX, False), (mx.MX_SOFTMAX, True), (mx.MX_SIGMOID, False),
                                          (mx.MX_SIGMOID, True)])
def test_choices_and_weights(E, K, dtype, score, biased):
    for T in (1, 9, 70):
        both(make(T, E, 3 * E + T, dtype), K, score=score, bias=bias_of(E, E) if biased else None, renormalise=T != 9,
             scale=2.5 if T == 9 else 1.0)


@pytest.mark.parametrize("E,groups,keep,K", [(16, 8, 3, 4), (64, 8, 4, 8), (96, 3, 2, 8), (60, 6, 2, 8), (72, 9, 4, 6),
                                             (160, 8, 3, 6), (256, 8, 4, 8), (256, 32, 5, 8), (480, 10, 3, 8), (512, 2, 1, 32),
                                             (26, 13, 12, 20)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score,biased", [(mx.MX_SOFTMAX, True), (mx.MX_SIGMOID, True), (mx.MX_SIGMOID, False),
                                          (mx.MX_SOFTMAX, False)])
def test_groups(E, groups, keep, K, best, score, biased):
    both(make(133, E, E + groups, "f32"), K, score=score, bias=bias_of(E, 7) if biased else None, n_groups=groups,
         topk_groups=keep, group_best=best, scale=2.0)


# one block, several, blocks of 32 tokens, joined blocks, blocks of more than 32 tokens
@pytest.mark.parametrize("T", [1, 7, 8, 9, 32, 33, 511, 2048, 2049, 4097, 16400, 120001])
@pytest.mark.parametrize("E,K", [(16, 3), (300, 2)])
def test_grouped_slots(T, E, K):
    both(make(T, E, T), K)


@pytest.mark.parametrize("K", [1, 8, 32])
def test_grouped_slots_of_full_choices(K):
    """Every token chooses every expert, or all choose the same."""
    import torch
    both(make(100, K, 1), K)
    x = torch.zeros(300, 64, device="cuda")
    x[:, 5:5 + K] = 3.0
    both(x, K)


def test_no_tokens():
    import torch
    idx, w, counts, offsets, perm = call(torch.zeros(0, 40, device="cuda"), 3)
    torch.cuda.synchronize()
    assert not counts.any() and not offsets.any()
    call(torch.zeros(0, 40, device="cuda"), 3, group=False)


@pytest.mark.parametrize("E", [8, 60, 256])
@pytest.mark.parametrize("score", [mx.MX_SOFTMAX, mx.MX_SIGMOID])
def test_equal_logits_go_to_the_lower_expert(E, score):
    import torch
    x = torch.randint(0, 3, (200, E), device="cuda", generator=gen(E)).float()
    x[:20] = 1.25
    x[20:30] = 0.0
    x[30:40] = torch.where(x[30:40] > 0, 0.0, -0.0)  # zeros of both signs are equal
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), -0.5, device="cuda")):
        both(x, 6, score=score, bias=bias)
        if E % 4 == 0:
            both(x, 4, score=score, bias=bias, n_groups=4, topk_groups=2, group_best=2 if E > 8 else 1)


@pytest.mark.parametrize("E,groups,best", [(64, 1, 1), (256, 8, 2), (60, 6, 2), (256, 8, 1)])
@pytest.mark.parametrize("score", [mx.MX_SOFTMAX, mx.MX_SIGMOID])
def test_scores_that_fp32_does_not_tell_apart(E, groups, best, score):
    """Biases that make many scores of a token equal but for roundings: the order is the exact one."""
    import torch
    T = 60
    base = make(1, E, 5 + E)
    s = torch.sigmoid(base.double()) if score == mx.MX_SIGMOID else torch.softmax(base.double(), 1)
    bias = (0.5 - s[0]).float()  # s + bias = 0.5 within half a step of fp32
    x = base.repeat(T, 1)
    # tokens that leave out some experts, and move others by single steps
    x[torch.rand(T, E, device="cuda", generator=gen(2)) < 0.3] = -6.0
    nudge = torch.randint(-1, 2, (T, E), device="cuda", generator=gen(3)).float()
    x = x * (1.0 + nudge * 2.0 ** -23)
    both(x, 6, score=score, bias=bias, n_groups=groups, topk_groups=max(1, groups // 2), group_best=best)


@pytest.mark.parametrize("score", [mx.MX_SOFTMAX, mx.MX_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_non_finite_logits(score, renorm):
    import torch
    x = make(64, 60, 9)
    x[0, 3] = x[0, 40] = math.nan
    x[1] = math.nan
    x[2] = -INF
    x[3] = -INF
    x[3, 17] = 1.0
    x[4, 5] = INF
    x[5, 5] = x[5, 50] = INF
    x[6, :] = INF
    x[7, ::2] = torch.finfo(torch.float32).min
    x[8, :] = torch.finfo(torch.float32).min
    x[9, :30] = -INF
    x[9, 30:] = math.nan
    x[10, 1:] = -200.0
    for kw in (dict(), dict(n_groups=6, topk_groups=2), dict(bias=bias_of(60, 1)),
               dict(bias=bias_of(60, 1), n_groups=6, topk_groups=2, group_best=2)):
        both(x, 8, score=score, renormalise=renorm, **kw)


@pytest.mark.parametrize("low", [-INF, -1e30, -3.4028234663852886e38, -1e9])
def test_biases_that_close_experts(low):
    """A mask of the type's lowest values leaves the others' order exact, also where it leaves too few."""
    import torch
    E = 128
    x, b = make(90, E, 4), bias_of(E, 4)
    for share in (0.5, 0.97, 1.0):
        bias = torch.where(torch.rand(E, device="cuda", generator=gen(6)) < share, low, b)
        both(x, 8, score=mx.MX_SIGMOID, bias=bias)
        both(x, 8, score=mx.MX_SIGMOID, bias=bias, n_groups=8, topk_groups=3, group_best=2)
        both(x, 8, score=mx.MX_SOFTMAX, bias=bias, n_groups=8, topk_groups=3, group_best=1)
    both(x, 8, score=mx.MX_SIGMOID, bias=torch.where(torch.arange(E, device="cuda") == 5, math.nan, b))
    both(x, 8, score=mx.MX_SIGMOID, bias=torch.where(torch.arange(E, device="cuda") == 5, INF, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,pitch,shift", [(256, 260, 0), (256, 257, 0), (256, 264, 1), (128, 130, 2), (60, 61, 0)])
def test_pitched_and_misaligned_rows(dtype, E, pitch, shift):
    wide = make(50, pitch + 8, 12, dtype).flatten()
    x = wide[shift:shift + 50 * pitch].view(50, pitch)[:, :E]
    both(x, 8, score=mx.MX_SIGMOID, bias=bias_of(E + 3, 1)[1:E + 1].clone() if shift else bias_of(E, 1))


def test_misaligned_bias():
    b = bias_of(257, 1)[1:]
    import torch
    assert b.data_ptr() % 16 and isinstance(b, torch.Tensor)
    both(make(40, 256, 3), 8, score=mx.MX_SIGMOID, bias=b)


def test_other_stream_and_shared_workspace():
    """Calls on a stream of their own; calls of different sizes that share a workspace, one after another."""
    import torch
    x, y = make(3000, 64, 1), make(500, 64, 2)
    r = mx.Router(64, 4)
    n = mx.route_logits_workspace_bytes(r, 3000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.workspace_init(ws, n, stream=s)
        got = [call(t, 4, ws=ws) for t in (x, y, x[:7], x)]
    s.synchronize()
    for t, g in zip((x, y, x[:7], x), got):
        check(t, 4, g)
    torch.cuda.current_stream().wait_stream(s)
    check(y, 4, call(y, 4, ws=ws, stream=torch.cuda.current_stream()))


@pytest.mark.parametrize("T", [5, 333, 2500])
def test_captured_and_replayed(T):
    import torch
    x = make(T, 160, 5)
    r = mx.Router(160, 6, score=mx.MX_SIGMOID, n_groups=8, topk_groups=3, group_best=2)
    n = mx.route_logits_workspace_bytes(r, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mx.workspace_init(ws, n, stream=torch.cuda.current_stream())
    out = [torch.empty(T, 6, dtype=torch.int32, device="cuda"), torch.empty(T, 6, device="cuda")]
    out += [torch.empty(k, dtype=torch.int32, device="cuda") for k in (160, 161, T * 6)]
    mx.route_logits(x, r, *out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.route_logits(x, r, *out, ws=ws)
        mx.route_logits(x, r, *out, ws=ws)
    for seed in (6, 7):
        x.copy_(make(T, 160, seed))
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(x, 6, out, score=mx.MX_SIGMOID, n_groups=8, topk_groups=3, group_best=2)


def test_logits_past_32_bits():
    """More than 2^31 logits: the last tokens are theirs."""
    import torch
    T, E = (1 << 31) // 512 + 5000, 512
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    got = call(x, 2, group=False)
    tail = slice(T - 300, T)
    check(x[tail], 2, (got[0][tail], got[1][tail]))
    check(x[:300], 2, (got[0][:300], got[1][:300]))
