"""FP8 block-scaled operators on the GPU against plain fp64 implementations.

Tolerances.  An fp32 product differs from the exact one by the rounding of its
sums: at most (K + 3 B) 2^-24 sum |terms| for K columns in B blocks; the tensor
core may truncate where fp32 rounds, which doubles the per-term bound.  A bf16
output adds half a step, 2^-8 of its value.  In the layer the hidden values are
quantised again: one that lies within its own rounding error (about
(D + 8) 2^-23 of its sum of |terms|) of a border between two e4m3 numbers may go
to either side, a step of at most 2^-3 of it, so the layer is compared with the
exact layer whose hidden values carry that uncertainty (see `layer_bound`)."""
from __future__ import annotations

import math

import numpy as np
import pytest

import expert_ffn_gb300 as mx

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126
U32 = 2.0 ** -24


def nb(n):
    return -(-n // 128)


# ------------------------------------------------- the definitions, in fp64

def ref_e4m3(v):
    import torch
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def ref_scale(a, pow2=False):
    """Scale of a block whose largest magnitude is a (fp64 holding fp32 numbers)."""
    import torch
    s = (a / 448.0).float().double()
    s = torch.where(s < TINY, torch.full_like(s, TINY), s)
    if pow2:
        m, _ = torch.frexp(s)
        s = torch.where(m == 0.5, s, s / m)  # s = m 2^e with m in [1/2, 1): 2^e, exactly
    return s


def ref_quantize(x, pow2=False):
    """(e4m3 values, scales) of fp64 rows."""
    import torch
    q, ss = torch.empty_like(x), []
    for lo in range(0, x.shape[1], 128):
        b = x[:, lo:lo + 128]
        s = ref_scale(b.abs().amax(1, keepdim=True), pow2)
        q[:, lo:lo + 128] = ref_e4m3((b / s).float().double())
        ss.append(s)
    return q, torch.cat(ss, 1)


def rows_value(q, s):
    v = q.double()
    for b in range(s.shape[1]):
        v[:, b * 128:(b + 1) * 128] *= s[:, b:b + 1].double()
    return v


def weight_value(w, s):
    v = w.double()
    for r in range(s.shape[-2]):
        for b in range(s.shape[-1]):
            v[..., r * 128:(r + 1) * 128, b * 128:(b + 1) * 128] *= s[..., r, b, None, None].double()
    return v


# ----------------------------------------------------------------- inputs

def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_rows(rows, cols, seed, row_major=False, spare=0):
    """Random e4m3 rows (any code but NaN) and scales."""
    import torch
    g = gen(seed)
    pitch = -(-cols // 16) * 16 + 16 * spare
    q = torch.randn(rows, pitch, device="cuda", generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)[:, :cols]
    s = torch.rand(rows, nb(cols), device="cuda", generator=g) + 0.25
    return q, (s if row_major else s.t().contiguous().t())


def make_weight(n, rows, cols, seed, spare=0):
    import torch
    g = gen(seed)
    pitch = -(-cols // 16) * 16 + 16 * spare
    w = torch.randn(n, rows, pitch, device="cuda", generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand(n, nb(rows), nb(cols), device="cuda", generator=g) + 0.25) / (100 * math.sqrt(cols))
    return w[..., :cols], s


def workspace(n):
    import torch
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mx.workspace_init(ws, n, stream=torch.cuda.current_stream())
    return ws


def check_product(out, x, w, K):
    """out against x @ w.T for fp64 x, w."""
    import torch
    exact, mag = x @ w.T, x.abs() @ w.abs().T
    tol = 2 * (K + 3 * nb(K)) * U32 * mag
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * exact.abs()
    bad = (out.double() - exact).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out.double() - exact).abs() / tol.clamp_min(1e-300)).max()))


# --------------------------------------------------------------- quantise

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pitch", [(1, 1, 0), (1, 2816, 0), (3, 127, 0), (33, 129, 0), (64, 704, 8),
                                             (31, 2112, 1), (257, 1040, 24)])
def test_quantize(rows, cols, pitch, dtype, pow2):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (torch.randn(rows, cols + pitch, device="cuda", generator=gen(rows + cols)) * 3).to(dt)[:, :cols]
    x[0, :: 7] = 0.0
    x[rows // 2, :128] = 0.0  # a block of zeros
    q = torch.zeros(rows, cols + pitch, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((nb(cols), rows), -1.0, device="cuda").t() if pitch != 1 else torch.full((rows, nb(cols)), -1.0, device="cuda")
    mx.fp8_quantize(x, q[:, :cols], s, pow2=pow2)
    rq, rs = ref_quantize(x.double(), pow2)
    assert torch.equal(s.double(), rs)
    assert torch.equal(q[:, :cols].double(), rq)
    assert not q[:, cols:].double().any()  # what lies behind the columns is left alone


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_extreme_values(dtype):
    """Subnormal, huge, infinite and NaN blocks; every block keeps to itself."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.ones(6, 256, device="cuda")
    x[0, :128] = torch.finfo(dt).tiny
    x[1, 5] = torch.finfo(dt).max
    x[2, 7] = math.inf
    x[3, 9] = math.nan
    x[4, :128] = 2.0 ** -130
    x[5, 3] = -448.0
    x = x.to(dt)
    q = torch.empty(6, 256, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(6, 2, device="cuda")
    mx.fp8_quantize(x, q, s)
    rows = [0, 1, 4, 5]
    rq, rs = ref_quantize(x[rows].double())
    assert torch.equal(s[rows].double(), rs) and torch.equal(q[rows].double(), rq)
    assert math.isinf(s[2, 0].item()) and math.isnan(s[3, 0].item())
    v = rows_value(q, s)
    assert v[2, :128].isnan().all() and v[3, :128].isnan().all()
    assert torch.equal(v[:4, 128:], torch.ones_like(v[:4, 128:]).double()) or \
        (v[:4, 128:] - 1).abs().max() < 2.0 ** -4
    assert v[2:4, 128:].isfinite().all()


# ---------------------------------------------------------------- product

@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 2112, 2816), (2, 130, 16), (16, 128, 128), (17, 127, 129), (5, 4096, 700),
                                   (33, 257, 1037), (64, 704, 384), (65, 300, 2816), (129, 129, 640), (300, 1000, 256),
                                   (1000, 520, 333), (2999, 2600, 333)])
def test_matmul(m, n, k, out):
    import torch
    q, s = make_rows(m, k, 1, row_major=m % 2 == 1, spare=m % 3)
    w, ws = make_weight(1, n, k, 2, spare=k % 2)
    pitch = n + (3 if m == 33 else 0)
    buf = torch.full((m, pitch), 7.0, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    work = workspace(256)
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), buf[:, :n], work)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_product(buf[:, :n], rows_value(q, s), weight_value(w[0], ws[0]), k)
    assert (buf[:, n:] == 7.0).all()
    again = torch.empty_like(buf)
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), again[:, :n], work)
    assert torch.equal(again[:, :n], buf[:, :n])


def test_matmul_keeps_non_finite_rows_apart():
    """A NaN row and an infinite scale touch their own output rows alone."""
    import torch
    q, s = make_rows(40, 512, 3)
    q.view(torch.uint8)[7, 100] = 0x7F
    s[9, 2] = math.inf
    w, ws = make_weight(1, 200, 512, 4)
    out = torch.empty(40, 200, device="cuda")
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), out, workspace(256))
    assert out[7].isnan().all() and not out[9].isfinite().any()
    keep = [i for i in range(40) if i not in (7, 9)]
    check_product(out[keep], rows_value(q, s)[keep], weight_value(w[0], ws[0]), 512)


@pytest.mark.parametrize("m", [1, 7])
def test_matmul_few_rows_of_a_large_matrix(m):
    import torch
    n, k = 8200, 4104  # above the 32 MB from which few rows change kernels
    q, s = make_rows(m, k, 31)
    w, ws = make_weight(1, n, k, 32)
    out = torch.full((m, n), 7.0, device="cuda")
    work = workspace(256)
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), out, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_product(out, rows_value(q, s), weight_value(w[0], ws[0]), k)


@pytest.mark.parametrize("m", [1, 9, 40, 64])
@pytest.mark.parametrize("n,k", [(100, 1100), (1024, 2100), (1300, 1024), (3000, 1030)])
def test_matmul_split_over_clusters(m, n, k):
    """Inner blocks over clusters of eight, four and two, and not at all."""
    import torch
    q, s = make_rows(m, k, 33)
    w, ws = make_weight(1, n, k, 34)
    out = torch.full((m, n), 7.0, device="cuda", dtype=torch.bfloat16)
    work = workspace(256)
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), out, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_product(out, rows_value(q, s), weight_value(w[0], ws[0]), k)


# ---------------------------------------------------------------- grouped

GROUPS = {
    "even": [8, 8, 8, 8],
    "one": [1],
    "gaps": [0, 5, 0, 0, 300, 1, 0],
    "ragged": [17, 33, 129, 2, 64, 65, 16],
    "empty": [0, 0, 0],
    "many": [700, 0, 129, 300, 5, 256, 257, 900],
    "few": [1, 0, 3, 2, 0, 0, 18, 0, 1, 0, 0, 2],
    "sparse": [0] * 60 + [4, 33] + [0] * 40 + [1],
}


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(129, 272), (704, 640), (40, 1037), (2600, 400)])
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_grouped(groups, n, k, out):
    import torch
    counts = GROUPS[groups]
    total, spare = sum(counts), 5
    q, s = make_rows(total + spare, k, 5)
    w, ws = make_weight(len(counts), n, k, 6)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    buf = torch.full((total + spare, n), 7.0, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    work = workspace(256)
    mx.fp8_grouped_matmul(q, s, offsets, mx.Fp8Weight(w, ws), buf, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    at = 0
    for e, c in enumerate(counts):
        if c:
            check_product(buf[at:at + c], rows_value(q[at:at + c], s[at:at + c]), weight_value(w[e], ws[e]), k)
        at += c
    assert (buf[total:] == 7.0).all()


def test_grouped_offsets_outside_the_rows():
    """Offsets beyond the rows are cut to them, a decreasing pair is an empty group."""
    import torch
    q, s = make_rows(20, 256, 7)
    w, ws = make_weight(4, 100, 256, 8)
    offsets = torch.tensor([-3, 6, 2, 9, 1000], dtype=torch.int32, device="cuda")
    buf = torch.full((20, 100), 7.0, device="cuda")
    mx.fp8_grouped_matmul(q, s, offsets, mx.Fp8Weight(w, ws), buf, workspace(256))
    x = rows_value(q, s)
    # groups [0, 6), (6, 2): empty, [2, 9) over the first, [9, 20)
    check_product(buf[9:], x[9:], weight_value(w[3], ws[3]), 256)
    check_product(buf[6:9], x[6:9], weight_value(w[2], ws[2]), 256)
    check_product(buf[:2], x[:2], weight_value(w[0], ws[0]), 256)


def test_grouped_few_rows_between_others():
    """Few rows to a matrix: those before the first group and behind the last are left alone, bad offsets are cut."""
    import torch
    q, s = make_rows(22, 400, 51)
    w, ws = make_weight(9, 300, 400, 52)
    weight, work, x = mx.Fp8Weight(w, ws), workspace(256), rows_value(q, s)
    buf = torch.full((22, 300), 7.0, device="cuda")
    offsets = torch.tensor([2, 2, 5, 5, 5, 9, 9, 9, 9, 19], dtype=torch.int32, device="cuda")
    mx.fp8_grouped_matmul(q, s, offsets, weight, buf, work)
    for e, lo, hi in ((1, 2, 5), (4, 5, 9), (8, 9, 19)):
        check_product(buf[lo:hi], x[lo:hi], weight_value(w[e], ws[e]), 400)
    assert (buf[:2] == 7.0).all() and (buf[19:] == 7.0).all()
    offsets.copy_(torch.tensor([-7, 4, 1, 4, 4, 4, 4, 4, 10, 1 << 30], dtype=torch.int32))
    mx.fp8_grouped_matmul(q, s, offsets, weight, buf, work)
    mx.workspace_check(work, torch.cuda.current_stream())
    # groups [0, 4), (4, 1): empty, [1, 4) over the first's rows, [4, 10), [10, 22)
    check_product(buf[:1], x[:1], weight_value(w[0], ws[0]), 400)
    check_product(buf[4:10], x[4:10], weight_value(w[7], ws[7]), 400)
    check_product(buf[10:], x[10:], weight_value(w[8], ws[8]), 400)


# ------------------------------------------------------------------ layer

def make_layer(E, D, I, S, seed, top_k, act, dtype, lam=0.5):
    ws = [make_weight(E, I, D, seed), make_weight(E, I, D, seed + 1), make_weight(E, D, I, seed + 2)]
    sh = [make_weight(1, S, D, seed + 3), make_weight(1, S, D, seed + 4), make_weight(1, D, S, seed + 5)] if S else None
    layer = mx.Fp8Layer(*ws, shared=sh, top_k=top_k, act_dtype=mx.MX_BF16 if dtype == "bf16" else mx.MX_F32,
                        activation=act, layer_scalar=lam)
    return layer, ws, sh


def ref_expert(x, gate, up, down, act):
    """Exact expert of fp64 rows, and a bound on what fp32 sums of the hidden layer can change."""
    import torch
    wg, wu, wd = (weight_value(*w) for w in (gate, up, down))
    g, u = x @ wg.T, x @ wu.T
    if act == mx.MX_SILU:
        a = g * torch.sigmoid(g)
    else:
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    h = a * u
    # rounding of g and u: 2 (D + 3 B) 2^-24 sum |terms|; slope of either activation at most 1.13, the fast
    # exponential and division a few ulp more
    D = x.shape[1]
    eg, eu = (2 * (D + 3 * nb(D)) * U32 * (x.abs() @ w.abs().T) for w in (wg, wu))
    eh = 1.13 * eg * u.abs() + a.abs() * eu + eg * eu + 2.0 ** -18 * h.abs() + 2.0 ** -18 * (g * u).abs()
    q, s = ref_quantize(h)
    # hidden values that those errors (and half a rounding of the quotient) can carry over a border of e4m3
    b = torch.empty_like(h)
    for j in range(s.shape[1]):
        c = slice(128 * j, 128 * j + 128)
        top = h[:, c].abs().amax(1, keepdim=True)
        v = h[:, c] / s[:, j:j + 1]
        ev = eh[:, c] / s[:, j:j + 1] + v.abs() * (eh[:, c].amax(1, keepdim=True) / top.clamp_min(1e-300) + 2.0 ** -21)
        lo, hi = ref_e4m3(v - ev), ref_e4m3(v + ev)
        # value error: the flip, or the scale's own change
        b[:, c] = (torch.maximum((hi - q[:, c]).abs(), (lo - q[:, c]).abs()) * s[:, j:j + 1]
                   + q[:, c].abs() * s[:, j:j + 1] * (eh[:, c].amax(1, keepdim=True) / top.clamp_min(1e-300) + 2.0 ** -22))
    hv = rows_value(q, s)
    y = hv @ wd.T
    I = h.shape[1]
    return y, b @ wd.abs().T + 2 * (I + 3 * nb(I)) * U32 * (hv.abs() @ wd.abs().T)


def check_layer(out, x, idx, wts, ws, sh, act, lam, residual, top_k):
    import torch
    xv = rows_value(*ref_quantize(x.double()))
    y, tol = torch.zeros_like(xv), torch.zeros_like(xv)
    mag = torch.zeros_like(xv)
    for e in range(ws[0][0].shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            p, b = ref_expert(xv[t], *((w[0][e], w[1][e]) for w in ws), act)
            wt = wts[t, k].double()[:, None]
            y.index_add_(0, t, p * wt)
            tol.index_add_(0, t, b * wt.abs())
            mag.index_add_(0, t, (p * wt).abs())
    if sh:
        p, b = ref_expert(xv, *((w[0][0], w[1][0]) for w in sh), act)
        y, tol, mag = y + p, tol + b, mag + p.abs()
    tol = abs(lam) * (tol + (top_k + 4) * 2 * U32 * mag)
    exact = lam * y + (0 if residual is None else residual.double())
    tol = tol + 4 * U32 * exact.abs()
    if residual is not None:
        tol = tol + 2 * U32 * residual.double().abs()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * exact.abs()
    err = (out.double() - exact).abs()
    assert not (err > tol).any(), (int((err > tol).sum()), float((err / tol.clamp_min(1e-300)).max()))
    # That bound adds every error with the same sign.  In the 2-norm they add as independent ones: fp32 sums of some
    # thousand terms are off by about 2^-20 of them, so a share of at most 2 * 2^-20 / 2^-4 = 2^-15 of the hidden
    # values goes to the other side of a border, by at most 2^-3 of itself: 2^-10.5 of the outputs.  2^-9 leaves room
    # for the scatter of few flips; bf16 adds half a step.
    rel = 2.0 ** -9 + (2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0)
    assert err.norm() <= rel * exact.norm(), float(err.norm() / exact.norm())


def routing(T, E, K, seed, skew=0.0):
    import torch
    g = gen(seed)
    logits = torch.randn(T, E, device="cuda", generator=g) - skew * torch.arange(E, device="cuda").float().log1p()
    top, idx = logits.topk(K, -1)
    return idx.to(torch.int32), torch.softmax(top, -1).contiguous()


CASES = [  # T, E, K, D, I, S, act, dtype, residual
    (1, 16, 2, 256, 128, 128, mx.MX_GELU_TANH, "bf16", False),
    (1, 128, 8, 2816, 704, 2112, mx.MX_GELU_TANH, "bf16", True),
    (2, 8, 8, 272, 144, 0, mx.MX_SILU, "f32", True),
    (4, 16, 2, 256, 128, 128, mx.MX_GELU_TANH, "f32", False),
    (7, 60, 6, 1040, 200, 77, mx.MX_SILU, "bf16", False),
    (16, 5, 1, 640, 1024, 0, mx.MX_GELU_TANH, "bf16", True),
    (17, 32, 4, 333, 129, 200, mx.MX_SILU, "f32", False),
    (32, 64, 8, 512, 256, 512, mx.MX_SILU, "bf16", True),
    (33, 16, 2, 256, 704, 64, mx.MX_GELU_TANH, "bf16", False),
    (64, 128, 8, 384, 128, 256, mx.MX_GELU_TANH, "f32", True),
    (65, 16, 4, 320, 192, 128, mx.MX_GELU_TANH, "bf16", True),
    (200, 8, 2, 336, 100, 0, mx.MX_SILU, "f32", False),
    (513, 60, 6, 272, 256, 130, mx.MX_SILU, "bf16", False),
    (700, 4, 3, 512, 384, 512, mx.MX_GELU_TANH, "f32", True),
    (1500, 8, 2, 700, 520, 1100, mx.MX_SILU, "bf16", True),
    (900, 4, 2, 2048, 1040, 0, mx.MX_GELU_TANH, "f32", False),
]


@pytest.mark.parametrize("case", range(len(CASES)), ids=[f"T{c[0]}_E{c[1]}_K{c[2]}_D{c[3]}" for c in CASES])
def test_moe_forward(case):
    import torch
    T, E, K, D, I, S, act, dtype, res = CASES[case]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    layer, ws, sh = make_layer(E, D, I, S, 20 + case, K, act, dtype)
    x = torch.randn(T, D, device="cuda", generator=gen(40 + case)).to(dt)
    residual = torch.randn(T, D, device="cuda", generator=gen(60 + case)).to(dt) if res else None
    idx, wts = routing(T, E, K, 80 + case, skew=0.7 if case % 2 else 0.0)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    out = torch.full((T, D), 7.0, device="cuda", dtype=dt)
    mx.fp8_moe_forward(x, idx, wts, layer, out, work, residual=residual)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_layer(out, x, idx, wts, ws, sh, act, 0.5, residual, K)
    again = torch.empty_like(out)
    mx.fp8_moe_forward(x, idx, wts, layer, again, work, residual=residual)
    assert torch.equal(out, again)


# Every split of the inner blocks over a cluster (by d_model and the tile of tokens), one token with more hidden
# blocks than run at once, many slots, many experts to a token, the smallest layers.
MORE = [
    (1, 40, 32, 300, 130, 0, mx.MX_SILU, "f32", False),
    (1, 4, 4, 512, 2560, 0, mx.MX_GELU_TANH, "bf16", True),
    (1, 2, 1, 5, 3, 0, mx.MX_SILU, "f32", True),
    (1, 16, 8, 1022, 144, 72, mx.MX_SILU, "bf16", True),
    (3, 2, 2, 1, 1, 1, mx.MX_GELU_TANH, "f32", False),
    (8, 128, 8, 2816, 320, 256, mx.MX_SILU, "bf16", True),
    (9, 40, 32, 300, 130, 50, mx.MX_GELU_TANH, "bf16", False),
    (10, 4, 2, 4096, 640, 0, mx.MX_SILU, "bf16", False),
    (20, 4, 2, 5120, 640, 128, mx.MX_GELU_TANH, "f32", True),
    (30, 6, 3, 8192, 512, 0, mx.MX_SILU, "bf16", False),
    (12, 4, 2, 13056, 512, 0, mx.MX_GELU_TANH, "f32", False),
    (50, 4, 2, 2816, 640, 0, mx.MX_SILU, "bf16", True),
    (50, 4, 2, 4096, 640, 64, mx.MX_SILU, "f32", True),
    (64, 6, 3, 8192, 512, 0, mx.MX_GELU_TANH, "bf16", False),
    (40, 4, 2, 20000, 256, 0, mx.MX_SILU, "bf16", False),
    (70, 2, 1, 5, 3, 2, mx.MX_SILU, "f32", True),
    (120, 40, 12, 272, 128, 0, mx.MX_SILU, "bf16", False),
    (1100, 16, 4, 256, 128, 64, mx.MX_GELU_TANH, "bf16", True),
]


@pytest.mark.parametrize("case", range(len(MORE)), ids=[f"T{c[0]}_E{c[1]}_K{c[2]}_D{c[3]}" for c in MORE])
def test_moe_forward_splits_and_limits(case):
    import torch
    T, E, K, D, I, S, act, dtype, res = MORE[case]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    layer, ws, sh = make_layer(E, D, I, S, 120 + case, K, act, dtype)
    x = torch.randn(T, D, device="cuda", generator=gen(140 + case)).to(dt)
    residual = torch.randn(T, D, device="cuda", generator=gen(160 + case)).to(dt) if res else None
    idx, wts = routing(T, E, K, 180 + case)
    n = mx.fp8_moe_workspace_bytes(layer, T)
    work = workspace(n + 4096)
    work[n:] = 0x5A  # (what lies behind the workspace is not this call's)
    out = torch.full((T, D), 7.0, device="cuda", dtype=dt)
    mx.fp8_moe_forward(x, idx, wts, layer, out, work[:n], residual=residual)
    mx.workspace_check(work, torch.cuda.current_stream())
    check_layer(out, x, idx, wts, ws, sh, act, 0.5, residual, K)
    assert (work[n:] == 0x5A).all()


@pytest.mark.parametrize("T", [1, 6, 40, 90])
def test_moe_odd_routings(T):
    """Indices outside the experts add nothing, repeated ones count twice, a token may have no expert at all, one
    expert may take every token."""
    import torch
    E, K, D, I = 12, 4, 384, 160
    layer, ws, _ = make_layer(E, D, I, 0, 5, K, mx.MX_SILU, "f32")
    x = torch.randn(T, D, device="cuda", generator=gen(6))
    idx, wts = routing(T, E, K, 7)
    idx[:, 1] = 3
    idx[:, 2] = 3
    idx[T // 2, 0] = -1
    idx[T - 1] = torch.tensor([-5, E, 1 << 30, -1], device="cuda", dtype=torch.int32)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    out = torch.full((T, D), 7.0, device="cuda")
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    check_layer(out, x, idx, wts, ws, None, mx.MX_SILU, 0.5, None, K)
    assert not out[T - 1].any()
    # no expert anywhere: out = residual
    idx.fill_(-1)
    mx.fp8_moe_forward(x, idx, wts, layer, out, work, residual=x)
    assert torch.equal(out, x)


@pytest.mark.parametrize("T", [3, 100])
def test_moe_in_place_and_other_stream(T):
    """out may be the residual itself; a call on a side stream with a captured and replayed graph gives the same."""
    import torch
    E, K, D, I, S = 16, 2, 512, 256, 128
    layer, ws, sh = make_layer(E, D, I, S, 9, K, mx.MX_GELU_TANH, "bf16")
    x = torch.randn(T, D, device="cuda", generator=gen(10)).bfloat16()
    idx, wts = routing(T, E, K, 11)
    n = mx.fp8_moe_workspace_bytes(layer, T)
    out = torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, out, workspace(n), residual=x)
    same = x.clone()
    mx.fp8_moe_forward(same, idx, wts, layer, same, workspace(n), residual=same)
    assert torch.equal(same, out)
    side, work = torch.cuda.Stream(), workspace(n)
    side.wait_stream(torch.cuda.current_stream())
    buf = torch.zeros_like(x)
    with torch.cuda.stream(side):
        mx.fp8_moe_forward(x, idx, wts, layer, buf, work, residual=x)  # (first call: loads the kernels)
        side.synchronize()
        buf.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mx.fp8_moe_forward(x, idx, wts, layer, buf, work, residual=x)
    torch.cuda.synchronize()
    x2 = x.clone()
    for _ in range(3):
        buf.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, out)
    x.mul_(2)  # new values in the captured buffers
    graph.replay()
    torch.cuda.synchronize()
    check_layer(buf, x2 * 2, idx, wts, ws, sh, mx.MX_GELU_TANH, 0.5, x2 * 2, K)


@pytest.mark.parametrize("T", [4, 40, 90])
def test_moe_non_finite_tokens_stay_apart(T):
    """A NaN or an infinity in a token makes that token's output NaN and leaves the others' bits as they were."""
    import torch
    E, K, D, I, S = 6, 3, 384, 160, 128
    layer, _, _ = make_layer(E, D, I, S, 45, K, mx.MX_GELU_TANH, "bf16")
    x = torch.randn(T, D, device="cuda", generator=gen(46)).bfloat16()
    idx, wts = routing(T, E, K, 47)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, T))
    clean, out = torch.empty_like(x), torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, clean, work)
    x[1, 5], x[T - 1, 300] = math.nan, -math.inf
    mx.fp8_moe_forward(x, idx, wts, layer, out, work)
    assert out[1].isnan().all() and out[T - 1].isnan().all()
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(out[keep], clean[keep]) and clean.isfinite().all()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_moe_non_finite_single_token(value):
    """One token with a NaN or an infinity: NaN throughout, and nothing of it in the workspace's next call."""
    import torch
    E, K, D, I, S = 6, 3, 384, 160, 128
    layer, _, _ = make_layer(E, D, I, S, 45, K, mx.MX_SILU, "f32")
    x = torch.randn(1, D, device="cuda", generator=gen(48))
    idx, wts = routing(1, E, K, 49)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, 1))
    clean, out, again = (torch.empty_like(x) for _ in range(3))
    mx.fp8_moe_forward(x, idx, wts, layer, clean, work)
    bad = x.clone()
    bad[0, 200] = value
    mx.fp8_moe_forward(bad, idx, wts, layer, out, work)
    mx.fp8_moe_forward(x, idx, wts, layer, again, work)
    assert out.isnan().all() and clean.isfinite().all() and torch.equal(again, clean)


@pytest.mark.parametrize("T", [1, 20, 90])
def test_two_calls_at_once(T):
    """Two streams with a workspace each, call upon call, give what one alone gives."""
    import torch
    E, K, D, I, S = 16, 4, 1024, 256, 128
    layer, _, _ = make_layer(E, D, I, S, 35, K, mx.MX_SILU, "bf16")
    n = mx.fp8_moe_workspace_bytes(layer, T)
    runs = []
    for i in range(2):
        x = torch.randn(T, D, device="cuda", generator=gen(36 + i)).bfloat16()
        idx, wts = routing(T, E, K, 38 + i)
        alone = torch.empty_like(x)
        mx.fp8_moe_forward(x, idx, wts, layer, alone, workspace(n))
        runs.append((x, idx, wts, alone, workspace(n), torch.cuda.Stream(), [torch.zeros_like(x) for _ in range(8)]))
    torch.cuda.synchronize()
    for j in range(8):
        for x, idx, wts, _, work, stream, outs in runs:
            mx.fp8_moe_forward(x, idx, wts, layer, outs[j], work, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, alone, work, stream, outs in runs:
        mx.workspace_check(work, stream)
        assert all(torch.equal(o, alone) for o in outs)


def test_captured_quantize_and_products():
    """A graph of quantiser, product and grouped product follows its buffers' new values and offsets."""
    import torch
    x = torch.randn(30, 512, device="cuda", generator=gen(41)).bfloat16()
    q, s = torch.empty(30, 512, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(4, 30, device="cuda").t()
    w, ws = make_weight(3, 200, 512, 42)
    one, all_ = mx.Fp8Weight(w[0], ws[0]), mx.Fp8Weight(w, ws)
    offsets = torch.tensor([0, 10, 10, 30], dtype=torch.int32, device="cuda")
    out, grp, work = torch.empty(30, 200, device="cuda"), torch.full((30, 200), 7.0, device="cuda"), workspace(256)

    def run():
        mx.fp8_quantize(x, q, s)
        mx.fp8_matmul(q, s, one, out, work)
        mx.fp8_grouped_matmul(q, s, offsets, all_, grp, work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    x.copy_(torch.randn(30, 512, device="cuda", generator=gen(43)))
    offsets.copy_(torch.tensor([2, 2, 19, 25], dtype=torch.int32))  # (rows 0, 1 and 25 on belong to nobody)
    grp.fill_(7.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    v = rows_value(*ref_quantize(x.double()))
    check_product(out, v, weight_value(w[0], ws[0]), 512)
    check_product(grp[2:19], v[2:19], weight_value(w[1], ws[1]), 512)
    check_product(grp[19:25], v[19:25], weight_value(w[2], ws[2]), 512)
    assert (grp[:2] == 7.0).all() and (grp[25:] == 7.0).all()


def test_moe_tokens_do_not_depend_on_their_batch():
    """A token's output alone is its output in a batch of 64, up to hidden values next to a border of e4m3."""
    import torch
    E, K, D, I, S = 16, 4, 640, 256, 128
    layer, _, _ = make_layer(E, D, I, S, 13, K, mx.MX_SILU, "f32")
    x = torch.randn(64, D, device="cuda", generator=gen(14))
    idx, wts = routing(64, E, K, 15)
    work = workspace(mx.fp8_moe_workspace_bytes(layer, 64))
    full = torch.empty_like(x)
    mx.fp8_moe_forward(x, idx, wts, layer, full, work)
    err = 0.0
    for t in (0, 13, 63):
        one = torch.empty(1, D, device="cuda")
        mx.fp8_moe_forward(x[t:t + 1].contiguous(), idx[t:t + 1].contiguous(), wts[t:t + 1].contiguous(), layer, one, work)
        err = max(err, float((one[0] - full[t]).norm() / full[t].norm()))
    assert err < 0.02  # (the split of the sums differs; hidden values next to a border may round the other way)


def test_route_then_experts():
    """The framework's router followed by the FP8 layer, as a decoder runs them, chained through two layers."""
    import torch

    import synth
    from tests.gpu_util import to_dev
    cfg = synth.small_config(T=5, D=256, E=16, K=2, I=128, S=128, act="bf16", seed=3)
    dev = mx.DeviceLayer(synth.make_layer(cfg), mx.MX_BF16)
    layer, ws, sh = make_layer(16, 256, 128, 128, 16, 2, mx.MX_GELU_TANH, "bf16")
    x = to_dev(synth.make_x(cfg)).view(torch.bfloat16)
    T, E, K = 5, 16, 2
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    n_route, n_moe = mx.workspace_bytes(dev.layout, T), mx.fp8_moe_workspace_bytes(layer, T)
    w_route, w_moe = workspace(n_route), workspace(n_moe)
    stream = torch.cuda.current_stream()
    for _ in range(2):
        idx, wts = i32(T, K), torch.zeros(T, K, device="cuda")
        mx.route(x, T, dev, idx, wts, i32(E), i32(E + 1), i32(T * K), w_route, n_route, stream=stream)
        out = torch.empty_like(x)
        mx.fp8_moe_forward(x, idx, wts, layer, out, w_moe, residual=x)
        check_layer(out, x, idx, wts, ws, sh, mx.MX_GELU_TANH, 0.5, x, K)
        x = out


def test_quantize_then_matmul():
    """Activations through the quantiser into a projection: the exact product of the quantised values."""
    import torch
    x = torch.randn(50, 700, device="cuda", generator=gen(17)).bfloat16()
    q = torch.empty(50, 704, device="cuda", dtype=torch.float8_e4m3fn)[:, :700]
    s = torch.empty(6, 50, device="cuda").t()
    mx.fp8_quantize(x, q, s)
    w, ws = make_weight(1, 300, 700, 18)
    out = torch.empty(50, 300, device="cuda")
    mx.fp8_matmul(q, s, mx.Fp8Weight(w[0], ws[0]), out, workspace(256))
    rq, rs = ref_quantize(x.double())
    check_product(out, rows_value(rq, rs), weight_value(w[0], ws[0]), 700)


def test_no_rows():
    import torch
    q, s = make_rows(4, 256, 1)
    w, ws = make_weight(1, 100, 256, 2)
    out = torch.empty(0, 100, device="cuda")
    mx.fp8_matmul(q[:0], s[:0], mx.Fp8Weight(w[0], ws[0]), out, workspace(256))
    mx.fp8_quantize(torch.empty(0, 256, device="cuda"), q[:0], s[:0])
