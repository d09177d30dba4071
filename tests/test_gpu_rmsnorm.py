"""RMS norm with the residual's addition and an e4m3 output, on the GPU, bit for bit against its definition in fp64.

The sum with the residual, r, both products and the quotient before e4m3 are defined as fp32 numbers.  r alone is not
always the nearest one: its statistic carries about 48 bits, so a row whose exact r lies within 2^-38 of it of a
border between two fp32 numbers may have either."""
from __future__ import annotations

import math

import pytest

import expert_ffn_gb300 as mx

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def same(a, b):
    """Equal bit for bit, NaN for NaN."""
    import torch
    a, b = a.double(), b.double()
    return (a == b) & (torch.signbit(a) == torch.signbit(b)) | (a.isnan() & b.isnan())


def quantised(y, pow2):
    """(e4m3 values, scales) of fp64 rows that hold fp32 numbers."""
    import torch
    q, ss = torch.empty_like(y), []
    for lo in range(0, y.shape[1], 128):
        b = y[:, lo:lo + 128]
        a = b.abs().amax(1, keepdim=True)
        a = torch.where(b.isnan().any(1, keepdim=True), math.nan, a)
        s = (a / 448.0).float().double()
        s = torch.where(s < TINY, torch.full_like(s, TINY), s)
        if pow2:
            m, _ = torch.frexp(s)
            s = torch.where(s.isfinite() & (m != 0.5), s / m, s)
        v = (b / s).float().double()
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        q[:, lo:lo + 128] = (torch.round(v / step) * step).clamp(-448.0, 448.0)
        ss.append(s)
    return q, torch.cat(ss, 1)


def reference(x, weight, residual, eps, offset, out_dtype, pow2):
    """{name: values} twice: with r rounded to nearest, and with the other neighbour in rows where r is near a border."""
    import torch
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(x.dtype)
    h64 = h.double()
    r = 1.0 / torch.sqrt(h64.pow(2).sum(1, keepdim=True) / x.shape[1] + torch.tensor(eps).float().double().item())
    r32 = r.float()
    err = r - r32.double()
    other = torch.where(err > 0, torch.nextafter(r32, torch.full_like(r32, math.inf)), torch.nextafter(r32, -torch.full_like(r32, math.inf)))
    near = ((r32.double() + other.double()) / 2 - r).abs() <= 2.0 ** -38 * r
    w = None if weight is None else (torch.tensor(offset).float().item() + weight.double()).float().double()
    res = []
    for rr in (r32, torch.where(near, other, r32)):
        y = (h64 * rr.double()).float().double()
        if w is not None:
            y = (y * w).float().double()
        q, s = quantised(y, pow2)
        res.append({"sum": h, "out": y.float().to(out_dtype), "q": q, "scales": s})
    return res


def run(x, weight=None, residual=None, eps=1e-6, offset=0.0, out_dtype=None, pow2=False, sum_=True, q=True, pitch=0,
        stream=None, into=None):
    import torch
    rows, cols = x.shape
    t = {}
    if sum_:
        t["sum"] = torch.full((rows, cols + pitch), 3.0, dtype=x.dtype, device="cuda")[:, :cols]
    if out_dtype is not None:
        t["out"] = torch.full((rows, cols + pitch), 3.0, dtype=out_dtype, device="cuda")[:, :cols]
    if q:
        t["q"] = torch.full((rows, cols + pitch), 3.0, device="cuda").to(torch.float8_e4m3fn)[:, :cols]
        t["scales"] = torch.full((-(-cols // 128), rows), 3.0, device="cuda").t()
    mx.fp8_rmsnorm(x, weight, eps=eps, weight_offset=offset, residual=residual, residual_out=t.get("sum"), out=t.get("out"),
                   q=t.get("q"), scales=t.get("scales"), pow2=pow2, stream=stream)
    return t


def check(got, want):
    import torch
    ok = [torch.ones(next(iter(got.values())).shape[0], dtype=torch.bool, device="cuda") for _ in want]
    for name, t in got.items():
        for o, w in zip(ok, want):
            o &= same(t, w[name].to(t.dtype) if name == "out" else w[name]).all(1)
    assert (ok[0] | ok[1]).all(), {n: int((~same(t, want[0][n])).sum()) for n, t in got.items()}


def make(rows, cols, seed, dtype, scale=1.0):
    import torch
    x = torch.randn(rows, cols, device="cuda", generator=gen(seed)) * scale
    x[:, ::97] *= 12
    return x.to(dt(dtype))


# one to several pieces a thread, ragged ends, whole and partial blocks of 128
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 127), (1, 128), (9, 129), (4, 1000), (1, 2816), (33, 2112),
                                       (700, 704), (3, 4096), (3, 4097), (2, 8192), (2, 8200), (2, 16384), (2, 16390),
                                       (2, 32768), (1500, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, cols, dtype, residual):
    x, w = make(rows, cols, cols, dtype), make(1, cols, 5, dtype)[0]
    r = make(rows, cols, 6, dtype) if residual else None
    got = run(x, w, r, out_dtype=dt(dtype))
    check(got, reference(x, w, r, 1e-6, 0.0, dt(dtype), False))


@pytest.mark.parametrize("dtype,wdtype,odtype", [("bf16", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "bf16", "f32")])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_types_powers_and_offset(dtype, wdtype, odtype, pow2, offset):
    x, w, r = make(40, 1000, 1, dtype), make(1, 1000, 2, wdtype)[0], make(40, 1000, 3, dtype)
    got = run(x, w, r, offset=offset, out_dtype=dt(odtype), pow2=pow2)
    check(got, reference(x, w, r, 1e-6, offset, dt(odtype), pow2))


@pytest.mark.parametrize("keep", [("sum",), ("out",), ("q",), ("sum", "q"), ("out", "q")])
def test_any_of_the_outputs(keep):
    x, r = make(20, 640, 1, "bf16"), make(20, 640, 2, "bf16")
    got = run(x, None, r, out_dtype=dt("bf16") if "out" in keep else None, sum_="sum" in keep, q="q" in keep)
    check(got, reference(x, None, r, 1e-6, 0.0, dt("bf16"), False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,shift", [(8, 0), (1, 0), (5, 3), (16, 1)])
def test_pitched_and_misaligned(dtype, pitch, shift):
    """Rows at any address; nothing behind them is written."""
    import torch
    rows, cols = 30, 777
    flat = make(1, (rows + 1) * (cols + pitch) + 8, 7, dtype)[0]
    x = flat[shift:shift + rows * (cols + pitch)].view(rows, cols + pitch)[:, :cols]
    w = make(1, cols + shift, 5, dtype)[0][shift:]
    r = make(rows, cols + pitch, 6, dtype)[:, :cols]
    got = run(x, w.clone() if shift == 3 else w, r, out_dtype=dt(dtype), pitch=pitch)
    check(got, reference(x, w, r, 1e-6, 0.0, dt(dtype), False))
    for name in ("sum", "out", "q"):
        t = got[name]
        whole = torch.as_strided(t, (rows, cols + pitch), t.stride())
        assert (whole[:, cols:].float() == 3.0).all(), name


@pytest.mark.parametrize("where", ["sum is residual", "sum is x", "out is x", "out is residual"])
def test_in_place(where):
    x, r, w = make(50, 1024, 1, "bf16"), make(50, 1024, 2, "bf16"), make(1, 1024, 3, "bf16")[0]
    want = reference(x, w, r, 1e-6, 0.0, dt("bf16"), False)
    x2, r2 = x.clone(), r.clone()
    kw = {"sum is residual": dict(residual_out=r2), "sum is x": dict(residual_out=x2), "out is x": dict(out=x2),
          "out is residual": dict(out=r2)}[where]
    mx.fp8_rmsnorm(x2, w, residual=r2, **kw)
    check({"sum" if "sum" in where else "out": next(iter(kw.values()))}, want)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-12, 1e18, 1e22, 3e37])
def test_extreme_magnitudes(scale):
    """Squares that fp32 does not hold."""
    x = make(6, 500, 4, "f32", scale)
    x = x.clamp(-3.3e38, 3.3e38)
    for eps in (0.0, 1e-6):
        got = run(x, None, None, eps=eps, out_dtype=dt("f32"), sum_=False)
        check(got, reference(x, None, None, eps, 0.0, dt("f32"), False))


def test_zeros_infinities_and_nan():
    import torch
    x = make(8, 300, 4, "f32")
    x[0] = 0
    x[1, 200] = math.inf
    x[2, 3] = math.nan
    x[3, 0], x[3, 299] = math.inf, -math.inf
    x[4] = -0.0
    got = run(x, None, None, out_dtype=dt("f32"), sum_=False)
    torch.cuda.synchronize()
    assert (got["out"][0] == 0).all() and (got["q"][0].float() == 0).all()
    assert got["out"][1, 200].isnan() and (got["out"][1, :200] == 0).all()
    assert (got["scales"][1].isnan() == torch.tensor([False, True, False], device="cuda")).all()
    assert got["out"][2].isnan().all() and got["scales"][2].isnan().all()
    assert got["out"][3, 0].isnan() and got["out"][3, 299].isnan() and (got["out"][3, 1:299] == 0).all()
    assert torch.signbit(got["out"][4]).all()
    clean = run(x[5:], None, None, out_dtype=dt("f32"), sum_=False)
    for n in ("out", "scales"):
        assert torch.equal(got[n][5:], clean[n])
    zero = run(x[:1], None, None, eps=0.0, out_dtype=dt("f32"), sum_=False)
    assert zero["out"].isnan().all()


def test_same_rows_as_the_quantiser():
    """q and scales are what fp8_quantize makes of the fp32 output."""
    import torch
    x, w = make(64, 2816, 8, "bf16"), make(1, 2816, 9, "bf16")[0]
    got = run(x, w, None, out_dtype=dt("f32"), sum_=False)
    q, s = torch.empty_like(got["q"]), torch.empty_like(got["scales"])
    mx.fp8_quantize(got["out"], q, s)
    assert torch.equal(q.view(torch.uint8), got["q"].view(torch.uint8)) and torch.equal(s, got["scales"])


def test_captured_replayed_and_on_another_stream():
    import torch
    x, w, r = make(17, 704, 1, "bf16"), make(1, 704, 2, "bf16")[0], make(17, 704, 3, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(x, w, r, out_dtype=dt("bf16"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mx.fp8_rmsnorm(x, w, residual=r, residual_out=got["sum"], out=got["out"], q=got["q"], scales=got["scales"])
    for seed in (4, 5):
        x.copy_(make(17, 704, seed, "bf16"))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        check(got, reference(x, w, r, 1e-6, 0.0, dt("bf16"), False))


def test_rows_past_32_bits():
    import torch
    rows, cols = 70000, 32768  # 2.3e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(1))
    out = torch.empty_like(x)
    mx.fp8_rmsnorm(x, out=out)
    for part in (slice(0, 5), slice(rows - 5, rows)):
        check({"out": out[part]}, reference(x[part], None, None, 1e-6, 0.0, dt("bf16"), False))
