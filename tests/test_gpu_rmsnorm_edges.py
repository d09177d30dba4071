"""The RMS norm at both ends of its types' range and of more rows than there are CTAs, bit for bit against its definition
in fp64 (as in its own tests)."""
from __future__ import annotations

import pytest

import expert_ffn_gb300 as mx
from tests.test_gpu_rmsnorm import check, dt, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [500, 4100, 8192, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e17, 3e20, 1e35, 3e37, 9e37, 1.3e38, 2e38, 3e38])
def test_rows_whose_squares_overflow(cols, dtype, scale):
    """Up to the largest numbers, whose r is subnormal."""
    import torch
    rows = [make(3, cols, 4, "f32", scale).clamp(-3.3e38, 3.3e38), torch.full((1, cols), scale, device="cuda"),
            torch.where(torch.arange(cols, device="cuda") == cols - 1, -scale, 1.0)[None]]
    x = torch.cat(rows).to(dt(dtype))
    assert x.isfinite().all()
    for eps in (0.0, 1e-6, 1e30):
        got = run(x, None, None, eps=eps, out_dtype=dt("f32"), sum_=False)
        check(got, reference(x, None, None, eps, 0.0, dt("f32"), False))
        assert got["out"].isfinite().all() and (got["out"][3].abs() > 0.5).all()


@pytest.mark.parametrize("cols", [500, 4100, 8192, 32768])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-9, 1e-14, 1e-16, 1e-20, 1e-30, 1e-34, 1e-36, 1e-37, 3e-38, 1e-38])
def test_rows_whose_squares_underflow(cols, dtype, scale):
    """Without eps, and with one as small as the squares or far above them, down to subnormal values."""
    import torch
    x = torch.cat([make(4, cols, 5, "f32", scale), torch.full((1, cols), scale, device="cuda")]).to(dt(dtype))
    for eps in (0.0, 1e-45, 1e-36, scale * scale, 1e-24, 1e-6):
        got = run(x, None, None, eps=eps, out_dtype=dt("f32"), sum_=False)
        check(got, reference(x, None, None, eps, 0.0, dt("f32"), False))


def test_rows_of_subnormal_values():
    """r itself leaves fp32's range below an rms of 2^-128."""
    import torch
    x = torch.stack([torch.full((300,), v, device="cuda") for v in (1e-38, 5e-39, 2.94e-39, 2.9e-39, 1e-40, 1e-45)])
    got = run(x, None, None, eps=0.0, out_dtype=dt("f32"), sum_=False, q=False)
    check(got, reference(x, None, None, 0.0, 0.0, dt("f32"), False))
    assert (got["out"][:2] > 0.99).all() and (got["out"][4:] == float("inf")).all()


# more rows than CTAs, for one to eight pieces of eight columns a thread, whole and ragged
@pytest.mark.parametrize("rows,cols", [(16000, 256), (16000, 251), (1000, 4096), (1000, 4090), (400, 4104), (400, 5001), (330, 8192),
                                       (330, 8200), (330, 16383), (320, 16400), (320, 20003)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["apart", "sum is residual", "sum is x, out is residual", "out is x"])
def test_several_rows_to_a_block(rows, cols, dtype, where):
    """A row's loads are under way while the one before is worked on, and may be written where that one's were."""
    import torch
    x, r, w = make(rows, cols, 1, dtype), make(rows, cols, 2, dtype), make(1, cols, 3, "bf16")[0]
    want = reference(x, w, r, 1e-6, 0.0, dt(dtype), False)
    if where == "apart":
        check(run(x, w, r, out_dtype=dt(dtype)), want)
        return
    kw = {"sum is residual": dict(residual_out=r), "sum is x, out is residual": dict(residual_out=x, out=r), "out is x": dict(out=x)}[where]
    mx.fp8_rmsnorm(x, w, residual=r, **kw)
    torch.cuda.synchronize()
    check({"sum" if k == "residual_out" else k: t for k, t in kw.items()}, want)
