"""Host-side argument checks of routing from logits, the RMS norm and the 4-bit operators, of the C calls and of the torch
binding (no GPU: they run before any CUDA call)."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import pytest

import expert_ffn_gb300 as mx
from expert_ffn_gb300 import build as mxbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4
FAKE = 0x7F0000000000  # aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    mxbuild.build()
    return mx.lib()


@pytest.mark.parametrize("name,cls", [("mx_rmsnorm", mx.RmsnormStruct), ("mx_fp4_matrix", mx.Fp4Matrix),
                                      ("mx_fp4_rows", mx.Fp4Rows), ("mx_router", mx.RouterStruct)])
def test_structs_match_the_header(tmp_path, name, cls):
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "off.c"
    body = "".join(f'    printf("{f} %zu\\n", offsetof({name}, {f}));\n' for f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mx_moe.h"\nint main(void) {\n' + body
                   + f'    printf("size %zu\\n", sizeof({name}));\n    return 0;\n}}\n')
    exe = tmp_path / "off"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f
    assert int(got["size"]) == C.sizeof(cls)


def test_packed_descriptors_have_the_structs_sizes():
    assert mx._NORM.size == C.sizeof(mx.RmsnormStruct)
    assert mx._FP4.size == C.sizeof(mx.Fp4Rows)


# ------------------------------------------------------------------- routing

def router(**kw):
    r = mx.RouterStruct(64, 4, mx.MX_SIGMOID, 8, 2, 2, 1, 1.0, FAKE)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def route(L, r=None, T=4, logits=FAKE, ld=64, dtype=mx.MX_F32, idx=FAKE, w=FAKE, counts=FAKE, offsets=FAKE, perm=FAKE,
          ws=FAKE, n=1 << 20):
    return L.mx_route_logits(logits, ld, dtype, T, C.byref(r) if r is not None else None, idx, w, counts, offsets, perm,
                             None, ws, n)


@pytest.mark.parametrize("field,status", [
    (dict(n_experts=0), UNSUP), (dict(n_experts=513), UNSUP), (dict(n_groups=0), INVALID), (dict(n_groups=33), INVALID),
    (dict(n_groups=7), INVALID), (dict(topk_groups=0), INVALID), (dict(topk_groups=9), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=17), INVALID), (dict(n_groups=1, topk_groups=1, top_k=33), INVALID), (dict(score=2), INVALID),
    (dict(group_best=0), INVALID), (dict(group_best=3), INVALID), (dict(n_experts=32, n_groups=32, topk_groups=8), INVALID),
    (dict(renormalise=2), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(bias=FAKE + 2), ALIGN),
])
def test_router_refusals(L, field, status):
    r = router(**field)
    assert route(L, r, ld=1024) == status
    assert L.mx_route_logits_workspace_bytes(C.byref(r), 4) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(T=1 << 30), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(ld=63), INVALID), (dict(ld=1 << 40), UNSUP),
    (dict(dtype=2), INVALID), (dict(logits=0), INVALID), (dict(idx=0), INVALID), (dict(w=0), INVALID),
    (dict(counts=0), INVALID), (dict(offsets=0), INVALID), (dict(perm=0), INVALID), (dict(counts=0, offsets=0), INVALID),
    (dict(logits=FAKE + 2), ALIGN), (dict(logits=FAKE + 1, dtype=mx.MX_BF16), ALIGN), (dict(idx=FAKE + 2), ALIGN),
    (dict(w=FAKE + 2), ALIGN), (dict(counts=FAKE + 2), ALIGN), (dict(offsets=FAKE + 1), ALIGN), (dict(perm=FAKE + 2), ALIGN),
    (dict(ws=0), WS), (dict(n=255), WS), (dict(ws=FAKE + 128), ALIGN),
])
def test_route_refusals(L, kw, status):
    assert route(L, router(), **kw) == status


def test_route_needs_a_router_and_no_workspace_without_grouping(L):
    assert route(L, None) == INVALID
    assert route(L, router(), T=0, counts=0, offsets=0, perm=0, ws=0, n=0) == OK  # no tokens: nothing is launched
    assert L.mx_route_logits_workspace_bytes(C.byref(router()), -1) == 0


@pytest.mark.parametrize("E", [1, 60, 256, 257, 512])
def test_route_workspace_holds_any_fewer_tokens(L, E):
    r = router(n_experts=E, n_groups=1, topk_groups=1, group_best=1, top_k=1)
    need = lambda T: L.mx_route_logits_workspace_bytes(C.byref(r), T)  # noqa: E731
    sizes = [0, 1, 8, 9, 64, 2047, 2048, 2049, 2100, 4096, 8192, 16384, 16385, 30000, 114688, 114689, 200000, 1 << 20]
    got = [need(T) for T in sizes]
    assert got == sorted(got) and got[0] >= 256
    for T, n in zip(sizes, got):  # what the call asks for is never above what the query said for more tokens
        assert route(L, r, T=T, ld=512, ws=FAKE + 1, n=n) != WS
        assert route(L, r, T=T, ld=512, ws=FAKE + 1, n=255) == WS


# ---------------------------------------------------------------------- norm

def norm(L, **kw):
    n = mx.RmsnormStruct(FAKE, 256, FAKE + (1 << 20), 256, FAKE + (2 << 20), FAKE + (3 << 20), 256, FAKE + (4 << 20), 256,
                         mx.Fp8Rows(FAKE + (5 << 20), FAKE + (6 << 20), 4, 256, 256, 1, 4), 4, 256, mx.MX_BF16, mx.MX_BF16,
                         mx.MX_BF16, 0, 1e-6, 0.0)
    for k, v in kw.items():
        obj = n
        *path, last = k.split("__")
        for p in path:
            obj = getattr(obj, p)
        setattr(obj, last, v)
    return L.mx_fp8_rmsnorm(C.byref(n), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(weight_dtype=-1), INVALID), (dict(out_dtype=3), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=0), UNSUP), (dict(cols=32769), UNSUP), (dict(pow2=2), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(eps=1.1e30), INVALID), (dict(weight_offset=NAN), INVALID), (dict(x=0), INVALID),
    (dict(sum=0, out=0, q__q=0), INVALID), (dict(q__rows=3), INVALID), (dict(q__cols=255), INVALID),
    (dict(q__scales=0), INVALID), (dict(q__ld=255), INVALID), (dict(q__scale_row=-1), INVALID),
    (dict(q__scale_block=-1), INVALID), (dict(q__ld=1 << 40), UNSUP), (dict(q__scales=FAKE + 2), ALIGN),
    (dict(ldx=255), INVALID), (dict(ldr=255), INVALID), (dict(lds=255), INVALID), (dict(ldo=255), INVALID),
    (dict(ldx=1 << 40), UNSUP), (dict(x=FAKE + 1), ALIGN), (dict(residual=FAKE + 1), ALIGN), (dict(weight=FAKE + 1), ALIGN),
    (dict(weight=FAKE + 2, weight_dtype=mx.MX_F32), ALIGN), (dict(sum=FAKE + 1), ALIGN),
    (dict(out=FAKE + 2, out_dtype=mx.MX_F32), ALIGN),
    # in place with other rows or types, and outputs in one another's place
    (dict(sum=FAKE, lds=264), INVALID), (dict(sum=FAKE + (1 << 20), lds=264), INVALID), (dict(out=FAKE, ldo=264), INVALID),
    (dict(out=FAKE, out_dtype=mx.MX_F32), INVALID), (dict(out=FAKE + (1 << 20), out_dtype=mx.MX_F32), INVALID),
    (dict(out=FAKE + (3 << 20)), INVALID), (dict(q__q=FAKE), INVALID), (dict(q__q=FAKE + (3 << 20)), INVALID),
    (dict(q__q=FAKE + (4 << 20)), INVALID),
])
def test_norm_refusals(L, kw, status):
    assert norm(L, **kw) == status


def test_norm_of_no_rows_is_done(L):
    assert norm(L, rows=0, q__rows=0) == OK
    assert norm(L, rows=0, x=0, sum=0, out=0, q__q=0) == OK  # (tensors without rows have no address)
    assert L.mx_fp8_rmsnorm(None, None) == INVALID


# --------------------------------------------------------------------- 4 bits

def rows4(**kw):
    r = mx.Fp4Rows(FAKE, FAKE + (1 << 20), None, 4, 512, mx.MX_FP4_E4M3, 256)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def matrix4(**kw):
    m = mx.Fp4Matrix(FAKE + (2 << 20), FAKE + (3 << 20), None, 64, 512, 1, mx.MX_FP4_E4M3, 256)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


ROWS4 = [(dict(rows=-1), INVALID), (dict(rows=(1 << 28) + 1), INVALID), (dict(cols=0), UNSUP),
         (dict(cols=(1 << 20) + 1, ld=1 << 20), UNSUP), (dict(format=2), INVALID), (dict(ld=255), INVALID),
         (dict(ld=1 << 23), UNSUP), (dict(q=0), INVALID), (dict(scales=0), INVALID), (dict(scales=FAKE + 8), ALIGN),
         (dict(tensor_scale=FAKE + 2), ALIGN), (dict(format=mx.MX_FP4_E8M0, tensor_scale=FAKE), INVALID)]


@pytest.mark.parametrize("field,status", ROWS4)
def test_quantize4_refuses_rows(L, field, status):
    assert L.mx_fp4_quantize(FAKE, 1 << 20, mx.MX_BF16, C.byref(rows4(**field)), None) == status


@pytest.mark.parametrize("kw,status", [(dict(x=0), INVALID), (dict(x=FAKE + 1), ALIGN), (dict(x=FAKE + 2, dtype=mx.MX_F32), ALIGN),
                                       (dict(ldx=511), INVALID), (dict(ldx=1 << 40), UNSUP), (dict(dtype=2), INVALID)])
def test_quantize4_refusals(L, kw, status):
    a = dict(x=FAKE, ldx=512, dtype=mx.MX_BF16)
    a.update(kw)
    assert L.mx_fp4_quantize(a["x"], a["ldx"], a["dtype"], C.byref(rows4()), None) == status
    assert L.mx_fp4_quantize(0, 512, mx.MX_BF16, C.byref(rows4(rows=0)), None) == OK
    assert L.mx_fp4_quantize(FAKE, 512, mx.MX_BF16, None, None) == INVALID


def product4(L, x=None, w=None, out=FAKE + (4 << 20), ldo=64, dtype=mx.MX_BF16, ws=FAKE, n=256, grouped=False,
             offsets=FAKE):
    a = C.byref(x or rows4()), C.byref(w or matrix4()), out, ldo, dtype, None, ws, n
    return L.mx_fp4_grouped_matmul(a[0], offsets, *a[1:]) if grouped else L.mx_fp4_matmul(*a)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("field,status", ROWS4 + [(dict(q=FAKE + 8), ALIGN), (dict(ld=264), ALIGN), (dict(cols=510), INVALID),
                                                  (dict(format=mx.MX_FP4_E8M0), INVALID)])
def test_product4_refuses_rows(L, grouped, field, status):
    assert product4(L, x=rows4(**field), grouped=grouped) == status


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("field,status", [
    (dict(rows=0), UNSUP), (dict(rows=(1 << 20) + 1), UNSUP), (dict(cols=0), UNSUP), (dict(count=0), None),
    (dict(count=513), None), (dict(format=-1), INVALID), (dict(ld=255), INVALID), (dict(ld=264), ALIGN), (dict(q=0), INVALID),
    (dict(scales=0), INVALID), (dict(q=FAKE + 8), ALIGN), (dict(scales=FAKE + 4), ALIGN), (dict(tensor_scale=FAKE + 1), ALIGN),
    (dict(format=mx.MX_FP4_E8M0, tensor_scale=FAKE), INVALID),
])
def test_product4_refuses_matrices(L, grouped, field, status):
    m = matrix4(**field)
    want = status if status is not None else (UNSUP if grouped else INVALID)
    assert product4(L, w=m, grouped=grouped) == want
    assert L.mx_fp4_matmul_workspace_bytes(C.byref(m), 4) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(ldo=63), INVALID), (dict(ldo=1 << 40), UNSUP), (dict(dtype=2), INVALID), (dict(out=0), INVALID),
    (dict(out=FAKE + 1), ALIGN), (dict(out=FAKE + 2, dtype=mx.MX_F32), ALIGN), (dict(ws=0), WS), (dict(n=255), WS),
    (dict(ws=FAKE + 64), ALIGN), (dict(grouped=True, offsets=0), INVALID), (dict(grouped=True, offsets=FAKE + 2), ALIGN),
])
def test_product4_refusals(L, kw, status):
    assert product4(L, **kw) == status


def test_product4_of_no_rows_and_pointers(L):
    assert product4(L, x=rows4(rows=0), ws=0, n=0) == OK
    assert product4(L, w=matrix4(count=2)) == INVALID
    assert L.mx_fp4_matmul(None, C.byref(matrix4()), FAKE, 64, 1, None, FAKE, 256) == INVALID
    assert L.mx_fp4_matmul(C.byref(rows4()), None, FAKE, 64, 1, None, FAKE, 256) == INVALID
    assert L.mx_fp4_matmul_workspace_bytes(C.byref(matrix4()), 1000) >= 256
    assert L.mx_fp4_matmul_workspace_bytes(C.byref(matrix4()), -1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(scales=0), INVALID), (dict(out=0), INVALID), (dict(out=FAKE + 8), ALIGN), (dict(ld=31), INVALID),
    (dict(ld=1 << 23), UNSUP), (dict(rows=0), UNSUP), (dict(cols=0), UNSUP), (dict(count=0), UNSUP), (dict(count=513), UNSUP),
    (dict(format=2), INVALID),
])
def test_pack_refusals(L, kw, status):
    a = dict(scales=FAKE, ld=32, rows=64, cols=512, count=1, format=mx.MX_FP4_E4M3, out=FAKE)
    a.update(kw)
    assert L.mx_fp4_pack_scales(a["scales"], a["ld"], a["rows"], a["cols"], a["count"], a["format"], a["out"], None) == status
    if any(k in kw for k in ("rows", "cols", "count", "format")):
        assert L.mx_fp4_pack_bytes(a["rows"], a["cols"], a["count"], a["format"]) == 0


def test_pack_bytes(L):
    for rows, cols, count, fmt in [(1, 1, 1, 0), (128, 256, 1, 1), (129, 257, 3, 1), (2112, 2816, 2, 0)]:
        per = 512 * (4 if fmt == mx.MX_FP4_E4M3 else 2)
        assert L.mx_fp4_pack_bytes(rows, cols, count, fmt) == count * -(-rows // 128) * -(-cols // 256) * per


# -------------------------------------------------------------------- binding

def test_binding_refuses_before_any_call():
    import torch
    x = torch.zeros(4, 256)
    q, s = mx.fp4_empty(4, 256, 16, device="cpu")
    assert q.shape == (4, 128) and s.shape == (1, 4, 16) and s.dtype is torch.float8_e4m3fn
    q3, s3 = mx.fp4_empty(3, 1037, 32, device="cpu")
    assert q3.shape == (3, 519) and q3.stride(0) == 528 and s3.shape == (5, 3, 8) and s3.dtype is torch.float8_e8m0fnu
    router = mx.Router(8, 2)
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    logits = torch.zeros(4, 8)
    bad = [
        lambda: mx.fp4_empty(4, 256, 8, device="cpu"),
        lambda: mx.fp4_quantize(x, q.to(torch.int32), s),
        lambda: mx.fp4_quantize(x, q[:, :100], s),
        lambda: mx.fp4_quantize(x[:3], q, s),
        lambda: mx.fp4_quantize(x, q, s.view(torch.uint8)),
        lambda: mx.fp4_quantize(x, q, s[:, :3]),
        lambda: mx.fp4_quantize(x.half(), q, s),
        lambda: mx.fp4_quantize(x, q, s),  # (not on a GPU)
        lambda: mx.Fp4Weight(torch.zeros(64, 128), torch.zeros(64, 16).to(torch.float8_e4m3fn)),
        lambda: mx.Fp4Weight(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 16)),
        lambda: mx.Fp4Weight(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 15).to(torch.float8_e4m3fn)),
        lambda: mx.Fp4Weight(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 16).to(torch.float8_e4m3fn), cols=254),
        lambda: mx.Fp4Weight(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 16).to(torch.float8_e4m3fn), torch.ones(2)),
        lambda: mx.fp8_rmsnorm(x),
        lambda: mx.fp8_rmsnorm(x.double(), out=x),
        lambda: mx.fp8_rmsnorm(x, out=x[:3]),
        lambda: mx.fp8_rmsnorm(x, out=x.t()),
        lambda: mx.fp8_rmsnorm(x, torch.ones(255), out=x),
        lambda: mx.fp8_rmsnorm(x, residual=x.bfloat16(), out=x),
        lambda: mx.fp8_rmsnorm(x, residual_out=x.bfloat16()),
        lambda: mx.fp8_rmsnorm(x, q=x.to(torch.float8_e4m3fn)),
        lambda: mx.fp8_rmsnorm(x, q=x.to(torch.float8_e4m3fn), scales=torch.zeros(4, 3)),
        lambda: mx.Router(8, 2, bias=torch.zeros(7)),
        lambda: mx.Router(8, 2, bias=torch.zeros(8, dtype=torch.float64)),
        lambda: mx.route_logits(logits[:, :7], router, idx, w),
        lambda: mx.route_logits(logits, router, idx.long(), w),
        lambda: mx.route_logits(logits, router, idx, w[:, :1]),
        lambda: mx.route_logits(logits, router, idx, w, counts=torch.zeros(8, dtype=torch.int32)),
        lambda: mx.route_logits(logits, router, idx, w),  # (not on a GPU)
    ]
    for i, call in enumerate(bad):
        with pytest.raises(mx.MxError):
            call()
            raise AssertionError(f"call {i} was not refused")
