"""Host-side argument checks of the FP8 block-scaled entry points (no GPU: they run before any CUDA call)."""
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


@pytest.fixture(scope="module")
def L():
    mxbuild.build()
    return mx.lib()


def rows(**kw):
    r = mx.Fp8Rows(FAKE, FAKE + 0x100000, 4, 256, 256, 1, 4)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def matrix(rows_=64, cols=256, count=1, **kw):
    m = mx.Fp8Matrix(FAKE + 0x200000, FAKE + 0x300000, rows_, cols, count, -(-cols // 16) * 16)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def layer(E=4, D=256, I=128, S=64, **kw):
    l = mx.Fp8LayerStruct()
    l.gate, l.up, l.down = matrix(I, D, E), matrix(I, D, E), matrix(D, I, E)
    if S:
        l.shared_gate, l.shared_up, l.shared_down = matrix(S, D), matrix(S, D), matrix(D, S)
    l.top_k, l.act_dtype, l.activation, l.layer_scalar = 2, mx.MX_BF16, mx.MX_SILU, 1.0
    for k, v in kw.items():
        setattr(l, k, v)
    return l


@pytest.mark.parametrize("name,fields", [
    ("mx_fp8_matrix", ("w", "scales", "rows", "cols", "count", "ld")),
    ("mx_fp8_rows", ("q", "scales", "rows", "cols", "ld", "scale_row", "scale_block")),
    ("mx_fp8_layer", ("gate", "up", "down", "shared_gate", "shared_up", "shared_down", "top_k", "act_dtype",
                      "activation", "layer_scalar")),
])
def test_structs_match_the_header(tmp_path, name, fields):
    cls = {"mx_fp8_matrix": mx.Fp8Matrix, "mx_fp8_rows": mx.Fp8Rows, "mx_fp8_layer": mx.Fp8LayerStruct}[name]
    src = tmp_path / "off.c"
    body = "".join(f'    printf("{f} %zu\\n", offsetof({name}, {f}));\n' for f in fields)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mx_moe.h"\nint main(void) {\n' + body
                   + f'    printf("size %zu\\n", sizeof({name}));\n    return 0;\n}}\n')
    exe = tmp_path / "off"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert [f for f, _ in cls._fields_] == list(fields)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f
    assert int(got["size"]) == C.sizeof(cls)


# ------------------------------------------------------------------ quantise

def quantize(L, r=None, x=FAKE, ldx=256, dtype=mx.MX_BF16, pow2=0):
    return L.mx_fp8_quantize(x, ldx, dtype, pow2, C.byref(r or rows()), None)


@pytest.mark.parametrize("kw,field,status", [
    (dict(x=0), {}, INVALID), (dict(x=FAKE + 1), {}, ALIGN), (dict(x=FAKE + 2, dtype=mx.MX_F32), {}, ALIGN),
    (dict(ldx=255), {}, INVALID), (dict(dtype=2), {}, INVALID), (dict(pow2=2), {}, INVALID),
    ({}, dict(rows=-1), INVALID), ({}, dict(cols=0), UNSUP), ({}, dict(cols=1 << 21, ld=1 << 21), UNSUP),
    ({}, dict(ld=255), INVALID), ({}, dict(q=0), INVALID), ({}, dict(scales=0), INVALID),
    ({}, dict(scales=FAKE + 2), ALIGN), ({}, dict(scale_row=-1), INVALID),
])
def test_quantize_rejections(L, kw, field, status):
    assert quantize(L, rows(**field), **kw) == status
    assert len(L.mx_last_error_string()) > 0


def test_calls_without_rows_do_nothing(L):
    assert quantize(L, rows(rows=0, q=0, scales=0), x=0) == OK
    assert matmul(L, rows(rows=0, q=0, scales=0), out=0, ws=None, nb=0) == OK
    assert moe(L, layer(), T=0) == OK


# ------------------------------------------------------------------ products

def matmul(L, r=None, m=None, out=FAKE + 0x400000, ldo=64, dtype=mx.MX_BF16, ws=FAKE + 0x500000, nb=256, offsets=None):
    a = [C.byref(r or rows())]
    if offsets is not None:
        return L.mx_fp8_grouped_matmul(*a, offsets, C.byref(m or matrix()), out, ldo, dtype, None, ws, nb)
    return L.mx_fp8_matmul(*a, C.byref(m or matrix()), out, ldo, dtype, None, ws, nb)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("kw,r,m,status", [
    (dict(out=0), {}, {}, INVALID), (dict(out=FAKE + 1), {}, {}, ALIGN), (dict(ldo=63), {}, {}, INVALID),
    (dict(dtype=5), {}, {}, INVALID), (dict(ws=None), {}, {}, WS), (dict(nb=255), {}, {}, WS),
    (dict(ws=FAKE + 128), {}, {}, ALIGN), ({}, dict(q=FAKE + 8), {}, ALIGN), ({}, dict(ld=264), {}, ALIGN),
    ({}, dict(ld=240), {}, INVALID), ({}, dict(cols=128), {}, INVALID), ({}, {}, dict(w=0), INVALID),
    ({}, {}, dict(scales=0), INVALID), ({}, {}, dict(w=FAKE + 4), ALIGN), ({}, {}, dict(ld=250), INVALID),
    ({}, {}, dict(ld=260), ALIGN), ({}, {}, dict(rows=0), UNSUP), ({}, {}, dict(count=0), None),
    ({}, {}, dict(count=513), None),
])
def test_product_rejections(L, kw, r, m, status, grouped):
    if grouped:
        kw = dict(kw, offsets=FAKE + 0x600000)
    if status is None:  # a wrong number of matrices
        status = UNSUP if grouped else INVALID
    assert matmul(L, rows(**r), matrix(**m), **kw) == status
    assert len(L.mx_last_error_string()) > 0


def test_grouped_offsets_pointer(L):
    assert matmul(L, offsets=0) == INVALID
    assert matmul(L, offsets=FAKE + 2) == ALIGN
    assert L.mx_fp8_matmul(C.byref(rows()), C.byref(matrix(count=2)), FAKE, 64, 1, None, FAKE, 256) == INVALID


def test_matmul_workspace(L):
    assert L.mx_fp8_matmul_workspace_bytes(C.byref(matrix()), 4096) >= 256
    assert L.mx_fp8_matmul_workspace_bytes(C.byref(matrix(rows=0)), 4) == 0


# --------------------------------------------------------------------- layer

def moe(L, l, T=4, x=FAKE, idx=FAKE + 0x1000000, w=FAKE + 0x1100000, res=None, out=FAKE + 0x1200000,
        ws=FAKE + 0x1300000, nb=None):
    if nb is None:
        nb = L.mx_fp8_moe_workspace_bytes(C.byref(l), T)
    return L.mx_fp8_moe_forward(x, T, idx, w, C.byref(l), res, out, None, ws, nb)


@pytest.mark.parametrize("change,status", [
    (dict(top_k=0), INVALID), (dict(top_k=33), INVALID), (dict(act_dtype=2), INVALID), (dict(activation=2), INVALID),
    (dict(up=matrix(64, 256, 4)), INVALID), (dict(down=matrix(256, 128, 3)), INVALID),
    (dict(shared_up=matrix(128, 256)), INVALID), (dict(shared_down=matrix(256, 64, 2)), INVALID),
    (dict(shared_gate=matrix(64, 272)), INVALID), (dict(gate=matrix(128, 256, 513)), UNSUP),
])
def test_layer_rejections(L, change, status):
    assert moe(L, layer(**change), nb=1 << 40) == status
    assert L.mx_fp8_moe_workspace_bytes(C.byref(layer(**change)), 4) == 0


@pytest.mark.parametrize("T", [4, 64, 65])
def test_moe_pointer_and_workspace_rejections(L, T):
    l = layer()
    need = L.mx_fp8_moe_workspace_bytes(C.byref(l), T)
    assert need > 0
    for kw in (dict(x=0), dict(idx=0), dict(w=0), dict(out=0), dict(T=-1, nb=1 << 40)):
        assert moe(L, l, **dict(dict(T=T), **kw)) == INVALID
    for kw in (dict(x=FAKE + 8), dict(out=FAKE + 0x1200008), dict(res=FAKE + 4), dict(idx=FAKE + 2), dict(ws=FAKE + 128)):
        assert moe(L, l, **dict(dict(T=T), **kw)) == ALIGN
    assert moe(L, l, T=T, nb=need - 1) == WS
    assert moe(L, l, T=T, ws=None) == WS
    assert moe(L, l, T=T, out=FAKE + 256) == INVALID  # overlaps x without being it
    assert moe(L, l, T=T, res=FAKE + 0x1200100) == INVALID


def test_moe_workspace_grows(L):
    l = layer()
    sizes = [L.mx_fp8_moe_workspace_bytes(C.byref(l), t) for t in (0, 1, 16, 17, 64, 65, 4096)]
    assert sizes == sorted(sizes)
    assert L.mx_fp8_moe_workspace_bytes(C.byref(l), -1) == 0


# ------------------------------------------------------------------- binding

def test_binding_checks_tensors():
    import torch
    f8 = torch.float8_e4m3fn
    w, s = torch.zeros(64, 256).to(f8), torch.zeros(1, 2)
    weight = mx.Fp8Weight(w, s)
    assert (weight.c.rows, weight.c.cols, weight.c.count, weight.c.ld) == (64, 256, 1, 256)
    for bad in ((w.float(), s), (w, s.double()), (w, torch.zeros(2, 2)), (w.t(), s), (w, torch.zeros(2, 4)[:1, ::2])):
        with pytest.raises(mx.MxError):
            mx.Fp8Weight(*bad)
    q, qs, out, ws = torch.zeros(4, 256).to(f8), torch.zeros(4, 2), torch.zeros(4, 64), torch.zeros(256, dtype=torch.uint8)
    for args in ((q, qs, weight, out[:, :63], ws), (q, qs[:3], weight, out, ws), (q.float(), qs, weight, out, ws),
                 (q, qs, weight, out.half(), ws), (q, qs, weight, out, ws)):  # (the last one: not on a GPU)
        with pytest.raises(mx.MxError):
            mx.fp8_matmul(*args)
    with pytest.raises(mx.MxError):
        mx.fp8_grouped_matmul(q, qs, torch.zeros(3, dtype=torch.int32), weight, out, ws)
    with pytest.raises(mx.MxError):
        mx.fp8_quantize(torch.zeros(4, 255), q, qs)
    big, down = torch.zeros(2, 128, 256).to(f8), torch.zeros(2, 256, 128).to(f8)
    pair, dpair = (big, torch.zeros(2, 1, 2)), (down, torch.zeros(2, 2, 1))
    lay = mx.Fp8Layer(pair, pair, dpair, top_k=2)
    x, idx, wt = torch.zeros(4, 256).bfloat16(), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args in ((x.float(), idx, wt, lay, x, ws), (x[:, :128], idx, wt, lay, x, ws), (x, idx.long(), wt, lay, x, ws),
                 (x, idx, wt[:3], lay, x, ws), (x, idx, wt, lay, x, ws)):
        with pytest.raises(mx.MxError):
            mx.fp8_moe_forward(*args)
