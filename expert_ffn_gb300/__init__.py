"""Python binding of ``libmx_moe.so`` -- the GB300 routed-MoE FFN block.

Argument marshalling only: every step of the block runs in the library's CUDA
kernels.  The library must have been built (``expert_ffn_gb300.build.build()``
or ``__graft_entry__.build()``); if it is missing, loading raises -- there is
no fallback path.  PyTorch provides device memory and streams.
"""
from __future__ import annotations

import ctypes as C
import os
import struct as _struct
import threading

from .build import LIB as LIB_PATH

__all__ = ["MxError", "lib", "QLinear", "Ffn", "Sub", "Layout", "Options", "LAYOUT_MAGIC", "LAYOUT_VERSION",
           "MX_F32", "MX_BF16", "DeviceLayer", "layer_forward", "layer_forward_ex", "route", "stack_forward",
           "workspace_bytes", "stack_workspace_bytes", "workspace_init", "layer_forward_static", "EXPORTED",
           "down_sb_bytes", "pack_down_sb",
           "MX_GELU_TANH", "MX_SILU", "Fp8Matrix", "Fp8Rows", "Fp8LayerStruct", "Fp8Weight", "Fp8Layer",
           "fp8_quantize", "fp8_matmul", "fp8_grouped_matmul", "fp8_moe_forward", "fp8_matmul_workspace_bytes",
           "fp8_moe_workspace_bytes",
           "RmsnormStruct", "fp8_rmsnorm",
           "MX_FP4_E8M0", "MX_FP4_E4M3", "Fp4Matrix", "Fp4Rows", "Fp4Weight", "fp4_empty", "fp4_quantize", "fp4_matmul",
           "fp4_grouped_matmul", "fp4_matmul_workspace_bytes",
           "MX_SOFTMAX", "MX_SIGMOID", "RouterStruct", "Router", "route_logits", "route_logits_workspace_bytes"]

LAYOUT_MAGIC = 0x4D584D45
LAYOUT_VERSION = 3
MX_F32, MX_BF16 = 0, 1
MX_GELU_TANH, MX_SILU = 0, 1
MX_FP4_E8M0, MX_FP4_E4M3 = 0, 1
MX_SOFTMAX, MX_SIGMOID = 0, 1

# Every symbol include/mx_moe.h declares.
EXPORTED = ("mx_moe_layer_forward", "mx_moe_layer_forward_ex", "mx_moe_workspace_bytes", "mx_moe_workspace_init",
            "mx_moe_route", "mx_moe_stack_forward", "mx_moe_stack_workspace_bytes", "mx_status_string",
            "mx_last_error_string", "mx_version", "mx_moe_profile_enable", "mx_moe_profile_read",
            "mx_moe_workspace_check", "mx_moe_layer_forward_static", "mx_moe_down_sb_bytes", "mx_moe_pack_down_sb",
            "mx_fp8_quantize", "mx_fp8_matmul", "mx_fp8_grouped_matmul", "mx_fp8_matmul_workspace_bytes",
            "mx_fp8_moe_forward", "mx_fp8_moe_workspace_bytes", "mx_fp8_rmsnorm", "mx_fp4_quantize",
            "mx_fp4_matmul", "mx_fp4_grouped_matmul", "mx_fp4_matmul_workspace_bytes", "mx_fp4_pack_bytes",
            "mx_fp4_pack_scales", "mx_route_logits",
            "mx_route_logits_workspace_bytes")


class MxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status}: {msg}")
        self.status = status


class QLinear(C.Structure):
    _fields_ = [("w", C.c_void_p), ("scales", C.c_void_p), ("biases", C.c_void_p),
                ("rows", C.c_int32), ("cols", C.c_int32), ("bits", C.c_int32)]


class Ffn(C.Structure):
    _fields_ = [("gate", QLinear), ("up", QLinear), ("down", QLinear)]


class Sub(C.Structure):
    _fields_ = [("w", C.c_uint64), ("s", C.c_uint64), ("b", C.c_uint64)]


class Layout(C.Structure):
    _fields_ = [("magic", C.c_uint32), ("version", C.c_uint32), ("d_model", C.c_int32), ("d_expert", C.c_int32),
                ("n_experts", C.c_int32), ("top_k", C.c_int32), ("d_shared", C.c_int32), ("group", C.c_int32),
                ("bits", C.c_int32), ("record_stride", C.c_uint64), ("gate", Sub), ("up", Sub), ("down", Sub),
                ("act_dtype", C.c_int32), ("layer_scalar", C.c_float), ("per_expert_scale", C.c_void_p),
                # version 2: optional parts of the layer (NULL = absent)
                ("expert_slot", C.c_void_p), ("n_slots", C.c_int32), ("router_scale", C.c_void_p),
                ("post_norm", C.c_void_p), ("post_eps", C.c_float), ("shared_expert_gate", C.c_void_p),
                # version 3: the packed down-projection scale / bias words (NULL = absent)
                ("down_sb", C.c_void_p)]


class Options(C.Structure):
    _fields_ = [("residual", C.c_void_p), ("pre_rmsnorm", C.c_int32), ("rms_eps", C.c_float)]


class Fp8Matrix(C.Structure):
    _fields_ = [("w", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int32), ("cols", C.c_int32),
                ("count", C.c_int32), ("ld", C.c_int64)]


class Fp8Rows(C.Structure):
    _fields_ = [("q", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int32), ("cols", C.c_int32),
                ("ld", C.c_int64), ("scale_row", C.c_int64), ("scale_block", C.c_int64)]


class Fp8LayerStruct(C.Structure):
    _fields_ = [(name, Fp8Matrix) for name in ("gate", "up", "down", "shared_gate", "shared_up", "shared_down")] + [
        ("top_k", C.c_int32), ("act_dtype", C.c_int32), ("activation", C.c_int32), ("layer_scalar", C.c_float)]


class RmsnormStruct(C.Structure):
    _fields_ = [("x", C.c_void_p), ("ldx", C.c_int64), ("residual", C.c_void_p), ("ldr", C.c_int64),
                ("weight", C.c_void_p), ("sum", C.c_void_p), ("lds", C.c_int64), ("out", C.c_void_p),
                ("ldo", C.c_int64), ("q", Fp8Rows), ("rows", C.c_int32), ("cols", C.c_int32),
                ("dtype", C.c_int32), ("weight_dtype", C.c_int32), ("out_dtype", C.c_int32), ("pow2", C.c_int32),
                ("eps", C.c_float), ("weight_offset", C.c_float)]


class Fp4Matrix(C.Structure):
    _fields_ = [("q", C.c_void_p), ("scales", C.c_void_p), ("tensor_scale", C.c_void_p), ("rows", C.c_int32),
                ("cols", C.c_int32), ("count", C.c_int32), ("format", C.c_int32), ("ld", C.c_int64)]


class Fp4Rows(C.Structure):
    _fields_ = [("q", C.c_void_p), ("scales", C.c_void_p), ("tensor_scale", C.c_void_p), ("rows", C.c_int32),
                ("cols", C.c_int32), ("format", C.c_int32), ("ld", C.c_int64)]


class RouterStruct(C.Structure):
    _fields_ = [("n_experts", C.c_int32), ("top_k", C.c_int32), ("score", C.c_int32), ("n_groups", C.c_int32),
                ("topk_groups", C.c_int32), ("group_best", C.c_int32), ("renormalise", C.c_int32),
                ("scale", C.c_float), ("bias", C.c_void_p)]


_lock = threading.Lock()
_lib = None


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with expert_ffn_gb300.build.build()")
            L = C.CDLL(LIB_PATH)
            P, I32, SZ = C.c_void_p, C.c_int, C.c_size_t
            L.mx_moe_layer_forward.argtypes = [P, I32, C.POINTER(QLinear), C.POINTER(Ffn), P, C.POINTER(Layout),
                                               P, P, P]
            L.mx_moe_layer_forward_ex.argtypes = L.mx_moe_layer_forward.argtypes + [C.POINTER(Options), P, P, SZ]
            L.mx_moe_layer_forward_static.argtypes = L.mx_moe_layer_forward.argtypes + [C.POINTER(Options), P]
            L.mx_moe_workspace_bytes.argtypes = [C.POINTER(Layout), I32]
            L.mx_moe_workspace_bytes.restype = SZ
            L.mx_moe_stack_workspace_bytes.argtypes = [C.POINTER(Layout), I32]
            L.mx_moe_stack_workspace_bytes.restype = SZ
            L.mx_moe_workspace_init.argtypes = [P, SZ, P]
            L.mx_moe_down_sb_bytes.argtypes = [C.POINTER(Layout)]
            L.mx_moe_down_sb_bytes.restype = SZ
            L.mx_moe_pack_down_sb.argtypes = [C.POINTER(Layout), P, C.POINTER(QLinear), P, P]
            L.mx_moe_route.argtypes = [P, I32, C.POINTER(QLinear), C.POINTER(Layout), P, P, P, P, P, P,
                                       C.POINTER(Options), P, P, SZ]
            L.mx_moe_stack_forward.argtypes = [P, I32, I32, C.POINTER(QLinear), C.POINTER(Ffn), C.POINTER(P),
                                               C.POINTER(Layout), P, P, C.c_float, P, P, SZ]
            L.mx_status_string.argtypes = [I32]
            L.mx_status_string.restype = C.c_char_p
            L.mx_last_error_string.restype = C.c_char_p
            L.mx_version.restype = C.c_char_p
            L.mx_moe_profile_enable.argtypes = [I32]
            L.mx_moe_workspace_check.argtypes = [P, P]
            L.mx_moe_profile_read.argtypes = [C.POINTER(C.c_double), C.POINTER(C.c_int), I32]
            I64 = C.c_int64
            L.mx_fp8_quantize.argtypes = [P, I64, I32, I32, P, P]  # (P: an Fp8Rows, by reference or packed)
            L.mx_fp8_matmul.argtypes = [P, C.POINTER(Fp8Matrix), P, I64, I32, P, P, SZ]
            L.mx_fp8_grouped_matmul.argtypes = [P, P, C.POINTER(Fp8Matrix), P, I64, I32, P, P, SZ]
            L.mx_fp8_matmul_workspace_bytes.argtypes = [C.POINTER(Fp8Matrix), I32]
            L.mx_fp8_matmul_workspace_bytes.restype = SZ
            L.mx_fp8_moe_forward.argtypes = [P, I32, P, P, C.POINTER(Fp8LayerStruct), P, P, P, P, SZ]
            L.mx_fp8_moe_workspace_bytes.argtypes = [C.POINTER(Fp8LayerStruct), I32]
            L.mx_fp8_moe_workspace_bytes.restype = SZ
            L.mx_fp8_rmsnorm.argtypes = [P, P]  # (P: a RmsnormStruct, by reference or packed)
            L.mx_fp4_quantize.argtypes = [P, I64, I32, P, P]  # (P: an Fp4Rows, likewise)
            L.mx_fp4_matmul.argtypes = [P, C.POINTER(Fp4Matrix), P, I64, I32, P, P, SZ]
            L.mx_fp4_grouped_matmul.argtypes = [P, P, C.POINTER(Fp4Matrix), P, I64, I32, P, P, SZ]
            L.mx_fp4_pack_bytes.argtypes = [I32, I32, I32, I32]
            L.mx_fp4_pack_bytes.restype = SZ
            L.mx_fp4_pack_scales.argtypes = [P, I64, I32, I32, I32, I32, P, P]
            L.mx_fp4_matmul_workspace_bytes.argtypes = [C.POINTER(Fp4Matrix), I32]
            L.mx_fp4_matmul_workspace_bytes.restype = SZ
            L.mx_route_logits.argtypes = [P, I64, I32, I32, C.POINTER(RouterStruct), P, P, P, P, P, P, P, SZ]
            L.mx_route_logits_workspace_bytes.argtypes = [C.POINTER(RouterStruct), I32]
            L.mx_route_logits_workspace_bytes.restype = SZ
            for name in ("mx_fp8_rmsnorm", "mx_fp4_quantize", "mx_fp4_matmul", "mx_fp4_grouped_matmul",
                         "mx_fp4_pack_scales", "mx_route_logits",
                         "mx_fp8_quantize", "mx_fp8_matmul", "mx_fp8_grouped_matmul", "mx_fp8_moe_forward",
                         "mx_moe_layer_forward", "mx_moe_layer_forward_ex", "mx_moe_layer_forward_static",
                         "mx_moe_workspace_init", "mx_moe_pack_down_sb",
                         "mx_moe_route", "mx_moe_stack_forward", "mx_moe_profile_enable", "mx_moe_profile_read",
                         "mx_moe_workspace_check"):
                getattr(L, name).restype = C.c_int
            _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        L = lib()
        raise MxError(status, f"{L.mx_status_string(status).decode()}: {L.mx_last_error_string().decode()}")


def _ptr(t):
    """Device (or host) address of a tensor, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_handle(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------- structs

def make_qlinear(w, s, b, rows: int, cols: int, bits: int) -> QLinear:
    return QLinear(_ptr(w), _ptr(s), _ptr(b), rows, cols, bits)


def make_layout(D, I, E, K, S, stride, offsets, act_dtype, lam, per_expert_scale=None, expert_slot=None,
                n_slots=0, router_scale=None, post_norm=None, post_eps=0.0, shared_expert_gate=None,
                down_sb=None) -> Layout:
    L = Layout()
    L.magic, L.version = LAYOUT_MAGIC, LAYOUT_VERSION
    L.d_model, L.d_expert, L.n_experts, L.top_k, L.d_shared = D, I, E, K, S
    L.group, L.bits = 64, 4
    L.record_stride = stride
    for name in ("gate", "up", "down"):
        w, s, b = offsets[name]
        setattr(L, name, Sub(w, s, b))
    L.act_dtype = act_dtype
    L.layer_scalar = lam
    L.per_expert_scale = _ptr(per_expert_scale)
    L.expert_slot = _ptr(expert_slot)
    L.n_slots = n_slots if expert_slot is not None else 0
    L.router_scale = _ptr(router_scale)
    L.post_norm = _ptr(post_norm)
    L.post_eps = post_eps
    L.shared_expert_gate = _ptr(shared_expert_gate)
    L.down_sb = _ptr(down_sb)
    return L


class DeviceLayer:
    """Device copy of one MoE layer given as host arrays.

    ``host`` is any object with attributes D, E, K, I, S, lam, router, shared_gate,
    shared_up, shared_down (each with .w .s .b .rows .cols .bits numpy arrays),
    blob, stride, offsets and optionally per_expert_scale and the layer's
    optional parts expert_slot (int16 [E]) with n_slots, router_scale,
    post_norm (with post_eps) and shared_expert_gate (BF16 bits [D]).

    ``pack_down_sb`` (default on) also builds the layout's packed
    down-projection scale / bias table (mx_moe_pack_down_sb) on the device."""

    def __init__(self, host, act_dtype: int, device="cuda", pack_down_sb: bool = True):
        import numpy as np
        import torch
        self.host = host
        self.act_dtype = act_dtype

        def dev(a):
            return torch.from_numpy(a.reshape(-1).view("uint8")).to(device, non_blocking=False)

        def q(m):
            ts = (dev(m.w), dev(m.s), dev(m.b))
            return ts, make_qlinear(*ts, m.rows, m.cols, m.bits)

        self._router_t, self.router = q(host.router)
        sg_t, sg = q(host.shared_gate)
        su_t, su = q(host.shared_up)
        sd_t, sd = q(host.shared_down)
        self._shared_t = (sg_t, su_t, sd_t)
        self.shared = Ffn(sg, su, sd)
        self.blob = torch.from_numpy(host.blob).to(device)
        assert self.blob.data_ptr() % 256 == 0
        pes = getattr(host, "per_expert_scale", None)
        self.pes = None if pes is None else torch.from_numpy(pes.astype("float32")).to(device)
        def opt(name, dtype):
            a = getattr(host, name, None)
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(device)

        self.expert_slot = opt("expert_slot", np.int16)
        self.router_scale = opt("router_scale", np.uint16)
        self.post_norm = opt("post_norm", np.uint16)
        self.shared_expert_gate = opt("shared_expert_gate", np.uint16)
        self.layout = make_layout(host.D, host.I, host.E, host.K, host.S, host.stride, host.offsets, act_dtype,
                                  host.lam, self.pes, self.expert_slot, int(getattr(host, "n_slots", 0) or 0),
                                  self.router_scale, self.post_norm, float(getattr(host, "post_eps", 0.0)),
                                  self.shared_expert_gate)
        self.down_sb = None
        if pack_down_sb:
            self.down_sb = _pack_down_sb(self.layout, self.blob, self.shared.down, device=device)
            self.layout.down_sb = self.down_sb.data_ptr()

    def set_layer_scalar(self, lam: float):
        self.layout.layer_scalar = lam


# --------------------------------------------------------------- entry points

def down_sb_bytes(layout: Layout) -> int:
    return lib().mx_moe_down_sb_bytes(C.byref(layout))


def _pack_down_sb(layout: Layout, blob, shared_down: QLinear, device="cuda", stream=None):
    """The layout's packed down-projection (scale | bias << 16) words as a new
    device uint8 tensor (mx_moe_pack_down_sb); the copy is done when this
    returns."""
    import torch
    n = down_sb_bytes(layout)
    if n == 0:
        _check(-1)
    out = torch.empty(n, dtype=torch.uint8, device=device)
    _check(lib().mx_moe_pack_down_sb(C.byref(layout), _ptr(blob), C.byref(shared_down), _ptr(out),
                                     _stream_handle(stream)))
    torch.cuda.synchronize(out.device)
    return out


pack_down_sb = _pack_down_sb


def workspace_bytes(layout: Layout, T: int) -> int:
    return lib().mx_moe_workspace_bytes(C.byref(layout), T)


def stack_workspace_bytes(layout: Layout, T: int) -> int:
    return lib().mx_moe_stack_workspace_bytes(C.byref(layout), T)


def workspace_init(ws, nbytes: int, stream=None):
    _check(lib().mx_moe_workspace_init(_ptr(ws), nbytes, _stream_handle(stream)))


def workspace_check(ws, stream=None):
    """Raise MxError(MX_ERR_DEVICE_TIMEOUT) if a device-side wait gave up."""
    _check(lib().mx_moe_workspace_check(_ptr(ws), _stream_handle(stream)))


def layer_forward(x, T, layer: DeviceLayer, out, topk_idx, topk_w):
    _check(lib().mx_moe_layer_forward(_ptr(x), T, C.byref(layer.router), C.byref(layer.shared),
                                      _ptr(layer.blob), C.byref(layer.layout), _ptr(out), _ptr(topk_idx),
                                      _ptr(topk_w)))


def layer_forward_ex(x, T, layer: DeviceLayer, out, topk_idx, topk_w, ws, ws_bytes, stream=None, residual=None,
                     pre_rmsnorm=False, rms_eps=1e-6):
    opt = Options(_ptr(residual), 1 if pre_rmsnorm else 0, rms_eps)
    _check(lib().mx_moe_layer_forward_ex(_ptr(x), T, C.byref(layer.router), C.byref(layer.shared),
                                         _ptr(layer.blob), C.byref(layer.layout), _ptr(out), _ptr(topk_idx),
                                         _ptr(topk_w), C.byref(opt), _stream_handle(stream), _ptr(ws), ws_bytes))


def layer_forward_static(x, T, layer: DeviceLayer, out, topk_idx, topk_w, stream=None, residual=None,
                         pre_rmsnorm=False, rms_eps=1e-6):
    """The block for T <= 4 with the library's fixed device scratch (no workspace, no allocation)."""
    opt = Options(_ptr(residual), 1 if pre_rmsnorm else 0, rms_eps)
    _check(lib().mx_moe_layer_forward_static(_ptr(x), T, C.byref(layer.router), C.byref(layer.shared),
                                             _ptr(layer.blob), C.byref(layer.layout), _ptr(out), _ptr(topk_idx),
                                             _ptr(topk_w), C.byref(opt), _stream_handle(stream)))


def route(x, T, layer: DeviceLayer, topk_idx, topk_w, counts, offsets, perm, ws, ws_bytes, logits=None,
          stream=None, pre_rmsnorm=False, rms_eps=1e-6):
    opt = Options(None, 1 if pre_rmsnorm else 0, rms_eps)
    _check(lib().mx_moe_route(_ptr(x), T, C.byref(layer.router), C.byref(layer.layout), _ptr(topk_idx),
                              _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(logits), C.byref(opt),
                              _stream_handle(stream), _ptr(ws), ws_bytes))


class Stack:
    """Arrays of per-layer C structs for mx_moe_stack_forward."""

    def __init__(self, layers: list[DeviceLayer]):
        n = len(layers)
        self.layers = layers
        self.routers = (QLinear * n)(*[l.router for l in layers])
        self.shareds = (Ffn * n)(*[l.shared for l in layers])
        self.blobs = (C.c_void_p * n)(*[l.blob.data_ptr() for l in layers])
        self.layouts = (Layout * n)(*[l.layout for l in layers])


def stack_forward(x_io, T, stack: Stack, topk_idx, topk_w, ws, ws_bytes, rms_eps=1e-6, stream=None):
    _check(lib().mx_moe_stack_forward(_ptr(x_io), T, len(stack.layers), stack.routers, stack.shareds, stack.blobs,
                                      stack.layouts, _ptr(topk_idx), _ptr(topk_w), rms_eps, _stream_handle(stream),
                                      _ptr(ws), ws_bytes))


PROFILE_STAGES = ("route", "gate_up", "down")


def profile_enable(on: bool):
    _check(lib().mx_moe_profile_enable(1 if on else 0))


def profile_read(reset: bool = True) -> dict:
    """Per-stage summed milliseconds and launch counts since the last reset."""
    ms = (C.c_double * 3)()
    n = (C.c_int * 3)()
    _check(lib().mx_moe_profile_read(ms, n, 1 if reset else 0))
    return {name: (ms[i], n[i]) for i, name in enumerate(PROFILE_STAGES)}


# ------------------------------------------- FP8 block-scaled operators
#
# Tensors carry their own shapes and strides here, so these calls check them: a
# wrong one raises MxError(-1) like a wrong argument of the library.  Work goes
# to `stream`, by default the current stream of the tensors' device.  A call for
# a single token runs for a few microseconds on the GPU, so the marshalling
# keeps to cheap operations: the row descriptor is packed bytes, devices are
# compared by index.

_ROWS = _struct.Struct("@PPiiqqq")  # Fp8Rows
_NORM = _struct.Struct("@PqPqPPqPqPPiiqqqiiiiiiff")  # RmsnormStruct
_FP4 = _struct.Struct("@PPPiiiq")  # Fp4Rows
_t = None  # names of torch, filled on first use


class _Torch:
    def __init__(self):
        import torch
        self.f8, self.f32, self.i32 = torch.float8_e4m3fn, torch.float32, torch.int32
        self.codes = {torch.float32: MX_F32, torch.bfloat16: MX_BF16}
        self.sizes = {MX_F32: 4, MX_BF16: 2}
        self.device = torch.cuda.device
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
        L = lib()
        self.quantize, self.matmul, self.grouped = L.mx_fp8_quantize, L.mx_fp8_matmul, L.mx_fp8_grouped_matmul
        self.moe = L.mx_fp8_moe_forward
        self.norm, self.route = L.mx_fp8_rmsnorm, L.mx_route_logits
        self.quantize4, self.matmul4, self.grouped4 = L.mx_fp4_quantize, L.mx_fp4_matmul, L.mx_fp4_grouped_matmul
        self.u8, self.e8m0 = torch.uint8, torch.float8_e8m0fnu


def _torch():
    global _t
    if _t is None:
        _t = _Torch()
    return _t


def _need(ok, msg):
    if not ok:
        raise MxError(-1, msg)


def _dtype_code(t, name):
    code = _torch().codes.get(t.dtype)
    if code is None:
        raise MxError(-1, f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _on(dev, fn, *args):
    """fn(*args) with the tensors' device current."""
    if dev < 0:
        raise MxError(-1, "tensors must be on a CUDA device")
    if _t.current_device() == dev:
        status = fn(*args)
    else:
        with _t.device(dev):
            status = fn(*args)
    if status:
        _check(status)


def _stream_on(dev, stream):
    """The handle of `stream`, by default of the device's current one."""
    if stream is None:
        return _t.stream(dev) if dev >= 0 else None
    return _stream_handle(stream)


def _bytes_on(dev, stream, n, device):
    """n bytes for the work of `stream`, from that stream's own pool: a block of the current stream's may still be in
    use there, and goes back to it when the tensor goes, whatever `stream` still does with it."""
    import torch
    if dev < 0 or stream is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=device)


def _fp8_matrix(w, scales, name):
    t = _torch()
    _need(w.dtype is t.f8 and w.dim() in (2, 3), f"{name} must be float8_e4m3fn [count,] rows, cols")
    rows, cols = w.shape[-2:]
    count = w.shape[0] if w.dim() == 3 else 1
    ld = w.stride(-2) if rows > 1 else -(-max(cols, w.stride(-2)) // 16) * 16
    _need(w.stride(-1) == 1 or cols == 1, f"{name} must have contiguous rows")
    _need(count == 1 or w.stride(0) == rows * ld, f"{name}: the matrices must follow one another")
    want = (-(-rows // 128), -(-cols // 128))
    _need(scales.dtype is t.f32 and scales.is_contiguous() and tuple(scales.shape[-2:]) == want
          and scales.numel() == count * want[0] * want[1],
          f"{name}: scales must be contiguous float32 [{count}, {want[0]}, {want[1]}]")
    _need(scales.device == w.device, f"{name}: scales must be on {w.device}")
    return Fp8Matrix(w.data_ptr(), scales.data_ptr(), rows, cols, count, ld)


def _fp8_rows(t, q, scales, dev, operand):
    """(rows, columns, packed Fp8Rows) of a pair of tensors."""
    if q.dtype is not t.f8 or scales.dtype is not t.f32:
        raise MxError(-1, "q must be float8_e4m3fn, scales float32")
    shape, strides = q.shape, q.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise MxError(-1, "q must be [rows, cols] with contiguous rows")
    rows, cols = shape
    if scales.shape != (rows, (cols + 127) // 128):
        raise MxError(-1, f"scales must be [{rows}, {(cols + 127) // 128}]")
    if q.get_device() != dev or scales.get_device() != dev:
        raise MxError(-1, "all tensors must be on one device")
    ld = strides[0]
    if rows <= 1:  # (the stride of a single row means nothing)
        ld = (cols + 15) // 16 * 16 if operand else cols
    return rows, cols, _ROWS.pack(q.data_ptr(), scales.data_ptr(), rows, cols, ld, *scales.stride())


class Fp8Weight:
    """Block-scaled e4m3 matrices on the device: ``w`` float8_e4m3fn [rows, cols] or [count, rows, cols], rows at
    multiples of 16 bytes; ``scales`` float32 [count,] ceil(rows / 128), ceil(cols / 128).  The tensors are kept and
    read by every call, not copied."""

    def __init__(self, w, scales):
        self.w, self.scales = w, scales
        self.c = _fp8_matrix(w, scales, "w")
        self.ref, self.rows, self.count, self.dev = C.byref(self.c), self.c.rows, self.c.count, w.get_device()


class Fp8Layer:
    """One MoE layer with FP8 weights.  ``gate``, ``up`` ([E, I, D]), ``down`` ([E, D, I]) and the three of
    ``shared`` ([1, S, D], [1, S, D], [1, D, S], or None) are (w, scales) pairs as for Fp8Weight."""

    def __init__(self, gate, up, down, shared=None, top_k=8, act_dtype=MX_BF16, activation=MX_GELU_TANH,
                 layer_scalar=1.0):
        _need(not shared or len(shared) == 3, "shared must be the (w, scales) pairs of gate, up and down")
        self.tensors = [gate, up, down, *(shared or [])]
        c = Fp8LayerStruct()
        names = ("gate", "up", "down", "shared_gate", "shared_up", "shared_down")
        for name, pair in zip(names, self.tensors):
            setattr(c, name, _fp8_matrix(*pair, name))
            _need(pair[0].device == gate[0].device, f"{name} must be on {gate[0].device}")
        c.top_k, c.act_dtype, c.activation, c.layer_scalar = top_k, act_dtype, activation, layer_scalar
        self.c = c
        self.ref, self.dev, self.d_model, self.top_k = C.byref(c), gate[0].get_device(), c.gate.cols, top_k
        self.dtype = {v: k for k, v in _torch().codes.items()}.get(act_dtype)


def fp8_quantize(x, q, scales, pow2=False, stream=None):
    """Quantise the rows of ``x`` (float32 or bfloat16 [rows, cols]) into ``q`` (float8_e4m3fn) and ``scales``
    (float32 [rows, ceil(cols / 128)], any strides; ``empty(blocks, rows).t()`` suits the products best)."""
    t = _t or _torch()
    dev = x.get_device()
    rows, cols, r = _fp8_rows(t, q, scales, dev, False)
    ldx, one = x.stride() if x.dim() == 2 else (0, 0)
    if x.shape != (rows, cols) or (one != 1 and cols > 1):
        raise MxError(-1, f"x must be [{rows}, {cols}] with contiguous rows")
    _on(dev, t.quantize, x.data_ptr(), ldx if rows > 1 else cols, _dtype_code(x, "x"), 1 if pow2 else 0, r,
        _stream_on(dev, stream))


def fp8_matmul_workspace_bytes(weight: Fp8Weight, rows: int) -> int:
    return lib().mx_fp8_matmul_workspace_bytes(weight.ref, rows)


def _out_pitch(rows, weight, out, ws):
    if out.get_device() != weight.dev or ws.get_device() != weight.dev:
        raise MxError(-1, "all tensors must be on one device")
    n = weight.rows
    ldo, one = out.stride() if out.dim() == 2 else (0, 0)
    if out.shape != (rows, n) or (one != 1 and n > 1):
        raise MxError(-1, f"out must be [{rows}, {n}] with contiguous rows")
    return ldo if rows > 1 else n


def fp8_matmul(q, scales, weight: Fp8Weight, out, ws, stream=None):
    """out = (q, scales) times the transposed ``weight``; out float32 or bfloat16 [rows, weight rows]; ws a
    uint8 workspace of fp8_matmul_workspace_bytes, prepared by workspace_init."""
    t = _t or _torch()
    dev = weight.dev
    rows, _, r = _fp8_rows(t, q, scales, dev, True)
    ldo = _out_pitch(rows, weight, out, ws)
    _on(dev, t.matmul, r, weight.ref, out.data_ptr(), ldo, _dtype_code(out, "out"), _stream_on(dev, stream),
        ws.data_ptr(), ws.nbytes)


def fp8_grouped_matmul(q, scales, offsets, weight: Fp8Weight, out, ws, stream=None):
    """The same with rows [offsets[e], offsets[e + 1]) against matrix e; offsets int32 [count + 1] on the device."""
    t = _t or _torch()
    dev = weight.dev
    rows, _, r = _fp8_rows(t, q, scales, dev, True)
    ldo = _out_pitch(rows, weight, out, ws)
    if (offsets.dtype is not t.i32 or offsets.shape != (weight.count + 1,) or not offsets.is_contiguous()
            or offsets.get_device() != dev):
        raise MxError(-1, f"offsets must be contiguous int32 [{weight.count + 1}] on the weight's device")
    _on(dev, t.grouped, r, offsets.data_ptr(), weight.ref, out.data_ptr(), ldo, _dtype_code(out, "out"),
        _stream_on(dev, stream), ws.data_ptr(), ws.nbytes)


def fp8_moe_workspace_bytes(layer: Fp8Layer, T: int) -> int:
    return lib().mx_fp8_moe_workspace_bytes(layer.ref, T)


def fp8_moe_forward(x, topk_idx, topk_w, layer: Fp8Layer, out, ws, residual=None, stream=None):
    """The block after its routing (mx_fp8_moe_forward): x, out and residual [T, D] of the layer's act_dtype,
    topk_idx int32 and topk_w float32 [T, top_k], all contiguous; ws a uint8 workspace of
    fp8_moe_workspace_bytes, prepared by workspace_init."""
    t = _t or _torch()
    dev, shape = layer.dev, x.shape
    T = shape[0]
    for a in (x, out) if residual is None else (x, out, residual):
        if a.dtype is not layer.dtype or a.shape != (T, layer.d_model) or not a.is_contiguous() or a.get_device() != dev:
            raise MxError(-1, f"x, out and residual must be contiguous [T, {layer.d_model}] tensors of the layer's "
                              "act_dtype on its device")
    k = (T, layer.top_k)
    if (topk_idx.dtype is not t.i32 or topk_idx.shape != k or not topk_idx.is_contiguous() or topk_w.dtype is not t.f32
            or topk_w.shape != k or not topk_w.is_contiguous()):
        raise MxError(-1, f"topk_idx and topk_w must be contiguous int32 and float32 [{T}, {layer.top_k}]")
    if topk_idx.get_device() != dev or topk_w.get_device() != dev or ws.get_device() != dev:
        raise MxError(-1, "all tensors must be on one device")
    _on(dev, t.moe, x.data_ptr(), T, topk_idx.data_ptr(), topk_w.data_ptr(), layer.ref,
        None if residual is None else residual.data_ptr(), out.data_ptr(), _stream_on(dev, stream), ws.data_ptr(),
        ws.nbytes)


# ------------------------------------------------------------- RMS norm

def _rows2d(t, shape, dev, name):
    """Row pitch of a tensor of the given shape with contiguous rows."""
    if t.shape != shape:
        raise MxError(-1, f"{name} must be {list(shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise MxError(-1, f"{name} must have contiguous rows")
    if t.get_device() != dev:
        raise MxError(-1, "all tensors must be on one device")
    return ld if shape[0] > 1 else shape[1]  # (the stride of a single row means nothing)


def fp8_rmsnorm(x, weight=None, eps=1e-6, weight_offset=0.0, residual=None, residual_out=None, out=None, q=None,
                scales=None, pow2=False, stream=None):
    """RMS norm of the rows of ``x`` (float32 or bfloat16 [rows, cols]) plus ``residual``, times ``weight_offset +
    weight`` (mx_fp8_rmsnorm).  ``residual_out`` gets the sum (it may be ``residual`` or ``x`` itself), ``out`` the
    normed rows, ``q`` and ``scales`` the same in e4m3 as fp8_quantize makes them; at least one of the three."""
    t = _t or _torch()
    dev, dtype, shape = x.get_device(), x.dtype, x.shape
    if len(shape) != 2:
        raise MxError(-1, "x must be [rows, cols]")
    rows, cols = shape
    dt = _dtype_code(x, "x")
    ldx = _rows2d(x, shape, dev, "x")
    rp = wp = sp = op = qp = cp = ldr = lds = ldo = ldq = wd = od = sr = sb = 0
    if residual is not None:
        ldr, rp = _rows2d(residual, shape, dev, "residual"), residual.data_ptr()
        if residual.dtype is not dtype:
            raise MxError(-1, "residual must have x's dtype")
    if residual_out is not None:
        lds, sp = _rows2d(residual_out, shape, dev, "residual_out"), residual_out.data_ptr()
        if residual_out.dtype is not dtype:
            raise MxError(-1, "residual_out must have x's dtype")
    if weight is not None:
        if weight.shape != (cols,) or not weight.is_contiguous() or weight.get_device() != dev:
            raise MxError(-1, f"weight must be contiguous [{cols}] on x's device")
        wd, wp = _dtype_code(weight, "weight"), weight.data_ptr()
    if out is not None:
        ldo, op, od = _rows2d(out, shape, dev, "out"), out.data_ptr(), _dtype_code(out, "out")
    if q is not None and scales is not None:
        if q.dtype is not t.f8 or scales.dtype is not t.f32 or scales.shape != (rows, (cols + 127) // 128):
            raise MxError(-1, f"q must be float8_e4m3fn, scales float32 [{rows}, {(cols + 127) // 128}]")
        if scales.get_device() != dev:
            raise MxError(-1, "all tensors must be on one device")
        ldq, qp, cp = _rows2d(q, shape, dev, "q"), q.data_ptr(), scales.data_ptr()
        sr, sb = scales.stride()
    elif q is not None or scales is not None:
        raise MxError(-1, "q and scales come together")
    _on(dev, t.norm, _NORM.pack(x.data_ptr(), ldx, rp, ldr, wp, sp, lds, op, ldo, qp, cp, rows, cols, ldq, sr, sb, rows,
                                cols, dt, wd, od, 1 if pow2 else 0, eps, weight_offset), _stream_on(dev, stream))


# ------------------------------------------- microscaled 4-bit operators

def _fp4_format(t, scales, name):
    if scales.dtype is t.f8:
        return MX_FP4_E4M3, 16
    if scales.dtype is t.e8m0:
        return MX_FP4_E8M0, 32
    raise MxError(-1, f"{name}: scales must be float8_e4m3fn (blocks of 16) or float8_e8m0fnu (of 32)")


def _up(n, m):
    return -(-n // m) * m


def _fp4_rows(t, q, scales, cols, factor, dev):
    """(rows, packed Fp4Rows) of quantised activations."""
    kind = scales.dtype
    if kind is t.f8:
        fmt, per = MX_FP4_E4M3, 16
    elif kind is t.e8m0:
        fmt, per = MX_FP4_E8M0, 8
    else:
        fmt, per = _fp4_format(t, scales, "q")
    nbytes = (cols + 1) // 2
    shape = q.shape
    if len(shape) != 2 or shape[1] != nbytes or q.dtype is not t.u8:
        raise MxError(-1, f"q must be uint8 [rows, {nbytes}]")
    rows = shape[0]
    ld, one = q.stride()
    if one != 1 and nbytes > 1:
        raise MxError(-1, "q must have contiguous rows")
    if scales.shape != ((cols + 255) // 256, rows, per) or not scales.is_contiguous():
        raise MxError(-1, f"scales must be contiguous [{(cols + 255) // 256}, {rows}, {per}]")
    if q.get_device() != dev or scales.get_device() != dev:
        raise MxError(-1, "all tensors must be on one device")
    if rows <= 1:  # (the stride of a single row means nothing)
        ld = (nbytes + 15) // 16 * 16
    return rows, _FP4.pack(q.data_ptr(), scales.data_ptr(), 0 if factor is None else _factor(t, factor, 1, fmt, dev), rows,
                           cols, fmt, ld)


def _factor(t, factor, count, fmt, dev):
    """Address of the tensors' fp32 factors, 0 without."""
    if factor is None:
        return 0
    if (fmt != MX_FP4_E4M3 or factor.dtype is not t.f32 or factor.numel() != count or factor.get_device() != dev
            or (count > 1 and not factor.is_contiguous())):
        raise MxError(-1, f"tensor_scale must be {count} contiguous float32 on the tensors' device, with e4m3 scales")
    return factor.data_ptr()


class Fp4Weight:
    """Microscaled e2m1 matrices on the device: ``w`` uint8 [count,] rows, ceil(cols / 2), two numbers to a byte, rows
    at multiples of 16 bytes; ``scales`` float8_e4m3fn (a block of 16 columns each) or float8_e8m0fnu (32) [count,]
    rows, blocks; ``tensor_scale`` float32 [count] or None (e4m3 only).  ``cols`` is needed where it is odd.  ``w`` and
    ``tensor_scale`` are kept and read by every call; of ``scales`` the products read a copy in their own order, made
    here on ``stream`` (mx_fp4_pack_scales) in memory of that stream: products on others come after it, and the handle
    is kept until they have ended."""

    def __init__(self, w, scales, tensor_scale=None, cols=None, stream=None):
        t = _t or _torch()
        _need(w.dtype is t.u8 and w.dim() in (2, 3), "w must be uint8 [count,] rows, bytes")
        fmt, block = _fp4_format(t, scales, "w")
        rows, nbytes = w.shape[-2:]
        count = w.shape[0] if w.dim() == 3 else 1
        cols = 2 * nbytes if cols is None else cols
        _need((cols + 1) // 2 == nbytes, f"w has {nbytes} bytes a row, {cols} columns need {(cols + 1) // 2}")
        nb = -(-cols // block)
        _need(tuple(scales.shape) == (*w.shape[:-1], nb), f"scales must be [{count}, {rows}, {nb}]")
        ld = w.stride(-2) if rows > 1 else w.stride(0) if count > 1 else _up(nbytes, 16)
        lds = scales.stride(-2) if rows > 1 else scales.stride(0) if count > 1 else nb
        _need((w.stride(-1) == 1 or nbytes == 1) and (scales.stride(-1) == 1 or nb == 1), "rows must be contiguous")
        _need(count == 1 or (w.stride(0) == rows * ld and scales.stride(0) == rows * lds),
              "the matrices must follow one another")
        dev = w.get_device()
        _need(scales.get_device() == dev, f"scales must be on {w.device}")
        factor = _factor(t, tensor_scale, count, fmt, dev)
        n = lib().mx_fp4_pack_bytes(rows, cols, count, fmt)
        if n == 0:
            _check(-1)
        self.w, self.tensor_scale = w, tensor_scale
        self.packed = _bytes_on(dev, stream, n, w.device)
        _on(dev, lib().mx_fp4_pack_scales, scales.data_ptr(), lds, rows, cols, count, fmt, self.packed.data_ptr(),
            _stream_on(dev, stream))
        self.c = Fp4Matrix(w.data_ptr(), self.packed.data_ptr(), factor or None, rows, cols, count, fmt, ld)
        self.ref, self.rows, self.cols, self.count, self.dev = C.byref(self.c), rows, cols, count, dev


def fp4_empty(rows: int, cols: int, block: int, device="cuda"):
    """Uninitialised (q, scales) for fp4_quantize as the products want them: q uint8 [rows, ceil(cols / 2)], rows at
    multiples of 16 bytes; scales [ceil(cols / 256), rows, 256 / block], float8_e4m3fn for block 16, float8_e8m0fnu for
    32."""
    import torch
    _need(block in (16, 32) and rows >= 0 and cols >= 1, "block must be 16 or 32, rows >= 0, cols >= 1")
    nbytes = (cols + 1) // 2
    q = torch.empty(rows, _up(nbytes, 16), dtype=torch.uint8, device=device)[:, :nbytes]
    s = torch.empty(-(-cols // 256), rows, 256 // block, dtype=torch.uint8, device=device)
    return q, s.view(torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu)


def fp4_quantize(x, q, scales, tensor_scale=None, stream=None):
    """Quantise the rows of ``x`` (float32 or bfloat16 [rows, cols]) into ``q`` and ``scales`` of fp4_empty: e4m3 scales
    for blocks of 16 columns, with the optional float32 ``tensor_scale`` on the device, or e8m0 scales for blocks of
    32."""
    t = _t or _torch()
    dev, shape = x.get_device(), x.shape
    if len(shape) != 2:
        raise MxError(-1, "x must be [rows, cols]")
    cols = shape[1]
    n, r = _fp4_rows(t, q, scales, cols, tensor_scale, dev)
    ldx, one = x.stride()
    if shape[0] != n or (one != 1 and cols > 1):
        raise MxError(-1, f"x must be [{n}, cols] with contiguous rows")
    _on(dev, t.quantize4, x.data_ptr(), ldx if n > 1 else cols, _dtype_code(x, "x"), r, _stream_on(dev, stream))


def fp4_matmul_workspace_bytes(weight: Fp4Weight, rows: int) -> int:
    return lib().mx_fp4_matmul_workspace_bytes(weight.ref, rows)


def fp4_matmul(q, scales, weight: Fp4Weight, out, ws, tensor_scale=None, stream=None):
    """out = (q, scales, tensor_scale) times the transposed ``weight``; out float32 or bfloat16 [rows, weight rows]; ws
    a uint8 workspace of fp4_matmul_workspace_bytes, prepared by workspace_init."""
    t = _t or _torch()
    dev = weight.dev
    rows, r = _fp4_rows(t, q, scales, weight.cols, tensor_scale, dev)
    ldo = _out_pitch(rows, weight, out, ws)
    _on(dev, t.matmul4, r, weight.ref, out.data_ptr(), ldo, _dtype_code(out, "out"), _stream_on(dev, stream),
        ws.data_ptr(), ws.nbytes)


def fp4_grouped_matmul(q, scales, offsets, weight: Fp4Weight, out, ws, tensor_scale=None, stream=None):
    """The same with rows [offsets[e], offsets[e + 1]) against matrix e; offsets int32 [count + 1] on the device."""
    t = _t or _torch()
    dev = weight.dev
    rows, r = _fp4_rows(t, q, scales, weight.cols, tensor_scale, dev)
    ldo = _out_pitch(rows, weight, out, ws)
    if (offsets.dtype is not t.i32 or offsets.shape != (weight.count + 1,) or not offsets.is_contiguous()
            or offsets.get_device() != dev):
        raise MxError(-1, f"offsets must be contiguous int32 [{weight.count + 1}] on the weight's device")
    _on(dev, t.grouped4, r, offsets.data_ptr(), weight.ref, out.data_ptr(), ldo, _dtype_code(out, "out"),
        _stream_on(dev, stream), ws.data_ptr(), ws.nbytes)


# ------------------------------------------------------ routing from logits

class Router:
    """How tokens choose experts by their logits (mx_route_logits): scores MX_SOFTMAX or MX_SIGMOID; ``bias`` float32
    [n_experts] on the device, added for the choice alone; the best ``topk_groups`` of ``n_groups`` runs of experts, by
    their ``group_best`` (1 or 2) highest scores; the weights of the ``top_k`` chosen divided by their sum
    (``renormalise``) and times ``scale``."""

    def __init__(self, n_experts, top_k, score=MX_SOFTMAX, bias=None, n_groups=1, topk_groups=1, group_best=1,
                 renormalise=True, scale=1.0):
        t = _t or _torch()
        _need(bias is None or (bias.dtype is t.f32 and bias.shape == (n_experts,) and bias.is_contiguous()),
              f"bias must be contiguous float32 [{n_experts}]")
        self.bias = bias
        self.c = RouterStruct(n_experts, top_k, score, n_groups, topk_groups, group_best, 1 if renormalise else 0, scale,
                              _ptr(bias))
        self.ref, self.n_experts, self.top_k = C.byref(self.c), n_experts, top_k
        self.dev = None if bias is None else bias.get_device()


def route_logits_workspace_bytes(router: Router, T: int) -> int:
    return lib().mx_route_logits_workspace_bytes(router.ref, T)


def route_logits(logits, router: Router, topk_idx, topk_w, counts=None, offsets=None, perm=None, ws=None, stream=None):
    """Choose the experts of each row of ``logits`` (float32 or bfloat16 [T, n_experts]): topk_idx int32 and topk_w
    float32 [T, top_k].  With counts, offsets and perm (int32 [n_experts], [n_experts + 1], [T * top_k]) the slots are
    grouped by expert as route() does; ws is then a uint8 workspace of route_logits_workspace_bytes, prepared by
    workspace_init."""
    t = _t or _torch()
    dev, shape = logits.get_device(), logits.shape
    E, K = router.n_experts, router.top_k
    if len(shape) != 2 or shape[1] != E:
        raise MxError(-1, f"logits must be [T, {E}]")
    T = shape[0]
    ld, one = logits.stride()
    if one != 1 and E > 1:
        raise MxError(-1, "logits must have contiguous rows")
    chosen = (T, K)
    if (topk_idx.dtype is not t.i32 or topk_w.dtype is not t.f32 or topk_idx.shape != chosen or topk_w.shape != chosen
            or not topk_idx.is_contiguous() or not topk_w.is_contiguous()):
        raise MxError(-1, f"topk_idx and topk_w must be contiguous int32 and float32 [{T}, {K}]")
    if topk_idx.get_device() != dev or topk_w.get_device() != dev or (router.dev is not None and router.dev != dev):
        raise MxError(-1, "all tensors must be on one device")
    cp = op = pp = wp = None
    n = 0
    if counts is not None or offsets is not None or perm is not None:
        if counts is None or offsets is None or perm is None or ws is None:
            raise MxError(-1, "counts, offsets, perm and ws come together")
        for a, size in ((counts, E), (offsets, E + 1), (perm, T * K)):
            if a.dtype is not t.i32 or a.numel() != size or not a.is_contiguous() or a.get_device() != dev:
                raise MxError(-1, f"counts, offsets and perm must be contiguous int32 [{E}], [{E + 1}] and [{T * K}] on "
                                  "the logits' device")
        if ws.get_device() != dev:
            raise MxError(-1, "all tensors must be on one device")
        cp, op, pp, wp, n = counts.data_ptr(), offsets.data_ptr(), perm.data_ptr(), ws.data_ptr(), ws.nbytes
    _on(dev, t.route, logits.data_ptr(), ld if T > 1 else E, _dtype_code(logits, "logits"), T, router.ref,
        topk_idx.data_ptr(), topk_w.data_ptr(), cp, op, pp, _stream_on(dev, stream), wp, n)
