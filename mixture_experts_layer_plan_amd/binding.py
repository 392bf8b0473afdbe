"""ctypes binding of libmoe.so (include/moe.h), same names as the C entry points.

Marshalling only: torch tensors become device pointers, ``None`` becomes NULL and
the current torch stream becomes the hipStream_t.  Every step of the layer runs in
the library's HIP kernels; there is no Python or CPU fallback.  A missing library
raises ``MoeLibraryMissing``.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8}


class MoeLibraryMissing(RuntimeError):
    pass


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn}: status {code} ({msg})")
        self.code = code


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("T_minibatch", ctypes.c_int32), ("flags", ctypes.c_int32)]


class moe_plan_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("counts", "offsets", "src_token", "src_slot", "pos",
                                                "tiles", "n_tiles", "err_flag", "active",
                                                "n_active", "tile_first", "wtiles",
                                                "n_wtiles", "scratch",
                                                "sub_plan_bytes", "total_bytes")] + \
               [(n, ctypes.c_int32) for n in ("tile_m", "max_tiles", "chunk_pairs", "n_chunks",
                                              "n_minibatch", "T_minibatch", "wtile_m",
                                              "max_wtiles")]


class moe_scoring(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


class moe_lora_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H_in", ctypes.c_int32), ("H_out", ctypes.c_int32),
                ("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32)]


class moe_norm_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class moe_balance(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_seq", ctypes.c_int32), ("coef", ctypes.c_float)]


class moe_adamw_shape(ctypes.Structure):
    _fields_ = [("elements", ctypes.c_int64), ("n_tensors", ctypes.c_int32),
                ("p_type", ctypes.c_int32), ("g_type", ctypes.c_int32),
                ("master", ctypes.c_int32), ("state_bits", ctypes.c_int32)]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "grad", "param", "m", "v", "master", "m_scale", "v_scale", "param_out", "m_out", "v_out",
        "master_out", "m_scale_out", "v_scale_out")] + \
        [("n", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)]


class moe_adamw_hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in (
        "lr", "beta1", "one_minus_beta1", "beta2", "one_minus_beta2", "eps", "corr1", "corr2",
        "grad_scale")] + [("seed", ctypes.c_uint32)]


_P = ctypes.c_void_p
_NS = ctypes.POINTER(moe_norm_shape)
_BA = ctypes.POINTER(moe_balance)
_AS = ctypes.POINTER(moe_adamw_shape)
_AH = ctypes.POINTER(moe_adamw_hyper)
_S = ctypes.POINTER(moe_shape)
_SC = ctypes.POINTER(moe_scoring)
_LS = ctypes.POINTER(moe_lora_shape)
_Z = ctypes.c_size_t
_I = ctypes.c_int

class moe_trace(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)),
                ("names", ctypes.POINTER(ctypes.c_char_p)),
                ("capacity", ctypes.c_int32), ("count", ctypes.c_int32)]


# name -> (restype, argtypes)
_SIGS = {
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_trace_set": (None, [ctypes.POINTER(moe_trace)]),
    "moe_set_cu_budget": (None, [ctypes.c_int32]),
    "moe_plan_layout_of": (ctypes.c_int, [_S, ctypes.POINTER(moe_plan_layout)]),
    "moe_plan_bytes": (_Z, [_S]),
    "moe_saved_bytes": (_Z, [_S, _I]),
    "moe_workspace_bytes": (_Z, [_S, _I, _I]),
    "moe_router_logits_f32": (_I, [_S, _P, _P, _P, _P]),
    "moe_route": (_I, [_S, _P, _P, _P, _P]),
    "moe_route_backward": (_I, [_S, _P, _P, _P, _P, _P]),
    "moe_router_backward_f32": (_I, [_S, _P, _P, _P, _P, _P, _P]),
    "moe_route_scored": (_I, [_S, _SC, _P, _P, _P, _P, _P]),
    "moe_route_scored_backward": (_I, [_S, _SC, _P, _P, _P, _P, _P]),
    "moe_router_workspace_bytes": (_Z, [_S, _I]),
    "moe_router_logits_bf16": (_I, [_S, _P, _P, _P, _P, _Z, _P]),
    "moe_router_backward_bf16": (_I, [_S] + [_P] * 7 + [_Z, _P]),
    "moe_lora_plan_bytes": (_Z, [_LS]),
    "moe_lora_plan": (_I, [_LS, _P, _P, _P]),
    "moe_lora_saved_bytes": (_Z, [_LS]),
    "moe_lora_workspace_bytes": (_Z, [_LS, _I]),
    "moe_lora_bf16": (_I, [_LS] + [_P] * 9 + [_Z, _P]),
    "moe_lora_backward_bf16": (_I, [_LS] + [_P] * 12 + [_Z, _P]),
    "moe_norm_bf16": (_I, [_NS] + [_P] * 8),
    "moe_norm_f32": (_I, [_NS] + [_P] * 8),
    "moe_norm_backward_bf16": (_I, [_NS] + [_P] * 9 + [_Z, _P]),
    "moe_norm_backward_f32": (_I, [_NS] + [_P] * 9 + [_Z, _P]),
    "moe_norm_workspace_bytes": (_Z, [_NS]),
    "moe_balance_loss": (_I, [_S, _BA] + [_P] * 7 + [_Z, _P]),
    "moe_balance_loss_backward": (_I, [_S, _BA] + [_P] * 9),
    "moe_balance_workspace_bytes": (_Z, [_S, _BA]),
    "moe_adamw_table_bytes": (_Z, [_AS]),
    "moe_adamw_table": (_I, [_AS, ctypes.POINTER(moe_adamw_tensor), _P, _P]),
    "moe_adamw_hyper_of": (_I, [ctypes.c_double] * 4 + [ctypes.c_int64, ctypes.c_double,
                                                       ctypes.c_uint32, _AH]),
    "moe_adamw_step": (_I, [_AS, _P, _AH, _P, _P]),
    "moe_adamw_values": (_I, [ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P]),
    "moe_plan": (_I, [_S, _P, _P, _P]),
    "moe_dispatch_bf16": (_I, [_S, _P, _P, _P, _P]),
    "moe_dispatch_f32": (_I, [_S, _P, _P, _P, _P]),
    "moe_combine_bf16": (_I, [_S, _P, _P, _P, _P, _P, _P]),
    "moe_combine_f32": (_I, [_S, _P, _P, _P, _P, _P, _P]),
    "moe_reverse_combine_bf16": (_I, [_S, _P, _P, _P, _P]),
    "moe_reverse_dispatch_bf16": (_I, [_S, _P, _P, _P, _P, _P]),
    "moe_forward_bf16": (_I, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_forward_f32": (_I, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_forward_bf16_noalloc": (_I, [_S] + [_P] * 12),
    "moe_backward_bf16": (_I, [_S] + [_P] * 20 + [_Z, _P]),
    "moe_backward_f32": (_I, [_S] + [_P] * 20 + [_Z, _P]),
    "moe_mx_weights_bytes": (_Z, [_S]),
    "moe_quantize_weights_mxfp8": (_I, [_S, _P, _P, _P, _P, _P]),
    "moe_quantize_mxfp8": (_I, [_P, ctypes.c_int64, ctypes.c_int64, _I, _P, _P, _P]),
    "moe_quantize_mxfp8_f32": (_I, [_P, ctypes.c_int64, ctypes.c_int64, _I, _P, _P, _P]),
    "moe_forward_mxfp8": (_I, [_S] + [_P] * 10 + [_Z, _P]),
    "moe_backward_mxfp8": (_I, [_S] + [_P] * 18 + [_Z, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeLibraryMissing(
                f"{LIB_PATH} is missing: build it with `python -m mixture_experts_layer_plan_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_names() -> list[str]:
    return list(_SIGS)


MOE_REPLAY = 1
MOE_FUSED_FORWARD = 2


def shape(T, H, I, E, k, I_shared=0, T_minibatch=0, flags=0) -> moe_shape:
    return moe_shape(int(T), int(H), int(I), int(E), int(k), int(I_shared), int(T_minibatch),
                     int(flags))


def _ptr(t, dtype=None, numel=None):
    """Device pointer of a contiguous tensor (None -> NULL).  ``dtype`` and ``numel``,
    when given, are checked: the library reads and writes through raw pointers, so a
    tensor of another element type or size would be over-read or overrun."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"expected a {dtype} tensor, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"expected {numel} elements, got {t.numel()}")
    return t.data_ptr()


_F32 = torch.float32
_BF16 = torch.bfloat16


def _f32(t, numel=None):
    return _ptr(t, _F32, numel)


def _bf16(t, numel=None):
    return _ptr(t, _BF16, numel)


# The current stream's handle without building a torch.cuda.Stream (0.1 us against 2.7):
# what a call of a few microseconds on the GPU is measured by.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# And the current device without torch.cuda's check that it has been started (0.06 us against
# 0.25): a device tensor among the arguments has started it.
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(name, *args):
    rc = getattr(lib(), name)(*args)
    if rc != 0:
        raise MoeError(name, rc, lib().moe_status_str(rc).decode())


def moe_set_cu_budget(cus: int) -> None:
    lib().moe_set_cu_budget(int(cus))


def moe_status_str(code: int) -> str:
    return lib().moe_status_str(code).decode()


def moe_plan_layout_of(s: moe_shape) -> moe_plan_layout:
    out = moe_plan_layout()
    _call("moe_plan_layout_of", ctypes.byref(s), ctypes.byref(out))
    return out


def moe_plan_bytes(s: moe_shape) -> int:
    return lib().moe_plan_bytes(ctypes.byref(s))


def moe_saved_bytes(s: moe_shape, dtype: int) -> int:
    return lib().moe_saved_bytes(ctypes.byref(s), dtype)


def moe_workspace_bytes(s: moe_shape, dtype: int, backward: bool) -> int:
    return lib().moe_workspace_bytes(ctypes.byref(s), dtype, int(backward))


def moe_router_logits_f32(s, x, w_router, logits, stream=None):
    _call("moe_router_logits_f32", ctypes.byref(s), _f32(x, s.T * s.H), _f32(w_router, s.E * s.H),
          _f32(logits, s.T * s.E), _stream(stream))


def moe_route(s, logits, topk_idx, topk_w, stream=None):
    _call("moe_route", ctypes.byref(s), _f32(logits, s.T * s.E), _ptr(topk_idx, torch.int32, s.T * s.k),
          _f32(topk_w, s.T * s.k), _stream(stream))


def moe_route_backward(s, topk_idx, topk_w, d_topk_w, d_logits, stream=None):
    _call("moe_route_backward", ctypes.byref(s), _ptr(topk_idx, torch.int32, s.T * s.k),
          _f32(topk_w, s.T * s.k), _f32(d_topk_w, s.T * s.k), _f32(d_logits, s.T * s.E),
          _stream(stream))


def moe_router_backward_f32(s, x, w_router, d_logits, dw_router, dx, stream=None):
    _call("moe_router_backward_f32", ctypes.byref(s), _f32(x, s.T * s.H), _f32(w_router, s.E * s.H),
          _f32(d_logits, s.T * s.E), _f32(dw_router, s.E * s.H), _f32(dx, s.T * s.H),
          _stream(stream))


def moe_plan(s, topk_idx, plan, stream=None):
    _call("moe_plan", ctypes.byref(s), _ptr(topk_idx), _ptr(plan), _stream(stream))


def moe_dispatch_bf16(s, plan, x, X, stream=None):
    _call("moe_dispatch_bf16", ctypes.byref(s), _ptr(plan), _ptr(x), _ptr(X), _stream(stream))


def moe_dispatch_f32(s, plan, x, X, stream=None):
    _call("moe_dispatch_f32", ctypes.byref(s), _ptr(plan), _f32(x, s.T * s.H), _f32(X, s.T * s.k * s.H),
          _stream(stream))


def moe_combine_bf16(s, plan, Y, topk_w, shared_out, y, stream=None):
    _call("moe_combine_bf16", ctypes.byref(s), _ptr(plan), _ptr(Y), _ptr(topk_w),
          _ptr(shared_out), _ptr(y), _stream(stream))


def moe_combine_f32(s, plan, Y, topk_w, shared_out, y, stream=None):
    _call("moe_combine_f32", ctypes.byref(s), _ptr(plan), _f32(Y, s.T * s.k * s.H),
          _f32(topk_w, s.T * s.k), _f32(shared_out, s.T * s.H), _f32(y, s.T * s.H), _stream(stream))


def moe_reverse_combine_bf16(s, plan, dy, dYu, stream=None):
    _call("moe_reverse_combine_bf16", ctypes.byref(s), _ptr(plan), _ptr(dy), _ptr(dYu),
          _stream(stream))


def moe_reverse_dispatch_bf16(s, plan, dX, shared_dx, dx, stream=None):
    _call("moe_reverse_dispatch_bf16", ctypes.byref(s), _ptr(plan), _ptr(dX), _ptr(shared_dx),
          _ptr(dx), _stream(stream))


def _fwd(name, s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y, saved, ws,
         stream):
    dt = _F32 if name.endswith("_f32") else _BF16
    nw, ns = s.E * s.I * s.H, s.I_shared * s.H
    _call(name, ctypes.byref(s), _ptr(plan), _ptr(x, dt, s.T * s.H), _f32(topk_w, s.T * s.k),
          _ptr(w_gate, dt, nw), _ptr(w_up, dt, nw), _ptr(w_down, dt, nw), _ptr(s_gate, dt, ns),
          _ptr(s_up, dt, ns), _ptr(s_down, dt, ns), _ptr(y, dt, s.T * s.H), _ptr(saved), _ptr(ws),
          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))


def moe_forward_bf16(s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y, saved,
                     ws, stream=None):
    _fwd("moe_forward_bf16", s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y,
         saved, ws, stream)


MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_forward_bf16_noalloc(s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y,
                             saved, stream=None):
    nw, ns, nt = s.E * s.I * s.H, s.I_shared * s.H, s.T * s.H
    _call("moe_forward_bf16_noalloc", ctypes.byref(s), _ptr(plan), _bf16(x, nt),
          _f32(topk_w, s.T * s.k), _bf16(w_gate, nw), _bf16(w_up, nw), _bf16(w_down, nw),
          _bf16(s_gate, ns), _bf16(s_up, ns), _bf16(s_down, ns), _bf16(y, nt), _ptr(saved),
          _stream(stream))


def moe_forward_f32(s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y, saved,
                    ws, stream=None):
    _fwd("moe_forward_f32", s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, y,
         saved, ws, stream)


def _bwd(name, s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, saved, dy, dx,
         dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws, stream):
    dt = _F32 if name.endswith("_f32") else _BF16
    nw, ns, nt = s.E * s.I * s.H, s.I_shared * s.H, s.T * s.H
    _call(name, ctypes.byref(s), _ptr(plan), _ptr(x, dt, nt), _f32(topk_w, s.T * s.k),
          _ptr(w_gate, dt, nw), _ptr(w_up, dt, nw), _ptr(w_down, dt, nw), _ptr(s_gate, dt, ns),
          _ptr(s_up, dt, ns), _ptr(s_down, dt, ns), _ptr(saved), _ptr(dy, dt, nt), _ptr(dx, dt, nt),
          _ptr(dw_gate, dt, nw), _ptr(dw_up, dt, nw), _ptr(dw_down, dt, nw), _ptr(ds_gate, dt, ns),
          _ptr(ds_up, dt, ns), _ptr(ds_down, dt, ns), _f32(d_topk_w, s.T * s.k), _ptr(ws),
          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))


def moe_backward_bf16(s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, saved, dy,
                      dx, dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws,
                      stream=None):
    _bwd("moe_backward_bf16", s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down,
         saved, dy, dx, dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws, stream)


def moe_backward_f32(s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down, saved, dy,
                     dx, dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws,
                     stream=None):
    _bwd("moe_backward_f32", s, plan, x, topk_w, w_gate, w_up, w_down, s_gate, s_up, s_down,
         saved, dy, dx, dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws, stream)


def moe_mx_weights_bytes(s: moe_shape) -> int:
    return lib().moe_mx_weights_bytes(ctypes.byref(s))


def moe_quantize_weights_mxfp8(s, w_gate, w_up, w_down, wq, stream=None):
    nw = s.E * s.I * s.H
    _call("moe_quantize_weights_mxfp8", ctypes.byref(s), _bf16(w_gate, nw), _bf16(w_up, nw),
          _bf16(w_down, nw), _ptr(wq, torch.uint8, moe_mx_weights_bytes(s)), _stream(stream))


def moe_quantize_mxfp8(src, rows, cols, axis, q, scales, stream=None):
    _call("moe_quantize_mxfp8", _ptr(src), int(rows), int(cols), int(axis), _ptr(q), _ptr(scales),
          _stream(stream))


def moe_quantize_mxfp8_f32(src, rows, cols, axis, q, scales, stream=None):
    n = int(rows) * int(cols)
    _call("moe_quantize_mxfp8_f32", _f32(src, n), int(rows), int(cols), int(axis),
          _ptr(q, torch.uint8, n), _ptr(scales, torch.uint8, n // 32), _stream(stream))


def moe_forward_mxfp8(s, plan, x, topk_w, wq, s_gate, s_up, s_down, y, saved, ws, stream=None):
    ns, nt = s.I_shared * s.H, s.T * s.H
    _call("moe_forward_mxfp8", ctypes.byref(s), _ptr(plan), _bf16(x, nt), _f32(topk_w, s.T * s.k),
          _ptr(wq, torch.uint8, moe_mx_weights_bytes(s)), _bf16(s_gate, ns), _bf16(s_up, ns),
          _bf16(s_down, ns), _bf16(y, nt), _ptr(saved), _ptr(ws),
          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))


def moe_backward_mxfp8(s, plan, x, topk_w, wq, s_gate, s_up, s_down, saved, dy, dx, dw_gate,
                       dw_up, dw_down, ds_gate, ds_up, ds_down, d_topk_w, ws, stream=None):
    nw, ns, nt = s.E * s.I * s.H, s.I_shared * s.H, s.T * s.H
    _call("moe_backward_mxfp8", ctypes.byref(s), _ptr(plan), _bf16(x, nt), _f32(topk_w, s.T * s.k),
          _ptr(wq, torch.uint8, moe_mx_weights_bytes(s)), _bf16(s_gate, ns), _bf16(s_up, ns),
          _bf16(s_down, ns), _ptr(saved), _bf16(dy, nt), _bf16(dx, nt), _bf16(dw_gate, nw),
          _bf16(dw_up, nw), _bf16(dw_down, nw), _bf16(ds_gate, ns), _bf16(ds_up, ns),
          _bf16(ds_down, ns), _f32(d_topk_w, s.T * s.k), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))


# ------------------------------------------- scored routing, bf16 router, adapters
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


def scoring(score="softmax", n_groups=1, topk_groups=1, group_top=1, renormalise=True,
            scale=1.0) -> moe_scoring:
    if score not in SCORES:
        raise ValueError(f"unsupported score {score!r}")
    return moe_scoring(SCORES[score], int(n_groups), int(topk_groups), int(group_top),
                       int(bool(renormalise)), float(scale))


def lora_shape(T, H_in, H_out, n_adapters, rank) -> moe_lora_shape:
    return moe_lora_shape(int(T), int(H_in), int(H_out), int(n_adapters), int(rank))


def _here(t, dtype, numel, dev):
    """Device pointer of a contiguous tensor of the current device ``dev`` (None -> NULL).
    The launches go to the current device, so a tensor of another one is refused, as are
    another type or size (a call of a few microseconds: one pass of cheap checks)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"expected a tensor on cuda:{dev}, the current device, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"expected a {dtype} tensor, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"expected {numel} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _buf(t, nbytes, dev):
    """Pointer of a buffer the library lays out itself, of at least ``nbytes``."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"expected a tensor on cuda:{dev}, the current device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"buffer of {t.numel() * t.element_size()} bytes, {nbytes} needed")
    return t.data_ptr()


def _ws(t, dev):
    return _buf(t, 0, dev), 0 if t is None else t.numel() * t.element_size()


def _dev():
    return _raw_device()


@functools.lru_cache(maxsize=256)
def _lora_bytes(T, H_in, H_out, n, r):
    """(plan, saved) bytes of a lora shape"""
    s = lora_shape(T, H_in, H_out, n, r)
    return moe_lora_plan_bytes(s), moe_lora_saved_bytes(s)


def moe_route_scored(s, sc, logits, bias, topk_idx, topk_w, stream=None):
    T, E, k, d = s.T, s.E, s.k, _dev()
    _call("moe_route_scored", ctypes.byref(s), ctypes.byref(sc), _here(logits, _F32, T * E, d),
          _here(bias, _F32, E, d), _here(topk_idx, torch.int32, T * k, d),
          _here(topk_w, _F32, T * k, d), _stream(stream))


def moe_route_scored_backward(s, sc, logits, topk_idx, d_topk_w, d_logits, stream=None):
    T, E, k, d = s.T, s.E, s.k, _dev()
    _call("moe_route_scored_backward", ctypes.byref(s), ctypes.byref(sc),
          _here(logits, _F32, T * E, d), _here(topk_idx, torch.int32, T * k, d),
          _here(d_topk_w, _F32, T * k, d), _here(d_logits, _F32, T * E, d), _stream(stream))


def moe_router_workspace_bytes(s: moe_shape, backward: bool) -> int:
    return lib().moe_router_workspace_bytes(ctypes.byref(s), int(backward))


def moe_router_logits_bf16(s, x, w_router, logits, ws, stream=None):
    T, H, E, d = s.T, s.H, s.E, _dev()
    _call("moe_router_logits_bf16", ctypes.byref(s), _here(x, _BF16, T * H, d),
          _here(w_router, _BF16, E * H, d), _here(logits, _F32, T * E, d), *_ws(ws, d),
          _stream(stream))


def moe_router_backward_bf16(s, x, w_router, d_logits, dx_in, dw_router, dx, ws, stream=None):
    T, H, E, d = s.T, s.H, s.E, _dev()
    _call("moe_router_backward_bf16", ctypes.byref(s), _here(x, _BF16, T * H, d),
          _here(w_router, _BF16, E * H, d), _here(d_logits, _F32, T * E, d),
          _here(dx_in, _BF16, T * H, d), _here(dw_router, _BF16, E * H, d),
          _here(dx, _BF16, T * H, d), *_ws(ws, d), _stream(stream))


def moe_lora_plan_bytes(s: moe_lora_shape) -> int:
    return lib().moe_lora_plan_bytes(ctypes.byref(s))


def moe_lora_saved_bytes(s: moe_lora_shape) -> int:
    return lib().moe_lora_saved_bytes(ctypes.byref(s))


def moe_lora_workspace_bytes(s: moe_lora_shape, backward: bool) -> int:
    return lib().moe_lora_workspace_bytes(ctypes.byref(s), int(backward))


def moe_lora_plan(s, adapter_idx, plan, stream=None):
    d = _dev()
    _call("moe_lora_plan", ctypes.byref(s), _here(adapter_idx, torch.int32, s.T, d),
          _buf(plan, moe_lora_plan_bytes(s), d), _stream(stream))


def moe_lora_bf16(s, plan, x, lora_a, lora_b, scale, base, y, saved, ws, stream=None):
    T, hi, ho, n, r, d = s.T, s.H_in, s.H_out, s.n_adapters, s.rank, _dev()
    pb, sb = _lora_bytes(T, hi, ho, n, r)
    _call("moe_lora_bf16", ctypes.byref(s), _buf(plan, pb, d), _here(x, _BF16, T * hi, d),
          _here(lora_a, _BF16, n * r * hi, d), _here(lora_b, _BF16, n * r * ho, d),
          _here(scale, _F32, n, d), _here(base, _BF16, T * ho, d), _here(y, _BF16, T * ho, d),
          _buf(saved, sb, d), *_ws(ws, d), _stream(stream))


def moe_lora_backward_bf16(s, plan, x, lora_a, lora_b, scale, saved, dy, dx_in, dx, d_lora_a,
                           d_lora_b, ws, stream=None):
    T, hi, ho, n, r, d = s.T, s.H_in, s.H_out, s.n_adapters, s.rank, _dev()
    pb, sb = _lora_bytes(T, hi, ho, n, r)
    na, nb = n * r * hi, n * r * ho
    _call("moe_lora_backward_bf16", ctypes.byref(s), _buf(plan, pb, d), _here(x, _BF16, T * hi, d),
          _here(lora_a, _BF16, na, d), _here(lora_b, _BF16, nb, d), _here(scale, _F32, n, d),
          _buf(saved, sb, d), _here(dy, _BF16, T * ho, d), _here(dx_in, _BF16, T * hi, d),
          _here(dx, _BF16, T * hi, d), _here(d_lora_a, _BF16, na, d),
          _here(d_lora_b, _BF16, nb, d), *_ws(ws, d), _stream(stream))


# ---------------------------------- norm, balance of the experts, AdamW step
MOE_NORM_LAYER, MOE_NORM_RMS = 0, 1
NORMS = {"layer": MOE_NORM_LAYER, "rms": MOE_NORM_RMS}
MOE_ADAMW_M, MOE_ADAMW_V = 0, 1
MOE_ADAMW_MAX_TENSORS = 65536


def norm_shape(T, H, kind="layer", eps=1e-5) -> moe_norm_shape:
    if kind not in NORMS:
        raise ValueError(f"unsupported norm {kind!r}")
    return moe_norm_shape(int(T), int(H), NORMS[kind], float(eps))


def _norm(name, dt, s, x, residual, w, b, h, y, stats, stream):
    n, H, d = s.T * s.H, s.H, _dev()
    _call(name, ctypes.byref(s), _here(x, dt, n, d), _here(residual, dt, n, d), _here(w, dt, H, d),
          _here(b, dt, H, d), _here(h, dt, n, d), _here(y, dt, n, d), _here(stats, _F32, 2 * s.T, d),
          _stream(stream))


def _norm_backward(name, dt, s, h, w, stats, dy, dh_in, dx, dw, db, ws, stream):
    n, H, d = s.T * s.H, s.H, _dev()
    _call(name, ctypes.byref(s), _here(h, dt, n, d), _here(w, dt, H, d),
          _here(stats, _F32, 2 * s.T, d), _here(dy, dt, n, d), _here(dh_in, dt, n, d),
          _here(dx, dt, n, d), _here(dw, dt, H, d), _here(db, dt, H, d), *_ws(ws, d),
          _stream(stream))


def moe_norm_bf16(s, x, residual, w, b, h, y, stats, stream=None):
    _norm("moe_norm_bf16", _BF16, s, x, residual, w, b, h, y, stats, stream)


def moe_norm_f32(s, x, residual, w, b, h, y, stats, stream=None):
    _norm("moe_norm_f32", _F32, s, x, residual, w, b, h, y, stats, stream)


def moe_norm_backward_bf16(s, h, w, stats, dy, dh_in, dx, dw, db, ws, stream=None):
    _norm_backward("moe_norm_backward_bf16", _BF16, s, h, w, stats, dy, dh_in, dx, dw, db, ws, stream)


def moe_norm_backward_f32(s, h, w, stats, dy, dh_in, dx, dw, db, ws, stream=None):
    _norm_backward("moe_norm_backward_f32", _F32, s, h, w, stats, dy, dh_in, dx, dw, db, ws, stream)


def moe_norm_workspace_bytes(s: moe_norm_shape) -> int:
    return lib().moe_norm_workspace_bytes(ctypes.byref(s))


def balance(score="softmax", coef=0.01, n_seq=1) -> moe_balance:
    if score not in SCORES:
        raise ValueError(f"unsupported score {score!r}")
    return moe_balance(SCORES[score], int(n_seq), float(coef))


def moe_balance_workspace_bytes(s: moe_shape, ba: moe_balance) -> int:
    return lib().moe_balance_workspace_bytes(ctypes.byref(s), ctypes.byref(ba))


def moe_balance_loss(s, ba, logits, topk_idx, seq_start, loss, counts, scales, ws, stream=None):
    T, E, k, n, d = s.T, s.E, s.k, ba.n_seq, _dev()
    _call("moe_balance_loss", ctypes.byref(s), ctypes.byref(ba), _here(logits, _F32, T * E, d),
          _here(topk_idx, torch.int32, T * k, d), _here(seq_start, torch.int32, n + 1, d),
          _here(loss, _F32, 1, d), _here(counts, torch.int32, n * E, d), _here(scales, _F32, n, d),
          *_ws(ws, d), _stream(stream))


def moe_balance_loss_backward(s, ba, logits, topk_idx, seq_start, counts, scales, d_loss, d_in,
                              d_logits, stream=None):
    T, E, k, n, d = s.T, s.E, s.k, ba.n_seq, _dev()
    _call("moe_balance_loss_backward", ctypes.byref(s), ctypes.byref(ba),
          _here(logits, _F32, T * E, d), _here(topk_idx, torch.int32, T * k, d),
          _here(seq_start, torch.int32, n + 1, d), _here(counts, torch.int32, n * E, d),
          _here(scales, _F32, n, d), _here(d_loss, _F32, 1, d), _here(d_in, _F32, T * E, d),
          _here(d_logits, _F32, T * E, d), _stream(stream))


def adamw_shape(elements, n_tensors, p_type="bf16", g_type="bf16", master=False,
                state_bits=32) -> moe_adamw_shape:
    for t in (p_type, g_type):
        if t not in ("bf16", "f32"):
            raise ValueError(f"unsupported type {t!r}")
    return moe_adamw_shape(int(elements), int(n_tensors), DTYPES[p_type], DTYPES[g_type],
                           int(bool(master)), int(state_bits))


def adamw_hyper(lr, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=1.0, seed=None) -> moe_adamw_hyper:
    """A step's scalars; ``bytes(...)`` of it is what a device copy holds.  ``seed`` is ``step``
    if not given: with one seed for all steps an element would be rounded by the same random
    number every time, up or down for good."""
    out = moe_adamw_hyper()
    seed = step if seed is None else seed
    _call("moe_adamw_hyper_of", float(lr), float(beta1), float(beta2), float(eps), int(step),
          float(grad_scale), int(seed) & 0xFFFFFFFF, ctypes.byref(out))
    return out


def moe_adamw_table_bytes(s: moe_adamw_shape) -> int:
    return lib().moe_adamw_table_bytes(ctypes.byref(s))


def moe_adamw_table(s, tensors, table, stream=None):
    """``tensors``: a dict for each, with ``grad``, ``param``, ``m``, ``v`` and, where the shape
    has them, ``master``, ``m_scale`` and ``v_scale``; ``weight_decay`` (0 if absent); and for an
    output elsewhere than over its input its name with ``_out``.  The table holds their
    addresses: they have to stay where they are."""
    d = _dev()
    if len(tensors) != s.n_tensors:
        raise ValueError(f"expected {s.n_tensors} tensors, got {len(tensors)}")
    types = {MOE_F32: _F32, MOE_BF16: _BF16}
    state = _F32 if s.state_bits == 32 else torch.uint8
    kinds = {"param": types[s.p_type], "m": state, "v": state}
    if s.master:
        kinds["master"] = _F32
    if s.state_bits == 8:
        kinds["m_scale"] = kinds["v_scale"] = torch.uint8
    places = [(k, k + "_out", dt, k.endswith("scale")) for k, dt in kinds.items()]
    known = {"grad", "weight_decay"}.union(*(p[:2] for p in places))
    arr = (moe_adamw_tensor * s.n_tensors)()
    for a, t in zip(arr, tensors):
        if not t.keys() <= known:
            raise ValueError(f"no place for {sorted(t.keys() - known)} in this shape")
        grad = t["grad"]
        a.n = n = grad.numel()
        a.weight_decay = t.get("weight_decay", 0.0)
        a.grad = _here(grad, types[s.g_type], n, d)
        for k, k_out, dt, by_block in places:
            m = (n + 31) // 32 if by_block else n
            own = _here(t[k], dt, m, d)
            setattr(a, k, own)
            setattr(a, k_out, _here(t[k_out], dt, m, d) if k_out in t else own)
    _call("moe_adamw_table", ctypes.byref(s), arr, _buf(table, moe_adamw_table_bytes(s), d),
          _stream(stream))


def moe_adamw_step(s, table, hyper, stream=None):
    """``hyper``: an ``adamw_hyper`` of this step, or a device tensor of the bytes of one."""
    d = _dev()
    dev = isinstance(hyper, torch.Tensor)
    _call("moe_adamw_step", ctypes.byref(s), _buf(table, moe_adamw_table_bytes(s), d),
          None if dev else ctypes.byref(hyper),
          _buf(hyper, ctypes.sizeof(moe_adamw_hyper), d) if dev else None, _stream(stream))


def moe_adamw_values(which, codes, scales, out, stream=None):
    """``which``: "m" or "v"."""
    n, d = codes.numel(), _dev()
    _call("moe_adamw_values", {"m": MOE_ADAMW_M, "v": MOE_ADAMW_V}[which], n,
          _here(codes, torch.uint8, n, d), _here(scales, torch.uint8, (n + 31) // 32, d),
          _here(out, _BF16, n, d), _stream(stream))


# ------------------------------------------------------------ kernel timing
_hip = None


def _hiprt():
    global _hip
    if _hip is None:
        h = ctypes.CDLL("libamdhip64.so")
        h.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        h.hipEventDestroy.argtypes = [ctypes.c_void_p]
        h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                          ctypes.c_void_p]
        _hip = h
    return _hip


class KernelTrace:
    """Per-kernel HIP events around every launch the library makes from this
    thread while active (``with KernelTrace(n) as tr: ...``); ``records()`` gives
    (name, milliseconds) per launch after the stream has been synchronised."""

    def __init__(self, capacity: int):
        h = _hiprt()
        self.capacity = capacity
        self._events = (ctypes.c_void_p * (2 * capacity))()
        ev = ctypes.c_void_p()
        for i in range(2 * capacity):
            if h.hipEventCreate(ctypes.byref(ev)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self._events[i] = ev.value
        self._names = (ctypes.c_char_p * capacity)()
        self.t = moe_trace(ctypes.cast(self._events, ctypes.POINTER(ctypes.c_void_p)),
                           ctypes.cast(self._names, ctypes.POINTER(ctypes.c_char_p)),
                           capacity, 0)

    def __enter__(self):
        self.t.count = 0
        lib().moe_trace_set(ctypes.byref(self.t))
        return self

    def __exit__(self, *exc):
        lib().moe_trace_set(None)
        return False

    def records(self):
        h = _hiprt()
        out = []
        ms = ctypes.c_float()
        for i in range(self.t.count):
            if h.hipEventElapsedTime(ctypes.byref(ms), self._events[2 * i], self._events[2 * i + 1]) != 0:
                raise RuntimeError("hipEventElapsedTime failed")
            out.append((self._names[i].decode(), ms.value))
        return out

    def close(self):
        h = _hiprt()
        for i in range(2 * self.capacity):
            h.hipEventDestroy(self._events[i])
        self.capacity = 0


# ------------------------------------------------------------ buffer helpers
def plan_views(s: moe_shape, plan: torch.Tensor, minibatch: int = 0) -> dict:
    """int32 views of the arrays of one minibatch's table inside a plan buffer
    (uint8 tensor); ``T`` is that minibatch's token count."""
    L = moe_plan_layout_of(s)
    T = min(L.T_minibatch, s.T - minibatch * L.T_minibatch)
    R = T * s.k
    sub = plan[minibatch * L.sub_plan_bytes:(minibatch + 1) * L.sub_plan_bytes]

    def view(off, n):
        return sub[off:off + 4 * n].view(torch.int32)

    return {"counts": view(L.counts, s.E), "offsets": view(L.offsets, s.E + 1),
            "src_token": view(L.src_token, R), "src_slot": view(L.src_slot, R),
            "pos": view(L.pos, R).view(T, s.k), "tiles": view(L.tiles, 2 * L.max_tiles).view(-1, 2),
            "n_tiles": view(L.n_tiles, 1), "err_flag": view(L.err_flag, 1),
            "active": view(L.active, s.E), "n_active": view(L.n_active, 1),
            "tile_first": view(L.tile_first, s.E + 1), "tile_m": L.tile_m,
            "wtiles": view(L.wtiles, 2 * L.max_wtiles).view(-1, 2),
            "n_wtiles": view(L.n_wtiles, 1), "wtile_m": L.wtile_m, "T": T}
