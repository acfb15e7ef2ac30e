"""Thin Python binding of libusaf.so (ctypes): argument marshalling only.

Every function here has the name of the C entry point it calls, without the ``usaf_`` prefix.
Tensors are PyTorch CUDA tensors; the binding passes their device pointers and the current CUDA
stream. PyTorch allocates memory and owns streams; every step of the computation runs in the
library's kernels. If the library is missing the binding raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass

import torch

from . import build as _build

_LIB = None

F32, BF16 = 0, 1
ROW_ALIGN = 16
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace", 4: "CUDA error",
          5: "timeout"}
DEV_NONFINITE, DEV_SELECT_EXACT_PATH, DEV_TIMEOUT, DEV_BAD_INDEX = 1, 2, 4, 8
DEV_SKIP_MASK = DEV_NONFINITE | DEV_TIMEOUT | DEV_BAD_INDEX


class UsafError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({code})")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("I", ctypes.c_int64)]


class TraceEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


class _Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "expert_count",
                                               "expert_offset", "perm_tok", "perm_slot",
                                               "slot_row")]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_D = ctypes.c_double
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGS = {
    "usaf_abi_version": (ctypes.c_int, []),
    "usaf_status_string": (ctypes.c_char_p, [_INT]),
    "usaf_routed_rows_capacity": (_I64, [_P]),
    "usaf_route_topk_workspace_size": (_SZ, [_P]),
    "usaf_route_topk": (_INT, [_P, _P, _INT, _P, _P, _P, _INT, _P, _P, _P, _SZ, _P]),
    "usaf_route_topk_noalloc": (_INT, [_P, _P, _INT, _P, _P, _P, _INT, _P, _P, _P]),
    "usaf_moe_fwd_workspace_size": (_SZ, [_P, _INT]),
    "usaf_moe_fwd": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_moe_fwd_wait": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                 _P]),
    "usaf_moe_bwd_workspace_size": (_SZ, [_P, _INT, _I64]),
    "usaf_moe_bwd_sparse": (_INT, [_P, _INT, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_sparse_adam_step": (_INT, [_I64, _P, _P, _P, _P, _P, _P, _I64, _P, _INT, _D, _D, _D, _D,
                                     _I64, _INT, _P, _P]),
    "usaf_importance_select_workspace_size": (_SZ, [_I64, _I64]),
    "usaf_importance_select": (_INT, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "usaf_rigl_swap_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "usaf_trace_enable": (_INT, [_INT]),
    "usaf_launch_count": (_I64, []),
    "usaf_trace_summary": (_INT, [_P, _INT]),
    "usaf_rigl_swap": (_INT, [_P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _INT, _P, _P, _P,
                              _P, _P, _P, _P, _SZ, _P]),
    "usaf_moe_fwd_wait2": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                  _SZ, _P]),
    "usaf_moe_fwd_stage": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _P, _SZ,
                                  _P]),
    "usaf_scan_nonfinite": (_INT, [_P, _I64, _P, _P]),
    "usaf_select_and_swap_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "usaf_select_and_swap": (_INT, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P,
                                    _INT, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_moe_bwd_sparse_accumulate": (_INT, [_P, _INT, _INT, _P, _P, _P, _P, _P, _P, _P, _P,
                                              _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _SZ,
                                              _P]),
    "usaf_moe_bwd_dense": (_INT, [_P, _INT, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                  _INT, _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_validate_active": (_INT, [_P, _I64, _I64, _P, _P]),
    "usaf_shard_key_histogram": (_INT, [_P, _I64, _P, ctypes.c_uint32, _INT, _INT, _P, _P]),
    "usaf_shard_emit_workspace_size": (_SZ, [_I64, _I64]),
    "usaf_shard_emit": (_INT, [_P, _I64, _P, ctypes.c_uint32, _I64, _I64, _I64, _P, _P, _P, _SZ,
                               _P]),
    "usaf_active_bitmap": (_INT, [_P, _I64, _I64, _I64, _P, _P]),
    "usaf_rigl_apply_workspace_size": (_SZ, [_I64, _I64]),
    "usaf_rigl_apply": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P, _INT, _P, _P,
                               _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_reselect_carry_workspace_size": (_SZ, []),
    "usaf_reselect_carry": (_INT, [_P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _INT, _P,
                                   _P, _P, _P, _P, _P, _SZ, _P]),
    "usaf_masked_plan_size": (_SZ, [_P]),
    "usaf_masked_plan_build": (_INT, [_P, _P, _I64, _D, _P, _SZ, _P]),
    "usaf_moe_bwd_sparse_planned": (_INT, [_P, _INT, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _P, _I64, _P, _P, _P, _P, _INT, _P, _I64, _P, _P,
                                           _SZ, _P]),
    "usaf_moe_wgrad_dense": (_INT, [_P, _INT, _P, _P, _P, _P, _INT, _P, _P, _SZ, _P]),
    "usaf_moe_bwd_dlogit_offset": (_I64, [_P, _INT, _I64]),
    "usaf_diag_bounded_wait": (_INT, [_I64, _P, _P]),
    "usaf_reselect_full_workspace_size": (_SZ, [_I64, _I64]),
    "usaf_reselect_full": (_INT, [_P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _INT, _P,
                                  _P, _P, _P, _P, _P, _P, _SZ, _P]),
}

# include/usaf_train.h: auxiliary router losses, dense router gradient products, 8-bit activations
_TRAIN_SIGS = {
    "usaf_router_aux_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "usaf_router_aux_fwd": (_INT, [_I64, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _D, _D, _P, _P,
                                   _P, _P, _P, _P, _SZ, _P]),
    "usaf_router_aux_bwd": (_INT, [_I64, _I64, _I64, _P, _I64, _P, _P, _I64, _D, _D, _P, _P, _P,
                                   _P, _I64, _INT, _P, _P]),
    "usaf_router_grad_workspace_size": (_SZ, [_I64, _I64, _I64, _INT]),
    "usaf_router_grad": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P,
                                _SZ, _P]),
    "usaf_act8_save": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "usaf_act8_restore": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
}


def header_symbols() -> list:
    """Names of the functions include/usaf.h declares."""
    text = open(os.path.join(_build.ROOT, "include", "usaf.h")).read()
    return sorted(set(re.findall(r"\b(usaf_[a-z0-9_]+)\s*\(", text)))


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load libusaf.so (building it first if it is absent)."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path):
            _build.build()
        L = ctypes.CDLL(path)
        for name, (res, args) in (*_SIGS.items(), *_TRAIN_SIGS.items()):
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(name: str, code: int) -> None:
    if code != 0:
        raise UsafError(name, code)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def shape(T, H, E, k, I) -> Shape:
    return Shape(int(T), int(H), int(E), int(k), int(I))


def routed_rows_capacity(s: Shape) -> int:
    return int(lib().usaf_routed_rows_capacity(ctypes.byref(s)))


@dataclass
class Routing:
    """Device routing tables of one layer call (see usaf_routing in include/usaf.h)."""
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    expert_count: torch.Tensor
    expert_offset: torch.Tensor
    perm_tok: torch.Tensor
    perm_slot: torch.Tensor
    slot_row: torch.Tensor

    @staticmethod
    def empty(s: Shape, device="cuda") -> "Routing":
        R = s.T * s.k
        cap = routed_rows_capacity(s)
        i32 = dict(dtype=torch.int32, device=device)
        return Routing(torch.empty(R, **i32), torch.empty(R, dtype=torch.float32, device=device),
                       torch.empty(s.E, **i32), torch.empty(s.E + 1, **i32),
                       torch.empty(cap, **i32), torch.empty(cap, **i32), torch.empty(R, **i32))

    def c(self) -> _Routing:
        try:
            return _Routing(self.topk_idx.data_ptr(), self.topk_w.data_ptr(),
                            self.expert_count.data_ptr(), self.expert_offset.data_ptr(),
                            self.perm_tok.data_ptr(), self.perm_slot.data_ptr(),
                            self.slot_row.data_ptr())
        except AttributeError:  # a field that is None or an address
            return _Routing(*[_ptr(getattr(self, f)) for f, _ in _Routing._fields_])


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def route_topk_workspace_size(s: Shape) -> int:
    return int(lib().usaf_route_topk_workspace_size(ctypes.byref(s)))


def route_topk(s: Shape, x, w_router, rt: Routing, logits_in=None, logits_out=None, renorm=1,
               dev_status=None, ws=None, stream=None):
    dev = rt.topk_idx.device
    if ws is None:
        ws = _ws(route_topk_workspace_size(s), dev)
    xdt = _dt(x) if x is not None else F32
    r = rt.c()
    _check("usaf_route_topk", lib().usaf_route_topk(
        ctypes.byref(s), _ptr(x), xdt, _ptr(w_router), _ptr(logits_in), _ptr(logits_out),
        int(renorm), ctypes.byref(r), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def route_topk_noalloc(s: Shape, x, w_router, rt: Routing, logits_in=None, logits_out=None,
                       renorm=1, dev_status=None, stream=None):
    """usaf_route_topk_noalloc: no workspace argument; scratch is the library's fixed array."""
    xdt = _dt(x) if x is not None else F32
    r = rt.c()
    _check("usaf_route_topk_noalloc", lib().usaf_route_topk_noalloc(
        ctypes.byref(s), _ptr(x), xdt, _ptr(w_router), _ptr(logits_in), _ptr(logits_out),
        int(renorm), ctypes.byref(r), _ptr(dev_status), _stream(stream)))


def moe_fwd_workspace_size(s: Shape, dt: int) -> int:
    return int(lib().usaf_moe_fwd_workspace_size(ctypes.byref(s), dt))


def moe_fwd(s: Shape, x, w_gate_up, w_down, rt: Routing, x_perm, h, wa, y, ws=None, stream=None,
            weights_ready=None, dev_status=None, down_ready=None):
    """weights_ready: a recorded torch.cuda.Event that the reads of the expert weights wait for
    (the token gather before them does not); with down_ready, weights_ready is waited for before
    the gate_up GEMM and down_ready before the down GEMM (usaf_moe_fwd_wait2)."""
    dt = _dt(x)
    if ws is None:
        ws = _ws(moe_fwd_workspace_size(s, dt), x.device)
    r = rt.c()
    ev = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    if down_ready is None:
        _check("usaf_moe_fwd_wait", lib().usaf_moe_fwd_wait(
            ctypes.byref(s), dt, _ptr(x), _ptr(w_gate_up), _ptr(w_down), ctypes.byref(r),
            _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(y), ev(weights_ready), _ptr(dev_status),
            _ptr(ws), ws.numel(), _stream(stream)))
    else:
        _check("usaf_moe_fwd_wait2", lib().usaf_moe_fwd_wait2(
            ctypes.byref(s), dt, _ptr(x), _ptr(w_gate_up), _ptr(w_down), ctypes.byref(r),
            _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(y), ev(weights_ready), ev(down_ready),
            _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


FWD_GATHER, FWD_GATE_UP, FWD_DOWN = 1, 2, 4


def moe_fwd_stage(s: Shape, x, w_gate_up, w_down, rt: Routing, x_perm, h, wa, y, stages, ws,
                  stream=None, dev_status=None):
    """usaf_moe_fwd_stage: the forward's stages in the bit set `stages` (FWD_GATHER,
    FWD_GATE_UP, FWD_DOWN), in order, on the workspace the earlier stages used."""
    r = rt.c()
    _check("usaf_moe_fwd_stage", lib().usaf_moe_fwd_stage(
        ctypes.byref(s), _dt(x), _ptr(x), _ptr(w_gate_up), _ptr(w_down), ctypes.byref(r),
        _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(y), int(stages), _ptr(dev_status), _ptr(ws),
        ws.numel(), _stream(stream)))


def moe_bwd_workspace_size(s: Shape, dt: int, K: int) -> int:
    return int(lib().usaf_moe_bwd_workspace_size(ctypes.byref(s), dt, int(K)))


def moe_bwd_dlogit_offset(s: Shape, dt: int, K: int) -> int:
    """Byte offset in the backward workspace of dlogit at the selected experts ([T*k] fp32)."""
    return int(lib().usaf_moe_bwd_dlogit_offset(ctypes.byref(s), dt, int(K)))


def moe_bwd_sparse(s: Shape, x, w_router, w_gate_up, w_down, rt: Routing, x_perm, h, wa, dy,
                   act_idx, g_act, g_router, dx=None, dw_slot=None, logits=None, renorm=1,
                   dev_status=None, ws=None, stream=None):
    dt = _dt(x)
    K = 0 if act_idx is None else act_idx.numel()
    if ws is None:
        ws = _ws(moe_bwd_workspace_size(s, dt, K), x.device)
    r = rt.c()
    _check("usaf_moe_bwd_sparse", lib().usaf_moe_bwd_sparse(
        ctypes.byref(s), dt, int(renorm), _ptr(x), _ptr(w_router), _ptr(w_gate_up), _ptr(w_down),
        ctypes.byref(r), _ptr(logits), _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(dy), _ptr(act_idx),
        K, _ptr(g_act), _ptr(g_router), _ptr(dx), _ptr(dw_slot), _ptr(dev_status), _ptr(ws),
        ws.numel(), _stream(stream)))


def masked_plan_size(s: Shape) -> int:
    return int(lib().usaf_masked_plan_size(ctypes.byref(s)))


def masked_plan_build(s: Shape, act_idx, dense_density, plan, stream=None):
    """usaf_masked_plan_build; after the stream has run it, masked_plan_count(plan) reads the
    number of listed experts."""
    K = 0 if act_idx is None else act_idx.numel()
    _check("usaf_masked_plan_build", lib().usaf_masked_plan_build(
        ctypes.byref(s), _ptr(act_idx), K, float(dense_density), _ptr(plan), plan.numel(),
        _stream(stream)))


def masked_plan_count(plan) -> int:
    """The plan's first 8 bytes: the number of experts it lists (reads device memory)."""
    return int(plan[:8].view(torch.int64).item())


def moe_bwd_sparse_planned(s: Shape, x, w_router, w_gate_up, w_down, rt: Routing, x_perm, h, wa,
                           dy, act_idx, g_act, g_router, plan=None, n_dense=0, accumulate=0,
                           dx=None, dw_slot=None, logits=None, renorm=1, dev_status=None,
                           ws=None, stream=None):
    dt = _dt(x)
    K = 0 if act_idx is None else act_idx.numel()
    if ws is None:
        ws = _ws(moe_bwd_workspace_size(s, dt, K), x.device)
    r = rt.c()
    _check("usaf_moe_bwd_sparse_planned", lib().usaf_moe_bwd_sparse_planned(
        ctypes.byref(s), dt, int(renorm), _ptr(x), _ptr(w_router), _ptr(w_gate_up), _ptr(w_down),
        ctypes.byref(r), _ptr(logits), _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(dy), _ptr(act_idx),
        K, _ptr(g_act), _ptr(g_router), _ptr(dx), _ptr(dw_slot), int(accumulate), _ptr(plan),
        int(n_dense), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def moe_bwd_sparse_accumulate(s: Shape, x, w_router, w_gate_up, w_down, rt: Routing, x_perm,
                              h, wa, dy, act_idx, g_act, g_router, dx=None, dw_slot=None,
                              logits=None, renorm=1, dev_status=None, ws=None, stream=None):
    """moe_bwd_sparse that adds this micro-batch's g_act and g_router to the buffers."""
    dt = _dt(x)
    K = 0 if act_idx is None else act_idx.numel()
    if ws is None:
        ws = _ws(moe_bwd_workspace_size(s, dt, K), x.device)
    r = rt.c()
    _check("usaf_moe_bwd_sparse_accumulate", lib().usaf_moe_bwd_sparse_accumulate(
        ctypes.byref(s), dt, int(renorm), _ptr(x), _ptr(w_router), _ptr(w_gate_up), _ptr(w_down),
        ctypes.byref(r), _ptr(logits), _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(dy), _ptr(act_idx),
        K, _ptr(g_act), _ptr(g_router), _ptr(dx), _ptr(dw_slot), _ptr(dev_status), _ptr(ws),
        ws.numel(), _stream(stream)))


def moe_bwd_dense(s: Shape, x, w_router, w_gate_up, w_down, rt: Routing, x_perm, h, wa, dy,
                  g_dense, g_router, accumulate=0, dx=None, dw_slot=None, logits=None, renorm=1,
                  dev_status=None, ws=None, stream=None):
    dt = _dt(x)
    if ws is None:
        ws = _ws(moe_bwd_workspace_size(s, dt, 0), x.device)
    r = rt.c()
    _check("usaf_moe_bwd_dense", lib().usaf_moe_bwd_dense(
        ctypes.byref(s), dt, int(renorm), _ptr(x), _ptr(w_router), _ptr(w_gate_up), _ptr(w_down),
        ctypes.byref(r), _ptr(logits), _ptr(x_perm), _ptr(h), _ptr(wa), _ptr(dy), _ptr(g_dense),
        int(accumulate), _ptr(g_router), _ptr(dx), _ptr(dw_slot), _ptr(dev_status), _ptr(ws),
        ws.numel(), _stream(stream)))


def moe_wgrad_dense(s: Shape, rt: Routing, x_perm, wa, g_dense, ws, accumulate=0,
                    dev_status=None, stream=None):
    """usaf_moe_wgrad_dense: the dense expert gradient from the dh and permuted dy that the last
    backward call left in `ws` (that call's workspace)."""
    r = rt.c()
    _check("usaf_moe_wgrad_dense", lib().usaf_moe_wgrad_dense(
        ctypes.byref(s), _dt(x_perm), ctypes.byref(r), _ptr(x_perm), _ptr(wa), _ptr(g_dense),
        int(accumulate), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def sparse_adam_step(idx, g, p, m, v, w_seg0, n_seg0, w_seg1, lr, beta1, beta2, eps, step,
                     skip_if_nonfinite=0, dev_status=None, stream=None, n=None):
    n = g.numel() if n is None else n
    _check("usaf_sparse_adam_step", lib().usaf_sparse_adam_step(
        int(n), _ptr(idx), _ptr(g), _ptr(p), _ptr(m), _ptr(v), _ptr(w_seg0), int(n_seg0),
        _ptr(w_seg1), _dt(w_seg0), float(lr), float(beta1), float(beta2), float(eps), int(step),
        int(skip_if_nonfinite), _ptr(dev_status), _stream(stream)))


def scan_nonfinite(g, dev_status, stream=None, n=None):
    """usaf_scan_nonfinite: sets DEV_NONFINITE in dev_status when g[:n] holds a NaN or inf."""
    n = g.numel() if n is None else n
    _check("usaf_scan_nonfinite", lib().usaf_scan_nonfinite(_ptr(g), int(n), _ptr(dev_status),
                                                            _stream(stream)))


def importance_select_workspace_size(N: int, K: int) -> int:
    return int(lib().usaf_importance_select_workspace_size(int(N), int(K)))


def importance_select(g, K, out_idx, dev_status=None, ws=None, stream=None):
    N = g.numel()
    if ws is None:
        ws = _ws(importance_select_workspace_size(N, K), g.device)
    _check("usaf_importance_select", lib().usaf_importance_select(
        _ptr(g), N, int(K), _ptr(out_idx), _ptr(dev_status), _ptr(ws), ws.numel(),
        _stream(stream)))


def rigl_swap_workspace_size(N: int, K: int, D: int) -> int:
    return int(lib().usaf_rigl_swap_workspace_size(int(N), int(K), int(D)))


def rigl_swap(g, act_idx, D, p_in, m_in, v_in, w_seg0, n_seg0, w_seg1, new_idx, p_out, m_out,
              v_out, n_swapped, dev_status=None, ws=None, stream=None):
    N, K = g.numel(), act_idx.numel()
    if ws is None:
        ws = _ws(rigl_swap_workspace_size(N, K, D), g.device)
    _check("usaf_rigl_swap", lib().usaf_rigl_swap(
        _ptr(g), N, _ptr(act_idx), K, int(D), _ptr(p_in), _ptr(m_in), _ptr(v_in), _ptr(w_seg0),
        int(n_seg0), _ptr(w_seg1), _dt(w_seg0), _ptr(new_idx), _ptr(p_out), _ptr(m_out),
        _ptr(v_out), _ptr(n_swapped), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def select_and_swap_workspace_size(N: int, K_sel: int, K: int, D: int) -> int:
    return int(lib().usaf_select_and_swap_workspace_size(int(N), int(K_sel), int(K), int(D)))


def select_and_swap(g, sel_idx, act_idx, D, p_in, m_in, v_in, w_seg0, n_seg0, w_seg1, new_idx,
                    p_out, m_out, v_out, n_swapped, dev_status=None, ws=None, stream=None):
    """usaf_select_and_swap: importance_select into sel_idx (K_sel = its length) and rigl_swap of
    act_idx, from one pass over g."""
    N, K, K_sel = g.numel(), act_idx.numel(), sel_idx.numel()
    if ws is None:
        ws = _ws(select_and_swap_workspace_size(N, K_sel, K, D), g.device)
    _check("usaf_select_and_swap", lib().usaf_select_and_swap(
        _ptr(g), N, K_sel, _ptr(sel_idx), _ptr(act_idx), K, int(D), _ptr(p_in), _ptr(m_in),
        _ptr(v_in), _ptr(w_seg0), int(n_seg0), _ptr(w_seg1), _dt(w_seg0), _ptr(new_idx),
        _ptr(p_out), _ptr(m_out), _ptr(v_out), _ptr(n_swapped), _ptr(dev_status), _ptr(ws),
        ws.numel(), _stream(stream)))


def reselect_full_workspace_size(N: int, K: int) -> int:
    return int(lib().usaf_reselect_full_workspace_size(int(N), int(K)))


def reselect_full(g, K, old_idx, p_in, m_in, v_in, w_seg0, n_seg0, w_seg1, new_idx, p_out, m_out,
                  v_out, n_kept, dev_status=None, ws=None, stream=None):
    N, K_old = g.numel(), old_idx.numel()
    if ws is None:
        ws = _ws(reselect_full_workspace_size(N, K), g.device)
    _check("usaf_reselect_full", lib().usaf_reselect_full(
        _ptr(g), N, int(K), _ptr(old_idx), K_old, _ptr(p_in), _ptr(m_in), _ptr(v_in),
        _ptr(w_seg0), int(n_seg0), _ptr(w_seg1), _dt(w_seg0), _ptr(new_idx), _ptr(p_out),
        _ptr(m_out), _ptr(v_out), _ptr(n_kept), _ptr(dev_status), _ptr(ws), ws.numel(),
        _stream(stream)))


def validate_active(idx, N, dev_status, stream=None):
    """usaf_validate_active: sets DEV_BAD_INDEX in dev_status unless idx is strictly ascending in
    [0, N)."""
    K = 0 if idx is None else idx.numel()
    _check("usaf_validate_active", lib().usaf_validate_active(
        _ptr(idx), K, int(N), _ptr(dev_status), _stream(stream)))


def diag_bounded_wait(limit_cycles, dev_status, stream=None):
    """usaf_diag_bounded_wait: one CTA whose bounded mbarrier wait runs out after limit_cycles."""
    _check("usaf_diag_bounded_wait", lib().usaf_diag_bounded_wait(
        int(limit_cycles), _ptr(dev_status), _stream(stream)))


def shard_key_histogram(g, excl, prefix, shift, bits, hist, stream=None):
    """hist [2^bits] uint64 (int64 tensor) += digit counts of the part's keys (usaf.h)."""
    _check("usaf_shard_key_histogram", lib().usaf_shard_key_histogram(
        _ptr(g), g.numel(), _ptr(excl), int(prefix) & 0xFFFFFFFF, int(shift), int(bits),
        _ptr(hist), _stream(stream)))


def shard_emit(g, excl, tau, take_eq, count, base, out, dev_status=None, ws=None, stream=None):
    n = g.numel()
    if ws is None:
        ws = _ws(lib().usaf_shard_emit_workspace_size(n, int(count)), g.device)
    _check("usaf_shard_emit", lib().usaf_shard_emit(
        _ptr(g), n, _ptr(excl), int(tau) & 0xFFFFFFFF, int(take_eq), int(count), int(base),
        _ptr(out), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def active_bitmap(idx, lo, n, bitmap, stream=None):
    K = 0 if idx is None else idx.numel()
    _check("usaf_active_bitmap", lib().usaf_active_bitmap(
        _ptr(idx), K, int(lo), int(n), _ptr(bitmap), _stream(stream)))


def _n_entries(n_seg0, w_seg1):
    return int(n_seg0) + (0 if w_seg1 is None else w_seg1.numel())


def rigl_apply(act_idx, D, grown, p_in, m_in, v_in, w_seg0, n_seg0, w_seg1, new_idx, p_out,
               m_out, v_out, n_swapped, dev_status=None, ws=None, stream=None):
    """usaf_rigl_apply: RigL's drop and merge with the grow set given (chosen over ranks)."""
    K = act_idx.numel()
    if ws is None:
        ws = _ws(lib().usaf_rigl_apply_workspace_size(K, int(D)), act_idx.device)
    _check("usaf_rigl_apply", lib().usaf_rigl_apply(
        _ptr(act_idx), K, _n_entries(n_seg0, w_seg1), int(D), _ptr(grown), _ptr(p_in), _ptr(m_in), _ptr(v_in), _ptr(w_seg0),
        int(n_seg0), _ptr(w_seg1), _dt(w_seg0), _ptr(new_idx), _ptr(p_out), _ptr(m_out),
        _ptr(v_out), _ptr(n_swapped), _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


def reselect_carry(new_idx, old_idx, p_in, m_in, v_in, w_seg0, n_seg0, w_seg1, p_out, m_out,
                   v_out, n_kept, dev_status=None, ws=None, stream=None):
    """usaf_reselect_carry: the state of a full reselection for a new set chosen over ranks."""
    if ws is None:
        ws = _ws(lib().usaf_reselect_carry_workspace_size(), new_idx.device)
    _check("usaf_reselect_carry", lib().usaf_reselect_carry(
        _ptr(new_idx), new_idx.numel(), _n_entries(n_seg0, w_seg1), _ptr(old_idx),
        old_idx.numel(), _ptr(p_in), _ptr(m_in), _ptr(v_in), _ptr(w_seg0), int(n_seg0),
        _ptr(w_seg1), _dt(w_seg0), _ptr(p_out), _ptr(m_out), _ptr(v_out), _ptr(n_kept),
        _ptr(dev_status), _ptr(ws), ws.numel(), _stream(stream)))


# ---------------------------------------------------------------- usaf_train.h
ACT8_BLOCK = 16


_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8


def _refuse(name, t, dtype, shape, dev):
    """Say what is wrong with a tensor that _ok or _ok_rows turned down."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {list(shape)} {dtype}, got {list(t.shape)} {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: expected a tensor on CUDA device {max(dev, 0)}, got {t.device}")
    raise ValueError(f"{name}: expected contiguous rows that do not overlap")


# The library reads and writes bare pointers, so tensors of another dtype, shape, layout or device
# are refused before any launch. These run on every call of a step: attribute reads and no more.
def _ok(name, t, dtype, shape, dev):
    """The address of a contiguous tensor."""
    if (t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0
            or not t.is_contiguous()):
        _refuse(name, t, dtype, shape, dev)
    return t.data_ptr()


def _opt(name, t, dtype, shape, dev):
    return None if t is None else _ok(name, t, dtype, shape, dev)


def _ok_rows(name, t, dtype, shape, dev):
    """The address of a tensor whose rows may be a distance apart, and that distance (torch keeps
    any stride for a single row)."""
    if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev or dev < 0:
        _refuse(name, t, dtype, shape, dev)
    ld, step = t.stride()
    n = shape[1]
    if (step != 1 and n > 1) or (ld < n and shape[0] > 1):
        _refuse(name, t, dtype, shape, dev)
    return t.data_ptr(), (ld if ld >= n else n)


def _buf(name, t, dev, nbytes=1, dtype=None):
    """The address of a contiguous buffer of at least that many bytes; None and addresses pass."""
    if t is None or t.__class__ is int:
        return t
    if (t.nbytes < nbytes or t.get_device() != dev or not t.is_contiguous()
            or (dtype is not None and t.dtype is not dtype)):
        raise ValueError(f"{name}: expected at least {nbytes} contiguous bytes "
                         f"{'' if dtype is None else f'of {dtype} '}on CUDA device {dev}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _status(t, dev):
    return None if t is None else _buf("dev_status", t, dev, 4)


def _on(stream, dev):
    """The stream handle: the device's current stream unless one is given. The library launches on
    the current device, so the tensors have to be there."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on CUDA device {dev}, but the current one is "
                         f"{torch._C._cuda_getDevice()}: call within torch.cuda.device({dev})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _ws_on(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace of the stream that the call runs on: the allocator may hand its memory out again as
    soon as the call returns, and then only behind the call's work."""
    if stream is None:
        return _ws(nbytes, device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return _ws(nbytes, device)


def router_aux_workspace_size(T: int, E: int, k: int, G: int = 1) -> int:
    return int(lib().usaf_router_aux_workspace_size(int(T), int(E), int(k), int(G)))


def router_aux_fwd(logits, topk_idx, k, count, prob_sum, n_tok, loss, coef_balance, coef_z,
                   token_mask=None, group_offset=None, dev_status=None, ws=None, stream=None):
    """usaf_router_aux_fwd: balance loss, z-loss and per-expert counts of logits [T,E] (rows may be
    a stride apart); count and prob_sum [G,E], n_tok [G], loss [3] = (total, balance, z)."""
    T, E = logits.shape
    G, d = count.shape[0], logits.get_device()
    if topk_idx.dim() == 2:
        topk_idx = topk_idx.reshape(-1)
    lp, ld = _ok_rows("logits", logits, _f32, (T, E), d)
    ge = (G, E)
    if group_offset is None and G != 1:
        raise ValueError("group_offset is required")
    if ws is None:
        ws = _ws_on(router_aux_workspace_size(T, E, k, G), logits.device, stream)
    _check("usaf_router_aux_fwd", lib().usaf_router_aux_fwd(
        T, E, int(k), lp, ld, _ok("topk_idx", topk_idx, _i32, (T * k,), d),
        _opt("token_mask", token_mask, _u8, (T,), d),
        _opt("group_offset", group_offset, _i32, (G + 1,), d), G, float(coef_balance),
        float(coef_z), _ok("count", count, _i32, ge, d), _ok("prob_sum", prob_sum, _f32, ge, d),
        _ok("n_tok", n_tok, _i32, (G,), d), _ok("loss", loss, _f32, (3,), d), _status(dev_status, d),
        _buf("ws", ws, d), ws.nbytes, _on(stream, d)))


def router_aux_bwd(logits, k, count, n_tok, dlogit, coef_balance, coef_z, d_loss=None,
                   token_mask=None, group_offset=None, accumulate=0, dev_status=None,
                   stream=None):
    """usaf_router_aux_bwd: the gradient of the forward's loss[0] times d_loss ([1], None: 1) into
    dlogit [T,E] (accumulate = 1 adds); count and n_tok as the forward wrote them."""
    T, E = logits.shape
    G, d = count.shape[0], logits.get_device()
    lp, ld = _ok_rows("logits", logits, _f32, (T, E), d)
    op, ldo = _ok_rows("dlogit", dlogit, _f32, (T, E), d)
    if group_offset is None and G != 1:
        raise ValueError("group_offset is required")
    _check("usaf_router_aux_bwd", lib().usaf_router_aux_bwd(
        T, E, int(k), lp, ld, _opt("token_mask", token_mask, _u8, (T,), d),
        _opt("group_offset", group_offset, _i32, (G + 1,), d), G, float(coef_balance),
        float(coef_z), _ok("count", count, _i32, (G, E), d), _ok("n_tok", n_tok, _i32, (G,), d),
        _opt("d_loss", d_loss, _f32, (1,), d), op, ldo, int(accumulate), _status(dev_status, d),
        _on(stream, d)))


def router_grad_workspace_size(T: int, E: int, H: int, dtype) -> int:
    """dtype: torch.bfloat16 or torch.float32, of x and dx."""
    dt = BF16 if dtype == torch.bfloat16 else F32
    return int(lib().usaf_router_grad_workspace_size(int(T), int(E), int(H), dt))


def router_grad(dlogit, x, w_router, g_router=None, g_in=None, dx=None, dx_in=None,
                dev_status=None, ws=None, stream=None):
    """usaf_router_grad: g_router = g_in + dlogit^T x and dx = dx_in + dlogit w_router, each only
    where its output is given (g_in / dx_in None: zero; they may be the outputs themselves)."""
    T, E = dlogit.shape
    ref = x if x is not None else dx
    if ref is None or (x is None and g_router is not None):
        raise ValueError("x is required")
    H, d, dt = ref.shape[1], dlogit.get_device(), ref.dtype
    dp, ld = _ok_rows("dlogit", dlogit, _f32, (T, E), d)
    th, eh = (T, H), (E, H)
    if ws is None:
        ws = _ws_on(router_grad_workspace_size(T, E, H, dt), dlogit.device, stream)
    _check("usaf_router_grad", lib().usaf_router_grad(
        T, E, H, _dt(ref), dp, ld, _opt("x", x, dt, th, d),
        _opt("w_router", w_router, _f32, eh, d), _opt("g_in", g_in, _f32, eh, d),
        _opt("g_router", g_router, _f32, eh, d), _opt("dx_in", dx_in, dt, th, d),
        _opt("dx", dx, dt, th, d), _status(dev_status, d), _buf("ws", ws, d), ws.nbytes, _on(stream, d)))


@dataclass
class ActStore8:
    """A layer's x and h between its forward and its backward, as 8-bit codes with one exponent
    byte per 16 values (the format is in include/usaf_train.h)."""
    x_code: torch.Tensor
    x_exp: torch.Tensor
    h_code: torch.Tensor
    h_exp: torch.Tensor

    @staticmethod
    def shapes(s: Shape) -> tuple:
        cap = routed_rows_capacity(s)
        return ((s.T, s.H), (s.T, -(-s.H // ACT8_BLOCK)), (2 * s.I, cap),
                (2 * s.I, cap // ACT8_BLOCK))

    @staticmethod
    def empty(s: Shape, device="cuda") -> "ActStore8":
        dts = (torch.int8, torch.uint8, torch.int8, torch.uint8)
        return ActStore8(*[torch.empty(sh, dtype=dt, device=device)
                           for sh, dt in zip(ActStore8.shapes(s), dts)])

    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.x_code, self.x_exp, self.h_code, self.h_exp))

    def ptrs(self, sh: tuple, dev: int) -> tuple:
        """The addresses, checked against the shapes of ActStore8.shapes."""
        return (_ok("x_code", self.x_code, torch.int8, sh[0], dev),
                _ok("x_exp", self.x_exp, _u8, sh[1], dev),
                _ok("h_code", self.h_code, torch.int8, sh[2], dev),
                _ok("h_exp", self.h_exp, _u8, sh[3], dev))


def act8_save(s: Shape, x, h, rt: Routing, store: ActStore8, dev_status=None, stream=None):
    """usaf_act8_save: x [T,H] and h [2I,R_cap] of a forward into the store."""
    d, sh = x.get_device(), ActStore8.shapes(s)
    xp, hp = _ok("x", x, x.dtype, sh[0], d), _ok("h", h, x.dtype, sh[2], d)
    r = _Routing(expert_offset=_buf("expert_offset", rt.expert_offset, d, 4 * s.E + 4, _i32))
    _check("usaf_act8_save", lib().usaf_act8_save(
        ctypes.byref(s), _dt(x), xp, hp, ctypes.byref(r), *store.ptrs(sh, d), _status(dev_status, d),
        _on(stream, d)))


def act8_restore(s: Shape, store: ActStore8, rt: Routing, x_perm, h, wa, x=None, stream=None):
    """usaf_act8_restore: what the backward reads (x_perm, h, wa; x too unless None) from the
    store and the routing of that forward."""
    d, dt, sh = h.get_device(), h.dtype, ActStore8.shapes(s)
    cap = sh[2][1]
    ptrs = store.ptrs(sh, d)
    r = _Routing(None, _buf("topk_w", rt.topk_w, d, 4 * s.T * s.k, _f32), None,
                 _buf("expert_offset", rt.expert_offset, d, 4 * s.E + 4, _i32),
                 _buf("perm_tok", rt.perm_tok, d, 4 * cap, _i32),
                 _buf("perm_slot", rt.perm_slot, d, 4 * cap, _i32))
    _check("usaf_act8_restore", lib().usaf_act8_restore(
        ctypes.byref(s), _dt(h), *ptrs, ctypes.byref(r), _opt("x", x, dt, sh[0], d),
        _ok("x_perm", x_perm, dt, (s.H, cap), d), _ok("h", h, dt, sh[2], d),
        _ok("wa", wa, dt, (s.I, cap), d), _on(stream, d)))


def trace_enable(on: bool) -> None:
    _check("usaf_trace_enable", lib().usaf_trace_enable(1 if on else 0))


def trace_summary() -> list:
    """[(kernel name, launches, total ms)] of the launches recorded since trace_enable(True)."""
    L = lib()
    n = L.usaf_trace_summary(None, 0)
    if n < 0:
        raise UsafError("usaf_trace_summary", 4)
    arr = (TraceEntry * max(n, 1))()
    n = L.usaf_trace_summary(arr, n)
    return [(arr[i].name.decode(), int(arr[i].launches), float(arr[i].total_ms)) for i in range(n)]


def launch_count() -> int:
    """Kernel launches the library has issued since it was loaded."""
    return int(lib().usaf_launch_count())
