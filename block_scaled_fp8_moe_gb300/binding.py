"""Thin ctypes binding of libmoe (include/moe.h): argument marshalling only.

Every function takes torch tensors, checks dtype/device/contiguity/size on the host, and calls
the C entry point of the same name on the current CUDA stream. There is no fallback: if libmoe.so
is missing, importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
lib = ctypes.CDLL(LIB_PATH)

(MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT,
 MOE_ERR_DEVICE_INPUT) = range(7)

EXPORTED = [
    "moe_status_string", "moe_workspace_bytes", "moe_packed_w13_bytes", "moe_packed_w2_bytes",
    "moe_quant_mxfp4", "moe_pack_w13", "moe_pack_w2", "moe_route_topk", "moe_quant_mxfp8",
    "moe_w13_swiglu_grouped", "moe_w2_combine_grouped", "moe_forward", "moe_check_device_status",
    "moe_route_topk_noalloc", "moe_selftest_timeout", "moe_route_topk_anchored", "moe_forward_anchored",
    "moe_packed_shared_w13_bytes", "moe_packed_shared_w2_bytes", "moe_pack_shared_w13", "moe_pack_shared_w2",
    "moe_shared_workspace_bytes", "moe_forward_shared", "moe_dead_from_survival", "moe_w2_grouped", "moe_combine",
    "moe_probe_mma_rate", "moe_quant_mxfp8_plan", "moe_experts_grouped", "moe_add_rmsnorm_mxfp8", "moe_kv_append",
    "moe_paged_attention_workspace_bytes", "moe_paged_attention", "moe_prefill_attention",
    "moe_selftest_attention_hold", "moe_rotary_turns", "moe_rope", "moe_rope_kv_append",
]

MOE_FLAG_SWIGLU_DEBUG = 1
MOE_FLAG_X_PLAN_ORDER = 2


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32), ("flags", ctypes.c_int32)]


class MoeSharedExpert(ctypes.Structure):
    _fields_ = [("I", ctypes.c_int32), ("w13", ctypes.c_void_p), ("w13_s", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_s", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


class MoeIntermediates(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "expert_counts", "expert_offsets", "xq", "xs", "hq", "hs", "swiglu")]


class MoeKvCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("format", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_s", ctypes.c_void_p), ("v_s", ctypes.c_void_p)]


class MoeAttention(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeRotary(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("factor", ctypes.c_float), ("turns", ctypes.c_void_p),
                ("axis", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_SHP = ctypes.POINTER(MoeShape)

lib.moe_status_string.restype = ctypes.c_char_p
lib.moe_status_string.argtypes = [ctypes.c_int]
lib.moe_workspace_bytes.restype = _SZ
lib.moe_workspace_bytes.argtypes = [_SHP]
lib.moe_packed_w13_bytes.restype = _SZ
lib.moe_packed_w13_bytes.argtypes = [_SHP, ctypes.POINTER(_SZ)]
lib.moe_packed_w2_bytes.restype = _SZ
lib.moe_packed_w2_bytes.argtypes = [_SHP, ctypes.POINTER(_SZ)]
lib.moe_quant_mxfp4.argtypes = [_I32, _I32, _P, _P, _P, _P]
lib.moe_quant_mxfp8.argtypes = [_I32, _I32, _P, _P, _P, _P]
lib.moe_quant_mxfp8_plan.argtypes = [_SHP] + [_P] * 6 + [_P]
lib.moe_experts_grouped.argtypes = [_SHP] + [_P] * 12 + [_P, _SZ, _P]
lib.moe_dead_from_survival.argtypes = [_I32, _P, ctypes.c_float, _P, _P]
lib.moe_pack_w13.argtypes = [_SHP, _P, _P, _P, _P, _P]
lib.moe_pack_w2.argtypes = [_SHP, _P, _P, _P, _P, _P]
lib.moe_route_topk.argtypes = [_SHP] + [_P] * 10 + [_P, _SZ, _P]
lib.moe_w13_swiglu_grouped.argtypes = [_SHP] + [_P] * 9 + [_P, _SZ, _P]
lib.moe_w2_combine_grouped.argtypes = [_SHP] + [_P] * 10 + [_P, _SZ, _P]
lib.moe_w2_grouped.argtypes = [_SHP] + [_P] * 7 + [_P, _SZ, _P]
lib.moe_combine.argtypes = [_SHP] + [_P] * 5 + [_P, _SZ, _P]
lib.moe_probe_mma_rate.argtypes = [_I32, _I32, ctypes.POINTER(_I32), ctypes.POINTER(ctypes.c_int64), _P, _SZ, _P]
lib.moe_forward.argtypes = [_SHP] + [_P] * 9 + [ctypes.POINTER(MoeIntermediates), _P, _SZ, _P]
lib.moe_check_device_status.argtypes = [_P, _P]
lib.moe_route_topk_noalloc.argtypes = [_SHP] + [_P] * 10 + [_P]
lib.moe_selftest_timeout.argtypes = [_P, ctypes.c_uint64, _P]
lib.moe_selftest_attention_hold.argtypes = [ctypes.c_int32]
lib.moe_route_topk_anchored.argtypes = [_SHP] + [_P] * 11 + [_P, _SZ, _P]
lib.moe_forward_anchored.argtypes = [_SHP] + [_P] * 10 + [ctypes.POINTER(MoeIntermediates), _P, _SZ, _P]
lib.moe_packed_shared_w13_bytes.restype = _SZ
lib.moe_packed_shared_w13_bytes.argtypes = [_SHP, ctypes.POINTER(_SZ)]
lib.moe_packed_shared_w2_bytes.restype = _SZ
lib.moe_packed_shared_w2_bytes.argtypes = [_SHP, ctypes.POINTER(_SZ)]
lib.moe_pack_shared_w13.argtypes = [_SHP, _P, _P, _P, _P, _P]
lib.moe_pack_shared_w2.argtypes = [_SHP, _P, _P, _P, _P, _P]
lib.moe_shared_workspace_bytes.restype = _SZ
lib.moe_shared_workspace_bytes.argtypes = [_SHP, _I32]
lib.moe_forward_shared.argtypes = ([_SHP] + [_P] * 9 + [ctypes.POINTER(MoeSharedExpert), _P,
                                   ctypes.POINTER(MoeIntermediates), _P, _SZ, _P, _P])
_I64 = ctypes.c_int64
_ATT = ctypes.POINTER(MoeAttention)
_KVC = ctypes.POINTER(MoeKvCache)
lib.moe_add_rmsnorm_mxfp8.argtypes = [_I32, _I32, _P, _P, _P, ctypes.c_float] + [_P] * 5
lib.moe_kv_append.argtypes = [_KVC, _I32, _P, _I64, _P, _I64, _P, _P, _SZ, _P]
lib.moe_paged_attention_workspace_bytes.restype = _SZ
lib.moe_paged_attention_workspace_bytes.argtypes = [_ATT, _I32, _I32]
lib.moe_paged_attention.argtypes = [_ATT, _KVC, _I32, _I32, _P, _I64, _P, _I32, _P, _P, _P, _SZ, _P]
lib.moe_prefill_attention.argtypes = [_ATT, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]
_ROT = ctypes.POINTER(MoeRotary)
lib.moe_rotary_turns.argtypes = [_I32, _P, _P]
lib.moe_rope.argtypes = [_ROT, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P]
lib.moe_rope_kv_append.argtypes = [_ROT, _KVC, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64,
                                   _P, _SZ, _P]
for _n in EXPORTED:
    if _n not in ("moe_status_string", "moe_workspace_bytes", "moe_packed_w13_bytes", "moe_packed_w2_bytes",
                  "moe_packed_shared_w13_bytes", "moe_packed_shared_w2_bytes", "moe_shared_workspace_bytes",
                  "moe_paged_attention_workspace_bytes"):
        getattr(lib, _n).restype = ctypes.c_int


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {lib.moe_status_string(code).decode()} ({code})")
        self.code = code


def _check(code: int, where: str) -> None:
    if code != MOE_OK:
        raise MoeError(code, where)


def shape(T, H, E, k, I, flags=0) -> MoeShape:
    return MoeShape(int(T), int(H), int(E), int(k), int(I), int(flags))


def _ptr(t: torch.Tensor | None, dtype=None, numel=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} needs {numel} elements, has {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def hs_pitch(I: int) -> int:
    return (I + 127) // 128 * 128 // 32


def moe_workspace_bytes(shp: MoeShape) -> int:
    return int(lib.moe_workspace_bytes(ctypes.byref(shp)))


def alloc_workspace(shp: MoeShape, device="cuda") -> torch.Tensor:
    n = moe_workspace_bytes(shp)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_packed_w13_bytes(shp: MoeShape) -> tuple[int, int]:
    sb = _SZ(0)
    n = lib.moe_packed_w13_bytes(ctypes.byref(shp), ctypes.byref(sb))
    return int(n), int(sb.value)


def moe_packed_w2_bytes(shp: MoeShape) -> tuple[int, int]:
    sb = _SZ(0)
    n = lib.moe_packed_w2_bytes(ctypes.byref(shp), ctypes.byref(sb))
    return int(n), int(sb.value)


def moe_quant_mxfp4(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None, stream=None):
    rows, cols = w.reshape(-1, w.shape[-1]).shape
    q = torch.empty(rows * cols // 2, dtype=torch.uint8, device=w.device) if q is None else q
    s = torch.empty(rows * cols // 32, dtype=torch.uint8, device=w.device) if s is None else s
    _check(lib.moe_quant_mxfp4(rows, cols, _ptr(w, torch.float32, name="w"), _ptr(q, torch.uint8, rows * cols // 2),
                               _ptr(s, torch.uint8, rows * cols // 32), _stream(stream)), "moe_quant_mxfp4")
    return q.view(*w.shape[:-1], cols // 2), s.view(*w.shape[:-1], cols // 32)


def moe_quant_mxfp8(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None, stream=None):
    rows, cols = x.reshape(-1, x.shape[-1]).shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device) if q is None else q
    s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device) if s is None else s
    _check(lib.moe_quant_mxfp8(rows, cols, _ptr(x, torch.bfloat16, name="x"), _ptr(q, torch.uint8, rows * cols),
                               _ptr(s, torch.uint8, rows * cols // 32), _stream(stream)), "moe_quant_mxfp8")
    return q, s


def moe_quant_mxfp8_plan(shp: MoeShape, x, plan: "Plan", xq_plan=None, xs_plan=None, xq=None, xs=None,
                         stream=None):
    """MXFP8 codes/scales written to plan rows ([T*k, H] / [T*k, H/32]); token order too if given."""
    S = shp.T * shp.k
    xq_plan = torch.empty(max(S, 1), shp.H, dtype=torch.uint8, device=x.device) if xq_plan is None else xq_plan
    xs_plan = torch.empty(max(S, 1), shp.H // 32, dtype=torch.uint8, device=x.device) if xs_plan is None else xs_plan
    _check(lib.moe_quant_mxfp8_plan(
        ctypes.byref(shp), _ptr(x, torch.bfloat16, shp.T * shp.H, "x"), _ptr(plan.row_of_slot, torch.int32, S),
        _ptr(xq_plan, torch.uint8, S * shp.H), _ptr(xs_plan, torch.uint8, S * shp.H // 32),
        _ptr(xq, torch.uint8, shp.T * shp.H), _ptr(xs, torch.uint8, shp.T * shp.H // 32), _stream(stream)),
        "moe_quant_mxfp8_plan")
    return xq_plan, xs_plan


SURVIVAL_THRESHOLD = 0.2


def moe_dead_from_survival(p_survive: torch.Tensor, threshold: float = SURVIVAL_THRESHOLD,
                           dead: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """u8 [T] dead-row mask: 1 where the fp32 survival estimate is below the threshold."""
    T = p_survive.numel()
    dead = torch.empty(T, dtype=torch.uint8, device=p_survive.device) if dead is None else dead
    _check(lib.moe_dead_from_survival(T, _ptr(p_survive, torch.float32, T, "p_survive"), float(threshold),
                                      _ptr(dead, torch.uint8, T, "dead"), _stream(stream)), "moe_dead_from_survival")
    return dead


def moe_pack_w13(shp: MoeShape, q: torch.Tensor, s: torch.Tensor, stream=None):
    nq, ns = moe_packed_w13_bytes(shp)
    qp = torch.empty(nq, dtype=torch.uint8, device=q.device)
    sp = torch.empty(ns, dtype=torch.uint8, device=q.device)
    _check(lib.moe_pack_w13(ctypes.byref(shp), _ptr(q, torch.uint8, shp.E * 2 * shp.I * shp.H // 2),
                            _ptr(s, torch.uint8, shp.E * 2 * shp.I * shp.H // 32), _ptr(qp), _ptr(sp),
                            _stream(stream)), "moe_pack_w13")
    return qp, sp


def moe_pack_w2(shp: MoeShape, q: torch.Tensor, s: torch.Tensor, stream=None):
    nq, ns = moe_packed_w2_bytes(shp)
    qp = torch.empty(nq, dtype=torch.uint8, device=q.device)
    sp = torch.empty(ns, dtype=torch.uint8, device=q.device)
    _check(lib.moe_pack_w2(ctypes.byref(shp), _ptr(q, torch.uint8, shp.E * shp.H * shp.I // 2),
                           _ptr(s, torch.uint8, shp.E * shp.H * shp.I // 32), _ptr(qp), _ptr(sp),
                           _stream(stream)), "moe_pack_w2")
    return qp, sp


class Plan:
    """Device tensors written by moe_route_topk."""

    def __init__(self, shp: MoeShape, device):
        T, k, E = shp.T, shp.k, shp.E
        self.topk_idx = torch.empty(T, k, dtype=torch.int32, device=device)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=device)
        self.expert_counts = torch.empty(E, dtype=torch.int32, device=device)
        self.expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.slot_of_row = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)
        self.row_of_slot = torch.empty(max(T * k, 1), dtype=torch.int32, device=device)


def moe_route_topk(shp: MoeShape, x, w_router, bias, dead, ws, plan: Plan | None = None, stream=None,
                   anchor=None) -> Plan:
    """anchor (optional int32 [T]): -1 routes the row itself, a >= 0 reuses row a's experts."""
    plan = Plan(shp, x.device) if plan is None else plan
    T, H, E = shp.T, shp.H, shp.E
    _check(lib.moe_route_topk_anchored(
        ctypes.byref(shp), _ptr(x, torch.bfloat16, T * H, "x"), _ptr(w_router, torch.bfloat16, E * H, "w_router"),
        _ptr(bias, torch.float32, E, "bias"), _ptr(dead, torch.uint8, T, "dead"),
        _ptr(anchor, torch.int32, T, "anchor"),
        _ptr(plan.topk_idx), _ptr(plan.topk_w), _ptr(plan.expert_counts), _ptr(plan.expert_offsets),
        _ptr(plan.slot_of_row), _ptr(plan.row_of_slot), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_route_topk_anchored")
    return plan


def moe_route_topk_noalloc(shp: MoeShape, x, w_router, bias, dead, plan: Plan | None = None,
                           stream=None) -> Plan:
    """moe_route_topk without a workspace (scratch inside the library; see include/moe.h)."""
    plan = Plan(shp, x.device) if plan is None else plan
    T, H, E = shp.T, shp.H, shp.E
    _check(lib.moe_route_topk_noalloc(
        ctypes.byref(shp), _ptr(x, torch.bfloat16, T * H, "x"), _ptr(w_router, torch.bfloat16, E * H, "w_router"),
        _ptr(bias, torch.float32, E, "bias"), _ptr(dead, torch.uint8, T, "dead"),
        _ptr(plan.topk_idx), _ptr(plan.topk_w), _ptr(plan.expert_counts), _ptr(plan.expert_offsets),
        _ptr(plan.slot_of_row), _ptr(plan.row_of_slot), _stream(stream)), "moe_route_topk_noalloc")
    return plan


def moe_w13_swiglu_grouped(shp: MoeShape, xq, xs, w13p, w13sp, plan: Plan, ws, hq=None, hs=None, debug=None,
                           stream=None):
    """xq/xs in token order, or in plan order when shp.flags has MOE_FLAG_X_PLAN_ORDER."""
    S = shp.T * shp.k
    dev = xq.device
    rows = S if shp.flags & MOE_FLAG_X_PLAN_ORDER else shp.T
    hq = torch.empty(max(S, 1), shp.I, dtype=torch.uint8, device=dev) if hq is None else hq
    hs = torch.empty(max(S, 1), hs_pitch(shp.I), dtype=torch.uint8, device=dev) if hs is None else hs
    _check(lib.moe_w13_swiglu_grouped(
        ctypes.byref(shp), _ptr(xq, torch.uint8, rows * shp.H), _ptr(xs, torch.uint8, rows * shp.H // 32),
        _ptr(w13p, torch.uint8), _ptr(w13sp, torch.uint8), _ptr(plan.expert_offsets), _ptr(plan.slot_of_row),
        _ptr(hq, torch.uint8, S * shp.I), _ptr(hs, torch.uint8, S * hs_pitch(shp.I)),
        _ptr(debug, torch.float32, S * shp.I), _ptr(ws), ws.numel(), _stream(stream)), "moe_w13_swiglu_grouped")
    return hq, hs


def moe_w2_combine_grouped(shp: MoeShape, hq, hs, w2p, w2sp, plan: Plan, ws, out=None, stream=None, dead=None):
    out = torch.empty(shp.T, shp.H, dtype=torch.bfloat16, device=hq.device) if out is None else out
    _check(lib.moe_w2_combine_grouped(
        ctypes.byref(shp), _ptr(hq, torch.uint8), _ptr(hs, torch.uint8), _ptr(w2p, torch.uint8),
        _ptr(w2sp, torch.uint8), _ptr(plan.topk_w), _ptr(plan.expert_offsets), _ptr(plan.slot_of_row),
        _ptr(plan.row_of_slot), _ptr(dead, torch.uint8, shp.T, "dead"),
        _ptr(out, torch.bfloat16, shp.T * shp.H, "out"), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_w2_combine_grouped")
    return out


def moe_w2_grouped(shp: MoeShape, hq, hs, w2p, w2sp, plan: Plan, ws, y=None, stream=None):
    """Down-projection GEMM alone: fp32 rows y [T*k, H] in plan order, before the routing weight."""
    S = shp.T * shp.k
    y = torch.empty(max(S, 1), shp.H, dtype=torch.float32, device=hq.device) if y is None else y
    _check(lib.moe_w2_grouped(
        ctypes.byref(shp), _ptr(hq, torch.uint8), _ptr(hs, torch.uint8), _ptr(w2p, torch.uint8),
        _ptr(w2sp, torch.uint8), _ptr(plan.expert_offsets), _ptr(plan.slot_of_row),
        _ptr(y, torch.float32, S * shp.H, "y"), _ptr(ws), ws.numel(), _stream(stream)), "moe_w2_grouped")
    return y


def moe_combine(shp: MoeShape, y, plan: Plan, ws, dead=None, out=None, stream=None):
    """Fixed-order combine alone: out[t] = bf16(((w_0 y[r_0] + w_1 y[r_1]) + ...)), dead rows +0."""
    out = torch.empty(shp.T, shp.H, dtype=torch.bfloat16, device=y.device) if out is None else out
    _check(lib.moe_combine(
        ctypes.byref(shp), _ptr(y, torch.float32, shp.T * shp.k * shp.H, "y"),
        _ptr(plan.topk_w, torch.float32, shp.T * shp.k, "topk_w"),
        _ptr(plan.row_of_slot, torch.int32, shp.T * shp.k, "row_of_slot"), _ptr(dead, torch.uint8, shp.T, "dead"),
        _ptr(out, torch.bfloat16, shp.T * shp.H, "out"), _ptr(ws), ws.numel(), _stream(stream)), "moe_combine")
    return out


def moe_experts_grouped(shp: MoeShape, xq, xs, w13p, w13sp, w2p, w2sp, plan: Plan, ws, hq=None, hs=None, y=None,
                        debug=None, stream=None):
    """Both expert GEMMs (one launch for decode-sized batches): hq / hs and plan-order fp32 y."""
    S = shp.T * shp.k
    dev = xq.device
    rows = S if shp.flags & MOE_FLAG_X_PLAN_ORDER else shp.T
    hq = torch.empty(max(S, 1), shp.I, dtype=torch.uint8, device=dev) if hq is None else hq
    hs = torch.empty(max(S, 1), hs_pitch(shp.I), dtype=torch.uint8, device=dev) if hs is None else hs
    y = torch.empty(max(S, 1), shp.H, dtype=torch.float32, device=dev) if y is None else y
    _check(lib.moe_experts_grouped(
        ctypes.byref(shp), _ptr(xq, torch.uint8, rows * shp.H), _ptr(xs, torch.uint8, rows * shp.H // 32),
        _ptr(w13p, torch.uint8), _ptr(w13sp, torch.uint8), _ptr(w2p, torch.uint8), _ptr(w2sp, torch.uint8),
        _ptr(plan.expert_offsets), _ptr(plan.slot_of_row), _ptr(hq, torch.uint8, S * shp.I),
        _ptr(hs, torch.uint8, S * hs_pitch(shp.I)), _ptr(debug, torch.float32, S * shp.I),
        _ptr(y, torch.float32, S * shp.H, "y"), _ptr(ws), ws.numel(), _stream(stream)), "moe_experts_grouped")
    return hq, hs, y


class SharedExpert:
    """A shared expert's packed MXFP8 weights on the device (canonical E4M3 codes and UE8M0 scales
    in, see include/moe.h) and its per-T scratch."""

    def __init__(self, H: int, I: int, q13, s13, q2, s2, stream=None):
        self.H, self.I = H, I
        dev = q13.device
        shp = shape(1, H, 1, 1, I)
        sb = ctypes.c_size_t(0)
        n = lib.moe_packed_shared_w13_bytes(ctypes.byref(shp), ctypes.byref(sb))
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_packed_shared_w13_bytes")
        self.w13p = torch.empty(n, dtype=torch.uint8, device=dev)
        self.w13sp = torch.empty(sb.value, dtype=torch.uint8, device=dev)
        _check(lib.moe_pack_shared_w13(ctypes.byref(shp), _ptr(q13, torch.uint8, 2 * I * H), _ptr(s13, torch.uint8),
                                       _ptr(self.w13p), _ptr(self.w13sp), _stream(stream)), "moe_pack_shared_w13")
        n = lib.moe_packed_shared_w2_bytes(ctypes.byref(shp), ctypes.byref(sb))
        self.w2p = torch.empty(n, dtype=torch.uint8, device=dev)
        self.w2sp = torch.empty(sb.value, dtype=torch.uint8, device=dev)
        _check(lib.moe_pack_shared_w2(ctypes.byref(shp), _ptr(q2, torch.uint8, H * I), _ptr(s2, torch.uint8),
                                      _ptr(self.w2p), _ptr(self.w2sp), _stream(stream)), "moe_pack_shared_w2")
        self._ws = {}

    def descriptor(self, shp: MoeShape) -> MoeSharedExpert:
        if shp.T not in self._ws:
            n = lib.moe_shared_workspace_bytes(ctypes.byref(shp), self.I)
            if n == 0:
                raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_shared_workspace_bytes")
            self._ws[shp.T] = torch.empty(n, dtype=torch.uint8, device=self.w13p.device)
        ws = self._ws[shp.T]
        return MoeSharedExpert(self.I, self.w13p.data_ptr(), self.w13sp.data_ptr(), self.w2p.data_ptr(),
                               self.w2sp.data_ptr(), ws.data_ptr(), ws.numel())


def moe_forward(shp: MoeShape, x, w_router, bias, dead, w13p, w13sp, w2p, w2sp, ws, out=None,
                inter: dict | None = None, stream=None, anchor=None, shared: SharedExpert | None = None,
                side_stream=None):
    out = torch.empty(shp.T, shp.H, dtype=torch.bfloat16, device=x.device) if out is None else out
    im = None
    if inter:
        im = MoeIntermediates(*[ctypes.c_void_p(inter[n].data_ptr()) if inter.get(n) is not None else None
                                for n, _ in MoeIntermediates._fields_])
    if shared is not None:
        desc = shared.descriptor(shp)
        _check(lib.moe_forward_shared(
            ctypes.byref(shp), _ptr(x, torch.bfloat16, shp.T * shp.H, "x"),
            _ptr(w_router, torch.bfloat16, shp.E * shp.H, "w_router"), _ptr(bias, torch.float32, shp.E, "bias"),
            _ptr(dead, torch.uint8, shp.T, "dead"), _ptr(anchor, torch.int32, shp.T, "anchor"),
            _ptr(w13p, torch.uint8), _ptr(w13sp, torch.uint8), _ptr(w2p, torch.uint8), _ptr(w2sp, torch.uint8),
            ctypes.byref(desc), _ptr(out, torch.bfloat16, shp.T * shp.H, "out"),
            ctypes.byref(im) if im is not None else None, _ptr(ws), ws.numel(), _stream(stream),
            _stream(side_stream) if side_stream is not None else None), "moe_forward_shared")
    elif anchor is None:
        _check(lib.moe_forward(
            ctypes.byref(shp), _ptr(x, torch.bfloat16, shp.T * shp.H, "x"),
            _ptr(w_router, torch.bfloat16, shp.E * shp.H, "w_router"), _ptr(bias, torch.float32, shp.E, "bias"),
            _ptr(dead, torch.uint8, shp.T, "dead"), _ptr(w13p, torch.uint8), _ptr(w13sp, torch.uint8),
            _ptr(w2p, torch.uint8), _ptr(w2sp, torch.uint8), _ptr(out, torch.bfloat16, shp.T * shp.H, "out"),
            ctypes.byref(im) if im is not None else None, _ptr(ws), ws.numel(), _stream(stream)), "moe_forward")
    else:
        _check(lib.moe_forward_anchored(
            ctypes.byref(shp), _ptr(x, torch.bfloat16, shp.T * shp.H, "x"),
            _ptr(w_router, torch.bfloat16, shp.E * shp.H, "w_router"), _ptr(bias, torch.float32, shp.E, "bias"),
            _ptr(dead, torch.uint8, shp.T, "dead"), _ptr(anchor, torch.int32, shp.T, "anchor"),
            _ptr(w13p, torch.uint8), _ptr(w13sp, torch.uint8),
            _ptr(w2p, torch.uint8), _ptr(w2sp, torch.uint8), _ptr(out, torch.bfloat16, shp.T * shp.H, "out"),
            ctypes.byref(im) if im is not None else None, _ptr(ws), ws.numel(), _stream(stream)),
            "moe_forward_anchored")
    return out


# --------------------------------------------------------------------------------------------------
# Residual norm, rotary positions, key/value cache, attention
# --------------------------------------------------------------------------------------------------
MOE_KV_BF16 = 0
MOE_KV_MXFP8 = 1
MOE_KV_MXFP4 = 4


# These calls run once or more per layer and step, where the host's time counts as much as the kernel's: addresses
# go to ctypes as plain integers, and descriptors and sizes are kept by their values.
def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _on(t: torch.Tensor, name: str, dtype, dev: int) -> int:
    """The address of a contiguous tensor of this type on device `dev`."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows_on(t: torch.Tensor, name: str, heads: int, D: int, dev: int) -> tuple[int, int]:
    """The address and the row stride of bf16 rows [rows, heads, D] (rows may lie apart; one row has no stride)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    n, h, d = t.shape
    if h != heads or d != D:
        raise ValueError(f"{name} must be [rows, {heads}, {D}], is {tuple(t.shape)}")
    row, head, one = t.stride()
    if n * h and ((one != 1 and d > 1) or (head != D and h > 1)):
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return t.data_ptr(), row if n > 1 else h * d


def _current(t: torch.Tensor, name: str) -> int:
    """t's device, which has to be the current one (launches go there)."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


_as_is = contextlib.nullcontext()


def _allocating(stream):
    """Where outputs are allocated: on the stream that will write them."""
    return _as_is if stream is None else torch.cuda.stream(stream)


def _sized(t: torch.Tensor, name: str, dtype, numel: int, dev: int) -> int:
    if t.numel() != numel:
        raise ValueError(f"{name} needs {numel} elements, has {t.numel()}")
    return _on(t, name, dtype, dev)


_scratch: dict[tuple[int, int], tuple[torch.Tensor, int, int]] = {}
# Buffers that a stream has outgrown. Kept: another thread may be about to launch with one.
_outgrown: dict[tuple[int, int], list[torch.Tensor]] = {}
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _workspace(nbytes: int, like: torch.Tensor, stream, dev: int, raw: int) -> tuple[int, int]:
    """Address and size of this stream's workspace of the attention and cache calls. Not for a graph: all that are
    captured share one stream, and would share their partial results when they are replayed on others."""
    if stream is None:
        captured = _capturing()
    else:
        with torch.cuda.stream(stream):
            captured = _capturing()
    if captured:
        raise ValueError(f"a captured call needs a workspace of its own: pass ws, uint8 of at least {max(nbytes, 256)} "
                         "zeros, which the graph's replays use and moe_check_device_status(ws) reads")
    have = _scratch.get((dev, raw))
    if have is None or have[2] < nbytes:
        have = _grown(have, nbytes, like, stream, (dev, raw))
    return have[1], have[2]


def _grown(have, nbytes: int, like: torch.Tensor, stream, key):
    """A larger workspace for that stream (at least twofold); its status word starts at zero."""
    size = max(nbytes, 4096, 0 if have is None else 2 * have[2])
    with _allocating(stream):
        ws = torch.empty(size, dtype=torch.uint8, device=like.device)
        ws[:256].zero_()
    if have is not None:
        _outgrown.setdefault(key, []).append(have[0])
    _scratch[key] = ws, ws.data_ptr(), size
    return _scratch[key]


def attention_status(device=None, stream=None) -> None:
    """Synchronises `stream` and raises what the attention and cache calls without a workspace of their own found
    invalid on the device there (a page, slot or length out of range) or gave up, then clears it."""
    s = torch.cuda.current_stream(device) if stream is None else stream
    found = None
    key = s.device_index, s.cuda_stream
    for ws in _outgrown.get(key, []) + [have[0] for have in (_scratch.get(key),) if have]:
        try:
            moe_check_device_status(ws, s)
        except MoeError as e:
            found = found or e
    if found:
        raise found


@functools.lru_cache(maxsize=4096)
def _attention(B: int, Hq: int, Hkv: int, D: int, window: int, sinks: int, scale: float | None):
    return ctypes.byref(MoeAttention(B, Hq, Hkv, D, window, sinks, D ** -0.5 if scale is None else scale))


@functools.lru_cache(maxsize=4096)
def _paged_bytes(a, rows: int, max_len: int) -> int:
    return int(lib.moe_paged_attention_workspace_bytes(a, rows, max_len))


def moe_add_rmsnorm_mxfp8(x, weight, residual=None, eps: float = 1e-6, sum_out=None, y=None, q=None, s=None,
                          quant: bool = True, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight and y's MXFP8 codes and scales, for bf16 rows [..., cols].

    Returns (y, sum, q, s): bf16(y), bf16(h), u8 codes and u8 scales [..., cols / 32]. sum_out and y may be x or residual
    themselves. With quant=False, q and s are None. residual has x's shape, or its rows in another number of dimensions."""
    dev = _current(x, "x")
    bf16, u8 = torch.bfloat16, torch.uint8
    shape_ = x.shape
    cols = shape_[-1]
    n = x.numel()
    rows = n // cols if cols else 0
    px, pw = _on(x, "x", bf16, dev), _on(weight, "weight", bf16, dev)
    if weight.numel() != cols:
        raise ValueError(f"weight needs {cols} elements, has {weight.numel()}")
    pr = None
    if residual is not None:
        pr = _on(residual, "residual", bf16, dev)
        if residual.shape != shape_ and (residual.numel() != n or residual.dim() == x.dim() or
                                         residual.dim() > 1 and residual.shape[-1] != cols):
            raise ValueError(f"residual must be {tuple(shape_)}, is {tuple(residual.shape)}")
    if not quant and (q is not None or s is not None):
        raise ValueError("q and s are not written with quant=False")

    with _allocating(stream):
        if sum_out is None:
            sum_out = torch.empty_like(x)
            psum = sum_out.data_ptr()
        else:
            psum = _sized(sum_out, "sum_out", bf16, n, dev)
        if y is None:
            y = torch.empty_like(x)
            py = y.data_ptr()
        else:
            py = _sized(y, "y", bf16, n, dev)
        pq = ps = None
        if quant:
            if q is None:
                q = torch.empty_like(x, dtype=u8)
                pq = q.data_ptr()
            else:
                pq = _sized(q, "q", u8, n, dev)
            if s is None:
                s = torch.empty(shape_[:-1] + (cols // 32,), dtype=u8, device=x.device)
                ps = s.data_ptr()
            else:
                ps = _sized(s, "s", u8, rows * (cols // 32), dev)
    rc = lib.moe_add_rmsnorm_mxfp8(rows, cols, px, pr, pw, eps, psum, py, pq, ps, _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_add_rmsnorm_mxfp8")
    return y, sum_out, q, s


class KvCache:
    """A paged key/value cache: k and v [pages, Hkv, page_size, D] in bf16, or u8 codes with u8 UE8M0 scales k_s and v_s
    [pages, Hkv, page_size, D/32]: E4M3, or E2M1 two to a byte, [pages, Hkv, page_size, D/2] (see include/moe.h).
    The scales tell which it is, one for 32 bytes or for 16; format, MOE_KV_*, refuses tensors of another one. Holds the
    tensors it is given."""

    def __init__(self, k, v, k_s=None, v_s=None, format: int | None = None):
        dev = _current(k, "k")
        mx = k_s is not None
        if k.dim() != 4 or v.shape != k.shape or (mx != (v_s is not None)):
            raise ValueError("k and v must be [pages, Hkv, page_size, D], with both scale tensors or none")
        pages, Hkv, page_size, D = k.shape
        # codes of 4 bits have a scale for 16 bytes, codes of 8 bits one for 32
        four = mx and k_s.dim() == 4 and k_s.shape[3] > 0 and D == 16 * k_s.shape[3]
        if four:
            D *= 2
        self.format = MOE_KV_MXFP4 if four else MOE_KV_MXFP8 if mx else MOE_KV_BF16
        if format is not None and format != self.format:
            raise ValueError(f"k, v and their scales are a cache of format {self.format}, not {format}")
        dtype = torch.uint8 if mx else torch.bfloat16
        ptrs = [_on(k, "k", dtype, dev), _on(v, "v", dtype, dev), None, None]
        if mx:
            for i, (t, name) in enumerate(((k_s, "k_s"), (v_s, "v_s"))):
                if tuple(t.shape) != (pages, Hkv, page_size, D // 32):
                    raise ValueError(f"{name} must be [pages, Hkv, page_size, D/32], is {tuple(t.shape)}")
                ptrs[2 + i] = _on(t, name, torch.uint8, dev)
        self.k, self.v, self.k_s, self.v_s, self.dev = k, v, k_s, v_s, dev
        self.pages, self.page_size, self.Hkv, self.D = pages, page_size, Hkv, D
        self.desc = MoeKvCache(pages, page_size, Hkv, D, self.format, *ptrs)
        self.ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, pages: int, page_size: int, Hkv: int, D: int, mxfp8: bool = False, device="cuda", mxfp4: bool = False):
        if mxfp8 and mxfp4:
            raise ValueError("a cache has one format: mxfp8 or mxfp4")
        shp = (pages, Hkv, page_size, D // 2 if mxfp4 else D)
        if not mxfp8 and not mxfp4:
            return cls(*(torch.zeros(shp, dtype=torch.bfloat16, device=device) for _ in range(2)))
        k, v = (torch.zeros(shp, dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, *(torch.zeros(*shp[:3], D // 32, dtype=torch.uint8, device=device) for _ in range(2)))


def moe_kv_append(cache: KvCache, k, v, slots, ws=None, stream=None) -> None:
    """Stores the bf16 rows k and v [T, Hkv, D] (rows may lie apart) at slots i32 [T] (page * page_size + place;
    -1 = not stored; the others must differ). ws: at least 256 bytes of uint8, zeros at first; one per stream is kept where
    it is not given (inside a graph's capture it has to be)."""
    dev = _current(k, "k")
    if cache.dev != dev:
        raise ValueError("cache and k must be on the same CUDA device")
    pk, sk = _rows_on(k, "k", cache.Hkv, cache.D, dev)
    pv, sv = _rows_on(v, "v", cache.Hkv, cache.D, dev)
    T = slots.numel()
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"k and v need {T} rows, have {k.shape[0]} and {v.shape[0]}")
    ps = _on(slots, "slots", torch.int32, dev)
    raw = _raw_stream(stream, dev)
    pws, nws = _workspace(256, k, stream, dev, raw) if ws is None else (_on(ws, "ws", torch.uint8, dev), ws.numel())
    rc = lib.moe_kv_append(cache.ref, T, pk, sk, pv, sv, ps, pws, nws, raw)
    if rc:
        _check(rc, "moe_kv_append")


class Rotary:
    """Rotary positions: the frequencies of a head's pairs (a tensor or a sequence of numbers, taken in 64 bits), which axis each
    turns by (`axis`, a sequence of indexes; all 0 where it is not given) of `axes` positions a token has, whether pairs are
    neighbours (2i, 2i + 1) or (i, i + dim/2), and a factor on cosines and sines (see include/moe.h). Holds its tables on
    `device`."""

    def __init__(self, inv_freq, axis=None, axes: int | None = None, interleaved: bool = False, factor: float = 1.0,
                 device="cuda"):
        freq = torch.as_tensor(inv_freq, dtype=torch.float64).cpu().contiguous()
        if freq.dim() != 1 or not len(freq):
            raise ValueError("inv_freq must be one frequency for every pair")
        n = len(freq)
        turns = torch.empty(n, dtype=torch.int64)
        _check(lib.moe_rotary_turns(n, freq.data_ptr(), turns.data_ptr()), "moe_rotary_turns")
        self.axis = None
        if axis is not None:
            which = torch.as_tensor(axis).cpu()
            if which.dim() != 1 or len(which) != n or which.is_floating_point():
                raise ValueError(f"axis needs {n} indexes, one for every pair")
            axes = int(which.max()) + 1 if axes is None else axes
            if int(which.min()) < 0 or int(which.max()) >= axes:
                raise ValueError(f"axis must hold indexes below {axes}")
            self.axis = which.to(torch.uint8).to(device)
        self.turns = turns.to(device)
        self.dim, self.axes, self.dev = 2 * n, 1 if axes is None else axes, self.turns.get_device()
        self.refs = [ctypes.byref(MoeRotary(2 * n, self.axes, bool(interleaved), back, factor, self.turns.data_ptr(),
                                            None if self.axis is None else self.axis.data_ptr())) for back in (0, 1)]


def _positions(rotary: Rotary, pos, T: int, dev: int) -> int:
    if rotary.dev != dev:
        raise ValueError(f"rotary must be on device {dev}")
    if pos.shape != (rotary.axes, T) and (rotary.axes > 1 or pos.shape != (T,)):
        raise ValueError(f"pos must be [{rotary.axes}, {T}], is {tuple(pos.shape)}")
    return _on(pos, "pos", torch.int32, dev)


def _tokens_on(t: torch.Tensor, name: str, T: int, heads: int, D: int, dev: int) -> tuple[int, int]:
    """As _rows_on, of so many rows."""
    at, stride = _rows_on(t, name, heads, D, dev)
    if t.shape[0] != T:
        raise ValueError(f"{name} needs {T} rows, has {t.shape[0]}")
    return at, stride


def _not_across(out: int, so: int, x: int, sx: int, n: int, name: str) -> None:
    """Rows are turned to rows of their own or where they are, not to the same place at another spacing."""
    if out == x and so != sx and n:
        raise ValueError(f"{name} must not overlap what is read, or be the same rows")


def moe_rope(rotary: Rotary, q, k, pos, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Turns q bf16 [T, Hq, D] and k bf16 [T, Hkv, D] (or None; rows may lie apart) by the positions pos i32 [T] or [axes, T].
    Returns (q_out, k_out), which may be q and k themselves (turned where they are). inverse: turns back, which is also
    the gradient: of q and k, from that of the results."""
    dev = _current(q, "q")
    T, Hq, D = q.shape
    pq, sq = _rows_on(q, "q", Hq, D, dev)
    Hkv, pk, sk, pko, sko = 0, None, 0, None, 0
    if k is not None:
        Hkv = k.shape[1]
        pk, sk = _tokens_on(k, "k", T, Hkv, D, dev)
    elif k_out is not None:
        raise ValueError("k_out is not written without k")
    pp = _positions(rotary, pos, T, dev)
    if q_out is None or (k_out is None and k is not None):
        with _allocating(stream):
            if q_out is None:
                q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
            if k_out is None and k is not None:
                k_out = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=q.device)
    pqo, sqo = _tokens_on(q_out, "q_out", T, Hq, D, dev)
    _not_across(pqo, sqo, pq, sq, T * Hq, "q_out")
    if k is not None:
        pko, sko = _tokens_on(k_out, "k_out", T, Hkv, D, dev)
        _not_across(pko, sko, pk, sk, T * Hkv, "k_out")
    rc = lib.moe_rope(rotary.refs[bool(inverse)], T, Hq, Hkv, D, pq, sq, pk, sk, pp, T, pqo, sqo, pko, sko,
                      _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_rope")
    return q_out, k_out


def moe_rope_kv_append(rotary: Rotary, cache: KvCache, q, k, v, pos, slots, q_out=None, k_out=None, ws=None, stream=None):
    """moe_kv_append of k and v [T, Hkv, D] with the keys turned on the way, and q [T, Hq, D] turned into q_out (which may be q
    itself); pos as for moe_rope, slots and ws as for moe_kv_append. Where k_out is given (k itself, or rows of its own), the
    turned keys go there too, for a prompt's own attention. Returns q_out."""
    dev = _current(q, "q")
    if cache.dev != dev:
        raise ValueError("cache and q must be on the same CUDA device")
    T, Hq, _ = q.shape
    Hkv, D = cache.Hkv, cache.D
    pq, sq = _rows_on(q, "q", Hq, D, dev)
    pk, sk = _tokens_on(k, "k", T, Hkv, D, dev)
    pv, sv = _tokens_on(v, "v", T, Hkv, D, dev)
    if slots.numel() != T:
        raise ValueError(f"slots needs {T} entries, has {slots.numel()}")
    pp = _positions(rotary, pos, T, dev)
    ps = _on(slots, "slots", torch.int32, dev)
    if q_out is None:
        with _allocating(stream):
            q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    pqo, sqo = _tokens_on(q_out, "q_out", T, Hq, D, dev)
    _not_across(pqo, sqo, pq, sq, T * Hq, "q_out")
    pko, sko = None, 0
    if k_out is not None:
        pko, sko = _tokens_on(k_out, "k_out", T, Hkv, D, dev)
        _not_across(pko, sko, pk, sk, T * Hkv, "k_out")
    raw = _raw_stream(stream, dev)
    pws, nws = _workspace(256, q, stream, dev, raw) if ws is None else (_on(ws, "ws", torch.uint8, dev), ws.numel())
    rc = lib.moe_rope_kv_append(rotary.refs[0], cache.ref, T, Hq, pq, sq, pk, sk, pv, sv, pp, T, ps, pqo, sqo, pko, sko,
                                pws, nws, raw)
    if rc:
        _check(rc, "moe_rope_kv_append")
    return q_out


def moe_paged_attention_workspace_bytes(B: int, rows: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    return _paged_bytes(_attention(B, Hq, Hkv, D, 0, 0, 1.0), rows, max_len)


def moe_paged_attention(q, cache: KvCache, block_table, seq_lens, max_len: int, scale: float | None = None,
                        window: int = 0, sinks: int = 0, out=None, ws=None, stream=None):
    """Attention of q bf16 [B, rows, Hq, D] (each sequence's newest rows) over the paged cache. block_table i32
    [B, width], seq_lens i32 [B] (the new rows counted), max_len >= every seq_len. Returns bf16 [B, rows, Hq, D]. ws:
    moe_paged_attention_workspace_bytes of uint8, zeros at first; one per stream is kept where it is not given (inside a
    graph's capture it has to be)."""
    dev = _current(q, "q")
    if cache.dev != dev:
        raise ValueError("cache and q must be on the same CUDA device")
    B, rows, Hq, D = q.shape
    width = block_table.shape[-1]
    if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError(f"block_table must be [{B}, width] and seq_lens [{B}]")
    if q.is_contiguous():
        pq, sq = _on(q, "q", torch.bfloat16, dev), Hq * D
    else:
        if rows > 1 and B > 1 and q.stride(0) != rows * q.stride(1):
            raise ValueError("q: rows must be evenly spaced")
        pq, sq = _rows_on(q[:, 0] if rows == 1 else q[0], "q", Hq, D, dev)
        if rows > 1 and B > 1:
            sq = q.stride(1)
    a = _attention(B, Hq, cache.Hkv, D, window, sinks, scale)
    if out is None:
        with _allocating(stream):
            out = torch.empty((B, rows, Hq, D), dtype=torch.bfloat16, device=q.device)
    pout = _sized(out, "out", torch.bfloat16, q.numel(), dev)
    raw = _raw_stream(stream, dev)
    if ws is None:
        pws, nws = _workspace(_paged_bytes(a, rows, max_len), q, stream, dev, raw)
    else:
        pws, nws = _on(ws, "ws", torch.uint8, dev), ws.numel()
    rc = lib.moe_paged_attention(a, cache.ref, rows, max_len, pq, sq, _on(block_table, "block_table", torch.int32, dev),
                                 width, _on(seq_lens, "seq_lens", torch.int32, dev),
                                 pout, pws, nws, raw)
    if rc:
        _check(rc, "moe_paged_attention")
    return out


def moe_prefill_attention(q, k, v, cu_q, cu_k=None, scale: float | None = None, window: int = 0, sinks: int = 0,
                          out=None, ws=None, stream=None):
    """Attention of packed prompts: q bf16 [Tq, Hq, D], k and v bf16 [Tk, Hkv, D] (rows may lie apart), cu_q and cu_k
    i32 [B + 1] the sequences' bounds (cu_k None: the same). Returns bf16 [Tq, Hq, D]; rows outside every sequence are
    left as they are in `out`. ws: as for moe_kv_append."""
    dev = _current(q, "q")
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    pq, sq = _rows_on(q, "q", Hq, D, dev)
    pk, sk = _rows_on(k, "k", Hkv, D, dev)
    pv, sv = _rows_on(v, "v", Hkv, D, dev)
    if v.shape[0] != Tk:
        raise ValueError(f"v needs {Tk} rows, has {v.shape[0]}")
    B = cu_q.numel() - 1
    if B < 0 or (cu_k is not None and cu_k.numel() != B + 1):
        raise ValueError("cu_q and cu_k need one entry more than there are sequences")
    if cu_k is None and Tq != Tk:
        raise ValueError("without cu_k, k and v need as many rows as q")
    if out is None:
        with _allocating(stream):
            out = torch.empty((Tq, Hq, D), dtype=torch.bfloat16, device=q.device)
    pout = _sized(out, "out", torch.bfloat16, q.numel(), dev)
    raw = _raw_stream(stream, dev)
    pws, nws = _workspace(256, q, stream, dev, raw) if ws is None else (_on(ws, "ws", torch.uint8, dev), ws.numel())
    rc = lib.moe_prefill_attention(
        _attention(B, Hq, Hkv, D, window, sinks, scale), Tq, Tk, pq, sq, pk, sk, pv, sv,
        _on(cu_q, "cu_q", torch.int32, dev), None if cu_k is None else _on(cu_k, "cu_k", torch.int32, dev),
        pout, pws, nws, raw)
    if rc:
        _check(rc, "moe_prefill_attention")
    return out


def moe_probe_mma_rate(iters: int, ws, mode: int = 0, stream=None) -> tuple[int, int]:
    """Launch the block-scaled MMA rate probe (time it with events on `stream`); returns
    (CTAs, FLOPs of the launch). mode: see include/moe.h (0 = the tensor-peak denominator)."""
    ctas = _I32(0)
    flops = ctypes.c_int64(0)
    _check(lib.moe_probe_mma_rate(int(iters), int(mode), ctypes.byref(ctas), ctypes.byref(flops), _ptr(ws),
                                  ws.numel(), _stream(stream)), "moe_probe_mma_rate")
    return int(ctas.value), int(flops.value)


def moe_selftest_timeout(ws, limit_ns: int, stream=None) -> None:
    _check(lib.moe_selftest_timeout(_ptr(ws), int(limit_ns), _stream(stream)), "moe_selftest_timeout")


def moe_selftest_attention_hold(load: int = -1) -> None:
    """Test hook: which load of every block never completes in the calls that follow (-1: none)."""
    _check(lib.moe_selftest_attention_hold(int(load)), "moe_selftest_attention_hold")


def moe_check_device_status(ws, stream=None) -> None:
    _check(lib.moe_check_device_status(_ptr(ws), _stream(stream)), "moe_check_device_status")


class MoeLayer:
    """One routed-expert layer with packed MXFP4 weights resident on the device."""

    def __init__(self, H, E, k, I, w_router, bias, w13p, w13sp, w2p, w2sp):
        self.H, self.E, self.k, self.I = H, E, k, I
        self.w_router, self.bias = w_router, bias
        self.w13p, self.w13sp, self.w2p, self.w2sp = w13p, w13sp, w2p, w2sp
        self._ws: dict[int, torch.Tensor] = {}

    @classmethod
    def from_fp32(cls, w_router, bias, w13, w2, k):
        """w13 fp32 [E, 2I, H], w2 fp32 [E, H, I] on the device -> quantise (MXFP4) and pack."""
        E, I2, H = w13.shape
        I = I2 // 2
        shp = shape(1, H, E, k, I)
        q13, s13 = moe_quant_mxfp4(w13)
        q2, s2 = moe_quant_mxfp4(w2)
        w13p, w13sp = moe_pack_w13(shp, q13, s13)
        w2p, w2sp = moe_pack_w2(shp, q2, s2)
        return cls(H, E, k, I, w_router, bias, w13p, w13sp, w2p, w2sp)

    def shape(self, T, flags=0) -> MoeShape:
        return shape(T, self.H, self.E, self.k, self.I, flags)

    def workspace(self, T) -> torch.Tensor:
        if T not in self._ws:
            self._ws[T] = alloc_workspace(self.shape(T), self.w_router.device)
        return self._ws[T]

    def forward(self, x, dead=None, out=None, inter=None, stream=None, anchor=None, shared=None, side_stream=None):
        T = x.shape[0]
        return moe_forward(self.shape(T), x, self.w_router, self.bias, dead, self.w13p, self.w13sp, self.w2p,
                           self.w2sp, self.workspace(T), out=out, inter=inter, stream=stream, anchor=anchor,
                           shared=shared, side_stream=side_stream)
