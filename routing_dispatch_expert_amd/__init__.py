"""Python binding of libmoe_hip.so, the MI355X (gfx950) MoE-layer hot path.

Thin ctypes marshalling over the C ABI in include/moe.h: every function below
has the C entry point's name and argument order, turns torch tensors (device
memory), ints and None into pointers and sizes, and raises MoeError on a
non-zero status. All computation happens in the HIP library; torch provides
device memory and streams only. There is no fallback: if the library is not
built, loading fails with an error that says so.

`forward()` is a convenience on top: it allocates outputs and the workspace
with torch and calls moe_layer_forward once.
"""
from __future__ import annotations

import ctypes
import functools
import os
from operator import index as _index

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_hip.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_Q4_U4, MOE_Q4_E2M1 = 0, 1
Q4_KINDS = {"u4": MOE_Q4_U4, "e2m1": MOE_Q4_E2M1}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
FEW_MAX_TOKENS = 64   # tokens of moe_layer_forward_few, rows of moe_q4_matvec
TOTALS = ("dropped", "fully_dropped_tokens", "padded_rows", "offrank_bytes")

EXPORTS = ("moe_capacity", "moe_workspace_size", "moe_layer_forward", "moe_backward_workspace_size",
           "moe_layer_backward", "moe_layer_backward_saved", "moe_replica_plan", "moe_replicated_workspace_size", "moe_layer_forward_replicated", "moe_router_workspace_size", "moe_router", "moe_route",
           "moe_permute_workspace_size", "moe_permute", "moe_permute_static", "moe_grouped_gemm_workspace_size",
           "moe_grouped_gemm", "moe_combine", "moe_q4_size", "moe_q4_quantize", "moe_q4_dequantize",
           "moe_q4_matvec_workspace_size", "moe_q4_matvec", "moe_few_workspace_size", "moe_layer_forward_few",
           "moe_layer_forward_few_q4", "moe_gate", "moe_gate_backward", "moe_layer_forward_routed", "moe_layer_backward_routed", "moe_mx8_size",
           "moe_mx8_quantize", "moe_mx8_dequantize", "moe_rmsnorm", "moe_rmsnorm_backward_workspace_size",
           "moe_rmsnorm_backward", "moe_experts_mx8_workspace_size", "moe_experts_mx8", "moe_set_stage_events", "moe_stage_ran", "moe_status_string", "moe_last_error")
STAGES = ("router", "route", "slots", "scatter", "gate_up", "down", "combine")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({detail})")


class moe_stats_t(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("slot", ctypes.c_void_p),
                ("src", ctypes.c_void_p), ("routed_count", ctypes.c_void_p),
                ("kept_count", ctypes.c_void_p), ("send_count", ctypes.c_void_p),
                ("totals", ctypes.c_void_p), ("buckets", ctypes.c_void_p), ("instance", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("u", ctypes.c_void_p), ("h", ctypes.c_void_p)]


_STATS = frozenset(name for name, _ in moe_stats_t._fields_)


class moe_q4_t(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("kind", ctypes.c_int32), ("group", ctypes.c_int32)]


class moe_gate_t(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class moe_mx8_t(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


_lib = None
_P, _I32, _I64, _F32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "moe_capacity": [_I64, _I32, _I32, _F32, _P],
    "moe_workspace_size": [_I64, _I64, _I64, _I32, _I32, _F32, _I32, ctypes.c_int, _P],
    "moe_layer_forward": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32, ctypes.c_int,
                          _P, ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_backward_workspace_size": [_I64, _I64, _I64, _I32, _I32, _F32, _I32, ctypes.c_int, _P],
    "moe_layer_backward": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32, ctypes.c_int,
                           _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_layer_backward_saved": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32,
                                 ctypes.c_int, ctypes.POINTER(moe_stats_t), _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_replica_plan": [_P, _I32, _I32, _P],
    "moe_replicated_workspace_size": [_I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32, ctypes.c_int, _P],
    "moe_layer_forward_replicated": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32, _P,
                                     _I32, ctypes.c_int, _P, ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_router_workspace_size": [_I64, _I64, _I32, ctypes.c_int, _P],
    "moe_router": [_P, _P, _P, _I64, _I64, _I32, _I32, _I32, _I32, ctypes.c_int, _P, _P, _P, _P, _SZ, _P],
    "moe_route": [_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P],
    "moe_permute_workspace_size": [_I64, _I32, _P],
    "moe_permute": [_P, _P, _I64, _I64, _I32, _I32, _I64, _I32, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P,
                    _P, _SZ, _P],
    "moe_permute_static": [_P, _P, _I64, _I64, _I32, _I32, _I64, _I32, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P,
                           _P],
    "moe_grouped_gemm_workspace_size": [_I32, _I64, _P],
    "moe_grouped_gemm": [_P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, ctypes.c_int, _P, _P, _P, _SZ, _P],
    "moe_combine": [_P, _P, _P, _P, _P, _I64, _I64, _I32, _I32, _I64, ctypes.c_int, _P, _P],
    "moe_q4_size": [_I32, _I64, _I64, _I32, _P, _P, _P],
    "moe_q4_quantize": [_P, _I32, _I64, _I64, ctypes.c_int, ctypes.POINTER(moe_q4_t), _P],
    "moe_q4_dequantize": [ctypes.POINTER(moe_q4_t), _I32, _I64, _I64, ctypes.c_int, _P, _P],
    "moe_q4_matvec_workspace_size": [_I32, _I64, ctypes.c_int, _P],
    "moe_q4_matvec": [_P, _P, ctypes.POINTER(moe_q4_t), _I32, _I32, _I64, _I64, ctypes.c_int, _P, _P, _SZ, _P],
    "moe_few_workspace_size": [_I64, _I64, _I64, _I32, _I32, _F32, _I32, ctypes.c_int, _I32, _P],
    "moe_layer_forward_few": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32, ctypes.c_int,
                              _P, ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_layer_forward_few_q4": [_P, _P, _P, ctypes.POINTER(moe_q4_t), ctypes.POINTER(moe_q4_t),
                                 ctypes.POINTER(moe_q4_t), _I64, _I64, _I64, _I32, _I32, _F32, _I32, _I32,
                                 ctypes.c_int, _P, ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_gate": [_P, _P, ctypes.POINTER(moe_gate_t), _I64, _I32, _I32, _P, _P, _P],
    "moe_gate_backward": [_P, _P, _P, _P, ctypes.POINTER(moe_gate_t), _I64, _I32, _I32, _P, _P],
    "moe_layer_forward_routed": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, ctypes.c_int, _P,
                                 ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_layer_backward_routed": [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _I32, _F32, _I32, ctypes.c_int,
                                  ctypes.POINTER(moe_stats_t), _P, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_mx8_size": [_I32, _I64, _I64, _P, _P],
    "moe_mx8_quantize": [_P, _I32, _I64, _I64, ctypes.c_int, ctypes.POINTER(moe_mx8_t), _P],
    "moe_mx8_dequantize": [ctypes.POINTER(moe_mx8_t), _I32, _I64, _I64, ctypes.c_int, _P, _P],
    "moe_rmsnorm": [_P, _P, _P, _F32, _I64, _I64, ctypes.c_int, _P, _P, ctypes.POINTER(moe_mx8_t), _P, _P],
    "moe_rmsnorm_backward_workspace_size": [_I64, _I64, ctypes.c_int, _P],
    "moe_rmsnorm_backward": [_P, _P, _P, _P, _P, _I64, _I64, ctypes.c_int, _P, _P, _P, _SZ, _P],
    "moe_experts_mx8_workspace_size": [_I64, _I64, _I64, _I32, _I32, _F32, ctypes.c_int, _P],
    "moe_experts_mx8": [ctypes.POINTER(moe_mx8_t), _P, _P, _P, ctypes.POINTER(moe_mx8_t), ctypes.POINTER(moe_mx8_t),
                        ctypes.POINTER(moe_mx8_t), _I64, _I64, _I64, _I32, _I32, _F32, ctypes.c_int, _P,
                        ctypes.POINTER(moe_stats_t), _P, _SZ, _P],
    "moe_set_stage_events": [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int],
    "moe_stage_ran": [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
}


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m routing_dispatch_expert_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_status_string(status: int) -> str:
    return status_string(status)


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where, moe_last_error())


def _ptr(a):
    """Device pointer of a torch tensor, an int address, or None (NULL)."""
    if a is None:
        return None
    if isinstance(a, int):
        return a or None
    return a.data_ptr() or None


@functools.lru_cache(maxsize=16)
def _dtype(dt) -> int:
    if isinstance(dt, int):
        return dt
    s = str(dt)
    if s in ("bf16", "torch.bfloat16"):
        return MOE_DTYPE_BF16
    if s in ("f32", "fp32", "torch.float32"):
        return MOE_DTYPE_F32
    raise ValueError(f"unsupported dtype {dt!r}")


def _stream(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


# ----------------------------------------------------------------- C entry points

def moe_capacity(T: int, E: int, k: int, cf: float) -> int:
    C = ctypes.c_int64(0)
    _check(lib().moe_capacity(T, E, k, cf, ctypes.byref(C)), "moe_capacity")
    return C.value


def moe_workspace_size(T, d, d_ff, E, k, cf, P, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(T, d, d_ff, E, k, cf, P, _dtype(dtype), ctypes.byref(n)),
           "moe_workspace_size")
    return n.value


def _stats(stats) -> "ctypes.POINTER(moe_stats_t) | None":
    if stats is None:
        return None
    s = moe_stats_t()
    for name, t in stats.items():
        if name in _STATS:
            setattr(s, name, _ptr(t))
    return ctypes.pointer(s)


def moe_layer_forward(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks,
                      dtype, out, stats, workspace, workspace_bytes, stream=None):
    """stats: None or a dict of moe_stats_t field name -> tensor (or None)."""
    _check(lib().moe_layer_forward(_ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
                                   _ptr(W_down), T, d, d_ff, E, k, cf, P, max_ranks, _dtype(dtype), _ptr(out),
                                   _stats(stats), _ptr(workspace), workspace_bytes, _stream(stream)),
           "moe_layer_forward")


def moe_backward_workspace_size(T, d, d_ff, E, k, cf, P, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_backward_workspace_size(T, d, d_ff, E, k, cf, P, _dtype(dtype), ctypes.byref(n)),
           "moe_backward_workspace_size")
    return n.value


def moe_layer_backward(x, W_router, router_bias, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P, max_ranks,
                       dtype, dx, dW_router, d_bias, dW_gate, dW_up, dW_down, workspace, workspace_bytes,
                       stream=None):
    _check(lib().moe_layer_backward(_ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
                                    _ptr(W_down), _ptr(dout), T, d, d_ff, E, k, cf, P, max_ranks, _dtype(dtype),
                                    _ptr(dx), _ptr(dW_router), _ptr(d_bias), _ptr(dW_gate), _ptr(dW_up),
                                    _ptr(dW_down), _ptr(workspace), workspace_bytes, _stream(stream)),
           "moe_layer_backward")


def moe_layer_backward_saved(x, W_router, router_bias, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P,
                             max_ranks, dtype, saved, dx, dW_router, d_bias, dW_gate, dW_up, dW_down, workspace,
                             workspace_bytes, stream=None):
    """saved: the stats dict of a moe_layer_forward call that kept g, u and h."""
    _check(lib().moe_layer_backward_saved(_ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
                                          _ptr(W_down), _ptr(dout), T, d, d_ff, E, k, cf, P, max_ranks,
                                          _dtype(dtype), _stats(saved), _ptr(dx), _ptr(dW_router), _ptr(d_bias),
                                          _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), _ptr(workspace),
                                          workspace_bytes, _stream(stream)),
           "moe_layer_backward_saved")


def moe_replica_plan(routed_count, extra):
    """Host-side replica counts (numpy int32 array of length E) from routed counts."""
    import numpy as np
    routed = np.ascontiguousarray(routed_count, dtype=np.int32)
    out = np.empty_like(routed)
    _check(lib().moe_replica_plan(routed.ctypes.data, routed.size, int(extra), out.ctypes.data), "moe_replica_plan")
    return out


def moe_replicated_workspace_size(T, d, d_ff, E, k, cf, P, R, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_replicated_workspace_size(T, d, d_ff, E, k, cf, P, R, _dtype(dtype), ctypes.byref(n)),
           "moe_replicated_workspace_size")
    return n.value


def moe_layer_forward_replicated(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks,
                                 replicas, R, dtype, out, stats, workspace, workspace_bytes, stream=None):
    _check(lib().moe_layer_forward_replicated(_ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
                                              _ptr(W_down), T, d, d_ff, E, k, cf, P, max_ranks, _ptr(replicas), R,
                                              _dtype(dtype), _ptr(out), _stats(stats), _ptr(workspace),
                                              workspace_bytes, _stream(stream)),
           "moe_layer_forward_replicated")


def moe_router_workspace_size(T, d, E, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_router_workspace_size(T, d, E, _dtype(dtype), ctypes.byref(n)), "moe_router_workspace_size")
    return n.value


def moe_router(x, W_router, router_bias, T, d, E, k, P, max_ranks, dtype, topk_idx, topk_w, logits_out,
               workspace, workspace_bytes, stream=None):
    _check(lib().moe_router(_ptr(x), _ptr(W_router), _ptr(router_bias), T, d, E, k, P, max_ranks, _dtype(dtype),
                            _ptr(topk_idx), _ptr(topk_w), _ptr(logits_out), _ptr(workspace),
                            workspace_bytes, _stream(stream)), "moe_router")


def moe_route(logits, T, E, k, P, max_ranks, topk_idx, topk_w, stream=None):
    _check(lib().moe_route(_ptr(logits), T, E, k, P, max_ranks, _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_route")


def moe_permute_workspace_size(T, E) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_permute_workspace_size(T, E, ctypes.byref(n)), "moe_permute_workspace_size")
    return n.value


def moe_permute(x, topk_idx, T, d, E, k, C, P, dtype, buckets, slot, src, routed_count, kept_count,
                send_count, totals, workspace, workspace_bytes, stream=None):
    _check(lib().moe_permute(_ptr(x), _ptr(topk_idx), T, d, E, k, C, P, _dtype(dtype), _ptr(buckets),
                             _ptr(slot), _ptr(src), _ptr(routed_count), _ptr(kept_count),
                             _ptr(send_count), _ptr(totals), _ptr(workspace), workspace_bytes,
                             _stream(stream)), "moe_permute")


def moe_permute_static(x, topk_idx, T, d, E, k, C, P, dtype, buckets, slot, src, routed_count, kept_count,
                       send_count, totals, stream=None):
    _check(lib().moe_permute_static(_ptr(x), _ptr(topk_idx), T, d, E, k, C, P, _dtype(dtype), _ptr(buckets),
                                    _ptr(slot), _ptr(src), _ptr(routed_count), _ptr(kept_count),
                                    _ptr(send_count), _ptr(totals), _stream(stream)), "moe_permute_static")


def moe_grouped_gemm_workspace_size(E, C) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_grouped_gemm_workspace_size(E, C, ctypes.byref(n)), "moe_grouped_gemm_workspace_size")
    return n.value


def moe_grouped_gemm(buckets, kept_count, W_gate, W_up, W_down, E, C, d, d_ff, dtype, h, y, workspace,
                     workspace_bytes, stream=None):
    _check(lib().moe_grouped_gemm(_ptr(buckets), _ptr(kept_count), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                  E, C, d, d_ff, _dtype(dtype), _ptr(h), _ptr(y), _ptr(workspace),
                                  workspace_bytes, _stream(stream)), "moe_grouped_gemm")


def moe_combine(x, y, topk_idx, topk_w, slot, T, d, E, k, C, dtype, out, stream=None):
    _check(lib().moe_combine(_ptr(x), _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(slot), T, d, E, k, C,
                             _dtype(dtype), _ptr(out), _stream(stream)), "moe_combine")


def moe_q4_size(E, N, K, group) -> tuple[int, int, int]:
    """Bytes of a 4-bit matrix stack's codes, scales and (where kept) zero points."""
    a, b, c = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_q4_size(E, N, K, group, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), "moe_q4_size")
    return a.value, b.value, c.value


def _q4(q) -> "ctypes.POINTER(moe_q4_t) | None":
    """q: None, a Q4Weights, or (codes, scale, zero, kind, group)."""
    if q is None:
        return None
    if isinstance(q, Q4Weights):
        return ctypes.pointer(moe_q4_t(_ptr(q._codes), _ptr(q._scale), _ptr(q._zero), Q4_KINDS[q._kind], q._group))
    codes, scale, zero, kind, group = q
    return ctypes.pointer(moe_q4_t(_ptr(codes), _ptr(scale), _ptr(zero), Q4_KINDS.get(kind, kind), group))


def moe_q4_quantize(W, E, N, K, dtype, q, stream=None):
    _check(lib().moe_q4_quantize(_ptr(W), E, N, K, _dtype(dtype), _q4(q), _stream(stream)), "moe_q4_quantize")


def moe_q4_dequantize(q, E, N, K, dtype, W, stream=None):
    _check(lib().moe_q4_dequantize(_q4(q), E, N, K, _dtype(dtype), _ptr(W), _stream(stream)), "moe_q4_dequantize")


def moe_q4_matvec_workspace_size(R, K, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_q4_matvec_workspace_size(R, K, _dtype(dtype), ctypes.byref(n)), "moe_q4_matvec_workspace_size")
    return n.value


def moe_q4_matvec(x, expert, W, R, E, N, K, dtype, out, workspace, workspace_bytes, stream=None):
    _check(lib().moe_q4_matvec(_ptr(x), _ptr(expert), _q4(W), R, E, N, K, _dtype(dtype), _ptr(out), _ptr(workspace),
                               workspace_bytes, _stream(stream)), "moe_q4_matvec")


def moe_few_workspace_size(T, d, d_ff, E, k, cf, P, dtype, q4) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_few_workspace_size(T, d, d_ff, E, k, cf, P, _dtype(dtype), q4, ctypes.byref(n)),
           "moe_few_workspace_size")
    return n.value


def moe_layer_forward_few(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks, dtype,
                          out, stats, workspace, workspace_bytes, stream=None):
    _check(lib().moe_layer_forward_few(_ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(W_gate), _ptr(W_up),
                                       _ptr(W_down), T, d, d_ff, E, k, cf, P, max_ranks, _dtype(dtype), _ptr(out),
                                       _stats(stats), _ptr(workspace), workspace_bytes, _stream(stream)),
           "moe_layer_forward_few")


def moe_layer_forward_few_q4(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks,
                             dtype, out, stats, workspace, workspace_bytes, stream=None):
    """W_gate, W_up, W_down: as for _q4 (a Q4Weights each)."""
    _check(lib().moe_layer_forward_few_q4(_ptr(x), _ptr(W_router), _ptr(router_bias), _q4(W_gate), _q4(W_up),
                                          _q4(W_down), T, d, d_ff, E, k, cf, P, max_ranks, _dtype(dtype), _ptr(out),
                                          _stats(stats), _ptr(workspace), workspace_bytes, _stream(stream)),
           "moe_layer_forward_few_q4")


@functools.lru_cache(maxsize=64)
def _gate_struct(score, groups, top_groups, group_best, renormalize, scale):
    return ctypes.pointer(moe_gate_t(score, groups, top_groups, group_best, renormalize, scale))


def _gate(gate) -> "ctypes.POINTER(moe_gate_t) | None":
    """gate: None or (score, groups, top_groups, group_best, renormalize, scale). The
    struct is remembered by plain numbers: a tensor is the same key whatever it holds."""
    if gate is None:
        return None
    score, groups, top_groups, group_best, renormalize, scale = gate
    return _gate_struct(SCORES.get(score, score), _index(groups), _index(top_groups), _index(group_best), int(renormalize),
                        float(scale))


def moe_gate(logits, bias, gate, T, E, k, topk_idx, topk_w, stream=None):
    _check(lib().moe_gate(_ptr(logits), _ptr(bias), _gate(gate), T, E, k, _ptr(topk_idx), _ptr(topk_w),
                          _stream(stream)), "moe_gate")


def moe_gate_backward(logits, topk_idx, d_topk_w, d_scores, gate, T, E, k, dlogits, stream=None):
    _check(lib().moe_gate_backward(_ptr(logits), _ptr(topk_idx), _ptr(d_topk_w), _ptr(d_scores), _gate(gate), T, E, k,
                                   _ptr(dlogits), _stream(stream)), "moe_gate_backward")


def moe_layer_forward_routed(x, residual, topk_idx, topk_w, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, dtype, out,
                             stats, workspace, workspace_bytes, stream=None):
    _check(lib().moe_layer_forward_routed(_ptr(x), _ptr(residual), _ptr(topk_idx), _ptr(topk_w), _ptr(W_gate), _ptr(W_up),
                                          _ptr(W_down), T, d, d_ff, E, k, cf, P, _dtype(dtype), _ptr(out), _stats(stats),
                                          _ptr(workspace), workspace_bytes, _stream(stream)), "moe_layer_forward_routed")


def moe_layer_backward_routed(x, topk_idx, topk_w, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P, dtype, saved, dx,
                              d_topk_w, dW_gate, dW_up, dW_down, workspace, workspace_bytes, stream=None):
    """saved: None, or the stats dict of a moe_layer_forward_routed call that kept buckets, g, u and h."""
    _check(lib().moe_layer_backward_routed(_ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                           _ptr(dout), T, d, d_ff, E, k, cf, P, _dtype(dtype), _stats(saved), _ptr(dx),
                                           _ptr(d_topk_w), _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), _ptr(workspace),
                                           workspace_bytes, _stream(stream)), "moe_layer_backward_routed")


def moe_mx8_size(E, N, K) -> tuple[int, int]:
    """Bytes of an 8-bit matrix stack's codes and scales."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_mx8_size(E, N, K, ctypes.byref(a), ctypes.byref(b)), "moe_mx8_size")
    return a.value, b.value


def _mx8(q):
    """q: None, an Mx8, or (codes, scale)."""
    if q is None:
        return None
    codes, scale = (q._codes, q._scale) if isinstance(q, Mx8) else q
    return ctypes.byref(moe_mx8_t(_ptr(codes), _ptr(scale)))


def moe_mx8_quantize(W, E, N, K, dtype, q, stream=None):
    _check(lib().moe_mx8_quantize(_ptr(W), E, N, K, _dtype(dtype), _mx8(q), _stream(stream)), "moe_mx8_quantize")


def moe_mx8_dequantize(q, E, N, K, dtype, W, stream=None):
    _check(lib().moe_mx8_dequantize(_mx8(q), E, N, K, _dtype(dtype), _ptr(W), _stream(stream)), "moe_mx8_dequantize")


def moe_rmsnorm(x, residual, weight, eps, R, d, dtype, h_out, y, y8, rstd, stream=None):
    _check(lib().moe_rmsnorm(_ptr(x), _ptr(residual), _ptr(weight), eps, R, d, _dtype(dtype), _ptr(h_out), _ptr(y),
                             _mx8(y8), _ptr(rstd), _stream(stream)), "moe_rmsnorm")


def moe_rmsnorm_backward_workspace_size(R, d, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_rmsnorm_backward_workspace_size(R, d, _dtype(dtype), ctypes.byref(n)),
           "moe_rmsnorm_backward_workspace_size")
    return n.value


def moe_rmsnorm_backward(dy, h, weight, rstd, dh_in, R, d, dtype, dh, dweight, workspace, workspace_bytes, stream=None):
    _check(lib().moe_rmsnorm_backward(_ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd), _ptr(dh_in), R, d, _dtype(dtype),
                                      _ptr(dh), _ptr(dweight), _ptr(workspace), workspace_bytes, _stream(stream)),
           "moe_rmsnorm_backward")


def moe_experts_mx8_workspace_size(T, d, d_ff, E, k, cf, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_experts_mx8_workspace_size(T, d, d_ff, E, k, cf, _dtype(dtype), ctypes.byref(n)),
           "moe_experts_mx8_workspace_size")
    return n.value


def moe_experts_mx8(x, residual, topk_idx, topk_w, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, dtype, out, stats,
                    workspace, workspace_bytes, stream=None):
    """x, W_gate, W_up, W_down: as for _mx8 (an Mx8 each)."""
    _check(lib().moe_experts_mx8(_mx8(x), _ptr(residual), _ptr(topk_idx), _ptr(topk_w), _mx8(W_gate), _mx8(W_up),
                                 _mx8(W_down), T, d, d_ff, E, k, cf, _dtype(dtype), _ptr(out), _stats(stats),
                                 _ptr(workspace), workspace_bytes, _stream(stream)), "moe_experts_mx8")


def moe_set_stage_events(events):
    """events: None (off) or 2 * len(STAGES) raw hipEvent_t handles (ints)."""
    if events is None:
        _check(lib().moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*events)
    _check(lib().moe_set_stage_events(arr, len(events)), "moe_set_stage_events")


def moe_stage_ran(stage: int) -> bool:
    """Whether the last layer call with stage events recorded this stage's events."""
    ran = ctypes.c_int32(0)
    _check(lib().moe_stage_ran(stage, ctypes.byref(ran)), "moe_stage_ran")
    return bool(ran.value)


# ----------------------------------------------------------------- convenience

def _require(t, name, torch_dtype, shape):
    if t.device.type != "cuda" or not t.is_contiguous() or t.dtype != torch_dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name}: need a contiguous {torch_dtype} cuda tensor of shape {shape}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def forward(x, W_router, W_gate, W_up, W_down, k, cf, P=1, router_bias=None, stream=None,
            want_buckets=False, want_src=False, workspace=None, max_ranks=0, keep_activations=False):
    """Run the layer once on torch device tensors; returns a dict of outputs.

    x [T, d]; W_router [E, d]; W_gate, W_up [E, d_ff, d]; W_down [E, d, d_ff]
    (bf16 or fp32, all the same dtype); router_bias [E] fp32 or None;
    max_ranks > 0 limits each token's experts to that many of the P ranks.
    keep_activations: also return the buckets and g, u, h [E, C, d_ff], the
    state backward(..., saved=result) takes instead of recomputing it.
    """
    import torch
    T, d = x.shape
    E = W_router.shape[0]
    d_ff = W_gate.shape[1]
    dt = x.dtype
    for t, n, s in ((x, "x", (T, d)), (W_router, "W_router", (E, d)), (W_gate, "W_gate", (E, d_ff, d)),
                    (W_up, "W_up", (E, d_ff, d)), (W_down, "W_down", (E, d, d_ff))):
        _require(t, n, dt, s)
    if router_bias is not None:
        _require(router_bias, "router_bias", torch.float32, (E,))
    C = moe_capacity(T, E, k, cf)
    dev = x.device
    i32 = dict(dtype=torch.int32, device=dev)
    res = {
        "C": C,
        "out": torch.empty_like(x),
        "topk_idx": torch.empty((T, k), **i32),
        "topk_w": torch.empty((T, k), dtype=torch.float32, device=dev),
        "slot": torch.empty((T, k), **i32),
        "routed_count": torch.empty(E, **i32),
        "kept_count": torch.empty(E, **i32),
        "send_count": torch.empty(P, **i32),
        "totals": torch.empty(4, dtype=torch.int64, device=dev),
    }
    if want_buckets or keep_activations:
        res["buckets"] = torch.empty((E, C, d), dtype=dt, device=dev)
    if want_src:
        res["src"] = torch.empty((E, C), **i32)
    if keep_activations:
        for name in ("g", "u", "h"):
            res[name] = torch.empty((E, C, d_ff), dtype=dt, device=dev)
    nbytes = moe_workspace_size(T, d, d_ff, E, k, cf, P, dt)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    moe_layer_forward(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks, dt,
                      res["out"], res, workspace, nbytes, stream)
    res["workspace"] = workspace
    return res


def backward(x, W_router, W_gate, W_up, W_down, dout, k, cf, P=1, router_bias=None, stream=None, max_ranks=0,
             workspace=None, want_d_bias=False, saved=None):
    """Gradients of the layer for dout on torch device tensors; returns a dict
    dx, dW_router, d_bias (fp32, when router_bias is given or want_d_bias),
    dW_gate, dW_up, dW_down, workspace. saved: the result of
    forward(..., keep_activations=True) on the same inputs, whose routing,
    buckets and activations are then used instead of being recomputed."""
    import torch
    T, d = x.shape
    E = W_router.shape[0]
    d_ff = W_gate.shape[1]
    dt = x.dtype
    for t, n, s in ((x, "x", (T, d)), (dout, "dout", (T, d)), (W_router, "W_router", (E, d)),
                    (W_gate, "W_gate", (E, d_ff, d)), (W_up, "W_up", (E, d_ff, d)), (W_down, "W_down", (E, d, d_ff))):
        _require(t, n, dt, s)
    if router_bias is not None:
        _require(router_bias, "router_bias", torch.float32, (E,))
    res = {"dx": torch.empty_like(x), "dW_router": torch.empty_like(W_router), "dW_gate": torch.empty_like(W_gate),
           "dW_up": torch.empty_like(W_up), "dW_down": torch.empty_like(W_down),
           "d_bias": (torch.empty(E, dtype=torch.float32, device=x.device)
                      if router_bias is not None or want_d_bias else None)}
    nbytes = moe_backward_workspace_size(T, d, d_ff, E, k, cf, P, dt)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    if saved is None:
        moe_layer_backward(x, W_router, router_bias, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P, max_ranks,
                           dt, res["dx"], res["dW_router"], res["d_bias"], res["dW_gate"], res["dW_up"],
                           res["dW_down"], workspace, nbytes, stream)
    else:
        moe_layer_backward_saved(x, W_router, router_bias, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P,
                                 max_ranks, dt, saved, res["dx"], res["dW_router"], res["d_bias"], res["dW_gate"],
                                 res["dW_up"], res["dW_down"], workspace, nbytes, stream)
    res["workspace"] = workspace
    return res


def forward_replicated(x, W_router, W_gate, W_up, W_down, k, cf, replicas, P=1, router_bias=None, stream=None,
                       want_buckets=False, want_src=False, workspace=None, max_ranks=0):
    """The layer with replicated experts; replicas is an int32 cuda tensor [E]
    (each >= 1). Returns a dict like forward(), with per-instance kept_count,
    src and buckets, and the instance of each copy."""
    import torch
    T, d = x.shape
    E = W_router.shape[0]
    d_ff = W_gate.shape[1]
    dt = x.dtype
    _require(replicas, "replicas", torch.int32, (E,))
    R = int(replicas.sum().item())
    C = moe_capacity(T, E, k, cf)
    dev = x.device
    i32 = dict(dtype=torch.int32, device=dev)
    res = {"C": C, "R": R, "out": torch.empty_like(x), "topk_idx": torch.empty((T, k), **i32),
           "topk_w": torch.empty((T, k), dtype=torch.float32, device=dev), "slot": torch.empty((T, k), **i32),
           "instance": torch.empty((T, k), **i32), "routed_count": torch.empty(E, **i32),
           "kept_count": torch.empty(R, **i32), "send_count": torch.empty(P, **i32),
           "totals": torch.empty(4, dtype=torch.int64, device=dev)}
    if want_buckets:
        res["buckets"] = torch.empty((R, C, d), dtype=dt, device=dev)
    if want_src:
        res["src"] = torch.empty((R, C), **i32)
    nbytes = moe_replicated_workspace_size(T, d, d_ff, E, k, cf, P, R, dt)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    moe_layer_forward_replicated(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks,
                                 replicas, R, dt, res["out"], res, workspace, nbytes, stream)
    res["workspace"] = workspace
    return res


# ---------------------------------------------------- few tokens, 4-bit weights

class Q4Weights:
    """A 4-bit matrix stack [E, N, K] (the layout of moe_q4_t in moe.h): codes
    uint8 [E, ceil(N/16), ceil(K/128), 1024], scale bfloat16 and zero uint8 (or
    None) [E, ceil(N/16), ceil(K/128) 128/group, 16]; kind "u4" or "e2m1". Made
    by quantize_q4(), or from a checkpoint laid out so. The tensors are kept
    and read in place: codes, scale and zero give views of them, whose values
    may be changed, but they are not exchanged for others (other tensors make
    another Q4Weights). Can be copied (copy.deepcopy) and pickled (torch.save)."""

    def __init__(self, codes, scale, zero, shape, group, kind):
        import torch
        E, N, K = (int(v) for v in shape)
        if kind not in Q4_KINDS:
            raise ValueError(f"kind: need one of {sorted(Q4_KINDS)}, got {kind!r}")
        moe_q4_size(E, N, K, group)   # checks the sizes
        nt, kt = -(-N // 16), -(-K // 128)
        _require(codes, "codes", torch.uint8, (E, nt, kt, 1024))
        _require(scale, "scale", torch.bfloat16, (E, nt, kt * (128 // group), 16))
        if zero is not None:
            _require(zero, "zero", torch.uint8, tuple(scale.shape))
            if kind == "e2m1":
                raise ValueError("zero: e2m1 codes take none")
        for t in (codes, scale, zero):
            if t is not None and t.device != codes.device:
                raise ValueError("codes, scale and zero must be on one device")
        # views: what becomes of the caller's tensor objects (x.data = ...) does not touch what was checked here
        self._set(codes.detach(), scale.detach(), None if zero is None else zero.detach(), (E, N, K), int(group), kind)

    def _set(self, codes, scale, zero, shape, group, kind):
        self._codes, self._scale, self._zero = codes, scale, zero
        self._shape, self._group, self._kind = shape, group, kind

    codes = property(lambda self: self._codes.detach())
    scale = property(lambda self: self._scale.detach())
    zero = property(lambda self: None if self._zero is None else self._zero.detach())
    shape = property(lambda self: self._shape)
    group = property(lambda self: self._group)
    kind = property(lambda self: self._kind)

    @property
    def device(self):
        return self._codes.device


class _On:
    """The device and stream of a call on `device`: the given stream, or
    torch's current one of that device. On another stream than torch's current
    one the call's tensors are marked as used there, so that torch does not hand
    their memory on before the call is done, and new ones come from that stream's
    own memory (the current stream's free blocks may still be in use by work
    that waits on it), marked as used on the current one. (The caller sees to it
    that the inputs are ready on that stream, and the results on the current one.)"""

    def __init__(self, device, stream):
        import torch
        self.torch, self.device = torch, device
        self.guard = torch.cuda.device(device) if torch.cuda.current_device() != device.index else None
        self.other = None
        self.current = torch.cuda.current_stream(device)
        if stream is None:
            stream = self.current
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device)
            elif stream.device != device:   # its kernels would run there, on memory that is not theirs
                raise ValueError(f"stream: need a stream of {device}, got one of {stream.device}")
            if stream.cuda_stream != self.current.cuda_stream:
                self.other = stream
        self.stream = stream

    def __enter__(self):
        if self.guard:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard:
            self.guard.__exit__(*exc)

    def empty(self, shape, dtype):
        if self.other is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.other):
            t = self.torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(self.current)
        return t

    def zero(self, t):
        with self.torch.cuda.stream(self.stream):
            t.zero_()

    def lent(self, t):
        if self.other is not None and t is not None:
            of = ((t._codes, t._scale, t._zero) if isinstance(t, Q4Weights) else
                  (t._codes, t._scale) if isinstance(t, Mx8) else (t,))
            for v in of:
                if v is not None:
                    v.record_stream(self.other)
        return t


class _Here:
    """_On for the usual call: on torch's current device and current stream, whose
    address is all that is needed. (Making torch's stream and device objects
    takes longer than a small kernel's launch.)"""
    other = None

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        pass

    def empty(self, shape, dtype):
        import torch
        return torch.empty(shape, dtype=dtype, device=self.device)

    def lent(self, t):
        return t

    def zero(self, t):
        t.zero_()


def _on(device, stream):
    """The device and stream of a call on tensors of `device`."""
    import torch
    if stream is None and device.index == torch._C._cuda_getDevice():
        return _Here(device, torch._C._cuda_getCurrentRawStream(device.index))
    return _On(device, stream)


def _same_device(device, names, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            name = names.split()[[v is t for v in tensors].index(True)]
            raise ValueError(f"{name}: need a tensor on {device}, got {t.device}")


def quantize_q4(W, group=128, kind="u4", zero_points=True, stream=None):
    """W [E, N, K] (bf16 or fp32) in 4 bits: a Q4Weights. kind "u4" keeps a zero
    point a group (zero_points) or is symmetric; "e2m1" has none. Runs on
    torch's current stream unless one is given."""
    import torch
    if W.dim() != 3:
        raise ValueError(f"W: need [E, N, K], got {tuple(W.shape)}")
    E, N, K = W.shape
    _require(W, "W", W.dtype, (E, N, K))
    dt = _dtype(W.dtype)
    if kind not in Q4_KINDS:
        raise ValueError(f"kind: need one of {sorted(Q4_KINDS)}, got {kind!r}")
    moe_q4_size(E, N, K, group)   # checks the sizes
    nt, kt = -(-N // 16), -(-K // 128)
    with _On(W.device, stream) as on:
        groups = (E, nt, kt * (128 // group), 16)
        q = Q4Weights.__new__(Q4Weights)   # of tensors that need no checks
        q._set(on.empty((E, nt, kt, 1024), torch.uint8), on.empty(groups, torch.bfloat16),
               on.empty(groups, torch.uint8) if kind == "u4" and zero_points else None, (E, N, K), int(group), kind)
        moe_q4_quantize(on.lent(W), E, N, K, dt, q, on.stream)
    return q


def dequantize_q4(q, dtype, stream=None):
    """The weights that a Q4Weights stands for, rounded to dtype: [E, N, K]."""
    import torch
    dt = _dtype(dtype)
    with _On(q.device, stream) as on:
        W = on.empty(q.shape, torch.bfloat16 if dt == MOE_DTYPE_BF16 else torch.float32)
        moe_q4_dequantize(on.lent(q), *q.shape, dt, W, on.stream)
    return W


def matvec_q4(x, W, expert=None, out=None, workspace=None, stream=None):
    """out[r] = W[expert[r]] x[r] for up to 64 rows x [R, K] and a Q4Weights W
    [E, N, K]; expert int32 [R], or None for matrix 0. Rows whose expert is
    outside [0, E) are left as they are in `out` (zero if it is not given).
    Returns a dict out, workspace, which may be passed in again (a workspace
    that is too small is replaced)."""
    import torch
    E, N, K = W.shape
    R = x.shape[0]
    dt = _dtype(x.dtype)
    _require(x, "x", x.dtype, (R, K))
    if expert is not None:
        _require(expert, "expert", torch.int32, (R,))
    dev = x.device
    _same_device(dev, "W expert out workspace", W, expert, out, workspace)
    if workspace is not None and not workspace.is_contiguous():   # its memory may be less than its size
        raise ValueError("workspace: need a contiguous tensor")
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((R, N), x.dtype)
            if expert is not None:
                with torch.cuda.stream(on.stream):
                    out.zero_()
        else:
            _require(out, "out", x.dtype, (R, N))
            on.lent(out)
        nbytes = 0 if dt == MOE_DTYPE_BF16 else moe_q4_matvec_workspace_size(R, K, dt)
        if workspace is None or workspace.nbytes < nbytes:
            workspace = on.empty(max(nbytes, 1), torch.uint8)
        else:
            on.lent(workspace)
        if on.other is not None:
            for t in (x, expert, W):
                on.lent(t)
        moe_q4_matvec(x, expert, W, R, E, N, K, dt, out, workspace, nbytes, on.stream)
    return {"out": out, "workspace": workspace}


class FewResult(dict):
    """What forward_few returns. Passed to a later call as `out` it lends that
    call the outputs and workspace that it was made with, and shows them again
    whatever became of its entries meanwhile."""


def forward_few(x, W_router, W_gate, W_up, W_down, k, cf, P=1, router_bias=None, stream=None, max_ranks=0, out=None):
    """The layer for up to 64 tokens, as forward(), reading each chosen expert's
    weights once for every 16 (or 32: moe.h) of its copies; W_gate, W_up and
    W_down are tensors of x's dtype or, all three, Q4Weights. Returns a dict as
    forward() does, without buckets or activations. out: the result of an
    earlier call with the same sizes, whose tensors this call writes instead of
    allocating new ones. Runs on torch's current stream unless one is given (a
    stream of x's device or its address, which outlives the call's tensors)."""
    import torch
    T, d = x.shape
    E = W_router.shape[0]
    q4 = isinstance(W_gate, Q4Weights)
    if any(isinstance(w, Q4Weights) != q4 for w in (W_up, W_down)):
        raise ValueError("W_gate, W_up, W_down: either all tensors or all Q4Weights")
    d_ff = W_gate.shape[1]
    dt, dev = x.dtype, x.device
    dtype = _dtype(dt)
    _require(x, "x", dt, (T, d))
    _require(W_router, "W_router", dt, (E, d))
    for w, n, s in ((W_gate, "W_gate", (E, d_ff, d)), (W_up, "W_up", (E, d_ff, d)), (W_down, "W_down", (E, d, d_ff))):
        if not q4:
            _require(w, n, dt, s)
        elif w.shape != s:
            raise ValueError(f"{n}: need 4-bit weights of shape {s}, got {w.shape}")
    if router_bias is not None:
        _require(router_bias, "router_bias", torch.float32, (E,))
    _same_device(dev, "W_router W_gate W_up W_down router_bias", W_router, W_gate, W_up, W_down, router_bias)
    k, cf, P = _index(k), float(cf), _index(P)   # as they are now: the key is held until a later call
    with _On(dev, stream) as on:
        key = (T, d, d_ff, E, k, cf, P, dt, q4, dev)
        if out is None:
            nbytes = moe_few_workspace_size(T, d, d_ff, E, k, cf, P, dtype, int(q4))
            i32 = torch.int32
            res = FewResult(C=moe_capacity(T, E, k, cf), out=on.empty((T, d), dt), topk_idx=on.empty((T, k), i32),
                            topk_w=on.empty((T, k), torch.float32), slot=on.empty((T, k), i32),
                            routed_count=on.empty(E, i32), kept_count=on.empty(E, i32), send_count=on.empty(P, i32),
                            totals=on.empty(4, torch.int64), workspace=on.empty(max(nbytes, 1), torch.uint8))
            if T == 0:   # nothing will be launched: the counts of no tokens
                with torch.cuda.stream(on.stream):
                    for name in ("routed_count", "kept_count", "send_count", "totals"):
                        res[name].zero_()
            # what a later call may write: held here, so that it stays valid whatever becomes of the dict's entries
            res._bound = (key, nbytes, dict(res))
        else:
            res = out
            if not isinstance(res, FewResult) or res._bound[0] != key:
                raise ValueError("out: need the result of a forward_few call with the same sizes, types and device")
            res.update(res._bound[2])   # entries that were replaced or removed are this call's outputs again
            for t in res._bound[2].values():
                if isinstance(t, torch.Tensor):
                    on.lent(t)
        if on.other is not None:
            for t in (x, W_router, router_bias, W_gate, W_up, W_down):
                on.lent(t)
        _, nbytes, t = res._bound
        call = moe_layer_forward_few_q4 if q4 else moe_layer_forward_few
        call(x, W_router, router_bias, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, max_ranks, dtype, t["out"], t,
             t["workspace"], nbytes, on.stream)
    return res


# ---------------------------------------------------- the gate

def _need(t, name, dtype, shape):
    """_require, for calls that take a few microseconds in all."""
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        _require(t, name, dtype, shape)

def _gate_rule(score, groups, top_groups, group_best, renormalize, scale):
    if score not in SCORES:
        raise ValueError(f"score: need one of {sorted(SCORES)}, got {score!r}")
    return score, groups, top_groups or groups, group_best, bool(renormalize), scale


def _lent_result(out, key, what):
    """The tensors of an earlier call's result, if it was of the same sizes."""
    if not isinstance(out, Result) or out._bound[0] != key:
        raise ValueError(f"out: need the result of a call of {what} with the same sizes, types and device")
    out.update(out._bound[1])   # entries that were replaced or removed are this call's outputs again
    return out


class Result(dict):
    """What gate, rmsnorm, experts_mx8, forward_mx8, forward_routed and their like return.
    Passed to a later call as `out` it lends that call the outputs and workspace
    that it was made with, and shows them again whatever became of its entries."""

    @classmethod
    def of(cls, key, **entries):
        res = cls(entries)
        res._bound = (key, dict(res))
        return res


def gate(logits, k, score="softmax", bias=None, groups=1, top_groups=0, group_best=1, renormalize=True, scale=1.0,
         out=None, stream=None):
    """The choice of k experts a token and their weights from logits [T, E] (fp32).

    score: "softmax" (over all experts) or "sigmoid". bias [E] fp32 or None is
    added to the scores for the choice only. groups > 1: the experts come from the
    top_groups (0: all) groups with the best sums of their group_best (1 or 2)
    largest scores. topk_w is scale * score, divided by the chosen scores' sum
    where renormalize. Ties go to the lower index (moe.h has the formulas).
    Returns a dict topk_idx int32 [T, k], topk_w fp32 [T, k]. out: the result of
    an earlier call with the same sizes, whose tensors this call writes. Runs on
    torch's current stream unless one is given."""
    import torch
    if logits.dim() != 2:
        raise ValueError(f"logits: need [T, E], got {tuple(logits.shape)}")
    T, E = logits.shape
    _need(logits, "logits", torch.float32, (T, E))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    rule = _gate_rule(score, groups, top_groups, group_best, renormalize, scale)
    dev = logits.device
    _same_device(dev, "bias", bias)
    k = _index(k)   # as it is now: the key is held until a later call
    key = ("gate", T, E, k, dev)
    with _on(dev, stream) as on:
        if out is None:
            res = Result.of(key, topk_idx=on.empty((T, k), torch.int32), topk_w=on.empty((T, k), torch.float32))
        else:
            res = _lent_result(out, key, "gate")
        if on.other is not None:
            for t in (*res._bound[1].values(), logits, bias):
                on.lent(t)
        t = res._bound[1]
        moe_gate(logits, bias, rule, T, E, k, t["topk_idx"], t["topk_w"], on.stream)
    return res


def gate_backward(logits, topk_idx, d_topk_w, score="softmax", renormalize=True, scale=1.0, d_scores=None, out=None,
                  stream=None):
    """The logits' gradient [T, E] of gate()'s weights' gradient d_topk_w [T, k] for
    the experts topk_idx that it chose and, optionally, of the scores' gradient
    d_scores [T, E] (a balance loss's); score, renormalize and scale as for gate().
    Written into `out` if it is given."""
    import torch
    if logits.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("logits, topk_idx: need [T, E] and [T, k]")
    T, E = logits.shape
    k = topk_idx.shape[1]
    _need(logits, "logits", torch.float32, (T, E))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(d_topk_w, "d_topk_w", torch.float32, (T, k))
    if d_scores is not None:
        _need(d_scores, "d_scores", torch.float32, (T, E))
    rule = _gate_rule(score, 1, 1, 1, renormalize, scale)
    dev = logits.device
    _same_device(dev, "topk_idx d_topk_w d_scores out", topk_idx, d_topk_w, d_scores, out)
    with _on(dev, stream) as on:
        if out is None:
            out = on.empty((T, E), torch.float32)
        else:
            _need(out, "out", torch.float32, (T, E))
            on.lent(out)
        if on.other is not None:
            for t in (logits, topk_idx, d_topk_w, d_scores):
                on.lent(t)
        moe_gate_backward(logits, topk_idx, d_topk_w, d_scores, rule, T, E, k, out, on.stream)
    return out


def _routed_shapes(x, topk_idx, topk_w, W_gate, W_up, W_down, others):
    import torch
    if x.dim() != 2 or topk_idx.dim() != 2 or W_gate.dim() != 3:
        raise ValueError("x, topk_idx, W_gate: need [T, d], [T, k] and [E, d_ff, d]")
    T, d = x.shape
    E, d_ff = W_gate.shape[:2]
    k = topk_idx.shape[1]
    dt = x.dtype
    for t, n, s in ((x, "x", (T, d)), (W_gate, "W_gate", (E, d_ff, d)), (W_up, "W_up", (E, d_ff, d)),
                    (W_down, "W_down", (E, d, d_ff)), *((t, n, (T, d)) for n, t in others.items())):
        _need(t, n, dt, s)
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_w, "topk_w", torch.float32, (T, k))
    _same_device(x.device, "topk_idx topk_w W_gate W_up W_down " + " ".join(others), topk_idx, topk_w, W_gate, W_up, W_down,
                 *others.values())
    return T, d, d_ff, E, k


def forward_routed(x, topk_idx, topk_w, W_gate, W_up, W_down, cf, residual=None, P=1, keep_activations=False, out=None,
                   stream=None):
    """The layer (bf16 or fp32) with a given routing, gate()'s or any other, and the
    residual of a transformer block: out = residual + the experts' outputs for x
    (residual None: x). Returns a dict out, slot [T, k], routed_count, kept_count,
    send_count [P], totals, workspace; with keep_activations also buckets and g, u, h,
    which backward_routed(..., saved=result) takes instead of recomputing them. out:
    the result of an earlier call with the same sizes, whose tensors this call writes."""
    import torch
    cf, P = float(cf), _index(P)   # as they are now: the key is held until a later call
    if residual is None:
        residual = x
    T, d, d_ff, E, k = _routed_shapes(x, topk_idx, topk_w, W_gate, W_up, W_down, {"residual": residual})
    dt, dev = x.dtype, x.device
    key = ("forward_routed", T, d, d_ff, E, k, cf, P, dt, dev, bool(keep_activations))
    with _on(dev, stream) as on:
        if out is None:
            nbytes, C, i32 = moe_workspace_size(T, d, d_ff, E, k, cf, P, dt), moe_capacity(T, E, k, cf), torch.int32
            kept = dict(buckets=on.empty((E, C, d), dt), **{n: on.empty((E, C, d_ff), dt) for n in "guh"}) if keep_activations else {}
            res = Result.of(key, C=C, out=on.empty((T, d), dt), slot=on.empty((T, k), i32), routed_count=on.empty((E,), i32),
                            kept_count=on.empty((E,), i32), send_count=on.empty((P,), i32), totals=on.empty((4,), torch.int64),
                            workspace=on.empty((max(nbytes, 1),), torch.uint8), **kept)
            if T == 0:   # nothing will be launched: the counts of no tokens
                for name in ("routed_count", "kept_count", "send_count", "totals"):
                    on.zero(res[name])
        else:
            res = _lent_result(out, key, "forward_routed")
        t = res._bound[1]
        if on.other is not None:
            for v in (*t.values(), x, topk_idx, topk_w, W_gate, W_up, W_down, residual):
                if not isinstance(v, int):
                    on.lent(v)
        if T:
            moe_layer_forward_routed(x, residual, topk_idx, topk_w, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, P, dt,
                                     t["out"], t, t["workspace"], t["workspace"].numel(), on.stream)
    return res


def backward_routed(x, topk_idx, topk_w, W_gate, W_up, W_down, dout, cf, P=1, saved=None, out=None, stream=None):
    """Gradients of forward_routed() for dout [T, d]: a dict dx (of the experts' path
    alone: residual's gradient is dout itself), d_topk_w fp32 [T, k] (for
    gate_backward()), dW_gate, dW_up, dW_down, workspace. saved: the result of
    forward_routed(..., keep_activations=True) on the same inputs. out: the result of
    an earlier call with the same sizes, whose tensors this call writes."""
    import torch
    cf, P = float(cf), _index(P)
    T, d, d_ff, E, k = _routed_shapes(x, topk_idx, topk_w, W_gate, W_up, W_down, {"dout": dout})
    dt, dev = x.dtype, x.device
    if saved is not None and (not isinstance(saved, Result) or
                              saved._bound[0] != ("forward_routed", T, d, d_ff, E, k, cf, P, dt, dev, True)):
        raise ValueError("saved: need the result of forward_routed(..., keep_activations=True) with the same sizes")
    key = ("backward_routed", T, d, d_ff, E, k, cf, P, dt, dev)
    with _on(dev, stream) as on:
        if out is None:
            nbytes = moe_backward_workspace_size(T, d, d_ff, E, k, cf, P, dt)
            res = Result.of(key, dx=on.empty((T, d), dt), d_topk_w=on.empty((T, k), torch.float32),
                            dW_gate=on.empty((E, d_ff, d), dt), dW_up=on.empty((E, d_ff, d), dt),
                            dW_down=on.empty((E, d, d_ff), dt), workspace=on.empty((max(nbytes, 1),), torch.uint8))
        else:
            res = _lent_result(out, key, "backward_routed")
        t, state = res._bound[1], None if saved is None else saved._bound[1]
        if on.other is not None:
            for v in (*t.values(), *(state or {}).values(), x, topk_idx, topk_w, W_gate, W_up, W_down, dout):
                if not isinstance(v, int):
                    on.lent(v)
        if T:
            moe_layer_backward_routed(x, topk_idx, topk_w, W_gate, W_up, W_down, dout, T, d, d_ff, E, k, cf, P, dt,
                                      state and {n: state[n] for n in ("buckets", "g", "u", "h")}, t["dx"], t["d_topk_w"],
                                      t["dW_gate"], t["dW_up"], t["dW_down"], t["workspace"], t["workspace"].numel(), on.stream)
        else:   # nothing will be launched: the gradients of no tokens
            for name in ("dW_gate", "dW_up", "dW_down"):
                on.zero(t[name])
    return res


# ---------------------------------------------------- 8-bit matrices, the norm

class Mx8:
    """8-bit matrices [E, N, K] or rows [R, K] (the layout of moe_mx8_t in moe.h):
    codes float8_e4m3fn of that shape, scale uint8 [E, ceil(K/128), N, 4] or
    [ceil(K/128), R, 4]. Made by quantize_mx8() or rmsnorm(), or from tensors laid
    out so, which are kept and read in place; codes and scale give views of them,
    whose values may be changed. Can be copied (copy.deepcopy) and pickled."""

    def __init__(self, codes, scale):
        import torch
        if codes.dim() not in (2, 3):
            raise ValueError(f"codes: need [E, N, K] or [R, K], got {tuple(codes.shape)}")
        lead, (N, K) = tuple(codes.shape[:-2]), codes.shape[-2:]
        moe_mx8_size(*lead or (1,), N, K)   # checks the sizes
        _need(codes, "codes", torch.float8_e4m3fn, tuple(codes.shape))
        _need(scale, "scale", torch.uint8, (*lead, -(-K // 128), N, 4))
        if scale.device != codes.device:
            raise ValueError("codes and scale must be on one device")
        self._set(codes.detach(), scale.detach())

    def _set(self, codes, scale):
        self._codes, self._scale, self._shape = codes, scale, tuple(codes.shape)

    @classmethod
    def _empty(cls, on, shape):
        """One of new memory; the sizes are checked where it is filled."""
        import torch
        q = cls.__new__(cls)
        q._set(on.empty(shape, torch.float8_e4m3fn), on.empty((*shape[:-2], -(-shape[-1] // 128), shape[-2], 4), torch.uint8))
        return q

    codes = property(lambda self: self._codes.detach())
    scale = property(lambda self: self._scale.detach())
    shape = property(lambda self: self._shape)

    @property
    def device(self):
        return self._codes.device


def quantize_mx8(W, stream=None):
    """W [E, N, K] or [R, K] (bf16 or fp32; K a multiple of 16) in 8 bits: an Mx8.
    Runs on torch's current stream unless one is given."""
    if W.dim() not in (2, 3):
        raise ValueError(f"W: need [E, N, K] or [R, K], got {tuple(W.shape)}")
    shape = tuple(W.shape)
    _need(W, "W", W.dtype, shape)
    dt = _dtype(W.dtype)
    E, N, K = shape if len(shape) == 3 else (1, *shape)
    with _on(W.device, stream) as on:   # the call checks the sizes
        q = Mx8._empty(on, shape)
        moe_mx8_quantize(on.lent(W), E, N, K, dt, q, on.stream)
    return q


def dequantize_mx8(q, dtype, stream=None):
    """The values that an Mx8 stands for, rounded to dtype, in its shape."""
    import torch
    dt = _dtype(dtype)
    E, N, K = q.shape if len(q.shape) == 3 else (1, *q.shape)
    with _on(q.device, stream) as on:
        W = on.empty(q.shape, torch.bfloat16 if dt == MOE_DTYPE_BF16 else torch.float32)
        moe_mx8_dequantize(on.lent(q), E, N, K, dt, W, on.stream)
    return W


def rmsnorm(x, weight, eps=1e-6, residual=None, want_y=True, mx8=False, out=None, stream=None):
    """The norm in front of the layer for rows x [R, d] (bf16 or fp32):
    h = x + residual (x itself without one), y = h / sqrt(mean(h^2) + eps) weight.

    Returns a dict h (x without a residual), y (unless want_y is false), y8 (an
    Mx8, with mx8) and rstd fp32 [R], which rmsnorm_backward takes. out: the result
    of an earlier call with the same sizes and outputs, whose tensors this call
    writes. Runs on torch's current stream unless one is given."""
    import torch
    if x.dim() != 2:
        raise ValueError(f"x: need [R, d], got {tuple(x.shape)}")
    R, d = x.shape
    dt, dev = x.dtype, x.device
    dtype = _dtype(dt)
    _need(x, "x", dt, (R, d))
    _need(weight, "weight", dt, (d,))
    if residual is not None:
        _need(residual, "residual", dt, (R, d))
    if mx8 and out is None:
        moe_mx8_size(1, R, d)   # checks the sizes
    _same_device(dev, "weight residual", weight, residual)
    key = ("rmsnorm", R, d, dt, dev, residual is not None, bool(want_y), bool(mx8))
    with _on(dev, stream) as on:
        if out is None:
            res = Result.of(key, h=on.empty((R, d), dt) if residual is not None else None,
                            y=on.empty((R, d), dt) if want_y else None, y8=Mx8._empty(on, (R, d)) if mx8 else None,
                            rstd=on.empty((R,), torch.float32))
        else:
            res = _lent_result(out, key, "rmsnorm")
        if on.other is not None:
            for t in (*res._bound[1].values(), x, weight, residual):
                on.lent(t)
        t = res._bound[1]
        moe_rmsnorm(x, residual, weight, eps, R, d, dtype, t["h"], t["y"], t["y8"], t["rstd"], on.stream)
    if residual is None:
        res["h"] = x
    return res


def rmsnorm_backward(dy, h, weight, rstd, dh=None, out=None, stream=None):
    """Gradient of rmsnorm(): of dy [R, d] for y and, if given, dh [R, d] that
    arrives at h otherwise. Returns a dict dh (the gradient of x and of residual
    both), dweight, workspace. out: the result of an earlier call with the same
    sizes, whose tensors this call writes."""
    import torch
    if dy.dim() != 2:
        raise ValueError(f"dy: need [R, d], got {tuple(dy.shape)}")
    R, d = dy.shape
    dt, dev = dy.dtype, dy.device
    dtype = _dtype(dt)
    for t, n, s in ((dy, "dy", (R, d)), (h, "h", (R, d)), (weight, "weight", (d,)), (dh, "dh", (R, d))):
        if t is not None:
            _need(t, n, dt, s)
    _need(rstd, "rstd", torch.float32, (R,))
    _same_device(dev, "h weight rstd dh", h, weight, rstd, dh)
    key = ("rmsnorm_backward", R, d, dt, dev)
    with _on(dev, stream) as on:
        if out is None:
            nbytes = moe_rmsnorm_backward_workspace_size(R, d, dtype)
            res = Result.of(key, dh=on.empty((R, d), dt), dweight=on.empty((d,), dt),
                            workspace=on.empty((max(nbytes, 1),), torch.uint8))
        else:
            res = _lent_result(out, key, "rmsnorm_backward")
        if on.other is not None:
            for t in (*res._bound[1].values(), dy, h, weight, rstd, dh):
                on.lent(t)
        t = res._bound[1]
        moe_rmsnorm_backward(dy, h, weight, rstd, dh, R, d, dtype, t["dh"], t["dweight"], t["workspace"],
                             t["workspace"].numel(), on.stream)
    return res


def experts_mx8(x, topk_idx, topk_w, W_gate, W_up, W_down, residual, cf, out=None, stream=None):
    """The experts from a given routing, with 8-bit rows x [T, d] and weights W_gate,
    W_up [E, d_ff, d] and W_down [E, d, d_ff] (an Mx8 each), added to residual
    [T, d] (bf16 or fp32): topk_idx int32 and topk_w fp32 [T, k] as gate() or the
    layer's router return them; cf = E / k drops nothing. Returns a dict out [T, d],
    slot [T, k], routed_count, kept_count [E], workspace. out: the result of an
    earlier call with the same sizes, whose tensors this call writes. Runs on
    torch's current stream unless one is given."""
    import torch
    for q, n, dims in ((x, "x", 2), (W_gate, "W_gate", 3), (W_up, "W_up", 3), (W_down, "W_down", 3)):
        if not isinstance(q, Mx8) or len(q.shape) != dims:
            raise ValueError(f"{n}: need an Mx8 of {dims} dimensions")
    T, d = x.shape
    E, d_ff = W_gate.shape[:2]
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx: need [T, k], got {tuple(topk_idx.shape)}")
    k = topk_idx.shape[1]
    for q, n, s in ((W_gate, "W_gate", (E, d_ff, d)), (W_up, "W_up", (E, d_ff, d)), (W_down, "W_down", (E, d, d_ff))):
        if q.shape != s:
            raise ValueError(f"{n}: need 8-bit weights of shape {s}, got {q.shape}")
    cf = float(cf)   # as it is now: the key is held until a later call
    dt, dev = residual.dtype, x.device
    dtype = _dtype(dt)
    _need(residual, "residual", dt, (T, d))
    _need(topk_idx, "topk_idx", torch.int32, (T, k))
    _need(topk_w, "topk_w", torch.float32, (T, k))
    _same_device(dev, "topk_idx topk_w W_gate W_up W_down residual", topk_idx, topk_w, W_gate, W_up, W_down, residual)
    key = ("experts_mx8", T, d, d_ff, E, k, cf, dt, dev)
    with _on(dev, stream) as on:
        if out is None:
            nbytes = moe_experts_mx8_workspace_size(T, d, d_ff, E, k, cf, dtype)
            i32 = torch.int32
            res = Result.of(key, out=on.empty((T, d), dt), slot=on.empty((T, k), i32), routed_count=on.empty((E,), i32),
                            kept_count=on.empty((E,), i32), workspace=on.empty((max(nbytes, 1),), torch.uint8))
            if T == 0:   # nothing will be launched: the counts of no tokens
                for name in ("routed_count", "kept_count"):
                    on.zero(res[name])
        else:
            res = _lent_result(out, key, "experts_mx8")
        if on.other is not None:
            for t in (*res._bound[1].values(), x, topk_idx, topk_w, W_gate, W_up, W_down, residual):
                on.lent(t)
        t = res._bound[1]
        stats = {"slot": t["slot"], "routed_count": t["routed_count"], "kept_count": t["kept_count"]}
        moe_experts_mx8(x, residual, topk_idx, topk_w, W_gate, W_up, W_down, T, d, d_ff, E, k, cf, dtype, t["out"], stats,
                        t["workspace"], t["workspace"].numel(), on.stream)
    return res


def forward_mx8(x, norm_weight, W_router, W_gate, W_up, W_down, k, cf, residual=None, eps=1e-6, score="softmax", bias=None,
                groups=1, top_groups=0, group_best=1, renormalize=True, scale=1.0, out=None, stream=None):
    """The layer as it stands in a transformer block, with 8-bit experts, for rows
    x [T, d] (bf16 or fp32):
      h = x + residual;  y = rmsnorm(h) norm_weight, also in 8 bits
      topk_idx, topk_w = gate(y W_router^T)        (score .. scale as for gate())
      out = h + the experts' outputs for the 8-bit y (as experts_mx8())
    W_router [E, d] and norm_weight [d] of x's dtype, W_gate, W_up, W_down an Mx8
    each. Returns a dict out, h (x without a residual), y, logits, topk_idx, topk_w,
    slot, routed_count, kept_count. out: the result of an earlier call with the same
    sizes, whose tensors and workspaces this call writes. Runs on torch's current
    stream unless one is given."""
    import torch
    for q, n in ((W_gate, "W_gate"), (W_up, "W_up"), (W_down, "W_down")):
        if not isinstance(q, Mx8) or len(q.shape) != 3:
            raise ValueError(f"{n}: need an Mx8 of 3 dimensions")
    if x.dim() != 2:
        raise ValueError(f"x: need [T, d], got {tuple(x.shape)}")
    T, d = x.shape
    E, d_ff = W_gate.shape[:2]
    dt, dev = x.dtype, x.device
    dtype = _dtype(dt)
    for q, n, s in ((W_gate, "W_gate", (E, d_ff, d)), (W_up, "W_up", (E, d_ff, d)), (W_down, "W_down", (E, d, d_ff))):
        if q.shape != s:
            raise ValueError(f"{n}: need 8-bit weights of shape {s}, got {q.shape}")
    _need(x, "x", dt, (T, d))
    _need(norm_weight, "norm_weight", dt, (d,))
    _need(W_router, "W_router", dt, (E, d))
    if residual is not None:
        _need(residual, "residual", dt, (T, d))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    rule = _gate_rule(score, groups, top_groups, group_best, renormalize, scale)
    _same_device(dev, "norm_weight W_router W_gate W_up W_down residual bias", norm_weight, W_router, W_gate, W_up, W_down,
                 residual, bias)
    k, cf = _index(k), float(cf)   # as they are now: the key is held until a later call
    key = ("forward_mx8", T, d, d_ff, E, k, cf, dt, dev, residual is not None)
    with _on(dev, stream) as on:
        if out is None:
            nbytes = moe_experts_mx8_workspace_size(T, d, d_ff, E, k, cf, dtype)
            rbytes = moe_router_workspace_size(T, d, E, dtype)
            i32, f32, u8 = torch.int32, torch.float32, torch.uint8
            res = Result.of(key, out=on.empty((T, d), dt), h=on.empty((T, d), dt) if residual is not None else None,
                            y=on.empty((T, d), dt), y8=Mx8._empty(on, (T, d)), logits=on.empty((T, E), f32),
                            top=on.empty((2, max(T, 1)), i32), topk_idx=on.empty((T, k), i32), topk_w=on.empty((T, k), f32),
                            slot=on.empty((T, k), i32), routed_count=on.empty((E,), i32), kept_count=on.empty((E,), i32),
                            router_workspace=on.empty((max(rbytes, 1),), u8), workspace=on.empty((max(nbytes, 1),), u8))
            if T == 0:   # nothing will be launched: the counts of no tokens
                for name in ("routed_count", "kept_count"):
                    on.zero(res[name])
        else:
            res = _lent_result(out, key, "forward_mx8")
        t = res._bound[1]
        if on.other is not None:
            for v in (*t.values(), x, norm_weight, W_router, W_gate, W_up, W_down, residual, bias):
                on.lent(v)
        h = x if residual is None else t["h"]
        moe_rmsnorm(x, residual, norm_weight, eps, T, d, dtype, t["h"], t["y"], t["y8"], None, on.stream)
        if T:   # the scores, with one best expert a token that nothing reads
            moe_router(t["y"], W_router, None, T, d, E, 1, 1, 0, dtype, t["top"][0], t["top"][1], t["logits"],
                       t["router_workspace"], t["router_workspace"].numel(), on.stream)
        moe_gate(t["logits"], bias, rule, T, E, k, t["topk_idx"], t["topk_w"], on.stream)
        stats = {"slot": t["slot"], "routed_count": t["routed_count"], "kept_count": t["kept_count"]}
        moe_experts_mx8(t["y8"], h, t["topk_idx"], t["topk_w"], W_gate, W_up, W_down, T, d, d_ff, E, k, cf, dtype, t["out"],
                        stats, t["workspace"], t["workspace"].numel(), on.stream)
    res["h"] = h
    return res
