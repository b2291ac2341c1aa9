"""Thin ctypes binding of ``include/strata_window.h``.

Argument marshalling only: the functions keep the C names
(``strata_window_create``, ``strata_moe_window_forward``, ``strata_window_sync``,
``strata_window_query``, ``strata_window_destroy``, ``strata_status_str``) and
every step of a window runs in the library's CUDA kernels.  Loading fails
loudly when the shared library has not been built; there is no fallback.

``Window`` wraps a handle for torch tensors (device memory and streams come
from PyTorch; nothing is computed by it).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libstrata_window.so")

STRATA_OK, STRATA_EINVAL, STRATA_ENOMEM, STRATA_ECUDA, STRATA_EUNSUPPORTED, STRATA_EDEVICE = range(6)

EXPORTED = ("strata_window_create", "strata_moe_window_forward", "strata_window_sync", "strata_window_query",
            "strata_window_set_profiling", "strata_window_timings", "strata_window_destroy", "strata_status_str",
            "strata_moe_window_forward_noalloc", "strata_moe_window_forward_graph", "strata_stack_create", "strata_stack_forward", "strata_stack_sync",
            "strata_stack_query", "strata_stack_set_profiling", "strata_stack_timings", "strata_stack_destroy",
            "strata_window_plan", "strata_tier_create", "strata_window_set_tier", "strata_tier_read",
            "strata_tier_destroy", "strata_head_create", "strata_head_forward", "strata_head_sync",
            "strata_head_query", "strata_head_set_profiling", "strata_head_timings", "strata_head_destroy",
            "strata_window_slots", "strata_stack_set_kv", "strata_stack_forward_kv", "strata_qknorm_create",
            "strata_qknorm_forward", "strata_qknorm_destroy", "strata_kv8_create", "strata_kv8_append",
            "strata_kv8_read", "strata_kv8_attend", "strata_kv8_sync", "strata_kv8_query", "strata_kv8_destroy",
            "strata_linear_create", "strata_linear_forward", "strata_linear_round_weights", "strata_linear_sync",
            "strata_linear_query", "strata_linear_destroy", "strata_sort_create", "strata_sort_route", "strata_sort_plan",
            "strata_sort_gather", "strata_sort_combine", "strata_sort_combine_backward", "strata_sort_destroy",
            "strata_blocknorm_create", "strata_blocknorm_forward", "strata_blocknorm_destroy")
STRATA_F32, STRATA_F16, STRATA_BF16 = range(3)
STRATA_KV8_E4M3, STRATA_KV8_INT8 = range(2)
STRATA_GATE_NONE, STRATA_GATE_CHANNEL, STRATA_GATE_ROW, STRATA_GATE_ELEMENT = range(4)
NOALLOC_SCRATCH_BYTES = 4 << 20


class StrataError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} ({status})")
        self.status = status


class strata_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("min", ctypes.c_void_p)]


class strata_moe_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "n_experts", "top_k", "ffn", "shared_ffn", "bits", "block",
                                              "max_rows", "renorm_topk")]


class strata_moe_weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_b", ctypes.c_void_p), ("gate", strata_qmat),
                ("up", strata_qmat), ("down", strata_qmat), ("shared_gate", strata_qmat),
                ("shared_up", strata_qmat), ("shared_down", strata_qmat)]


class strata_routing_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "counts", "offsets", "entries", "distinct",
                                               "n_distinct")]


class strata_window_info(ctypes.Structure):
    _fields_ = [("n_sm", ctypes.c_int32), ("stages", ctypes.c_int32), ("stage_bytes", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("packed_bytes", ctypes.c_int64),
                ("expert_bytes", ctypes.c_int64), ("shared_bytes", ctypes.c_int64), ("router_bytes", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64)]


class strata_attn_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "kv_heads", "head_dim")]


class strata_attn_weights(ctypes.Structure):
    _fields_ = [("q", strata_qmat), ("k", strata_qmat), ("v", strata_qmat), ("o", strata_qmat)]


class strata_stack_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "topk_idx", "topk_w", "n_distinct")]


class strata_stack_info(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_sm", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("stage_bytes", ctypes.c_int32), ("smem_bytes", ctypes.c_int32), ("dense_bytes", ctypes.c_int64),
                ("expert_bytes", ctypes.c_int64), ("shared_bytes", ctypes.c_int64), ("router_bytes", ctypes.c_int64)]


class strata_tier_desc(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("capacity", ctypes.c_int32), ("adapt_every", ctypes.c_int32),
                ("adapt_swaps", ctypes.c_int32), ("decay", ctypes.c_float), ("min_gain", ctypes.c_float)]


class strata_tier_stats(ctypes.Structure):
    _fields_ = [("windows", ctypes.c_int64), ("rounds", ctypes.c_int64), ("n_swaps", ctypes.c_int32)]


class strata_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_slots", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32)]


class strata_head_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "vocab", "bits", "block", "max_rows")]


class strata_draw_in(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("position", "seed", "temperature", "fed")]


class strata_draw_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens", "n_emit", "logits")]


class strata_qknorm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "kv_heads", "head_dim", "rotary_dim", "interleaved", "norm")] + \
        [("eps", ctypes.c_float)]


class strata_kv8_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "n_slots", "heads", "kv_heads", "head_dim", "max_ctx",
                                              "block", "format")]


class strata_kv8_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp")]


class strata_kv8_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seq", "n_rows", "max_rows")] + \
        [(n, ctypes.c_void_p) for n in ("row_start", "slot", "length")]


class strata_linear_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "in", "out", "bits", "block", "max_rows")]


class strata_sort_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_experts", "top_k", "renorm_topk")]


class strata_sort_order(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("counts", "offsets", "entries", "place")]


class strata_blocknorm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "after", "before", "gate", "sigmoid")] + \
        [(n, ctypes.c_float) for n in ("eps", "residual_scale", "block_scale")]


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with slot_decode_window_gb300.build.build() "
                           "(the window step has no non-CUDA implementation)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.strata_window_create.argtypes = [P(strata_moe_desc), P(strata_moe_weights), ctypes.c_void_p,
                                         P(ctypes.c_void_p)]
    lib.strata_window_create.restype = ctypes.c_int
    lib.strata_moe_window_forward.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                              P(strata_routing_out), ctypes.c_void_p]
    lib.strata_moe_window_forward.restype = ctypes.c_int
    lib.strata_moe_window_forward_graph.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                                    ctypes.c_void_p, ctypes.c_void_p]
    lib.strata_moe_window_forward_graph.restype = ctypes.c_int
    lib.strata_moe_window_forward_noalloc.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                                      ctypes.c_void_p, ctypes.c_void_p]
    lib.strata_moe_window_forward_noalloc.restype = ctypes.c_int
    lib.strata_stack_create.argtypes = [ctypes.c_int32, P(strata_moe_desc), P(strata_attn_desc),
                                        P(strata_moe_weights), P(strata_attn_weights), ctypes.c_void_p,
                                        P(ctypes.c_void_p)]
    lib.strata_stack_create.restype = ctypes.c_int
    lib.strata_stack_forward.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                         P(strata_stack_out), ctypes.c_void_p]
    lib.strata_stack_forward.restype = ctypes.c_int
    lib.strata_stack_sync.argtypes = [ctypes.c_void_p]
    lib.strata_stack_sync.restype = ctypes.c_int
    lib.strata_stack_query.argtypes = [ctypes.c_void_p, P(strata_stack_info)]
    lib.strata_stack_query.restype = ctypes.c_int
    lib.strata_stack_set_profiling.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.strata_stack_set_profiling.restype = ctypes.c_int
    lib.strata_stack_timings.argtypes = [ctypes.c_void_p, P(ctypes.c_float)]
    lib.strata_stack_timings.restype = ctypes.c_int
    lib.strata_stack_destroy.argtypes = [ctypes.c_void_p]
    lib.strata_stack_destroy.restype = ctypes.c_int
    lib.strata_window_sync.argtypes = [ctypes.c_void_p]
    lib.strata_window_sync.restype = ctypes.c_int
    lib.strata_window_query.argtypes = [ctypes.c_void_p, P(strata_window_info)]
    lib.strata_window_query.restype = ctypes.c_int
    lib.strata_window_plan.argtypes = [P(strata_moe_desc), ctypes.c_int32, P(strata_window_info)]
    lib.strata_window_plan.restype = ctypes.c_int
    lib.strata_window_set_profiling.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.strata_window_set_profiling.restype = ctypes.c_int
    lib.strata_window_timings.argtypes = [ctypes.c_void_p, P(ctypes.c_float)]
    lib.strata_window_timings.restype = ctypes.c_int
    lib.strata_window_destroy.argtypes = [ctypes.c_void_p]
    lib.strata_window_destroy.restype = ctypes.c_int
    lib.strata_tier_create.argtypes = [P(strata_tier_desc), ctypes.c_void_p, P(ctypes.c_void_p)]
    lib.strata_tier_create.restype = ctypes.c_int
    lib.strata_window_set_tier.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.strata_window_set_tier.restype = ctypes.c_int
    lib.strata_tier_read.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, P(strata_tier_stats)]
    lib.strata_tier_read.restype = ctypes.c_int
    lib.strata_tier_destroy.argtypes = [ctypes.c_void_p]
    lib.strata_tier_destroy.restype = ctypes.c_int
    lib.strata_head_create.argtypes = [P(strata_head_desc), P(strata_qmat), ctypes.c_void_p, P(ctypes.c_void_p)]
    lib.strata_head_create.restype = ctypes.c_int
    lib.strata_head_forward.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, P(strata_draw_in),
                                        P(strata_draw_out), ctypes.c_void_p]
    lib.strata_head_forward.restype = ctypes.c_int
    lib.strata_head_sync.argtypes = [ctypes.c_void_p]
    lib.strata_head_sync.restype = ctypes.c_int
    lib.strata_head_query.argtypes = [ctypes.c_void_p, P(ctypes.c_int64), P(ctypes.c_int64)]
    lib.strata_head_query.restype = ctypes.c_int
    lib.strata_head_set_profiling.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.strata_head_set_profiling.restype = ctypes.c_int
    lib.strata_head_timings.argtypes = [ctypes.c_void_p, P(ctypes.c_float)]
    lib.strata_head_timings.restype = ctypes.c_int
    lib.strata_head_destroy.argtypes = [ctypes.c_void_p]
    lib.strata_head_destroy.restype = ctypes.c_int
    lib.strata_window_slots.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_void_p, P(ctypes.c_int32), P(ctypes.c_int32)]
    lib.strata_window_slots.restype = ctypes.c_int
    lib.strata_stack_set_kv.argtypes = [ctypes.c_void_p, P(strata_kv_cache)]
    lib.strata_stack_set_kv.restype = ctypes.c_int
    lib.strata_stack_forward_kv.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, P(strata_stack_out), ctypes.c_void_p]
    lib.strata_stack_forward_kv.restype = ctypes.c_int
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.strata_qknorm_create.argtypes = [P(strata_qknorm_desc), vp, vp, vp, vp, P(vp)]
    lib.strata_qknorm_create.restype = ctypes.c_int
    lib.strata_qknorm_forward.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i32, vp]
    lib.strata_qknorm_forward.restype = ctypes.c_int
    lib.strata_qknorm_destroy.argtypes = [vp]
    lib.strata_qknorm_destroy.restype = ctypes.c_int
    lib.strata_kv8_create.argtypes = [P(strata_kv8_desc), P(strata_kv8_cache), P(vp)]
    lib.strata_kv8_create.restype = ctypes.c_int
    for fn in (lib.strata_kv8_append, lib.strata_kv8_read):
        fn.argtypes = [vp, i32, vp, i64, vp, i64, i32, P(strata_kv8_rows), vp]
        fn.restype = ctypes.c_int
    lib.strata_kv8_attend.argtypes = [vp, i32, vp, i64, vp, i64, i32, ctypes.c_float, P(strata_kv8_rows), vp]
    lib.strata_kv8_attend.restype = ctypes.c_int
    lib.strata_kv8_sync.argtypes = [vp]
    lib.strata_kv8_sync.restype = ctypes.c_int
    lib.strata_kv8_query.argtypes = [vp, P(i64), P(i64)]
    lib.strata_kv8_query.restype = ctypes.c_int
    lib.strata_kv8_destroy.argtypes = [vp]
    lib.strata_kv8_destroy.restype = ctypes.c_int
    lib.strata_linear_create.argtypes = [P(strata_linear_desc), P(strata_qmat), P(strata_qmat), vp, P(vp)]
    lib.strata_linear_forward.argtypes = [vp, vp, i64, vp, i64, i32, i32, vp, vp]
    lib.strata_linear_round_weights.argtypes = [vp, i32]
    lib.strata_linear_sync.argtypes = [vp]
    lib.strata_linear_query.argtypes = [vp, P(i64), P(i64)]
    lib.strata_linear_destroy.argtypes = [vp]
    lib.strata_sort_create.argtypes = [P(strata_sort_desc), P(vp)]
    lib.strata_sort_route.argtypes = [vp, vp, i64, vp, i32, vp, vp, vp]
    lib.strata_sort_plan.argtypes = [vp, vp, i32, P(strata_sort_order), vp]
    lib.strata_sort_gather.argtypes = [vp, vp, vp, i64, vp, i64, i32, i32, i32, vp]
    lib.strata_sort_combine.argtypes = [vp, vp, vp, i64, vp, vp, i64, vp, i64, i32, i32, i32, vp]
    lib.strata_sort_combine_backward.argtypes = [vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, i32, i32, i32, vp]
    lib.strata_sort_destroy.argtypes = [vp]
    lib.strata_blocknorm_create.argtypes = [P(strata_blocknorm_desc), vp, vp, vp, vp, P(vp)]
    lib.strata_blocknorm_forward.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, vp]
    lib.strata_blocknorm_destroy.argtypes = [vp]
    for name in ("linear_create", "linear_forward", "linear_round_weights", "linear_sync", "linear_query", "linear_destroy", "sort_create",
                 "sort_route", "sort_plan", "sort_gather", "sort_combine", "sort_combine_backward", "sort_destroy",
                 "blocknorm_create", "blocknorm_forward", "blocknorm_destroy"):
        getattr(lib, "strata_" + name).restype = ctypes.c_int
    lib.strata_status_str.argtypes = [ctypes.c_int]
    lib.strata_status_str.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().strata_status_str(status).decode()


# --- the C calls, same names ---------------------------------------------------


def strata_window_create(desc: strata_moe_desc, weights: strata_moe_weights, stream: int = 0):
    """Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_window_create(ctypes.byref(desc), ctypes.byref(weights), ctypes.c_void_p(stream),
                                     ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_moe_window_forward(handle, x_ptr: int, T: int, y_ptr: int, routing: Optional[strata_routing_out] = None,
                              stream: int = 0) -> int:
    return load().strata_moe_window_forward(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T,
                                            ctypes.c_void_p(y_ptr),
                                            ctypes.byref(routing) if routing is not None else None,
                                            ctypes.c_void_p(stream))


def strata_moe_window_forward_graph(handle, x_ptr: int, T: int, y_ptr: int, stream: int = 0) -> int:
    return load().strata_moe_window_forward_graph(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T,
                                                  ctypes.c_void_p(y_ptr), ctypes.c_void_p(stream))


def strata_moe_window_forward_noalloc(handle, x_ptr: int, T: int, y_ptr: int, stream: int = 0) -> int:
    return load().strata_moe_window_forward_noalloc(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T,
                                                    ctypes.c_void_p(y_ptr), ctypes.c_void_p(stream))


def strata_stack_create(n_layers: int, desc: strata_moe_desc, attn: strata_attn_desc, moe_w, attn_w,
                        stream: int = 0):
    """moe_w / attn_w: ctypes arrays of n_layers weight structs.  Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_stack_create(n_layers, ctypes.byref(desc), ctypes.byref(attn), moe_w, attn_w,
                                    ctypes.c_void_p(stream), ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_stack_forward(handle, x_ptr: int, T: int, y_ptr: int, out: Optional[strata_stack_out] = None,
                         stream: int = 0) -> int:
    return load().strata_stack_forward(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T, ctypes.c_void_p(y_ptr),
                                       ctypes.byref(out) if out is not None else None, ctypes.c_void_p(stream))


def strata_stack_sync(handle) -> int:
    return load().strata_stack_sync(ctypes.c_void_p(handle))


def strata_stack_query(handle):
    info = strata_stack_info()
    st = load().strata_stack_query(ctypes.c_void_p(handle), ctypes.byref(info))
    return st, info


def strata_stack_set_profiling(handle, enable: bool) -> int:
    return load().strata_stack_set_profiling(ctypes.c_void_p(handle), 1 if enable else 0)


def strata_stack_timings(handle):
    ms = ctypes.c_float()
    st = load().strata_stack_timings(ctypes.c_void_p(handle), ctypes.byref(ms))
    return st, ms.value


def strata_stack_destroy(handle) -> int:
    return load().strata_stack_destroy(ctypes.c_void_p(handle))


def strata_window_sync(handle) -> int:
    return load().strata_window_sync(ctypes.c_void_p(handle))


def strata_window_query(handle):
    info = strata_window_info()
    st = load().strata_window_query(ctypes.c_void_p(handle), ctypes.byref(info))
    return st, info


def strata_window_plan(desc: strata_moe_desc, smem_limit: int = 0):
    info = strata_window_info()
    st = load().strata_window_plan(ctypes.byref(desc), smem_limit, ctypes.byref(info))
    return st, info


def strata_window_set_profiling(handle, enable: bool) -> int:
    return load().strata_window_set_profiling(ctypes.c_void_p(handle), 1 if enable else 0)


def strata_window_timings(handle):
    """Returns (status, window kernel ms)."""
    ms = ctypes.c_float()
    st = load().strata_window_timings(ctypes.c_void_p(handle), ctypes.byref(ms))
    return st, ms.value


def strata_window_destroy(handle) -> int:
    return load().strata_window_destroy(ctypes.c_void_p(handle))


def strata_tier_create(desc: strata_tier_desc, initial=None):
    """initial: a sequence of expert ids or None.  Returns (status, tier or None)."""
    h = ctypes.c_void_p()
    arr = None
    if initial is not None:
        arr = (ctypes.c_int32 * len(initial))(*[int(e) for e in initial])
    st = load().strata_tier_create(ctypes.byref(desc), arr, ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_window_set_tier(handle, tier) -> int:
    return load().strata_window_set_tier(ctypes.c_void_p(handle), ctypes.c_void_p(tier) if tier else None)


def strata_tier_read(tier, n_experts: int):
    """Returns (status, dict of numpy arrays counters/resident/swap_in/swap_out and the stats)."""
    import numpy as np
    c = np.zeros(n_experts, np.float32)
    r = np.zeros(n_experts, np.int32)
    si = np.zeros(n_experts, np.int32)
    so = np.zeros(n_experts, np.int32)
    stats = strata_tier_stats()
    st = load().strata_tier_read(ctypes.c_void_p(tier), c.ctypes.data, r.ctypes.data, si.ctypes.data, so.ctypes.data,
                                 ctypes.byref(stats))
    return st, dict(counters=c, resident=r, swap_in=si[:stats.n_swaps], swap_out=so[:stats.n_swaps],
                    windows=stats.windows, rounds=stats.rounds, n_swaps=stats.n_swaps)


def strata_tier_destroy(tier) -> int:
    return load().strata_tier_destroy(ctypes.c_void_p(tier) if tier else None)


def strata_head_create(desc: strata_head_desc, weight: strata_qmat, stream: int = 0):
    """Returns (status, head or None)."""
    h = ctypes.c_void_p()
    st = load().strata_head_create(ctypes.byref(desc), ctypes.byref(weight), ctypes.c_void_p(stream), ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_head_forward(handle, x_ptr: int, T: int, draw_in: strata_draw_in, draw_out: strata_draw_out,
                        stream: int = 0) -> int:
    return load().strata_head_forward(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T, ctypes.byref(draw_in),
                                      ctypes.byref(draw_out), ctypes.c_void_p(stream))


def strata_head_sync(handle) -> int:
    return load().strata_head_sync(ctypes.c_void_p(handle))


def strata_head_query(handle):
    hb, wb = ctypes.c_int64(), ctypes.c_int64()
    st = load().strata_head_query(ctypes.c_void_p(handle), ctypes.byref(hb), ctypes.byref(wb))
    return st, hb.value, wb.value


def strata_head_set_profiling(handle, enable: bool) -> int:
    return load().strata_head_set_profiling(ctypes.c_void_p(handle), 1 if enable else 0)


def strata_head_timings(handle):
    ms = ctypes.c_float()
    st = load().strata_head_timings(ctypes.c_void_p(handle), ctypes.byref(ms))
    return st, ms.value


def strata_head_destroy(handle) -> int:
    return load().strata_head_destroy(ctypes.c_void_p(handle) if handle else None)


def strata_window_slots(rows_per_slot, start: int, max_rows: int = 8):
    """Returns (status, slots of the next window, next start)."""
    n = len(rows_per_slot)
    rows = (ctypes.c_int32 * max(n, 1))(*[int(r) for r in rows_per_slot])
    out = (ctypes.c_int32 * max(n, 1))()
    cnt, nxt = ctypes.c_int32(), ctypes.c_int32()
    st = load().strata_window_slots(n, rows if n else None, start, max_rows, out, ctypes.byref(cnt), ctypes.byref(nxt))
    return st, [out[i] for i in range(cnt.value)] if st == STRATA_OK else [], nxt.value


def strata_stack_set_kv(handle, kv) -> int:
    return load().strata_stack_set_kv(ctypes.c_void_p(handle), ctypes.byref(kv) if kv is not None else None)


def strata_stack_forward_kv(handle, x_ptr: int, T: int, y_ptr: int, slot_ptr: int, pos_ptr: int,
                            out: Optional["strata_stack_out"] = None, stream: int = 0) -> int:
    return load().strata_stack_forward_kv(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T, ctypes.c_void_p(y_ptr),
                                          ctypes.c_void_p(slot_ptr), ctypes.c_void_p(pos_ptr),
                                          ctypes.byref(out) if out is not None else None, ctypes.c_void_p(stream))


def strata_qknorm_create(desc: strata_qknorm_desc, q_gain_ptr=None, k_gain_ptr=None, freqs=None, stream: int = 0):
    """freqs: rotary_dim/2 radians per position, a sequence, an array or a tensor.  Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    arr = (ctypes.c_double * len(freqs))(*[float(f) for f in freqs]) if freqs is not None and len(freqs) > 0 else None
    st = load().strata_qknorm_create(ctypes.byref(desc), q_gain_ptr, k_gain_ptr, arr, stream, ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_qknorm_forward(handle, q_ptr, q_stride, k_ptr, k_stride, q_out_ptr, q_out_stride, k_out_ptr, k_out_stride,
                          dtype: int, position_ptr, T: int, stream: int = 0) -> int:
    return load().strata_qknorm_forward(handle, q_ptr, q_stride, k_ptr, k_stride, q_out_ptr, q_out_stride, k_out_ptr,
                                        k_out_stride, dtype, position_ptr, T, stream)


def strata_qknorm_destroy(handle) -> int:
    return load().strata_qknorm_destroy(handle)


def strata_kv8_create(desc: strata_kv8_desc, cache: strata_kv8_cache):
    """Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_kv8_create(ctypes.byref(desc), ctypes.byref(cache), ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_kv8_append(handle, layer: int, k_ptr, k_stride: int, v_ptr, v_stride: int, dtype: int,
                      rows: strata_kv8_rows, stream: int = 0) -> int:
    return load().strata_kv8_append(handle, layer, k_ptr, k_stride, v_ptr, v_stride, dtype, rows, stream)


def strata_kv8_read(handle, layer: int, k_ptr, k_stride: int, v_ptr, v_stride: int, dtype: int,
                    rows: strata_kv8_rows, stream: int = 0) -> int:
    return load().strata_kv8_read(handle, layer, k_ptr, k_stride, v_ptr, v_stride, dtype, rows, stream)


def strata_kv8_attend(handle, layer: int, q_ptr, q_stride: int, out_ptr, out_stride: int, dtype: int, scale: float,
                      rows: strata_kv8_rows, stream: int = 0) -> int:
    return load().strata_kv8_attend(handle, layer, q_ptr, q_stride, out_ptr, out_stride, dtype, scale, rows, stream)


def strata_kv8_sync(handle) -> int:
    return load().strata_kv8_sync(handle)


def strata_kv8_query(handle):
    """Returns (status, cache bytes, workspace bytes)."""
    cb, wb = ctypes.c_int64(), ctypes.c_int64()
    st = load().strata_kv8_query(handle, ctypes.byref(cb), ctypes.byref(wb))
    return st, cb.value, wb.value


def strata_kv8_destroy(handle) -> int:
    return load().strata_kv8_destroy(handle)


def strata_linear_create(desc: strata_linear_desc, weight: strata_qmat, up: Optional[strata_qmat] = None, stream: int = 0):
    """Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_linear_create(desc, weight, up, stream, ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_linear_forward(handle, x_ptr, x_stride: int, y_ptr, y_stride: int, dtype: int, T: int, offsets_ptr=None,
                          stream: int = 0) -> int:
    return load().strata_linear_forward(handle, x_ptr, x_stride, y_ptr, y_stride, dtype, T, offsets_ptr, stream)


def strata_linear_round_weights(handle, on: int) -> int:
    return load().strata_linear_round_weights(handle, on)


def strata_linear_sync(handle) -> int:
    return load().strata_linear_sync(handle)


def strata_linear_query(handle):
    """Returns (status, weight_bytes, workspace_bytes)."""
    a, b = ctypes.c_int64(), ctypes.c_int64()
    st = load().strata_linear_query(handle, ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


def strata_linear_destroy(handle) -> int:
    return load().strata_linear_destroy(handle)


def strata_sort_create(desc: strata_sort_desc):
    """Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_sort_create(desc, ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_sort_route(handle, logits_ptr, stride: int, bias_ptr, T: int, idx_ptr, w_ptr, stream: int = 0) -> int:
    return load().strata_sort_route(handle, logits_ptr, stride, bias_ptr, T, idx_ptr, w_ptr, stream)


def strata_sort_plan(handle, idx_ptr, T: int, order: strata_sort_order, stream: int = 0) -> int:
    return load().strata_sort_plan(handle, idx_ptr, T, order, stream)


def strata_sort_gather(handle, place_ptr, x_ptr, x_stride: int, xs_ptr, xs_stride: int, dtype: int, T: int, width: int,
                       stream: int = 0) -> int:
    return load().strata_sort_gather(handle, place_ptr, x_ptr, x_stride, xs_ptr, xs_stride, dtype, T, width, stream)


def strata_sort_combine(handle, place_ptr, z_ptr, z_stride: int, w_ptr, base_ptr, base_stride: int, y_ptr, y_stride: int,
                        dtype: int, T: int, width: int, stream: int = 0) -> int:
    return load().strata_sort_combine(handle, place_ptr, z_ptr, z_stride, w_ptr, base_ptr, base_stride, y_ptr, y_stride,
                                      dtype, T, width, stream)


def strata_sort_combine_backward(handle, place_ptr, dy_ptr, dy_stride: int, z_ptr, z_stride: int, w_ptr, dz_ptr,
                                 dz_stride: int, dw_ptr, dtype: int, T: int, width: int, stream: int = 0) -> int:
    return load().strata_sort_combine_backward(handle, place_ptr, dy_ptr, dy_stride, z_ptr, z_stride, w_ptr, dz_ptr,
                                               dz_stride, dw_ptr, dtype, T, width, stream)


def strata_sort_destroy(handle) -> int:
    return load().strata_sort_destroy(handle)


def strata_blocknorm_create(desc: strata_blocknorm_desc, after_ptr=None, before_ptr=None, channel_ptr=None,
                            stream: int = 0):
    """Returns (status, handle or None)."""
    h = ctypes.c_void_p()
    st = load().strata_blocknorm_create(desc, after_ptr, before_ptr, channel_ptr, stream, ctypes.byref(h))
    return st, (h.value if st == STRATA_OK else None)


def strata_blocknorm_forward(handle, x_ptr, x_stride: int, y_ptr, y_stride: int, gate_ptr, gate_stride: int, h_ptr,
                             h_stride: int, n_ptr, n_stride: int, dtype: int, T: int, stream: int = 0) -> int:
    return load().strata_blocknorm_forward(handle, x_ptr, x_stride, y_ptr, y_stride, gate_ptr, gate_stride, h_ptr,
                                           h_stride, n_ptr, n_stride, dtype, T, stream)


def strata_blocknorm_destroy(handle) -> int:
    return load().strata_blocknorm_destroy(handle)


def check(status: int, what: str) -> None:
    if status != STRATA_OK:
        raise StrataError(status, what)


# --- torch convenience -----------------------------------------------------------


def _qmat(q) -> strata_qmat:
    return strata_qmat(q.codes.data_ptr(), q.scale.data_ptr(), q.min.data_ptr())


def desc_of(spec, max_rows: int = 8) -> strata_moe_desc:
    return strata_moe_desc(spec.hidden, spec.n_experts, spec.top_k, spec.ffn, spec.shared_ffn, spec.bits, spec.block,
                           max_rows, spec.renorm_topk)


def weights_of(layer) -> strata_moe_weights:
    w = strata_moe_weights()
    w.router_w = layer.router_w.data_ptr()
    w.router_b = layer.router_b.data_ptr() if layer.router_b is not None else None
    w.gate, w.up, w.down = _qmat(layer.gate), _qmat(layer.up), _qmat(layer.down)
    if layer.shared_gate is not None:
        w.shared_gate, w.shared_up, w.shared_down = (_qmat(layer.shared_gate), _qmat(layer.shared_up),
                                                     _qmat(layer.shared_down))
    return w


class Window:
    """A handle for one MoE layer whose weights are CUDA torch tensors."""

    def __init__(self, layer, max_rows: int = 8, stream=None):
        import torch
        self.spec = layer.spec
        self.max_rows = max_rows
        s = (stream or torch.cuda.current_stream()).cuda_stream
        st, h = strata_window_create(desc_of(layer.spec, max_rows), weights_of(layer), s)
        check(st, "strata_window_create")
        self.handle = h

    def info(self) -> strata_window_info:
        st, info = strata_window_query(self.handle)
        check(st, "strata_window_query")
        return info

    def forward(self, x, y=None, routing: bool = False, stream=None):
        """Enqueue one window on x [T][d] (CUDA fp32); returns y (and routing tensors)."""
        import torch
        assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
        T, d = x.shape
        if y is None:
            y = torch.empty_like(x)
        r = None
        rt = None
        if routing:
            E, k = self.spec.n_experts, self.spec.top_k
            dev = x.device
            rt = dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=dev),
                      topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                      counts=torch.empty(E, dtype=torch.int32, device=dev),
                      offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                      entries=torch.empty(T * k, dtype=torch.int32, device=dev),
                      distinct=torch.full((E,), -1, dtype=torch.int32, device=dev),
                      n_distinct=torch.empty(1, dtype=torch.int32, device=dev))
            r = strata_routing_out(*(rt[n].data_ptr() for n in ("topk_idx", "topk_w", "counts", "offsets", "entries",
                                                               "distinct", "n_distinct")))
        s = (stream or torch.cuda.current_stream()).cuda_stream
        check(strata_moe_window_forward(self.handle, x.data_ptr(), T, y.data_ptr(), r, s),
              "strata_moe_window_forward")
        return (y, rt) if routing else y

    def forward_graph(self, x, y, stream=None):
        """Enqueue one window through the handle's graph cache (x, y fixed CUDA buffers)."""
        import torch
        assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous() and y.is_contiguous()
        s = (stream or torch.cuda.current_stream()).cuda_stream
        check(strata_moe_window_forward_graph(self.handle, x.data_ptr(), x.shape[0], y.data_ptr(), s),
              "strata_moe_window_forward_graph")
        return y

    def set_profiling(self, enable: bool) -> None:
        check(strata_window_set_profiling(self.handle, enable), "strata_window_set_profiling")

    def timings(self):
        st, ms = strata_window_timings(self.handle)
        check(st, "strata_window_timings")
        return ms

    def sync(self) -> None:
        check(strata_window_sync(self.handle), "strata_window_sync")

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_window_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def attn_desc_of(wl) -> strata_attn_desc:
    return strata_attn_desc(wl.heads, wl.kv_heads, wl.head_dim)


def attn_weights_of(dl) -> strata_attn_weights:
    return strata_attn_weights(_qmat(dl.q), _qmat(dl.k), _qmat(dl.v), _qmat(dl.o))


class Stack:
    """A handle for a stack of decoder layers whose weights are CUDA torch tensors.

    moe_layers / dense_layers: per-layer ``workloads.MoELayer`` / ``DenseLayer``;
    wl: the workload (attention shapes).  The handle keeps its own
    kernel-ordered copies, so the tensors may be freed after construction.
    """

    def __init__(self, wl, moe_layers, dense_layers, max_rows: int = 8, stream=None):
        import torch
        n = len(moe_layers)
        assert n == len(dense_layers) and n >= 1
        self.wl, self.n_layers, self.spec = wl, n, moe_layers[0].spec
        mw = (strata_moe_weights * n)(*[weights_of(m) for m in moe_layers])
        aw = (strata_attn_weights * n)(*[attn_weights_of(dl) for dl in dense_layers])
        s = (stream or torch.cuda.current_stream()).cuda_stream
        st, h = strata_stack_create(n, desc_of(self.spec, max_rows), attn_desc_of(wl), mw, aw, s)
        check(st, "strata_stack_create")
        self.handle = h

    def info(self) -> strata_stack_info:
        st, info = strata_stack_query(self.handle)
        check(st, "strata_stack_query")
        return info

    def set_kv(self, k, v, n_slots: int, max_ctx: int) -> None:
        """Attend over the fp16 caches k, v (CUDA tensors of
        [n_layers][n_slots][kv_heads][max_ctx][head_dim], float16) from now on
        (forward with slot and position); None drops them."""
        if k is None:
            check(strata_stack_set_kv(self.handle, None), "strata_stack_set_kv")
            self.kv = None
            return
        check(strata_stack_set_kv(self.handle, strata_kv_cache(k.data_ptr(), v.data_ptr(), n_slots, max_ctx)),
              "strata_stack_set_kv")
        self.kv = (k, v)

    def forward(self, x, y=None, outputs: bool = False, stream=None, slot=None, position=None):
        """Enqueue one window on x [T][d]; returns y (and per-layer q, k, routing).
        With slot and position (CUDA int32 [T]) the window attends over the caches set by set_kv."""
        import torch
        assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
        T, d = x.shape
        if y is None:
            y = torch.empty_like(x)
        o = None
        res = None
        if outputs:
            n, wl, k = self.n_layers, self.wl, self.spec.top_k
            dev = x.device
            res = dict(q=torch.empty(n, T, wl.heads * wl.head_dim, device=dev),
                       k=torch.empty(n, T, wl.kv_heads * wl.head_dim, device=dev),
                       topk_idx=torch.empty(n, T, k, dtype=torch.int32, device=dev),
                       topk_w=torch.empty(n, T, k, device=dev),
                       n_distinct=torch.empty(n, dtype=torch.int32, device=dev))
            o = strata_stack_out(*(res[m].data_ptr() for m in ("q", "k", "topk_idx", "topk_w", "n_distinct")))
        s = (stream or torch.cuda.current_stream()).cuda_stream
        if slot is not None:
            check(strata_stack_forward_kv(self.handle, x.data_ptr(), T, y.data_ptr(), slot.data_ptr(),
                                          position.data_ptr(), o, s), "strata_stack_forward_kv")
        else:
            check(strata_stack_forward(self.handle, x.data_ptr(), T, y.data_ptr(), o, s), "strata_stack_forward")
        return (y, res) if outputs else y

    def set_profiling(self, enable: bool) -> None:
        check(strata_stack_set_profiling(self.handle, enable), "strata_stack_set_profiling")

    def timings(self):
        st, ms = strata_stack_timings(self.handle)
        check(st, "strata_stack_timings")
        return ms

    def sync(self) -> None:
        check(strata_stack_sync(self.handle), "strata_stack_sync")

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Head:
    """The output head for a block-format weight ``QMat`` [1][V][d] on the GPU."""

    def __init__(self, weight, max_rows: int = 8, stream=None):
        import torch
        self.V, self.d = weight.rows, weight.cols
        s = (stream or torch.cuda.current_stream()).cuda_stream
        desc = strata_head_desc(weight.cols, weight.rows, weight.bits, weight.block, max_rows)
        st, h = strata_head_create(desc, _qmat(weight), s)
        check(st, "strata_head_create")
        self.handle = h

    def forward(self, x, position, seed, temperature, fed, logits: bool = False, stream=None):
        """Enqueue one window's head on x [T][d]; the per-row inputs are CUDA
        tensors (int32, int64 seeds, float32, int32).  Returns (tokens, n_emit,
        logits or None), int32 / float32 CUDA tensors."""
        import torch
        assert x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()
        T = x.shape[0]
        dev = x.device
        tokens = torch.empty(T, dtype=torch.int32, device=dev)
        n_emit = torch.empty(T, dtype=torch.int32, device=dev)
        lg = torch.empty(T, self.V, device=dev) if logits else None
        di = strata_draw_in(position.data_ptr(), seed.data_ptr(), temperature.data_ptr(), fed.data_ptr())
        do = strata_draw_out(tokens.data_ptr(), n_emit.data_ptr(), lg.data_ptr() if logits else None)
        s = (stream or torch.cuda.current_stream()).cuda_stream
        check(strata_head_forward(self.handle, x.data_ptr(), T, di, do, s), "strata_head_forward")
        return tokens, n_emit, lg

    def sync(self) -> None:
        check(strata_head_sync(self.handle), "strata_head_sync")

    def set_profiling(self, enable: bool) -> None:
        check(strata_head_set_profiling(self.handle, enable), "strata_head_set_profiling")

    def timings(self):
        st, ms = strata_head_timings(self.handle)
        check(st, "strata_head_timings")
        return ms

    def head_bytes(self) -> int:
        st, hb, _ = strata_head_query(self.handle)
        check(st, "strata_head_query")
        return hb

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_head_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# The calls below are short next to Python's own time (a window's take 2 to 16 us on the GPU), so their checks read each
# tensor property once and what they need of torch is looked up once, by the first handle.
_torch = None
_DTYPE = None  # torch dtype -> strata_dtype


def _with_torch():
    global _torch, _DTYPE
    if _torch is None:
        import torch
        _DTYPE = {torch.float32: STRATA_F32, torch.float16: STRATA_F16, torch.bfloat16: STRATA_BF16}
        _torch = torch
    return _torch


def _row_stride(t, shape, what: str) -> int:
    """The distance between rows, in elements, of a CUDA tensor of this shape [T][heads][head_dim]; raises for any
    layout whose rows are not contiguous."""
    st = t.stride()
    if t.shape != shape or st[2] != 1 or (st[1] != shape[2] and shape[1] != 1) or not t.is_cuda or \
            t.dtype not in _DTYPE:
        raise StrataError(STRATA_EINVAL, f"{what}: want a CUDA tensor [{shape[0]}][{shape[1]}][{shape[2]}] of float32, "
                                         "float16 or bfloat16 whose rows are contiguous")
    return st[0] if shape[0] > 1 else shape[1] * shape[2]


def _same(t, like, what: str) -> None:
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise StrataError(STRATA_EINVAL, f"{what}: type or device differ")


def _int32(t, n: int, device: int, what: str):
    """The pointer of a contiguous CUDA int32 tensor [n] of the device."""
    if t.dtype is not _torch.int32 or t.shape != (n,) or t.get_device() != device or (n > 1 and t.stride(0) != 1):
        raise StrataError(STRATA_EINVAL, f"{what}: want a contiguous CUDA int32 tensor [{n}] on the call's device")
    return t.data_ptr()


def _raw_stream(index: int, stream) -> int:
    """The cudaStream_t of a stream, or of the device's current one."""
    return stream.cuda_stream if stream is not None else _torch._C._cuda_getCurrentRawStream(index)


def _empty(shape, dtype, device, stream):
    """A new tensor of the stream that the call runs on."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


class QkNorm:
    """Norms of the query and key heads with the rotation by position.

    q_gain, k_gain: CUDA float32 [head_dim] or None (unit gain).  freqs:
    rotary_dim/2 radians per position (a sequence, an array or a tensor); None
    forms theta ** (-2 i / rotary_dim).
    """

    def __init__(self, heads: int, kv_heads: int, head_dim: int, rotary_dim: Optional[int] = None, freqs=None,
                 theta: float = 10000.0, interleaved: bool = False, norm: bool = True, eps: float = 1e-6,
                 q_gain=None, k_gain=None, device=None, stream=None):
        torch = _with_torch()
        rd = head_dim if rotary_dim is None else rotary_dim
        if freqs is None:
            freqs = [theta ** (-2.0 * i / rd) for i in range(rd // 2)] if rd > 0 else []
        if len(freqs) != max(rd, 0) // 2:
            raise StrataError(STRATA_EINVAL, "QkNorm: freqs has rotary_dim/2 entries")
        for g in (q_gain, k_gain):
            if g is not None:
                if not g.is_cuda or g.dtype != torch.float32 or tuple(g.shape) != (head_dim,) or \
                        not g.is_contiguous():
                    raise StrataError(STRATA_EINVAL, "QkNorm: a gain is a contiguous CUDA float32 [head_dim]")
                if device is None:
                    device = g.device
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        with torch.cuda.device(device):
            s = (stream or torch.cuda.current_stream()).cuda_stream
            self.device = torch.cuda.current_device()
            if any(g is not None and g.get_device() != self.device for g in (q_gain, k_gain)):
                raise StrataError(STRATA_EINVAL, "QkNorm: want the gains on the handle's device")
            st, h = strata_qknorm_create(
                strata_qknorm_desc(heads, kv_heads, head_dim, rd, int(interleaved), int(norm), eps),
                q_gain.data_ptr() if q_gain is not None else None, k_gain.data_ptr() if k_gain is not None else None,
                freqs, s)
        check(st, "strata_qknorm_create")
        self.handle = h
        self._forward = load().strata_qknorm_forward

    def forward(self, q, k, position, q_out=None, k_out=None, stream=None):
        """Enqueue q [T][heads][head_dim] and k [T][kv_heads][head_dim] at position (CUDA int32 [T]); returns
        (q_out, k_out), new tensors unless given (an output may be its own input)."""
        T, kv, hd = q.shape[0] if q.dim() == 3 else -1, self.kv_heads, self.head_dim
        shape = (T, self.heads, hd)
        qs = _row_stride(q, shape, "q")
        qos = self.heads * hd
        if q_out is None:
            q_out = _empty(shape, q.dtype, q.device, stream)
        else:
            qos = _row_stride(q_out, shape, "q_out")
            _same(q_out, q, "q_out")
        kp = ks = kop = kos = 0
        if kv > 0:
            if k is None:
                raise StrataError(STRATA_EINVAL, "k: wanted by kv_heads > 0")
            shape = (T, kv, hd)
            ks = _row_stride(k, shape, "k")
            _same(k, q, "k")
            kos = kv * hd
            if k_out is None:
                k_out = _empty(shape, k.dtype, k.device, stream)
            else:
                kos = _row_stride(k_out, shape, "k_out")
                _same(k_out, q, "k_out")
            kp, kop = k.data_ptr(), k_out.data_ptr()
        device = q.get_device()
        if device != self.device:
            raise StrataError(STRATA_EINVAL, "q: want a tensor on the handle's device")
        st = self._forward(self.handle, q.data_ptr(), qs, kp, ks, q_out.data_ptr(), qos, kop, kos, _DTYPE[q.dtype],
                           _int32(position, T, device, "position"), T, _raw_stream(device, stream))
        if st != STRATA_OK:
            check(st, "strata_qknorm_forward")
        return q_out, k_out

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_qknorm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KvRows:
    """The rows of a KvCache8 call: sequence i has rows row_start[i] to row_start[i+1] - 1, the last ones of the
    length[i] positions that slot[i] holds with them.  row_start [n_seq + 1], slot and length [n_seq] are CUDA int32
    tensors that the calls read on the device; n_rows is the rows of the value tensors (those behind the last
    sequence are left as they were), max_rows the most rows of one sequence."""

    def __init__(self, row_start, slot, length, n_rows: int, max_rows: int):
        _with_torch()
        n, device = slot.shape[0], slot.get_device()
        self.keep = (row_start, slot, length)
        self.n_rows, self.device = n_rows, device
        self.c = strata_kv8_rows(n, n_rows, max_rows, _int32(row_start, n + 1, device, "row_start"),
                                 _int32(slot, n, device, "slot"), _int32(length, n, device, "length"))


class KvCache8:
    """8-bit KV caches of the slots, one exponent per block of positions and kv head.

    The codes (k, v: uint8 [n_layers][n_slots][kv_heads][max_ctx][head_dim]) and exponent bytes (k_exp, v_exp:
    uint8 [...][ceil(max_ctx / block)]) are torch tensors, made here or given as ``buffers`` (contiguous, of these
    sizes).  format: "e4m3" or "int8".  Calls are asynchronous; sync() raises what the GPU recorded.

    attend() uses the handle's workspace: its calls on one KvCache8, whatever the layer, and replays of captured ones must
    not run at the same time.  On one stream they do not; across streams, order them with events.  (append() and read()
    need no such order.)  What an overlap may leave behind spoils later calls until sync() has raised it.
    """

    def __init__(self, n_layers: int, n_slots: int, heads: int, kv_heads: int, head_dim: int, max_ctx: int,
                 block: int = 64, format: str = "e4m3", buffers=None, device=None):
        torch = _with_torch()
        fmt = {"e4m3": STRATA_KV8_E4M3, "int8": STRATA_KV8_INT8}.get(format)
        if fmt is None:
            raise StrataError(STRATA_EINVAL, "KvCache8: format is e4m3 or int8")
        desc = strata_kv8_desc(n_layers, n_slots, heads, kv_heads, head_dim, max_ctx, block, fmt)
        if min(n_layers, n_slots, heads, kv_heads, head_dim, max_ctx, block) < 1:
            raise StrataError(STRATA_EINVAL, "KvCache8: sizes are positive")
        shape = (n_layers, n_slots, kv_heads, max_ctx, head_dim)
        eshape = shape[:3] + ((max_ctx + block - 1) // block,)
        if buffers is None:
            buffers = tuple(torch.empty(x, dtype=torch.uint8, device="cuda" if device is None else device)
                            for x in (shape, shape, eshape, eshape))
        for t, x in zip(buffers, (shape, shape, eshape, eshape)):
            n = 1
            for d in x:
                n *= d
            if not t.is_cuda or t.element_size() != 1 or t.numel() != n or not t.is_contiguous() or \
                    t.device != buffers[0].device:
                raise StrataError(STRATA_EINVAL, f"KvCache8: want contiguous 8-bit CUDA buffers of {shape}, {eshape}")
        self.heads, self.kv_heads, self.head_dim, self.n_layers = heads, kv_heads, head_dim, n_layers
        self.k, self.v, self.k_exp, self.v_exp = buffers
        self.scale = head_dim ** -0.5
        with torch.cuda.device(self.k.device):
            st, h = strata_kv8_create(desc, strata_kv8_cache(*(t.data_ptr() for t in buffers)))
        check(st, "strata_kv8_create")
        self.handle = h
        self.device = self.k.get_device()
        lib = load()
        self._append, self._read, self._attend = lib.strata_kv8_append, lib.strata_kv8_read, lib.strata_kv8_attend

    def _stride(self, rows, t, heads: int, what: str) -> int:
        if t.dim() != 3 or t.get_device() != self.device or rows.device != self.device:
            raise StrataError(STRATA_EINVAL, f"{what}: want [rows][heads][head_dim] on the cache's device")
        return _row_stride(t, (rows.n_rows, heads, self.head_dim), what)

    def append(self, layer: int, k, v, rows: KvRows, stream=None) -> None:
        """Enqueue the rows' keys and values [n_rows][kv_heads][head_dim] into the layer's caches."""
        ks, vs = self._stride(rows, k, self.kv_heads, "k"), self._stride(rows, v, self.kv_heads, "v")
        _same(v, k, "v")
        st = self._append(self.handle, layer, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPE[k.dtype], rows.c,
                          _raw_stream(self.device, stream))
        if st != STRATA_OK:
            check(st, "strata_kv8_append")

    def read(self, layer: int, rows: KvRows, dtype=None, k=None, v=None, stream=None):
        """Enqueue the rows' positions as values; returns (k, v), [n_rows][kv_heads][head_dim] of dtype (float32),
        new tensors unless given; rows of no sequence are not written."""
        shape = (rows.n_rows, self.kv_heads, self.head_dim)
        ks = vs = self.kv_heads * self.head_dim
        if k is None:
            k = _empty(shape, dtype or (v.dtype if v is not None else _torch.float32), self.k.device, stream)
            if k.dtype not in _DTYPE or rows.device != self.device:
                raise StrataError(STRATA_EINVAL, "read: want float32, float16 or bfloat16 and rows on the cache's device")
        else:
            ks = self._stride(rows, k, self.kv_heads, "k")
        if v is None:
            v = _empty(shape, k.dtype, self.k.device, stream)
        else:
            vs = self._stride(rows, v, self.kv_heads, "v")
            _same(v, k, "v")
        st = self._read(self.handle, layer, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPE[k.dtype], rows.c,
                        _raw_stream(self.device, stream))
        if st != STRATA_OK:
            check(st, "strata_kv8_read")
        return k, v

    def attend(self, layer: int, q, rows: KvRows, out=None, scale: Optional[float] = None, stream=None):
        """Enqueue the attention of q [n_rows][heads][head_dim] over the layer's caches; returns out, a new tensor
        unless given; rows of no sequence are not written.  scale: 1 / sqrt(head_dim) unless given.  Must not run at
        the same time as another attend() of this cache (see KvCache8)."""
        qs = self._stride(rows, q, self.heads, "q")
        if out is None:
            out = _empty((rows.n_rows, self.heads, self.head_dim), q.dtype, q.device, stream)
            os_ = self.heads * self.head_dim
        else:
            os_ = self._stride(rows, out, self.heads, "out")
            _same(out, q, "out")
        st = self._attend(self.handle, layer, q.data_ptr(), qs, out.data_ptr(), os_, _DTYPE[q.dtype],
                          self.scale if scale is None else scale, rows.c, _raw_stream(self.device, stream))
        if st != STRATA_OK:
            check(st, "strata_kv8_attend")
        return out

    def sync(self) -> None:
        check(strata_kv8_sync(self.handle), "strata_kv8_sync")

    def cache_bytes(self) -> int:
        st, cb, _ = strata_kv8_query(self.handle)
        check(st, "strata_kv8_query")
        return cb

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_kv8_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _rows(t, shape, what: str) -> int:
    """The distance between rows, in elements, of a CUDA tensor [T][width] whose rows are contiguous."""
    st = t.stride()
    if t.shape != shape or (st[1] != 1 and shape[1] > 1) or not t.is_cuda or t.dtype not in _DTYPE:
        raise StrataError(STRATA_EINVAL, f"{what}: want a CUDA tensor [{shape[0]}][{shape[1]}] of float32, float16 or "
                                         "bfloat16 whose rows are contiguous")
    return st[0] if shape[0] > 1 else shape[1]


def _on(t, device: int, what: str) -> None:
    if t.get_device() != device:
        raise StrataError(STRATA_EINVAL, f"{what}: want a tensor on the handle's device")


def _words(t, shape, dtype, device: int, what: str):
    """The pointer of a contiguous CUDA tensor of this shape and 4-byte type on the device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise StrataError(STRATA_EINVAL, f"{what}: want a contiguous {dtype} tensor {list(shape)} on the handle's device")
    return t.data_ptr()


class Linear:
    """Products with a stack of 4-bit matrices (block format: codes uint8 [n][rows][cols / 2], scale and min 16-bit
    [n][rows][cols / 32], on one CUDA device), as ``workloads.QMat``; with ``up`` (the same shape) silu(W x) * (U x).
    The handle keeps its own copy.  max_rows: most rows of a call.  rounded: calls of many bf16 rows take weights rounded to
    f16, faster (exact weights otherwise).

    Calls of more than 8 rows, or with offsets, may use the handle's workspace: they, and replays of captured ones, must not
    run at the same time.  On one stream they do not; across streams, order them with events.
    """

    def __init__(self, weight, up=None, max_rows: int = 8, stream=None, rounded: bool = False):
        torch = _with_torch()
        n, rows, cols = weight.codes.shape[0], weight.rows, weight.cols
        device = weight.codes.get_device()
        for q in (weight, up):
            if q is None:
                continue
            if (q.rows, q.cols, q.bits, q.block) != (rows, cols, weight.bits, weight.block) or q.bits < 1 or q.block < 1:
                raise StrataError(STRATA_EINVAL, "Linear: up has weight's shape and format")
            for t, size, width in ((q.codes, 1, cols * q.bits // 8), (q.scale, 2, cols // q.block),
                                   (q.min, 2, cols // q.block)):
                if not t.is_cuda or t.element_size() != size or t.shape != (n, rows, width) or not t.is_contiguous() or \
                        t.get_device() != device:
                    raise StrataError(STRATA_EINVAL, "Linear: want contiguous CUDA codes [n][rows][cols*bits/8] and 16-bit "
                                                     "scale, min [n][rows][cols/block] on one device")
        self.n, self.rows, self.cols, self.max_rows, self.device = n, rows, cols, max_rows, device
        with torch.cuda.device(device):
            s = (stream or torch.cuda.current_stream()).cuda_stream
            st, h = strata_linear_create(strata_linear_desc(n, cols, rows, weight.bits, weight.block, max_rows),
                                         _qmat(weight), _qmat(up) if up is not None else None, s)
        check(st, "strata_linear_create")
        self.handle = h
        check(strata_linear_round_weights(h, int(rounded)), "strata_linear_round_weights")
        self._forward = load().strata_linear_forward

    def forward(self, x, y=None, offsets=None, stream=None):
        """Enqueue x [T][cols]; returns y [T][rows] of the same type, a new tensor unless given.  offsets (CUDA int32
        [n + 1], wanted where n > 1): matrix i takes rows offsets[i] to offsets[i + 1] - 1; rows of no matrix are not
        written."""
        T = x.shape[0] if x.dim() == 2 else -1
        xs = _rows(x, (T, self.cols), "x")
        _on(x, self.device, "x")
        ys = self.rows
        if y is None:
            y = _empty((T, self.rows), x.dtype, x.device, stream)
        else:
            ys = _rows(y, (T, self.rows), "y")
            _same(y, x, "y")
        op = _int32(offsets, self.n + 1, self.device, "offsets") if offsets is not None else None
        st = self._forward(self.handle, x.data_ptr(), xs, y.data_ptr(), ys, _DTYPE[x.dtype], T, op,
                           _raw_stream(self.device, stream))
        if st != STRATA_OK:
            check(st, "strata_linear_forward")
        return y

    def sync(self) -> None:
        check(strata_linear_sync(self.handle), "strata_linear_sync")

    def bytes(self):
        """(bytes of the matrices, bytes of the workspace)."""
        st, a, b = strata_linear_query(self.handle)
        check(st, "strata_linear_query")
        return a, b

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SortPlan:
    """The order of T*k entries: counts [E], offsets [E + 1], entries [T*k] by expert, place [T*k] of each entry (-1: no
    expert's), CUDA int32 tensors (views of one, formed when they are asked for)."""

    def __init__(self, mem, n_experts: int, top_k: int, T: int):
        n = T * top_k
        self.mem, self.T, self.top_k, self._E, self._n = mem, T, top_k, n_experts, n
        at = mem.data_ptr()
        self.c = strata_sort_order(at, at + 4 * n_experts, at + 4 * (2 * n_experts + 1), at + 4 * (2 * n_experts + 1 + n))

    @property
    def counts(self):
        return self.mem[:self._E]

    @property
    def offsets(self):
        return self.mem[self._E:2 * self._E + 1]

    @property
    def entries(self):
        return self.mem[2 * self._E + 1:2 * self._E + 1 + self._n]

    @property
    def place(self):
        return self.mem[2 * self._E + 1 + self._n:]


class ExpertSort:
    """Tokens sorted by expert and back: the router's choice, the order of the entries, the rows in it, and the experts'
    results weighted back, with the gradient.  An entry t * k + j is row t's j-th expert."""

    def __init__(self, n_experts: int, top_k: int, renorm: bool = False, device=None):
        torch = _with_torch()
        with torch.cuda.device(device):
            self.device = torch.cuda.current_device()
            st, h = strata_sort_create(strata_sort_desc(n_experts, top_k, int(renorm)))
        check(st, "strata_sort_create")
        self.n_experts, self.top_k, self.handle = n_experts, top_k, h
        lib = load()
        self._route, self._plan, self._gather = lib.strata_sort_route, lib.strata_sort_plan, lib.strata_sort_gather
        self._combine, self._backward = lib.strata_sort_combine, lib.strata_sort_combine_backward

    def route(self, logits, bias=None, stream=None):
        """Enqueue the choice from logits float32 [T][E] (rows contiguous) with bias [E] or None; returns (topk_idx
        int32, topk_w float32) [T][k].  -inf and NaN are never chosen (-1, weight 0)."""
        E, k, dev = self.n_experts, self.top_k, self.device
        T = logits.shape[0] if logits.dim() == 2 else -1
        if logits.dtype is not _torch.float32:
            raise StrataError(STRATA_EINVAL, "logits: want float32")
        stride = _rows(logits, (T, E), "logits")
        _on(logits, dev, "logits")
        idx = _empty((T, k), _torch.int32, logits.device, stream)
        w = _empty((T, k), _torch.float32, logits.device, stream)
        st = self._route(self.handle, logits.data_ptr(), stride,
                         _words(bias, (E,), _torch.float32, dev, "bias") if bias is not None else None, T, idx.data_ptr(),
                         w.data_ptr(), _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_sort_route")
        return idx, w

    def plan(self, topk_idx, stream=None) -> SortPlan:
        """Enqueue the order of topk_idx int32 [T][k]; entries outside 0..E-1 are no expert's."""
        E, k, dev = self.n_experts, self.top_k, self.device
        T = topk_idx.shape[0]
        p = _words(topk_idx, (T, k), _torch.int32, dev, "topk_idx")
        plan = SortPlan(_empty((2 * E + 1 + 2 * T * k,), _torch.int32, topk_idx.device, stream), E, k, T)
        st = self._plan(self.handle, p, T, plan.c, _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_sort_plan")
        return plan

    def _place(self, plan: SortPlan) -> int:
        if plan.top_k != self.top_k or plan.mem.get_device() != self.device:
            raise StrataError(STRATA_EINVAL, "plan: want one of a sort with as many choices, on the handle's device")
        return plan.c.place

    def _weights(self, w, T: int):
        return _words(w, (T, self.top_k), _torch.float32, self.device, "w") if w is not None else None

    def gather(self, plan: SortPlan, x, out=None, stream=None):
        """Enqueue the rows of x [T][width] in the experts' order; returns [T*k][width], a new tensor unless given; rows
        behind the last expert's are not written.  Its gradient: combine(plan, dxs)."""
        T, dev, width = plan.T, self.device, x.shape[-1]
        xs = _rows(x, (T, width), "x")
        _on(x, dev, "x")
        os_ = width
        if out is None:
            out = _empty((T * self.top_k, width), x.dtype, x.device, stream)
        else:
            os_ = _rows(out, (T * self.top_k, width), "out")
            _same(out, x, "out")
        st = self._gather(self.handle, self._place(plan), x.data_ptr(), xs, out.data_ptr(), os_, _DTYPE[x.dtype], T,
                          width, _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_sort_gather")
        return out

    def combine(self, plan: SortPlan, z, w=None, base=None, out=None, stream=None):
        """Enqueue base[t] + sum_j w[t][j] z[place] (w float32 [T][k], None: ones; base [T][width] or None); returns
        [T][width], a new tensor unless given (it may be base)."""
        T, dev, width = plan.T, self.device, z.shape[-1]
        zs = _rows(z, (T * self.top_k, width), "z")
        _on(z, dev, "z")
        bs = os_ = width
        if base is not None:
            bs = _rows(base, (T, width), "base")
            _same(base, z, "base")
        if out is None:
            out = _empty((T, width), z.dtype, z.device, stream)
        else:
            os_ = _rows(out, (T, width), "out")
            _same(out, z, "out")
        st = self._combine(self.handle, self._place(plan), z.data_ptr(), zs, self._weights(w, T),
                           base.data_ptr() if base is not None else None, bs, out.data_ptr(), os_, _DTYPE[z.dtype], T,
                           width, _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_sort_combine")
        return out

    def combine_backward(self, plan: SortPlan, dy, z, w=None, dz=None, stream=None):
        """Enqueue combine's gradient for dy [T][width]: (dz [T*k][width], a new tensor unless given (it may be z), dw
        float32 [T][k]); rows of dz behind the last expert's are not written."""
        T, dev, width = plan.T, self.device, z.shape[-1]
        zs = _rows(z, (T * self.top_k, width), "z")
        ds = _rows(dy, (T, width), "dy")
        _on(z, dev, "z")
        _same(dy, z, "dy")
        os_ = width
        if dz is None:
            dz = _empty((T * self.top_k, width), z.dtype, z.device, stream)
        else:
            os_ = _rows(dz, (T * self.top_k, width), "dz")
            _same(dz, z, "dz")
        dw = _empty((T, self.top_k), _torch.float32, z.device, stream)
        st = self._backward(self.handle, self._place(plan), dy.data_ptr(), ds, z.data_ptr(), zs, self._weights(w, T),
                            dz.data_ptr(), os_, dw.data_ptr(), _DTYPE[z.dtype], T, width, _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_sort_combine_backward")
        return dz, dw

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_sort_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BlockNorm:
    """Norms after and before a block with the gate and the residual:
    h = residual_scale * x + block_scale * gate * norm(y) * after, and norm(h) * before.

    after, before: the gains, CUDA float32 [hidden], or True for ones, or None for no norm.  gate: "none", "channel"
    (channel_gate: CUDA float32 [hidden]), "row" or "element" (given to forward).  sigmoid: the gate is taken through it.
    """

    def __init__(self, hidden: int, after=None, before=None, gate: str = "none", channel_gate=None, sigmoid: bool = False,
                 eps: float = 1e-6, residual_scale: float = 1.0, block_scale: float = 1.0, device=None, stream=None):
        torch = _with_torch()
        kind = {"none": STRATA_GATE_NONE, "channel": STRATA_GATE_CHANNEL, "row": STRATA_GATE_ROW,
                "element": STRATA_GATE_ELEMENT}.get(gate)
        if kind is None or (channel_gate is not None) != (kind == STRATA_GATE_CHANNEL):
            raise StrataError(STRATA_EINVAL, "BlockNorm: gate is none, channel (with channel_gate), row or element")
        given = [g for g in (after, before, channel_gate) if g is not None and g is not True]
        for g in given:
            if not g.is_cuda or g.dtype != torch.float32 or tuple(g.shape) != (hidden,) or not g.is_contiguous():
                raise StrataError(STRATA_EINVAL, "BlockNorm: a gain or gate is a contiguous CUDA float32 [hidden]")
            if device is None:
                device = g.device
        self.hidden, self.gate, self.before = hidden, kind, before is not None
        with torch.cuda.device(device):
            s = (stream or torch.cuda.current_stream()).cuda_stream
            self.device = torch.cuda.current_device()
            if any(g.get_device() != self.device for g in given):
                raise StrataError(STRATA_EINVAL, "BlockNorm: want gains and gate on the handle's device")
            ptr = [g.data_ptr() if g is not None and g is not True else None for g in (after, before, channel_gate)]
            st, h = strata_blocknorm_create(
                strata_blocknorm_desc(hidden, int(after is not None), int(self.before), kind, int(sigmoid), eps,
                                      residual_scale, block_scale), *ptr, s)
        check(st, "strata_blocknorm_create")
        self.handle = h
        self._forward = load().strata_blocknorm_forward

    def forward(self, x, y=None, gate=None, h_out=None, n_out=None, keep: bool = True, stream=None):
        """Enqueue x and y [T][hidden] (y None where there is no after norm and no gate), gate float32 [T] ("row") or
        [T][hidden] of x's type ("element"); returns (h, n), new tensors unless given (each may be x or y).  keep False:
        h is not written (None); n is None without a before norm."""
        T, d, dev = x.shape[0] if x.dim() == 2 else -1, self.hidden, self.device
        shape = (T, d)
        xs = _rows(x, shape, "x")
        _on(x, dev, "x")
        ys = gs = hs = ns = d
        gp = None
        if y is not None:
            ys = _rows(y, shape, "y")
            _same(y, x, "y")
        if gate is not None:
            if self.gate == STRATA_GATE_ROW:
                gp = _words(gate, (T,), _torch.float32, dev, "gate")
            else:
                gs = _rows(gate, shape, "gate")
                _same(gate, x, "gate")
                gp = gate.data_ptr()
        if h_out is not None:
            hs = _rows(h_out, shape, "h_out")
            _same(h_out, x, "h_out")
        elif keep:
            h_out = _empty(shape, x.dtype, x.device, stream)
        if n_out is not None:
            ns = _rows(n_out, shape, "n_out")
            _same(n_out, x, "n_out")
        elif self.before:
            n_out = _empty(shape, x.dtype, x.device, stream)
        st = self._forward(self.handle, x.data_ptr(), xs, y.data_ptr() if y is not None else None, ys, gp, gs,
                           h_out.data_ptr() if h_out is not None else None, hs,
                           n_out.data_ptr() if n_out is not None else None, ns, _DTYPE[x.dtype], T,
                           _raw_stream(dev, stream))
        if st != STRATA_OK:
            check(st, "strata_blocknorm_forward")
        return h_out, n_out

    def close(self) -> None:
        if getattr(self, "handle", None):
            strata_blocknorm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
