"""GB300 (sm_103a) top-k routed MoE feed-forward layer: forward pass, 4-bit experts, and the
operators that train its router and experts.

Thin binding over the C ABI in ``include/moe.h`` (``libmoe_gb300.so``): the
functions below carry the same names and only marshal arguments (torch tensors
-> device pointers, the current CUDA stream).  Every step runs in the library's
CUDA kernels; there is no CPU path.  Importing fails loudly when the library has
not been built (``python moe_expert_layer_fp32_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python moe_expert_layer_fp32_gb300/build.py)")

_lib = ctypes.CDLL(LIB_PATH)

try:  # the tensor calls' fast path, built with the library against one torch's headers
    from . import _tensor_calls as _calls
    if _calls.torch_version != torch.__version__:
        raise ImportError(f"built with torch {_calls.torch_version}, this is {torch.__version__}")
    _calls.bind(LIB_PATH)
    NATIVE_TENSOR_CALLS = True
except ImportError as _e:
    warnings.warn(f"the native tensor calls are not available ({_e}): the same calls go through "
                  "Python, which takes longer on the host (build: python "
                  "moe_expert_layer_fp32_gb300/build.py)")
    NATIVE_TENSOR_CALLS = False

    class _calls:  # declines every call
        @staticmethod
        def _decline(*args):
            return None

        route_select = route_select_backward = mx4_quantize = mx4_expert_product = _decline
        grouped_product = grouped_weight_grad = swiglu = swiglu_backward = orthogonalize = _decline

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_MISALIGNED",
          4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_TIMEOUT",
          7: "MOE_ERR_DEVICE_CHECK"}

# Every symbol include/moe.h declares.
ABI_SYMBOLS = ("moe_workspace_bytes", "moe_packed_weight_bytes", "moe_route", "moe_load_stats",
               "moe_load_summary_host", "moe_permute", "moe_prepack_expert_weights",
               "moe_expert_ffn", "moe_combine", "moe_layer_fwd", "moe_layer_fwd_profiled",
               "moe_read_device_status", "moe_status_string", "moe_load_stats_noalloc",
               "moe_set_wait_limit", "moe_route_ex", "moe_combine_ex", "moe_layer_fwd_ex",
               "moe_load_stats_ex", "moe_lpt_placement_host", "moe_rank_load_summary_host",
               "moe_permute_ex", "moe_prepack_expert_weights_ex", "moe_combine_sharded",
               "moe_tree_reduce_bf16", "moe_shared_packed_bytes", "moe_prepack_shared_expert",
               "moe_shared_expert_workspace_bytes", "moe_shared_expert",
               "moe_sharded_workspace_bytes", "moe_layer_fwd_sharded",
               "moe_layer_fwd_sharded_profiled", "moe_expert_ffn_form",
               "moe_router_logits", "moe_select_workspace_bytes", "moe_route_select",
               "moe_route_select_bwd", "moe_mx4_quantize", "moe_mx4_packed_bytes",
               "moe_mx4_pack", "moe_mx4_prepack", "moe_mx4_product_workspace_bytes",
               "moe_mx4_expert_product", "moe_mx4_layer_workspace_bytes", "moe_mx4_layer_fwd",
               "moe_grouped_workspace_bytes", "moe_grouped_product", "moe_grouped_weight_grad",
               "moe_swiglu", "moe_swiglu_bwd", "moe_expert_ffn_bwd_workspace_bytes",
               "moe_expert_ffn_bwd", "moe_orthogonalize_workspace_bytes", "moe_orthogonalize")


class moe_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32)]

    def __repr__(self):
        return f"moe_dims(T={self.T}, H={self.H}, E={self.E}, k={self.k}, I={self.I})"


def dims(T, H, E, k, I) -> moe_dims:
    return moe_dims(T, H, E, k, I)


MOE_ROUTER_SOFTMAX, MOE_ROUTER_SIGMOID_BIAS_SELECT = 0, 1


class moe_router_opts(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("weights_bf16", ctypes.c_int32),
                ("route_scale", ctypes.c_float)]


def router_opts(kind=MOE_ROUTER_SOFTMAX, weights_bf16=False, route_scale=1.0) -> moe_router_opts:
    return moe_router_opts(int(kind), int(bool(weights_bf16)), float(route_scale))


MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1, 2
_DTYPES = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16,
           torch.float16: MOE_DTYPE_F16}


class moe_select_opts(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32)]


def select_opts(kind=MOE_ROUTER_SOFTMAX, n_group=1, topk_group=1, group_top=1,
                renorm=True) -> moe_select_opts:
    return moe_select_opts(int(kind), int(n_group), int(topk_group), int(group_top),
                           int(bool(renorm)))


def _opts(o):
    return None if o is None else ctypes.byref(o)


def _select(o):
    if o is not None and not isinstance(o, moe_select_opts):
        raise TypeError(f"opts: a select_opts, not {type(o).__name__}")
    return o


_vp, _sz, _i32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_sig = {
    "moe_workspace_bytes": (_sz, [moe_dims]),
    "moe_packed_weight_bytes": (_sz, [moe_dims]),
    "moe_route": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp, _vp]),
    "moe_load_stats": (ctypes.c_int, [_vp, moe_dims, _vp, _vp, _vp, _sz, _vp]),
    "moe_load_summary_host": (ctypes.c_int, [_vp, _i32, _vp, _vp]),
    "moe_permute": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_prepack_expert_weights": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _sz, _vp]),
    "moe_expert_ffn": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp, _sz, _vp]),
    "moe_combine": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp]),
    "moe_layer_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
    "moe_layer_fwd_profiled": (ctypes.c_int, [_vp, _vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp,
                                              _vp, _sz, _vp, _vp, _i32]),
    "moe_read_device_status": (ctypes.c_int, [_vp, _vp, _vp]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_load_stats_noalloc": (ctypes.c_int, [_vp, moe_dims, _vp, _vp, _vp, _vp]),
    "moe_set_wait_limit": (ctypes.c_int, [ctypes.c_longlong]),
    "moe_route_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, moe_dims, _vp, _vp, _vp]),
    "moe_combine_ex": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_float, moe_dims, _vp, _vp]),
    "moe_layer_fwd_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp,
                                        _vp, _sz, _vp]),
    "moe_load_stats_ex": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_lpt_placement_host": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp]),
    "moe_rank_load_summary_host": (ctypes.c_int, [_vp, _i32, _vp, _vp]),
    "moe_permute_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, moe_dims, _vp, _vp, _vp, _vp, _sz,
                                      _vp]),
    "moe_prepack_expert_weights_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, moe_dims, _vp, _sz,
                                                     _vp]),
    "moe_combine_sharded": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, ctypes.c_float, _vp,
                                           moe_dims, _vp, _vp, _vp]),
    "moe_tree_reduce_bf16": (ctypes.c_int, [_vp, _i32, ctypes.c_int64, _vp, _vp]),
    "moe_shared_packed_bytes": (_sz, [_i32, _i32]),
    "moe_expert_ffn_form": (ctypes.c_int, [moe_dims]),
    "moe_prepack_shared_expert": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _sz, _vp]),
    "moe_shared_expert_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_shared_expert": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _sz, _vp]),
    "moe_sharded_workspace_bytes": (_sz, [moe_dims, _i32, _i32]),
    "moe_layer_fwd_sharded": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                             moe_dims, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_layer_fwd_sharded_profiled": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                                      _i32, moe_dims, _vp, _vp, _vp, _vp, _vp,
                                                      _sz, _vp, _vp, _i32]),
    "moe_router_logits": (ctypes.c_int, [_vp, _vp, _vp, moe_dims, _vp, _vp]),
    "moe_select_workspace_bytes": (_sz, [_i32, _i32]),
    "moe_route_select": (ctypes.c_int, [_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp,
                                        _vp, _sz, _vp]),
    "moe_route_select_bwd": (ctypes.c_int, [_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                                            _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "moe_mx4_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp]),
    "moe_mx4_packed_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_mx4_pack": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, _sz, _vp]),
    "moe_mx4_prepack": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _sz, _vp]),
    "moe_mx4_product_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_mx4_expert_product": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                              _i32, _vp, _sz, _vp]),
    "moe_mx4_layer_workspace_bytes": (_sz, [moe_dims]),
    "moe_mx4_layer_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, moe_dims,
                                         _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_grouped_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_grouped_product": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _i64, _i64, _i32, _i32, _i32,
                                           _i32, _i32, _vp, _i64, _i32, _vp, _sz, _vp]),
    "moe_grouped_weight_grad": (ctypes.c_int, [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i32, _i32,
                                               _i32, _vp, _i64, _i64, _i32, _i32, _vp, _sz, _vp]),
    "moe_swiglu": (ctypes.c_int, [_vp, _i64, _vp, _i32, _i32, _i32, _vp, _i64, _vp]),
    "moe_swiglu_bwd": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _vp, _i64, _vp,
                                      _i64, _vp, _vp]),
    "moe_expert_ffn_bwd_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_expert_ffn_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                          _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _sz,
                                          _vp]),
    "moe_orthogonalize_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_orthogonalize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _i32,
                                         ctypes.c_float, ctypes.c_float, _vp, _i32, _i64, _i64, _vp,
                                         _sz, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class MoEError(RuntimeError):
    def __init__(self, name, code):
        self.code = code
        super().__init__(f"{name}: {STATUS.get(code, code)} "
                         f"({_lib.moe_status_string(code).decode()})")


def _check(name, code):
    if code != MOE_OK:
        raise MoEError(name, code)


def _ptr(t):
    """Device address of a tensor (None -> NULL); an int is taken as an address."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's address and the current device without the Python stream object
# (2.9 us against 0.1 us a call on the GB300's host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ws(ws):
    return (_ptr(ws), ws.numel() * ws.element_size()) if isinstance(ws, torch.Tensor) else ws


# ------------------------------------------------------------ raw ABI calls ---
def moe_workspace_bytes(d: moe_dims) -> int:
    return int(_lib.moe_workspace_bytes(d))


def moe_packed_weight_bytes(d: moe_dims) -> int:
    return int(_lib.moe_packed_weight_bytes(d))


def moe_route(x, w_router, bias, d, topk_idx, topk_w, stream=None):
    _check("moe_route", _lib.moe_route(_ptr(x), _ptr(w_router), _ptr(bias), d, _ptr(topk_idx),
                                       _ptr(topk_w), _stream(stream)))


def moe_route_ex(x, w_router, bias, opts, d, topk_idx, topk_w, stream=None):
    _check("moe_route_ex", _lib.moe_route_ex(_ptr(x), _ptr(w_router), _ptr(bias), _opts(opts), d,
                                             _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


def moe_combine_ex(y, topk_w, row_of_slot, route_scale, d, out, stream=None):
    _check("moe_combine_ex", _lib.moe_combine_ex(_ptr(y), _ptr(topk_w), _ptr(row_of_slot),
                                                 float(route_scale), d, _ptr(out),
                                                 _stream(stream)))


def moe_layer_fwd_ex(x, w_router, bias, opts, packed_weights, d, out, topk_idx_out, topk_w_out,
                     counts_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_layer_fwd_ex", _lib.moe_layer_fwd_ex(
        _ptr(x), _ptr(w_router), _ptr(bias), _opts(opts), _ptr(packed_weights), d, _ptr(out),
        _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), wp, wb, _stream(stream)))


def moe_load_stats(topk_idx, d, counts, offsets, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_load_stats", _lib.moe_load_stats(_ptr(topk_idx), d, _ptr(counts), _ptr(offsets),
                                                 wp, wb, _stream(stream)))


def moe_load_stats_noalloc(topk_idx, d, counts, offsets, device_status=None, stream=None):
    """moe_load_stats without a workspace, for callers that cannot allocate: the
    library's own fixed scratch array holds the partial counts (see include/moe.h
    for the size limit and the rule that overlapping calls race)."""
    _check("moe_load_stats_noalloc", _lib.moe_load_stats_noalloc(
        _ptr(topk_idx), d, _ptr(counts), _ptr(offsets), _ptr(device_status), _stream(stream)))


def moe_load_stats_ex(topk_idx, slot_of_expert, q, d, counts, offsets, weighted_counts,
                      workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_load_stats_ex", _lib.moe_load_stats_ex(
        _ptr(topk_idx), _ptr(slot_of_expert), _ptr(q), d, _ptr(counts), _ptr(offsets),
        _ptr(weighted_counts), wp, wb, _stream(stream)))


def moe_lpt_placement_host(loads, P):
    """(slot_of_expert [E] int32, rank_loads [P] int64) from host loads (RoutePack Alg. 1)."""
    import numpy as np
    L = np.ascontiguousarray(loads, dtype=np.int64)
    pi = np.empty(L.size, dtype=np.int32)
    G = np.empty(P, dtype=np.int64)
    _check("moe_lpt_placement_host", _lib.moe_lpt_placement_host(
        L.ctypes.data, int(L.size), int(P), pi.ctypes.data, G.ctypes.data))
    return pi, G


def moe_rank_load_summary_host(rank_loads):
    """(cv, eta_ep) of host rank loads."""
    import numpy as np
    G = np.ascontiguousarray(rank_loads, dtype=np.int64)
    cv, eta = ctypes.c_double(), ctypes.c_double()
    _check("moe_rank_load_summary_host", _lib.moe_rank_load_summary_host(
        G.ctypes.data, int(G.size), ctypes.addressof(cv), ctypes.addressof(eta)))
    return cv.value, eta.value


def moe_permute_ex(x, topk_idx, slot_of_expert, offsets, d, x_perm, row_of_slot, slot_of_row,
                   workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_permute_ex", _lib.moe_permute_ex(
        _ptr(x), _ptr(topk_idx), _ptr(slot_of_expert), _ptr(offsets), d, _ptr(x_perm),
        _ptr(row_of_slot), _ptr(slot_of_row), wp, wb, _stream(stream)))


def moe_prepack_expert_weights_ex(w_gate, w_up, w_down, slot_of_expert, d, packed, stream=None):
    nbytes = packed.numel() * packed.element_size() if isinstance(packed, torch.Tensor) else 1 << 62
    _check("moe_prepack_expert_weights_ex", _lib.moe_prepack_expert_weights_ex(
        _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(slot_of_expert), d, _ptr(packed), nbytes,
        _stream(stream)))


def moe_combine_sharded(y, topk_w, topk_idx, row_of_slot, owner, G, route_scale, shared, d, out,
                        partials=None, stream=None):
    """Per-rank BF16 partials (slots of other ranks as exact zeros, optional
    shared-expert shards [G, T, H] fp32) reduced by the fixed FP64 pairwise tree."""
    _check("moe_combine_sharded", _lib.moe_combine_sharded(
        _ptr(y), _ptr(topk_w), _ptr(topk_idx), _ptr(row_of_slot), _ptr(owner), int(G),
        float(route_scale), _ptr(shared), d, _ptr(partials), _ptr(out), _stream(stream)))


def moe_tree_reduce_bf16(partials, G, N, out, stream=None):
    """out [N] = bf16(FP64 pairwise tree over partials [G, N]) (bf16 tensors)."""
    _check("moe_tree_reduce_bf16", _lib.moe_tree_reduce_bf16(_ptr(partials), int(G), int(N),
                                                             _ptr(out), _stream(stream)))


def moe_shared_packed_bytes(H, Is) -> int:
    return int(_lib.moe_shared_packed_bytes(int(H), int(Is)))


def moe_shared_expert_workspace_bytes(T, H, Is, G) -> int:
    return int(_lib.moe_shared_expert_workspace_bytes(int(T), int(H), int(Is), int(G)))


def moe_prepack_shared_expert(w_gate, w_up, w_down, H, Is, G, packed, stream=None):
    nbytes = packed.numel() * packed.element_size() if isinstance(packed, torch.Tensor) else 1 << 62
    _check("moe_prepack_shared_expert", _lib.moe_prepack_shared_expert(
        _ptr(w_gate), _ptr(w_up), _ptr(w_down), int(H), int(Is), int(G), _ptr(packed), nbytes,
        _stream(stream)))


def moe_shared_expert(x, shared_packed, T, H, Is, G, shared_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_shared_expert", _lib.moe_shared_expert(
        _ptr(x), _ptr(shared_packed), int(T), int(H), int(Is), int(G), _ptr(shared_out), wp, wb,
        _stream(stream)))


def moe_sharded_workspace_bytes(d, G, Is=0) -> int:
    return int(_lib.moe_sharded_workspace_bytes(d, int(G), int(Is)))


def moe_layer_fwd_sharded(x, w_router, bias, opts, packed_weights, owner, G, shared_packed, Is, d,
                          out, topk_idx_out, topk_w_out, counts_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_layer_fwd_sharded", _lib.moe_layer_fwd_sharded(
        _ptr(x), _ptr(w_router), _ptr(bias), _opts(opts), _ptr(packed_weights), _ptr(owner),
        int(G), _ptr(shared_packed), int(Is), d, _ptr(out), _ptr(topk_idx_out), _ptr(topk_w_out),
        _ptr(counts_out), wp, wb, _stream(stream)))


def _event_array(events, stream):
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event on its first record
            e.record(torch.cuda.current_stream() if stream is None else stream)
    return (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])


def moe_layer_fwd_sharded_profiled(x, w_router, bias, opts, packed_weights, owner, G,
                                   shared_packed, Is, d, out, topk_idx_out, topk_w_out, counts_out,
                                   workspace, events, stream=None):
    """moe_layer_fwd_sharded with 7 torch.cuda.Event(enable_timing=True) recorded at
    the step boundaries (as moe_layer_fwd_profiled)."""
    wp, wb = _ws(workspace)
    arr = _event_array(events, stream)
    _check("moe_layer_fwd_sharded_profiled", _lib.moe_layer_fwd_sharded_profiled(
        _ptr(x), _ptr(w_router), _ptr(bias), _opts(opts), _ptr(packed_weights), _ptr(owner),
        int(G), _ptr(shared_packed), int(Is), d, _ptr(out), _ptr(topk_idx_out), _ptr(topk_w_out),
        _ptr(counts_out), wp, wb, _stream(stream), arr, len(events)))


def moe_load_summary_host(counts_host):
    """(imbalance max/mean - 1, cv) from host counts (sequence or numpy array)."""
    import numpy as np
    c = np.ascontiguousarray(counts_host, dtype=np.int32)
    imb, cv = ctypes.c_double(), ctypes.c_double()
    _check("moe_load_summary_host", _lib.moe_load_summary_host(
        c.ctypes.data, int(c.size), ctypes.addressof(imb), ctypes.addressof(cv)))
    return imb.value, cv.value


def moe_permute(x, topk_idx, offsets, d, x_perm, row_of_slot, slot_of_row, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_permute", _lib.moe_permute(_ptr(x), _ptr(topk_idx), _ptr(offsets), d, _ptr(x_perm),
                                           _ptr(row_of_slot), _ptr(slot_of_row), wp, wb,
                                           _stream(stream)))


def moe_prepack_expert_weights(w_gate, w_up, w_down, d, packed, stream=None):
    nbytes = packed.numel() * packed.element_size() if isinstance(packed, torch.Tensor) else 1 << 62
    _check("moe_prepack_expert_weights", _lib.moe_prepack_expert_weights(
        _ptr(w_gate), _ptr(w_up), _ptr(w_down), d, _ptr(packed), nbytes, _stream(stream)))


def moe_expert_ffn(x_perm, offsets, packed_weights, d, y, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_expert_ffn", _lib.moe_expert_ffn(_ptr(x_perm), _ptr(offsets), _ptr(packed_weights),
                                                 d, _ptr(y), wp, wb, _stream(stream)))


def moe_expert_ffn_form(d):
    """0: tile GEMMs, 1: swapped GEMMs (weight rows on the MMA's M side)."""
    r = _lib.moe_expert_ffn_form(d)
    if r < 0:
        raise MoEError("moe_expert_ffn_form", -r)
    return r


def moe_combine(y, topk_w, row_of_slot, d, out, stream=None):
    _check("moe_combine", _lib.moe_combine(_ptr(y), _ptr(topk_w), _ptr(row_of_slot), d, _ptr(out),
                                           _stream(stream)))


def moe_layer_fwd(x, w_router, bias, packed_weights, d, out, topk_idx_out, topk_w_out, counts_out,
                  workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_layer_fwd", _lib.moe_layer_fwd(
        _ptr(x), _ptr(w_router), _ptr(bias), _ptr(packed_weights), d, _ptr(out),
        _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), wp, wb, _stream(stream)))


def moe_layer_fwd_profiled(x, w_router, bias, packed_weights, d, out, topk_idx_out, topk_w_out,
                           counts_out, workspace, events, stream=None):
    """``events``: 7 torch.cuda.Event(enable_timing=True) recorded at the step
    boundaries (before route, after route, load stats, permute, gate/up GEMM,
    down GEMM, combine)."""
    wp, wb = _ws(workspace)
    arr = _event_array(events, stream)
    _check("moe_layer_fwd_profiled", _lib.moe_layer_fwd_profiled(
        _ptr(x), _ptr(w_router), _ptr(bias), _ptr(packed_weights), d, _ptr(out),
        _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), wp, wb, _stream(stream), arr,
        len(events)))


def moe_router_logits(x, w_router, bias, d, logits, stream=None):
    _check("moe_router_logits", _lib.moe_router_logits(_ptr(x), _ptr(w_router), _ptr(bias), d,
                                                       _ptr(logits), _stream(stream)))


def moe_select_workspace_bytes(T, E) -> int:
    return int(_lib.moe_select_workspace_bytes(int(T), int(E)))


def _ws_or_none(ws):
    return (None, 0) if ws is None else _ws(ws)


def moe_route_select(logits, dtype, ld, bias, opts, T, E, k, topk_idx, topk_w, prob_sum=None,
                     workspace=None, stream=None):
    wp, wb = _ws_or_none(workspace)
    _check("moe_route_select", _lib.moe_route_select(
        _ptr(logits), int(dtype), int(ld), _ptr(bias), _opts(_select(opts)), int(T), int(E), int(k),
        _ptr(topk_idx), _ptr(topk_w), _ptr(prob_sum), wp, wb, _stream(stream)))


def moe_route_select_bwd(logits, dtype, ld, bias, opts, T, E, k, topk_idx, d_topk_w, d_prob_sum,
                         d_logits, ld_d, d_bias=None, workspace=None, stream=None):
    wp, wb = _ws_or_none(workspace)
    _check("moe_route_select_bwd", _lib.moe_route_select_bwd(
        _ptr(logits), int(dtype), int(ld), _ptr(bias), _opts(_select(opts)), int(T), int(E), int(k),
        _ptr(topk_idx), _ptr(d_topk_w), _ptr(d_prob_sum), _ptr(d_logits), int(ld_d), _ptr(d_bias),
        wp, wb, _stream(stream)))


def moe_mx4_quantize(x, dtype, ld, R, K, codes, scales, values, stream=None):
    _check("moe_mx4_quantize", _lib.moe_mx4_quantize(
        _ptr(x), int(dtype), int(ld), int(R), int(K), _ptr(codes), _ptr(scales), _ptr(values),
        _stream(stream)))


def moe_mx4_packed_bytes(E, K, N) -> int:
    return int(_lib.moe_mx4_packed_bytes(int(E), int(K), int(N)))


def moe_mx4_pack(codes, scales, E, K, N, packed, stream=None):
    nbytes = packed.numel() * packed.element_size() if isinstance(packed, torch.Tensor) else 1 << 62
    _check("moe_mx4_pack", _lib.moe_mx4_pack(_ptr(codes), _ptr(scales), int(E), int(K), int(N),
                                             _ptr(packed), nbytes, _stream(stream)))


def moe_mx4_prepack(w, E, K, N, col0, N_total, packed, stream=None):
    nbytes = packed.numel() * packed.element_size() if isinstance(packed, torch.Tensor) else 1 << 62
    _check("moe_mx4_prepack", _lib.moe_mx4_prepack(_ptr(w), int(E), int(K), int(N), int(col0),
                                                   int(N_total), _ptr(packed), nbytes,
                                                   _stream(stream)))


def moe_mx4_product_workspace_bytes(R, K, E) -> int:
    return int(_lib.moe_mx4_product_workspace_bytes(int(R), int(K), int(E)))


def moe_mx4_expert_product(x, x_dtype, offsets, packed, R, K, N, E, y, y_dtype, workspace,
                           stream=None):
    wp, wb = _ws(workspace)
    _check("moe_mx4_expert_product", _lib.moe_mx4_expert_product(
        _ptr(x), int(x_dtype), _ptr(offsets), _ptr(packed), int(R), int(K), int(N), int(E),
        _ptr(y), int(y_dtype), wp, wb, _stream(stream)))


def moe_mx4_layer_workspace_bytes(d: moe_dims) -> int:
    return int(_lib.moe_mx4_layer_workspace_bytes(d))


def moe_mx4_layer_fwd(x, w_router, bias, opts, route_scale, packed_gate_up, packed_down, d, out,
                      topk_idx_out, topk_w_out, counts_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_mx4_layer_fwd", _lib.moe_mx4_layer_fwd(
        _ptr(x), _ptr(w_router), _ptr(bias), _opts(_select(opts)), float(route_scale),
        _ptr(packed_gate_up), _ptr(packed_down), d, _ptr(out), _ptr(topk_idx_out),
        _ptr(topk_w_out), _ptr(counts_out), wp, wb, _stream(stream)))


def moe_grouped_workspace_bytes(E, K, N) -> int:
    return int(_lib.moe_grouped_workspace_bytes(int(E), int(K), int(N)))


def moe_grouped_product(x, x_ld, dtype, offsets, w, w_ld, w_es, transposed, R, K, N, E, y, y_ld,
                        y_dtype, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_grouped_product", _lib.moe_grouped_product(
        _ptr(x), int(x_ld), int(dtype), _ptr(offsets), _ptr(w), int(w_ld), int(w_es),
        int(bool(transposed)), int(R), int(K), int(N), int(E), _ptr(y), int(y_ld), int(y_dtype), wp,
        wb, _stream(stream)))


def moe_grouped_weight_grad(x, x_ld, dy, dy_ld, dtype, offsets, R, K, N, E, d_w, w_ld, w_es,
                            w_dtype, accumulate, workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_grouped_weight_grad", _lib.moe_grouped_weight_grad(
        _ptr(x), int(x_ld), _ptr(dy), int(dy_ld), int(dtype), _ptr(offsets), int(R), int(K), int(N),
        int(E), _ptr(d_w), int(w_ld), int(w_es), int(w_dtype), int(bool(accumulate)), wp, wb,
        _stream(stream)))


def moe_swiglu(gate_up, gate_up_ld, row_w, dtype, R, I, h, h_ld, stream=None):
    _check("moe_swiglu", _lib.moe_swiglu(_ptr(gate_up), int(gate_up_ld), _ptr(row_w), int(dtype),
                                         int(R), int(I), _ptr(h), int(h_ld), _stream(stream)))


def moe_swiglu_bwd(gate_up, gate_up_ld, d_h, d_ld, row_w, dtype, R, I, d_gate_up, d_gate_up_ld,
                   h=None, h_ld=0, d_row_w=None, stream=None):
    _check("moe_swiglu_bwd", _lib.moe_swiglu_bwd(
        _ptr(gate_up), int(gate_up_ld), _ptr(d_h), int(d_ld), _ptr(row_w), int(dtype), int(R),
        int(I), _ptr(d_gate_up), int(d_gate_up_ld), _ptr(h), int(h_ld), _ptr(d_row_w),
        _stream(stream)))


def moe_expert_ffn_bwd_workspace_bytes(R, H, I, E) -> int:
    return int(_lib.moe_expert_ffn_bwd_workspace_bytes(int(R), int(H), int(I), int(E)))


def moe_expert_ffn_bwd(x_perm, offsets, w_gate_up, w_down, gate_up, row_w, d_y, dtype, R, H, I, E,
                       d_x_perm, d_x_dtype, d_w_gate_up, d_w_down, d_w_dtype, accumulate, d_row_w,
                       workspace, stream=None):
    wp, wb = _ws(workspace)
    _check("moe_expert_ffn_bwd", _lib.moe_expert_ffn_bwd(
        _ptr(x_perm), _ptr(offsets), _ptr(w_gate_up), _ptr(w_down), _ptr(gate_up), _ptr(row_w),
        _ptr(d_y), int(dtype), int(R), int(H), int(I), int(E), _ptr(d_x_perm), int(d_x_dtype),
        _ptr(d_w_gate_up), _ptr(d_w_down), int(d_w_dtype), int(bool(accumulate)), _ptr(d_row_w), wp,
        wb, _stream(stream)))


def moe_orthogonalize_workspace_bytes(E, rows, cols) -> int:
    return int(_lib.moe_orthogonalize_workspace_bytes(int(E), int(rows), int(cols)))


def moe_orthogonalize(m, dtype, ld, es, E, rows, cols, coefficients, steps, eps, scale, out,
                      out_dtype, out_ld, out_es, workspace, stream=None):
    wp, wb = _ws(workspace)
    co = None if coefficients is None else (ctypes.c_float * 3)(*coefficients)
    _check("moe_orthogonalize", _lib.moe_orthogonalize(
        _ptr(m), int(dtype), int(ld), int(es), int(E), int(rows), int(cols), co, int(steps),
        float(eps), float(scale), _ptr(out), int(out_dtype), int(out_ld), int(out_es), wp, wb,
        _stream(stream)))


def moe_set_wait_limit(cycles: int) -> None:
    """Diagnostics: bounded-wait limit of the GEMM kernels (<= 0: default)."""
    _check("moe_set_wait_limit", _lib.moe_set_wait_limit(int(cycles)))


def moe_read_device_status(workspace, stream=None) -> int:
    v = ctypes.c_int32()
    wp, _ = _ws(workspace)
    _check("moe_read_device_status", _lib.moe_read_device_status(wp, ctypes.addressof(v),
                                                                 _stream(stream)))
    return v.value


# ------------------------------------------------- allocation conveniences ---
# (torch's allocator supplies the memory; the library itself allocates nothing)
def new_workspace(d: moe_dims, device="cuda") -> torch.Tensor:
    """Zeroed workspace of moe_workspace_bytes(d) bytes (256-byte aligned by torch)."""
    n = moe_workspace_bytes(d)
    if n == 0:
        raise MoEError("moe_workspace_bytes", 2)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def prepack(w_gate, w_up, w_down, d, stream=None) -> torch.Tensor:
    packed = torch.empty(moe_packed_weight_bytes(d) // 2, dtype=torch.bfloat16,
                         device=w_gate.device)
    moe_prepack_expert_weights(w_gate, w_up, w_down, d, packed, stream)
    return packed


def layer_forward(x, w_router, bias, packed, d, workspace, stream=None, want_routing=False,
                  opts=None):
    """out [T, H] bf16 (and topk_idx, topk_w, counts if want_routing).  opts: a
    moe_router_opts (router variant, bf16 weights, routing scale) or None."""
    dev = x.device
    out = torch.empty((d.T, d.H), dtype=torch.bfloat16, device=dev)
    idx = w = counts = None
    if want_routing:
        idx = torch.empty((d.T, d.k), dtype=torch.int32, device=dev)
        w = torch.empty((d.T, d.k), dtype=torch.float32, device=dev)
        counts = torch.empty(d.E, dtype=torch.int32, device=dev)
    moe_layer_fwd_ex(x, w_router, bias, opts, packed, d, out, idx, w, counts, workspace, stream)
    return (out, idx, w, counts) if want_routing else out


def _dtype(name, t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: float32, bfloat16 or float16, not {t.dtype}")
    return code


def _rows(name, t, cols=None):
    """Row stride of a 2D tensor whose elements within a row are adjacent."""
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: a 2D tensor" + (f" of {cols} columns" if cols else "")
                         + f", not {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent (stride {t.stride()})")
    if t.shape[0] <= 1:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows must not overlap (stride {t.stride()})")
    return t.stride(0)


def _tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor, not {type(t).__name__}")
    return t


def _dense(name, t, dtype, shape):
    if _tensor(name, t).dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: a dense {dtype} tensor of shape {tuple(shape)}, not "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()}")
    return t


def _buffer(name, t, nbytes=None, of=""):
    """A dense tensor of any type; of exactly nbytes, if given."""
    if not _tensor(name, t).is_contiguous():
        raise ValueError(f"{name}: a dense tensor, not strides {t.stride()}")
    n = t.numel() * t.element_size()
    if nbytes is not None and n != nbytes:
        raise ValueError(f"{name}: {n} bytes, not the {nbytes} of {of}")
    return t


def _on_device(first, *rest):
    """All tensors on the current CUDA device (the one the library launches on)."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    if dev != _get_device():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{_get_device()}")


def _on_stream(stream):
    """Context in which `stream` (a torch stream or an address) is current: what a call
    allocates then belongs to the stream that its kernels run on."""
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream) if stream
                  else torch.cuda.default_stream())
    return torch.cuda.stream(stream)


# The tensor calls below first try _tensor_calls, which makes the whole call for arguments of
# the plain kind (dense tensors on the current device and stream); it returns None for others,
# which are then handled or refused here.  On small batches the host's part of a call is longer
# than the kernel's.
def _logits_args(logits, bias):
    """(type code, row stride, T, E) of logits [T, E]; refuses what a kernel would misread."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        _dtype("logits", logits)
    if logits.dim() == 2 and logits.is_contiguous():
        T, ld = logits.shape
    else:
        ld, T = _rows("logits", logits), logits.shape[0]
    E = logits.shape[1]
    if T >= 1 << 31:
        raise ValueError(f"logits: at most 2^31 - 1 tokens, not {T}")
    if bias is not None:
        _dense("bias", bias, torch.float32, (E,))
    return dt, ld, T, E


def _choice_args(name, T, E, k):
    """The library's limits on a choice of k of E experts, before anything of that size is allocated."""
    if E <= 0 or k <= 0 or k > E:
        raise MoEError(name, 1)
    if E > 256 or k > 16 or T * k >= 1 << 31:
        raise MoEError(name, 2)


def _made(name, r):
    """What a _tensor_calls function returned: its result, or the status of a refusal."""
    if type(r) is int:
        _check(name, r)
    return r


_default_opts = select_opts()


def route_select(logits, k, opts=None, bias=None, want_prob_sum=False, stream=None):
    """(topk_idx [T, k] int32, topk_w [T, k] fp32[, prob_sum [E] fp32]) from logits [T, E]
    (fp32, bf16 or fp16).  opts: a select_opts (default: softmax over all experts).

    Not part of autograd: the results carry no gradient, whatever the logits require.  A
    training step calls route_select_backward (as in examples/mx4_layer.py), or wraps the two
    in a torch.autograd.Function."""
    if stream is not None:
        with _on_stream(stream):
            return route_select(logits, k, opts, bias, want_prob_sum)
    opts = _default_opts if opts is None else _select(opts)
    r = _calls.route_select(logits, k, opts, bias, bool(want_prob_sum))
    if r is not None:
        return _made("moe_route_select", r)
    dt, ld, T, E = _logits_args(logits, bias)
    _choice_args("moe_route_select", T, E, k)
    _on_device(logits, bias)
    dev = logits.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    prob = pp = wp = None
    n = 0
    if want_prob_sum:
        prob = torch.empty(E, dtype=torch.float32, device=dev)
        n = moe_select_workspace_bytes(T, E)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pp, wp = prob.data_ptr(), ws.data_ptr()
    r = _lib.moe_route_select(
        logits.data_ptr(), dt, ld, None if bias is None else bias.data_ptr(),
        ctypes.byref(opts), T, E, k, idx.data_ptr(),
        w.data_ptr(), pp, wp, n, _stream(stream))
    if r:
        _check("moe_route_select", r)
    return (idx, w, prob) if want_prob_sum else (idx, w)


def route_select_backward(logits, topk_idx, d_topk_w, opts=None, bias=None, d_prob_sum=None,
                          want_d_bias=False, stream=None):
    """d_logits [T, E] in the logits' type (and d_bias [E] fp32 if want_d_bias, softmax only)
    for d_topk_w [T, k] and, if given, d_prob_sum [E], both fp32; the choice stays fixed.
    The gradient itself: nothing is recorded for or taken from autograd."""
    if stream is not None:
        with _on_stream(stream):
            return route_select_backward(logits, topk_idx, d_topk_w, opts, bias, d_prob_sum,
                                         want_d_bias)
    opts = _default_opts if opts is None else _select(opts)
    r = _calls.route_select_backward(logits, topk_idx, d_topk_w, opts, bias, d_prob_sum,
                                     bool(want_d_bias))
    if r is not None:
        return _made("moe_route_select_bwd", r)
    dt, ld, T, E = _logits_args(logits, bias)
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx: [T, k], not {tuple(topk_idx.shape)}")
    k = topk_idx.shape[1]
    _dense("topk_idx", topk_idx, torch.int32, (T, k))
    _dense("d_topk_w", d_topk_w, torch.float32, (T, k))
    if d_prob_sum is not None:
        _dense("d_prob_sum", d_prob_sum, torch.float32, (E,))
    _on_device(logits, topk_idx, d_topk_w, bias, d_prob_sum)
    dev = logits.device
    d_logits = torch.empty((T, E), dtype=logits.dtype, device=dev)
    d_bias = bp = wp = None
    n = 0
    if want_d_bias:
        d_bias = torch.empty(E, dtype=torch.float32, device=dev)
        n = moe_select_workspace_bytes(T, E)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        bp, wp = d_bias.data_ptr(), ws.data_ptr()
    r = _lib.moe_route_select_bwd(
        logits.data_ptr(), dt, ld, None if bias is None else bias.data_ptr(),
        ctypes.byref(opts), T, E, k, topk_idx.data_ptr(),
        d_topk_w.data_ptr(), None if d_prob_sum is None else d_prob_sum.data_ptr(),
        d_logits.data_ptr(), E, bp, wp, n, _stream(stream))
    if r:
        _check("moe_route_select_bwd", r)
    return (d_logits, d_bias) if want_d_bias else d_logits


def mx4_quantize(x, want_values=False, stream=None):
    """(codes [R, K/2] uint8, scales [R, K/32] uint8[, values [R, K] bf16]) of rows x [R, K]
    (fp32, bf16 or fp16), K a multiple of 32.  Not part of autograd."""
    if stream is not None:
        with _on_stream(stream):
            return mx4_quantize(x, want_values)
    r = _calls.mx4_quantize(x, bool(want_values))
    if r is not None:
        return _made("moe_mx4_quantize", r)
    dt, ld, R, K = _x_args(x)
    dev = x.device
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, K // 32), dtype=torch.uint8, device=dev)
    values = torch.empty((R, K), dtype=torch.bfloat16, device=dev) if want_values else None
    r = _lib.moe_mx4_quantize(x.data_ptr(), dt, ld, R, K, codes.data_ptr(), scales.data_ptr(),
                              values.data_ptr() if want_values else None, _stream(stream))
    if r:
        _check("moe_mx4_quantize", r)
    return (codes, scales, values) if want_values else (codes, scales)


def _x_args(x):
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        _dtype("x", x)
    if x.dim() == 2 and x.is_contiguous():
        R, K = x.shape
        ld = K
    else:
        ld = _rows("x", x)
        R, K = x.shape
    _on_device(x)
    return dt, ld, R, K


def mx4_pack(codes, scales, stream=None) -> torch.Tensor:
    """Packed operand from checkpoint tensors codes [E, N, K/2] and scales [E, N, K/32]."""
    if stream is not None:
        with _on_stream(stream):
            return mx4_pack(codes, scales)
    if codes.dim() != 3:
        raise ValueError(f"codes: [E, N, K/2], not {tuple(codes.shape)}")
    E, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    _dense("codes", codes, torch.uint8, (E, N, K // 2))
    _dense("scales", scales, torch.uint8, (E, N, K // 32))
    _on_device(codes, scales)
    n = moe_mx4_packed_bytes(E, K, N)
    if n == 0:
        raise MoEError("moe_mx4_packed_bytes", 2)
    packed = torch.empty(n, dtype=torch.uint8, device=codes.device)
    moe_mx4_pack(codes, scales, E, K, N, packed, stream)
    return packed


def mx4_prepack(*weights, stream=None) -> torch.Tensor:
    """Packed operand from bf16 weights [E, K, N_i] in the logical layout, quantised along K;
    several (gate, up) lie side by side in one operand of sum(N_i) columns."""
    if stream is not None:
        with _on_stream(stream):
            return mx4_prepack(*weights)
    if not weights or any(w.dim() != 3 for w in weights):
        raise ValueError("weights: one or more [E, K, N] tensors")
    E, K = weights[0].shape[:2]
    N_total = sum(w.shape[2] for w in weights)
    for w in weights:
        _dense("weights", w, torch.bfloat16, (E, K, w.shape[2]))
    _on_device(*weights)
    n = moe_mx4_packed_bytes(E, K, N_total)
    if n == 0:
        raise MoEError("moe_mx4_packed_bytes", 2)
    packed = torch.empty(n, dtype=torch.uint8, device=weights[0].device)
    col = 0
    for w in weights:
        moe_mx4_prepack(w, E, K, w.shape[2], col, N_total, packed, stream)
        col += w.shape[2]
    return packed


def _zeroed(n, name, device):
    if n == 0:
        raise MoEError(name, 2)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the status word; the rest is scratch
    return ws


def mx4_new_workspace(R, K, N, E, device="cuda") -> torch.Tensor:
    """Workspace of mx4_expert_product for up to R rows."""
    return _zeroed(moe_mx4_product_workspace_bytes(R, K, E), "moe_mx4_product_workspace_bytes",
                   device)


def mx4_expert_product(x, offsets, packed, N, workspace, dtype=torch.bfloat16, stream=None):
    """y [R, N] (bf16 or fp32): rows x [R, K] of each expert (offsets [E+1] int32) quantised to
    microscaled 4 bits, times the expert's packed weights."""
    if stream is not None:
        with _on_stream(stream):
            return mx4_expert_product(x, offsets, packed, N, workspace, dtype)
    if dtype is torch.bfloat16 or dtype is torch.float32:
        r = _calls.mx4_expert_product(x, offsets, packed, N, workspace, dtype is torch.bfloat16)
        if r is not None:
            return _made("moe_mx4_expert_product", r)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"x: a dense [R, K] tensor, not {tuple(x.shape)} strides {x.stride()}")
    dt = _dtype("x", x)
    if offsets.dim() != 1:
        raise ValueError(f"offsets: [E + 1], not {tuple(offsets.shape)}")
    E, (R, K) = offsets.numel() - 1, x.shape
    if R >= 1 << 31:
        raise ValueError(f"x: at most 2^31 - 1 rows, not {R}")
    _dense("offsets", offsets, torch.int32, (E + 1,))
    _buffer("packed", packed, moe_mx4_packed_bytes(E, K, N), f"{E} experts of {K} x {N}")
    _buffer("workspace", workspace)
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"y: float32 or bfloat16, not {dtype}")
    _on_device(x, offsets, packed, workspace)
    y = torch.empty((R, N), dtype=dtype, device=x.device)
    r = _lib.moe_mx4_expert_product(
        x.data_ptr(), dt, offsets.data_ptr(), packed.data_ptr(), R, K, N, E, y.data_ptr(),
        _DTYPES[dtype], workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream))
    if r:
        _check("moe_mx4_expert_product", r)
    return y


def mx4_new_layer_workspace(d: moe_dims, device="cuda") -> torch.Tensor:
    return _zeroed(moe_mx4_layer_workspace_bytes(d), "moe_mx4_layer_workspace_bytes", device)


def mx4_layer_forward(x, w_router, bias, packed_gate_up, packed_down, d, workspace, opts=None,
                      route_scale=1.0, want_routing=False, stream=None):
    """out [T, H] bf16 (and topk_idx, topk_w, counts if want_routing) of the layer with
    microscaled 4-bit experts."""
    if stream is not None:
        with _on_stream(stream):
            return mx4_layer_forward(x, w_router, bias, packed_gate_up, packed_down, d, workspace,
                                     opts, route_scale, want_routing)
    opts = _default_opts if opts is None else _select(opts)
    for name, t, dt, shape in (("x", x, torch.bfloat16, (d.T, d.H)),
                               ("w_router", w_router, torch.float32, (d.H, d.E)),
                               ("bias", bias, torch.float32, (d.E,))):
        if t is not None or name != "bias":
            _dense(name, _buffer(name, t), dt, shape)
    up, down = moe_mx4_packed_bytes(d.E, d.H, 2 * d.I), moe_mx4_packed_bytes(d.E, d.I, d.H)
    if up and down:  # (else the dims are outside the limits, which the call below refuses)
        _buffer("packed_gate_up", packed_gate_up, up, f"{d.E} experts of {d.H} x {2 * d.I}")
        _buffer("packed_down", packed_down, down, f"{d.E} experts of {d.I} x {d.H}")
        _buffer("workspace", workspace)
        _on_device(x, w_router, bias, packed_gate_up, packed_down, workspace)
    dev = x.device
    out = torch.empty((d.T, d.H), dtype=torch.bfloat16, device=dev)
    idx = w = counts = None
    if want_routing:
        idx = torch.empty((d.T, d.k), dtype=torch.int32, device=dev)
        w = torch.empty((d.T, d.k), dtype=torch.float32, device=dev)
        counts = torch.empty(d.E, dtype=torch.int32, device=dev)
    moe_mx4_layer_fwd(x, w_router, bias, opts, route_scale, packed_gate_up, packed_down, d, out, idx,
                      w, counts, workspace, stream)
    return (out, idx, w, counts) if want_routing else out


# ------------------------------------------------------ training the experts ---
# (as the calls above: not part of autograd; a training step calls the gradients itself)
def _stack(name, t, dtype, shape):
    """(row stride, matrix stride) of a 3D tensor of rows of adjacent elements."""
    _tensor(name, t)
    if (dtype is not None and t.dtype != dtype) or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    E, rows, cols = shape
    if cols > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent (stride {t.stride()})")
    ld = t.stride(1) if rows > 1 else cols
    es = t.stride(0) if E > 1 else rows * ld
    if ld < cols or es < rows * ld:
        raise ValueError(f"{name}: rows and matrices must not overlap (stride {t.stride()})")
    return ld, es


def _rows16(name, t, dtype, shape):
    """Row stride of a 2D tensor of this 16-bit type and shape."""
    _tensor(name, t)
    if t.dtype not in (torch.bfloat16, torch.float16) or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name}: {dtype or 'bfloat16 or float16'}, not {t.dtype}")
    if t.dim() != 2 or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: {tuple(shape)}, not {tuple(t.shape)}")
    if t.shape[0] >= 1 << 31 or t.shape[1] >= 1 << 31:
        raise ValueError(f"{name}: at most 2^31 - 1 rows and columns, not {tuple(t.shape)}")
    return _rows(name, t)


def _grouped_limits(name, R, E, K, N, widest=None):
    """The library's limits on grouped calls, before anything of that size is allocated.  widest: the widest
    product of the call, if not N."""
    n = N if widest is None else widest
    if (moe_grouped_workspace_bytes(E, K, N) == 0 or R > (1 << 31) - 512
            or (R // 128 + E + 1) * ((n + 127) // 128) >= 1 << 30):
        raise MoEError(name, 2)


def _offsets(offsets):
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: a tensor [E + 1]")
    _dense("offsets", offsets, torch.int32, (offsets.numel(),))
    return offsets.numel() - 1


def grouped_new_workspace(E, K, N, device="cuda") -> torch.Tensor:
    """Workspace of grouped_product and grouped_weight_grad with E experts of K x N (either way
    round), for any number of rows."""
    return _zeroed(moe_grouped_workspace_bytes(E, K, N), "moe_grouped_workspace_bytes", device)


def grouped_product(x, offsets, w, workspace, transposed=False, dtype=None, out=None, stream=None):
    """y [R, N] (fp32, bf16 or fp16; default: x's type): the rows x [R, K] (bf16 or fp16) of each
    expert (offsets [E+1] int32) times its matrix of w [E, K, N], or w [E, N, K] if transposed,
    of x's type.  out: written instead of a new tensor (no bytes of the inputs).  Not part of autograd:
    the gradients are this call with the other `transposed`, and grouped_weight_grad."""
    if stream is not None:
        with _on_stream(stream):
            return grouped_product(x, offsets, w, workspace, transposed, dtype, out)
    if out is None and isinstance(x, torch.Tensor):
        r = _calls.grouped_product(x, offsets, w, workspace, bool(transposed),
                                   _DTYPES.get(x.dtype if dtype is None else dtype))
        if r is not None:
            return _made("moe_grouped_product", r)
    E = _offsets(offsets)
    x_ld = _rows16("x", x, None, (None, None))
    R, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w: a tensor [E, K, N] or [E, N, K]")
    N = w.shape[1] if transposed else w.shape[2]
    w_ld, w_es = _stack("w", w, x.dtype, (E, N, K) if transposed else (E, K, N))
    _buffer("workspace", workspace)
    if out is None:
        _on_device(x, offsets, w, workspace)
        dtype = x.dtype if dtype is None else dtype
        if dtype not in _DTYPES:
            raise TypeError(f"y: float32, bfloat16 or float16, not {dtype}")
        _grouped_limits("moe_grouped_product", R, E, K, N)
        out, y_ld = torch.empty((R, N), dtype=dtype, device=x.device), N
    else:
        _on_device(x, offsets, w, workspace, _tensor("out", out))
        if dtype not in (None, out.dtype):
            raise TypeError(f"out: {dtype}, not {out.dtype}")
        _dtype("out", out)
        y_ld = _rows("out", out, N)
        if out.shape[0] != R:
            raise ValueError(f"out: {R} rows, not {out.shape[0]}")
    moe_grouped_product(x, x_ld, _DTYPES[x.dtype], offsets, w, w_ld, w_es, transposed, R, K, N, E,
                        out, y_ld, _DTYPES[out.dtype], workspace)
    return out


def grouped_weight_grad(x, dy, offsets, workspace, dtype=torch.float32, out=None, accumulate=False,
                        stream=None):
    """d_w [E, K, N] (fp32, bf16 or fp16): the sums over each expert's rows of x [R, K]^T dy [R, N]
    (both bf16 or both fp16); zeros for an expert without rows.  out: written instead of a new
    tensor, or, with accumulate (fp32 only), added to."""
    if stream is not None:
        with _on_stream(stream):
            return grouped_weight_grad(x, dy, offsets, workspace, dtype, out, accumulate)
    if out is None and not accumulate:
        r = _calls.grouped_weight_grad(x, dy, offsets, workspace, _DTYPES.get(dtype))
        if r is not None:
            return _made("moe_grouped_weight_grad", r)
    E = _offsets(offsets)
    x_ld = _rows16("x", x, None, (None, None))
    R, K = x.shape
    dy_ld = _rows16("dy", dy, x.dtype, (R, None))
    N = dy.shape[1]
    _buffer("workspace", workspace)
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out")
        _on_device(x, dy, offsets, workspace)
        if dtype not in _DTYPES:
            raise TypeError(f"d_w: float32, bfloat16 or float16, not {dtype}")
        _grouped_limits("moe_grouped_weight_grad", R, E, K, N)
        out, w_ld, w_es = torch.empty((E, K, N), dtype=dtype, device=x.device), N, K * N
    else:
        _on_device(x, dy, offsets, workspace, _tensor("out", out))
        _dtype("out", out)
        w_ld, w_es = _stack("out", out, None, (E, K, N))
    moe_grouped_weight_grad(x, x_ld, dy, dy_ld, _DTYPES[x.dtype], offsets, R, K, N, E, out, w_ld,
                            w_es, _DTYPES[out.dtype], accumulate, workspace)
    return out


def _gate_up_args(gate_up, row_weights):
    ld = _rows16("gate_up", gate_up, None, (None, None))
    R, n = gate_up.shape
    if n % 2:
        raise ValueError(f"gate_up: [R, 2 I], not {tuple(gate_up.shape)}")
    if n // 2 % 8 or n // 2 > 1 << 24:
        raise MoEError("moe_swiglu", 2)
    if row_weights is not None:
        _dense("row_weights", row_weights, torch.float32, (R,))
    return ld, R, n // 2


def swiglu(gate_up, row_weights=None, stream=None):
    """h [R, I] = row_weights * silu(gate) * up of gate_up [R, 2 I] (bf16 or fp16, gate first), one
    rounding."""
    if stream is not None:
        with _on_stream(stream):
            return swiglu(gate_up, row_weights)
    r = _calls.swiglu(gate_up, row_weights)
    if r is not None:
        return _made("moe_swiglu", r)
    ld, R, I = _gate_up_args(gate_up, row_weights)
    _on_device(gate_up, row_weights)
    h = torch.empty((R, I), dtype=gate_up.dtype, device=gate_up.device)
    moe_swiglu(gate_up, ld, row_weights, _DTYPES[gate_up.dtype], R, I, h, I)
    return h


def swiglu_backward(gate_up, d_h, row_weights=None, stream=None):
    """(d_gate_up [R, 2 I], h [R, I][, d_row_weights [R] fp32 if row_weights]) for d_h [R, I], the
    gradient of swiglu's result h, which is computed again."""
    if stream is not None:
        with _on_stream(stream):
            return swiglu_backward(gate_up, d_h, row_weights)
    r = _calls.swiglu_backward(gate_up, d_h, row_weights)
    if r is not None:
        return _made("moe_swiglu_bwd", r)
    ld, R, I = _gate_up_args(gate_up, row_weights)
    d_ld = _rows16("d_h", d_h, gate_up.dtype, (R, I))
    _on_device(gate_up, d_h, row_weights)
    d_gate_up = torch.empty((R, 2 * I), dtype=gate_up.dtype, device=gate_up.device)
    h = torch.empty((R, I), dtype=gate_up.dtype, device=gate_up.device)
    d_w = None if row_weights is None else torch.empty(R, dtype=torch.float32, device=gate_up.device)
    moe_swiglu_bwd(gate_up, ld, d_h, d_ld, row_weights, _DTYPES[gate_up.dtype], R, I, d_gate_up,
                   2 * I, h, I, d_w)
    return (d_gate_up, h) if d_w is None else (d_gate_up, h, d_w)


def expert_ffn_backward_new_workspace(R, H, I, E, device="cuda") -> torch.Tensor:
    """Workspace of expert_ffn_backward for up to R rows."""
    return _zeroed(moe_expert_ffn_bwd_workspace_bytes(R, H, I, E),
                   "moe_expert_ffn_bwd_workspace_bytes", device)


def expert_ffn_backward(x_perm, offsets, w_gate_up, w_down, d_y, workspace, row_weights=None,
                        gate_up=None, d_x_dtype=None, d_w_dtype=torch.float32, d_w_gate_up=None,
                        d_w_down=None, accumulate=False, stream=None):
    """(d_x_perm [R, H], d_w_gate_up [E, H, 2 I], d_w_down [E, I, H][, d_row_weights [R] fp32 if
    row_weights]): the experts' backward pass for d_y [R, H], the gradient of the layer's output
    for each row's token (moe_permute's rows of it).  x_perm [R, H], w_gate_up [E, H, 2 I] (gate
    columns first), w_down [E, I, H], all dense and bf16 or all fp16; gate_up [R, 2 I] as
    grouped_product gave it, or None: computed again.  d_w_gate_up and d_w_down: written instead
    of new tensors, or, with accumulate (fp32 only), added to."""
    if stream is not None:
        with _on_stream(stream):
            return expert_ffn_backward(x_perm, offsets, w_gate_up, w_down, d_y, workspace,
                                       row_weights, gate_up, d_x_dtype, d_w_dtype, d_w_gate_up,
                                       d_w_down, accumulate)
    E = _offsets(offsets)
    _rows16("x_perm", x_perm, None, (None, None))
    dt, (R, H) = x_perm.dtype, x_perm.shape
    if not isinstance(w_gate_up, torch.Tensor) or w_gate_up.dim() != 3 or w_gate_up.shape[2] % 2:
        raise ValueError("w_gate_up: a tensor [E, H, 2 I]")
    I = w_gate_up.shape[2] // 2
    for name, t, shape in (("x_perm", x_perm, (R, H)), ("d_y", d_y, (R, H)),
                           ("w_gate_up", w_gate_up, (E, H, 2 * I)), ("w_down", w_down, (E, I, H)),
                           ("gate_up", gate_up, (R, 2 * I))):
        if t is not None or name != "gate_up":
            _dense(name, _buffer(name, t), dt, shape)
    if row_weights is not None:
        _dense("row_weights", row_weights, torch.float32, (R,))
    _buffer("workspace", workspace)
    d_x_dtype = dt if d_x_dtype is None else d_x_dtype
    if d_x_dtype not in _DTYPES or d_w_dtype not in _DTYPES:
        raise TypeError("gradients: float32, bfloat16 or float16")
    given = [t for t in (d_w_gate_up, d_w_down) if t is not None]
    if accumulate and len(given) < 2:
        raise ValueError("accumulate: needs d_w_gate_up and d_w_down")
    for name, t, shape in (("d_w_gate_up", d_w_gate_up, (E, H, 2 * I)),
                           ("d_w_down", d_w_down, (E, I, H))):
        if t is not None:
            _dense(name, t, d_w_dtype, shape)
    _on_device(x_perm, offsets, w_gate_up, w_down, d_y, workspace, row_weights, gate_up, *given)
    if moe_expert_ffn_bwd_workspace_bytes(R, H, I, E) == 0:
        raise MoEError("moe_expert_ffn_bwd", 2)
    _grouped_limits("moe_expert_ffn_bwd", R, E, H, I, max(H, 2 * I))
    dev = x_perm.device
    d_x = torch.empty((R, H), dtype=d_x_dtype, device=dev)
    if d_w_gate_up is None:
        d_w_gate_up = torch.empty((E, H, 2 * I), dtype=d_w_dtype, device=dev)
    if d_w_down is None:
        d_w_down = torch.empty((E, I, H), dtype=d_w_dtype, device=dev)
    d_w = None if row_weights is None else torch.empty(R, dtype=torch.float32, device=dev)
    moe_expert_ffn_bwd(x_perm, offsets, w_gate_up, w_down, gate_up, row_weights, d_y, _DTYPES[dt], R,
                       H, I, E, d_x, _DTYPES[d_x_dtype], d_w_gate_up, d_w_down, _DTYPES[d_w_dtype],
                       accumulate, d_w, workspace)
    out = (d_x, d_w_gate_up, d_w_down)
    return out if d_w is None else out + (d_w,)


def orthogonalize_new_workspace(E, rows, cols, device="cuda") -> torch.Tensor:
    """Workspace of orthogonalize for a stack of E matrices (either way round)."""
    return _zeroed(moe_orthogonalize_workspace_bytes(E, rows, cols),
                   "moe_orthogonalize_workspace_bytes", device)


def orthogonalize(m, workspace, coefficients=(3.4445, -4.7750, 2.0315), steps=5, eps=1e-7,
                  scale=1.0, dtype=torch.bfloat16, out=None, stream=None):
    """[E, rows, cols] (bf16 or fp16): scale times the matrices m [E, rows, cols] (fp32, bf16 or
    fp16) orthogonalised by `steps` Newton-Schulz steps X <- a X + (b X X^T + c (X X^T)^2) X from
    X = m / (|m| + eps).  out: written instead of a new tensor (m itself, too)."""
    if stream is not None:
        with _on_stream(stream):
            return orthogonalize(m, workspace, coefficients, steps, eps, scale, dtype, out)
    if out is None and len(coefficients) == 3:
        r = _calls.orthogonalize(m, workspace, *coefficients, steps, eps, scale, _DTYPES.get(dtype))
        if r is not None:
            return _made("moe_orthogonalize", r)
    if not isinstance(m, torch.Tensor) or m.dim() != 3:
        raise ValueError("m: a tensor [E, rows, cols]")
    code = _dtype("m", m)
    E, rows, cols = m.shape
    if moe_orthogonalize_workspace_bytes(E, rows, cols) == 0:
        raise MoEError("moe_orthogonalize", 2)
    ld, es = _stack("m", m, m.dtype, m.shape)
    coefficients = tuple(float(v) for v in coefficients)
    if len(coefficients) != 3:
        raise ValueError(f"coefficients: three, not {len(coefficients)}")
    _buffer("workspace", workspace)
    if out is None:
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"out: bfloat16 or float16, not {dtype}")
        _on_device(m, workspace)
        out, o_ld, o_es = torch.empty((E, rows, cols), dtype=dtype, device=m.device), cols, rows * cols
    else:
        if _tensor("out", out).dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"out: bfloat16 or float16, not {out.dtype}")
        _on_device(m, workspace, out)
        o_ld, o_es = _stack("out", out, None, m.shape)
    moe_orthogonalize(m, code, ld, es, E, rows, cols, coefficients, steps, eps, scale, out,
                      _DTYPES[out.dtype], o_ld, o_es, workspace)
    return out


def layer_forward_host_batches(x_host_batches, w_router, bias, packed, d, out_host_batches,
                               workspace, stream=None, layer=None):
    """Forward a sequence of token batches that live in pinned host memory, writing each
    batch's output back to pinned host memory.

    Transfers overlap compute: batch i+1 is copied to the device on one copy stream
    while batch i runs (moe_layer_fwd on `stream`, default the current stream), and
    batch i's output is copied back on a second copy stream while batch i+1 runs.
    Two device buffers per direction rotate.  Every batch must have d.T tokens.
    layer: optional callable (x_dev, out_dev, stream) that runs one forward in place
    of moe_layer_fwd (e.g. moe_layer_fwd_sharded with its own arguments bound).
    Returns once all work is enqueued; synchronise `stream` (or the last event) to
    read the outputs.
    """
    compute = torch.cuda.current_stream() if stream is None else stream
    dev = torch.device("cuda", torch.cuda.current_device())
    h2d, d2h = torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev)
    h2d.wait_stream(compute)  # nothing starts before work already queued on the caller's stream
    x_dev = [torch.empty((d.T, d.H), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    o_dev = [torch.empty((d.T, d.H), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    copied_in = [torch.cuda.Event() for _ in range(2)]
    computed = [torch.cuda.Event() for _ in range(2)]
    copied_out = [torch.cuda.Event() for _ in range(2)]
    used = [False, False]
    for i, (xh, oh) in enumerate(zip(x_host_batches, out_host_batches)):
        b = i & 1
        if used[b]:
            h2d.wait_event(computed[b])        # batch i-2 no longer reads x_dev[b]
        with torch.cuda.stream(h2d):
            x_dev[b].copy_(xh, non_blocking=True)
            copied_in[b].record(h2d)
        compute.wait_event(copied_in[b])
        if used[b]:
            compute.wait_event(copied_out[b])  # batch i-2's output has left o_dev[b]
        if layer is None:
            moe_layer_fwd(x_dev[b], w_router, bias, packed, d, o_dev[b], None, None, None,
                          workspace, compute)
        else:
            layer(x_dev[b], o_dev[b], compute)
        computed[b].record(compute)
        d2h.wait_event(computed[b])
        with torch.cuda.stream(d2h):
            oh.copy_(o_dev[b], non_blocking=True)
            copied_out[b].record(d2h)
        used[b] = True
    for e in copied_out:
        compute.wait_event(e)                  # the caller's stream covers the last copies
    for t in x_dev + o_dev:
        t.record_stream(h2d)
        t.record_stream(d2h)
    return compute
