"""ctypes binding of ``libmoe_gb300.so`` (the C ABI in ``include/moe_gb300.h``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are ``torch`` CUDA tensors (device memory); ``None`` passes a
NULL pointer.  The stream defaults to torch's current stream.  A non-OK status
raises ``MoEError``.  There is no fallback: if the library is missing, importing
this module fails.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK = 0
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_CUDA",
          -4: "MOE_ERR_WORKSPACE_TOO_SMALL", -5: "MOE_ERR_TIMEOUT", -6: "MOE_ERR_DEVICE_BOUNDS",
          -7: "MOE_ERR_MISALIGNED", -8: "MOE_ERR_RANGE", -9: "MOE_ERR_BAD_PACK"}
DTYPES = {"f32": 0, "bf16": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
NORMS = {"none": 0, "l1": 1, "softmax_selected": 2, "lp": 3}
SHARED_MODES = {"none": 0, "const": 1, "gate": 2}
CAP_POLICIES = {"none": 0, "per_expert": 1, "rank_wide": 2}
H_FORMATS = {"bf16": 0, "f16": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LAYERNORM_KINDS = {"layer": 0, "rms": 1}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({_lib.moe_status_string(status).decode()})")


class moe_config(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d_model", c_int32), ("N", c_int32), ("K", c_int32),
                ("d_expert", c_int32), ("d_shared", c_int32), ("dtype", c_int32),
                ("score", c_int32), ("norm", c_int32), ("alpha", c_float),
                ("shared_mode", c_int32), ("shared_gain", c_float), ("cap_policy", c_int32),
                ("capacity_factor", c_double), ("num_ranks", c_int32), ("rho", POINTER(c_int32)),
                ("norm_p", c_float), ("h_format", c_int32), ("h_scale_log2", c_int32)]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("W_router", "router_bias", "selection_bias", "shared_gate_w",
                                        "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down")]


class moe_linear_config(ctypes.Structure):
    _fields_ = [("T", c_int64), ("in_features", c_int32), ("out_features", c_int32),
                ("dtype", c_int32), ("out_dtype", c_int32), ("act", c_int32), ("dx_dtype", c_int32),
                ("dw_dtype", c_int32), ("ldx", c_int64), ("ldw", c_int64), ("ldr", c_int64),
                ("ldy", c_int64)]


class moe_dropout_config(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("cols", c_int64), ("p", c_double), ("x_dtype", c_int32),
                ("residual_dtype", c_int32), ("y_dtype", c_int32), ("ldx", c_int64), ("ldr", c_int64),
                ("ldy", c_int64)]


class moe_layernorm_config(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d", c_int32), ("kind", c_int32), ("eps", c_float), ("x_dtype", c_int32),
                ("stream_dtype", c_int32), ("y_dtype", c_int32), ("w_dtype", c_int32), ("ldx", c_int64),
                ("ldr", c_int64), ("lds", c_int64), ("ldy", c_int64)]


class moe_embedding_config(ctypes.Structure):
    _fields_ = [("T", c_int64), ("V", c_int64), ("d", c_int32), ("ids_int64", c_int32),
                ("table_dtype", c_int32), ("out_dtype", c_int32), ("scale", c_float), ("ldt", c_int64),
                ("ldo", c_int64)]


class moe_tensor(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("rows", c_int64), ("cols", c_int64), ("ld", c_int64), ("dtype", c_int32)]


GRAD_FIELDS = ("dx", "dW_gate", "dW_up", "dW_down", "dWs_gate", "dWs_up", "dWs_down", "dW_router",
               "dshared_gate_w")


class moe_grads(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in GRAD_FIELDS]


OUTPUT_FIELDS = ("y", "topk_idx", "topk_w", "shared_coef", "logits", "counts_req", "counts_keep",
                 "offsets", "route_pos", "perm_src", "R_req", "R_keep", "drop_stats")


class moe_outputs(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in OUTPUT_FIELDS]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python routing_shared_expert_gb300/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    C = POINTER(moe_config)
    sig = {
        "moe_version": ([], c_char_p),
        "moe_status_string": ([c_int32], c_char_p),
        "moe_workspace_size": ([C, POINTER(c_size_t)], c_int32),
        "moe_workspace_init": ([P, c_size_t, P], c_int32),
        "moe_packed_weights_size": ([c_int64, POINTER(c_size_t)], c_int32),
        "moe_pack_weights": ([P, c_int64, P, c_size_t, P], c_int32),
        "moe_route": ([C, P, P, P, P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_balance_stats": ([C, P, P, P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_bias_update": ([c_int32, P, c_float, P, P], c_int32),
        "moe_permute": ([C, P, P, P, P, P, P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_permute_noalloc": ([C, P, P, P, P, P, P, P, P, P, P, P, P], c_int32),
        "moe_grouped_swiglu": ([C, P, P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_shared_mlp": ([C, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_combine": ([C, P, P, P, P, P, P, P], c_int32),
        "moe_layer_forward": ([C, POINTER(moe_weights), P, POINTER(moe_outputs), P, c_size_t, P], c_int32),
        "moe_layer_forward_profiled": ([C, POINTER(moe_weights), P, POINTER(moe_outputs), P, c_size_t, P,
                                        POINTER(c_void_p)], c_int32),
        "moe_merge_shared": ([c_int32, c_int32, c_int32, POINTER(c_int32), POINTER(c_void_p),
                              POINTER(c_void_p), POINTER(c_void_p), P, P, P, P], c_int32),
        "moe_read_status": ([P, POINTER(c_int32), P], c_int32),
        "moe_check_wait_bound": ([P, c_size_t, c_int64, P], c_int32),
        "moe_ep_keep_matrix": ([c_int32, c_int32, c_int32, POINTER(c_int32), c_int32, c_double, P, P,
                                P, P, P, P], c_int32),
        "moe_ep_place": ([c_int32, c_int32, c_int64, c_int32, c_int32, P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_ep_keep_matrix_host": ([c_int32, c_int32, c_int32, POINTER(c_int32), c_int32, c_double, P,
                                     P, P, P, P], c_int32),
        "moe_ep_place_host": ([c_int32, c_int32, c_int64, c_int32, c_int32, P, P, P, P], c_int32),
        "moe_ep_send_pos": ([c_int32, c_int32, c_int64, c_int32, c_int32, POINTER(c_int32), P, P, P,
                             P, P, P, P, c_size_t, P], c_int32),
        "moe_ep_recv_rows": ([c_int32, c_int32, c_int32, POINTER(c_int32), P, P, P, c_int64, P,
                              c_size_t, P], c_int32),
        "moe_rows_copy": ([P, c_int64, P, c_int64, P, c_int64, P, c_int64, c_int64, c_int32, P,
                           c_size_t, P], c_int32),
        "moe_ep_send_pos_host": ([c_int32, c_int32, c_int64, c_int32, c_int32, POINTER(c_int32), P,
                                  P, P, P, P, P], c_int32),
        "moe_ep_recv_rows_host": ([c_int32, c_int32, c_int32, POINTER(c_int32), P, P, P, c_int64],
                                  c_int32),
        "moe_rows_copy_host": ([P, c_int64, P, c_int64, P, c_int64, P, c_int64, c_int64, c_int32],
                               c_int32),
        "moe_backward_workspace_size": ([C, POINTER(c_size_t)], c_int32),
        "moe_layer_backward": ([C, POINTER(moe_weights), P, POINTER(moe_outputs), P, POINTER(moe_grads),
                                P, c_size_t, P], c_int32),
        "moe_layer_backward_aux": ([C, POINTER(moe_weights), P, POINTER(moe_outputs), P, P,
                                    POINTER(moe_grads), P, c_size_t, P], c_int32),
        "moe_linear_workspace_size": ([POINTER(moe_linear_config), POINTER(c_size_t)], c_int32),
        "moe_linear_forward": ([POINTER(moe_linear_config), P, P, P, P, P, P, P, c_size_t, P], c_int32),
        "moe_linear_backward": ([POINTER(moe_linear_config), P, P, P, P, P, P, P, P, c_size_t, P],
                                c_int32),
        "moe_dropout_add": ([POINTER(moe_dropout_config), P, P, P, P, P], c_int32),
        "moe_dropout_backward": ([POINTER(moe_dropout_config), P, P, P, P], c_int32),
        # the configurations of the calls below come packed by struct
        "moe_layernorm_forward": ([P, P, P, P, P, P, P, P, P, P], c_int32),
        "moe_layernorm_workspace_size": ([c_int64, c_int32, POINTER(c_size_t)], c_int32),
        "moe_layernorm_backward": ([P, P, P, P, P, P, P, P, P, P, P, c_size_t, P],
                                   c_int32),
        "moe_embedding_workspace_size": ([c_int64, c_int64, c_int32, POINTER(c_size_t)], c_int32),
        "moe_embedding_forward": ([P, P, P, P, P, c_size_t, P], c_int32),
        "moe_embedding_backward": ([P, P, P, P, c_int32, P, c_size_t, P], c_int32),
        "moe_grad_norm_workspace_size": ([POINTER(c_size_t)], c_int32),
        "moe_grad_norm": ([P, c_int32, c_float, P, P, c_size_t, P], c_int32),
        "moe_clip_grad_norm": ([P, P, c_int32, c_float, P, P, c_size_t, P], c_int32),
        "moe_balance_loss_workspace_size": ([C, c_int64, POINTER(c_size_t)], c_int32),
        "moe_balance_loss": ([C, P, P, P, c_int64, c_float, c_float, P, P, P, P, P, P, c_size_t, P],
                             c_int32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library():
    """The loaded ``ctypes.CDLL``."""
    return _lib


def version() -> str:
    return _lib.moe_version().decode()


def _enum(table, v):
    return table[v] if isinstance(v, str) else int(v)


def make_config(T, d_model, N, K, d_expert, d_shared, dtype="bf16", score="softmax", norm="l1",
                alpha=1.0, shared_mode="const", shared_gain=1.0, cap_policy="none",
                capacity_factor=1.0, num_ranks=1, rho=None, norm_p=2.0, h_format="bf16",
                h_scale_log2=0) -> moe_config:
    """Build a ``moe_config``; ``rho`` (host list) is kept alive on the returned object."""
    c = moe_config()
    c.T, c.d_model, c.N, c.K = int(T), int(d_model), int(N), int(K)
    c.d_expert, c.d_shared = int(d_expert), int(d_shared)
    c.dtype = _enum(DTYPES, dtype)
    c.score = _enum(SCORES, score)
    c.norm = _enum(NORMS, norm)
    c.alpha = float(alpha)
    c.shared_mode = _enum(SHARED_MODES, shared_mode)
    c.shared_gain = float(shared_gain)
    c.cap_policy = _enum(CAP_POLICIES, cap_policy)
    c.capacity_factor = float(capacity_factor)
    c.num_ranks = int(num_ranks)
    c.norm_p = float(norm_p)
    c.h_format = _enum(H_FORMATS, h_format)
    c.h_scale_log2 = int(h_scale_log2)
    if rho is not None:
        arr = (c_int32 * len(rho))(*[int(v) for v in rho])
        c._rho_keepalive = arr
        c.rho = ctypes.cast(arr, POINTER(c_int32))
    return c


def copy_config(cfg: moe_config, **changes) -> moe_config:
    """A copy of ``cfg`` (sharing its host ``rho`` array) with some fields changed."""
    c = moe_config()
    ctypes.memmove(ctypes.byref(c), ctypes.byref(cfg), ctypes.sizeof(moe_config))
    if hasattr(cfg, "_rho_keepalive"):
        c._rho_keepalive = cfg._rho_keepalive
    for k, v in changes.items():
        setattr(c, k, v)
    return c


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return c_void_p(t)
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        # the raw handle, without building a Stream object at every call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return c_void_p(stream)
    return c_void_p(stream.cuda_stream)


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status)


def moe_workspace_size(cfg: moe_config) -> int:
    n = c_size_t(0)
    _check("moe_workspace_size", _lib.moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def moe_workspace_init(workspace, stream=None):
    _check("moe_workspace_init", _lib.moe_workspace_init(_ptr(workspace), workspace.numel(), _stream(stream)))


def alloc_workspace(cfg: moe_config, device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) large enough for every entry point of ``cfg``."""
    import torch
    ws = torch.empty(max(moe_workspace_size(cfg), 256), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_packed_weights_size(elements: int) -> int:
    n = c_size_t(0)
    _check("moe_packed_weights_size", _lib.moe_packed_weights_size(int(elements), ctypes.byref(n)))
    return int(n.value)


def moe_pack_weights(W, packed, stream=None):
    """Pack the bf16 tensor W into ``packed`` (uint8 device tensor) for the fp16 intermediate."""
    _check("moe_pack_weights", _lib.moe_pack_weights(_ptr(W), W.numel(), _ptr(packed), packed.numel(),
                                                     _stream(stream)))


def pack_weights(W, stream=None):
    """A new packed buffer (uint8 device tensor) holding W for the fp16 intermediate."""
    import torch
    packed = torch.empty(moe_packed_weights_size(W.numel()), dtype=torch.uint8, device=W.device)
    moe_pack_weights(W, packed, stream)
    return packed


def moe_route(cfg, x, W_router, router_bias, selection_bias, shared_gate_w, topk_idx, topk_w,
              shared_coef, logits, workspace, stream=None):
    _check("moe_route", _lib.moe_route(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(router_bias), _ptr(selection_bias),
        _ptr(shared_gate_w), _ptr(topk_idx), _ptr(topk_w), _ptr(shared_coef), _ptr(logits),
        _ptr(workspace), workspace.numel(), _stream(stream)))


STATS = ("lbl", "imax_req", "imax_keep", "imax_rank_req", "imax_rank_keep", "ih_req", "ih_keep",
         "cv_req", "never_selected", "drop_fraction")


def moe_balance_stats(cfg, logits, counts_req, counts_keep, R_req, R_keep, P, f, stats, workspace,
                      stream=None):
    """stats: float32 [len(STATS)] device tensor, indexed as STATS."""
    _check("moe_balance_stats", _lib.moe_balance_stats(
        ctypes.byref(cfg), _ptr(logits), _ptr(counts_req), _ptr(counts_keep), _ptr(R_req),
        _ptr(R_keep), _ptr(P), _ptr(f), _ptr(stats), _ptr(workspace), workspace.numel(),
        _stream(stream)))


def moe_bias_update(N, counts, gamma, bias, stream=None):
    _check("moe_bias_update", _lib.moe_bias_update(int(N), _ptr(counts), float(gamma), _ptr(bias),
                                                    _stream(stream)))


def moe_permute(cfg, x, topk_idx, counts_req, counts_keep, offsets, route_pos, perm_src, x_perm,
                R_req, R_keep, drop_stats, workspace, stream=None):
    _check("moe_permute", _lib.moe_permute(
        ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(counts_req), _ptr(counts_keep),
        _ptr(offsets), _ptr(route_pos), _ptr(perm_src), _ptr(x_perm), _ptr(R_req), _ptr(R_keep),
        _ptr(drop_stats), _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_permute_noalloc(cfg, x, topk_idx, counts_req, counts_keep, offsets, route_pos, perm_src,
                        x_perm, R_req, R_keep, drop_stats, stream=None):
    """moe_permute for callers that cannot allocate: no workspace (see the C header)."""
    _check("moe_permute_noalloc", _lib.moe_permute_noalloc(
        ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(counts_req), _ptr(counts_keep),
        _ptr(offsets), _ptr(route_pos), _ptr(perm_src), _ptr(x_perm), _ptr(R_req), _ptr(R_keep),
        _ptr(drop_stats), _stream(stream)))


def moe_grouped_swiglu(cfg, x_rows, offsets, perm_src, W_gate, W_up, W_down, f, workspace,
                       stream=None):
    """x_rows is x_perm when perm_src is None, else x (rows gathered through perm_src)."""
    _check("moe_grouped_swiglu", _lib.moe_grouped_swiglu(
        ctypes.byref(cfg), _ptr(x_rows), _ptr(offsets), _ptr(perm_src), _ptr(W_gate), _ptr(W_up),
        _ptr(W_down), _ptr(f), _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_shared_mlp(cfg, x, Ws_gate, Ws_up, Ws_down, g, workspace, stream=None):
    _check("moe_shared_mlp", _lib.moe_shared_mlp(
        ctypes.byref(cfg), _ptr(x), _ptr(Ws_gate), _ptr(Ws_up), _ptr(Ws_down), _ptr(g),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_combine(cfg, f, route_pos, topk_w, g, shared_coef, y, stream=None):
    _check("moe_combine", _lib.moe_combine(
        ctypes.byref(cfg), _ptr(f), _ptr(route_pos), _ptr(topk_w), _ptr(g), _ptr(shared_coef),
        _ptr(y), _stream(stream)))


def make_weights(W_router, router_bias, shared_gate_w, W_gate, W_up, W_down, Ws_gate=None,
                 Ws_up=None, Ws_down=None, selection_bias=None) -> moe_weights:
    w = moe_weights()
    keep = []
    for name, t in (("W_router", W_router), ("router_bias", router_bias),
                    ("selection_bias", selection_bias),
                    ("shared_gate_w", shared_gate_w), ("W_gate", W_gate), ("W_up", W_up),
                    ("W_down", W_down), ("Ws_gate", Ws_gate), ("Ws_up", Ws_up), ("Ws_down", Ws_down)):
        p = _ptr(t)
        setattr(w, name, p.value if p is not None else None)
        keep.append(t)
    w._keepalive = keep
    return w


def make_outputs(**tensors) -> moe_outputs:
    o = moe_outputs()
    for name in OUTPUT_FIELDS:
        t = tensors.get(name)
        p = _ptr(t)
        setattr(o, name, p.value if p is not None else None)
    o._keepalive = list(tensors.values())
    return o


def moe_layer_forward(cfg, weights: moe_weights, x, outputs: moe_outputs, workspace, stream=None):
    _check("moe_layer_forward", _lib.moe_layer_forward(
        ctypes.byref(cfg), ctypes.byref(weights), _ptr(x), ctypes.byref(outputs), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def moe_layer_forward_profiled(cfg, weights: moe_weights, x, outputs: moe_outputs, workspace, events,
                               stream=None):
    """moe_layer_forward recording 5 torch.cuda.Event objects (created with enable_timing):
    before the router and after the router, the permutation, the routed experts and the
    shared expert + combine."""
    handles = []
    for ev in events:
        if ev.cuda_event == 0:       # torch creates the event on first record
            ev.record()
        handles.append(ev.cuda_event)
    arr = (c_void_p * 5)(*handles)
    _check("moe_layer_forward_profiled", _lib.moe_layer_forward_profiled(
        ctypes.byref(cfg), ctypes.byref(weights), _ptr(x), ctypes.byref(outputs), _ptr(workspace),
        workspace.numel(), _stream(stream), arr))


def moe_merge_shared(d_model, dtype, gate_parts, up_parts, down_parts, Ws_gate, Ws_up, Ws_down,
                     stream=None):
    n = len(gate_parts)
    widths = (c_int32 * n)(*[int(t.shape[0]) for t in gate_parts])
    gp = (c_void_p * n)(*[t.data_ptr() for t in gate_parts])
    up = (c_void_p * n)(*[t.data_ptr() for t in up_parts])
    dp = (c_void_p * n)(*[t.data_ptr() for t in down_parts])
    _check("moe_merge_shared", _lib.moe_merge_shared(
        int(d_model), _enum(DTYPES, dtype), n, widths, gp, up, dp, _ptr(Ws_gate), _ptr(Ws_up),
        _ptr(Ws_down), _stream(stream)))


def moe_read_status(workspace, stream=None) -> int:
    code = c_int32(0)
    _check("moe_read_status", _lib.moe_read_status(_ptr(workspace), ctypes.byref(code), _stream(stream)))
    return int(code.value)


def moe_check_wait_bound(workspace, limit_ns: int, stream=None):
    """Self-check of the device wait bound (see the C header): leaves MOE_ERR_TIMEOUT in the
    workspace status word once a barrier wait of limit_ns runs out."""
    _check("moe_check_wait_bound", _lib.moe_check_wait_bound(_ptr(workspace), workspace.numel(),
                                                               int(limit_ns), _stream(stream)))


def moe_backward_workspace_size(cfg: moe_config) -> int:
    n = c_size_t(0)
    _check("moe_backward_workspace_size", _lib.moe_backward_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def make_grads(**tensors) -> moe_grads:
    g = moe_grads()
    for name in GRAD_FIELDS:
        p = _ptr(tensors.get(name))
        setattr(g, name, p.value if p is not None else None)
    g._keepalive = list(tensors.values())
    return g


def moe_layer_backward(cfg, weights: moe_weights, x, fwd_outputs: moe_outputs, dy, grads: moe_grads,
                       workspace, stream=None):
    _check("moe_layer_backward", _lib.moe_layer_backward(
        ctypes.byref(cfg), ctypes.byref(weights), _ptr(x), ctypes.byref(fwd_outputs), _ptr(dy),
        ctypes.byref(grads), _ptr(workspace), workspace.numel(), _stream(stream)))



def moe_layer_backward_aux(cfg, weights: moe_weights, x, fwd_outputs: moe_outputs, dy, dlogits,
                           grads: moe_grads, workspace, stream=None):
    """moe_layer_backward with a further gradient of the router logits (fp32 [T][N], or None)."""
    _check("moe_layer_backward_aux", _lib.moe_layer_backward_aux(
        ctypes.byref(cfg), ctypes.byref(weights), _ptr(x), ctypes.byref(fwd_outputs), _ptr(dy),
        _mat("dlogits", dlogits, cfg.T, cfg.N, 0, DTYPES["f32"]), ctypes.byref(grads), _ptr(workspace), workspace.numel(), _stream(stream)))


# ---- the block around the layer ------------------------------------------------------

def make_linear_config(T, in_features, out_features, act="none", out_dtype="bf16", dx_dtype="bf16",
                       dw_dtype="bf16", dtype="bf16", ldx=0, ldw=0, ldr=0, ldy=0) -> moe_linear_config:
    """A ``moe_linear_config``; ``ld*`` are the elements between rows (0 = dense)."""
    c = moe_linear_config()
    c.T, c.in_features, c.out_features = int(T), int(in_features), int(out_features)
    c.dtype, c.out_dtype = _enum(DTYPES, dtype), _enum(DTYPES, out_dtype)
    c.dx_dtype, c.dw_dtype = _enum(DTYPES, dx_dtype), _enum(DTYPES, dw_dtype)
    c.act = _enum(ACTS, act)
    c.ldx, c.ldw, c.ldr, c.ldy = int(ldx), int(ldw), int(ldr), int(ldy)
    return c


_TORCH_DTYPES = {}     # torch dtype -> moe_dtype


def _dtypes():
    if not _TORCH_DTYPES:
        import torch
        _TORCH_DTYPES.update({torch.float32: 0, torch.bfloat16: 1})
    return _TORCH_DTYPES


def _dtype_of(t) -> int:
    try:
        return _dtypes()[t.dtype]
    except KeyError:
        raise ValueError(f"fp32 or bf16 tensors are expected, got {t.dtype}") from None


def _mat(name, t, rows, cols, ld, dtype):
    """Address of a row-strided [rows][cols] matrix, checked against what the call assumes."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if t.shape != (rows, cols) or _dtypes().get(t.dtype) != dtype:
        raise ValueError(f"{name}: expected [{rows}][{cols}] of "
                         f"{'fp32' if dtype == 0 else 'bf16'}, got {tuple(t.shape)} {t.dtype}")
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or (s0 != (ld or cols) and rows > 1):
        raise ValueError(f"{name}: strides {t.stride()} do not match a row stride of {ld or cols}")
    return t.data_ptr()


def _vec(name, t, n, dtype="float32"):
    """Address of n contiguous values."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    import torch
    if t.numel() != n or t.dtype is not getattr(torch, dtype) or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous values of {dtype}, "
                         f"got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def moe_linear_workspace_size(cfg: moe_linear_config) -> int:
    n = c_size_t(0)
    _check("moe_linear_workspace_size", _lib.moe_linear_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def alloc_linear_workspace(cfg: moe_linear_config, device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) for moe_linear_forward and moe_linear_backward."""
    import torch
    ws = torch.empty(moe_linear_workspace_size(cfg), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_linear_forward(cfg: moe_linear_config, x, W, bias, residual, pre, y, workspace, stream=None):
    """y = act(x W^T + bias) + residual; bias, residual and pre (z, for the backward pass) may
    be None.  Rows of x, W, residual and y may be strided as the configuration says."""
    T, i, o, od = cfg.T, cfg.in_features, cfg.out_features, cfg.out_dtype
    _check("moe_linear_forward", _lib.moe_linear_forward(
        ctypes.byref(cfg), _mat("x", x, T, i, cfg.ldx, cfg.dtype), _mat("W", W, o, i, cfg.ldw, cfg.dtype),
        _vec("bias", bias, o), _mat("residual", residual, T, o, cfg.ldr, od),
        _mat("pre", pre, T, o, 0, od), _mat("y", y, T, o, cfg.ldy, od), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def moe_linear_backward(cfg: moe_linear_config, x, W, pre, dy, dx, dW, dbias, workspace, stream=None):
    """dx, dW, dbias (each may be None) for the gradient dy of y; pre is the forward call's."""
    T, i, o, od = cfg.T, cfg.in_features, cfg.out_features, cfg.out_dtype
    _check("moe_linear_backward", _lib.moe_linear_backward(
        ctypes.byref(cfg), _mat("x", x, T, i, cfg.ldx, cfg.dtype), _mat("W", W, o, i, cfg.ldw, cfg.dtype),
        _mat("pre", pre, T, o, 0, od), _mat("dy", dy, T, o, cfg.ldy, od),
        _mat("dx", dx, T, i, 0, cfg.dx_dtype), _mat("dW", dW, o, i, 0, cfg.dw_dtype),
        _vec("dbias", dbias, o), _ptr(workspace), workspace.numel(), _stream(stream)))


def _rows_of(name, t, shape=None):
    """(rows, cols, row stride) of a contiguous tensor or a row-strided matrix."""
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dim() == 0:
        raise ValueError(f"{name}: a tensor with at least one dimension is expected")
    cols = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    if t.dim() == 2 and (t.stride(1) == 1 or cols == 1):
        ld = t.stride(0) if t.shape[0] > 1 else cols
        if ld < cols:   # expanded rows (a stride of 0 would mean dense ones) or overlapping ones
            raise ValueError(f"{name}: rows {ld} elements apart share memory, rows of {cols} elements of their "
                             "own are expected (an expanded tensor needs .contiguous())")
        return t.shape[0], cols, ld
    raise ValueError(f"{name}: contiguous tensors, or matrices of contiguous rows, are expected")


def _dropout_config(x, y, residual, p):
    rows, cols, ldx = _rows_of("x", x)
    ldy = _rows_of("y", y, x.shape)[2]
    ldr = _rows_of("residual", residual, x.shape)[2] if residual is not None else 0
    return moe_dropout_config(rows, cols, float(p), _dtype_of(x),
                              _dtype_of(residual) if residual is not None else 0, _dtype_of(y), ldx, ldr, ldy)


def moe_dropout_add(x, residual, p, rng_state, y, stream=None):
    """y = residual + keep * x / (1 - p); residual may be None.  rng_state: int64 [2] device
    tensor (seed, offset).  The mask depends on them and the element's number alone."""
    c = _dropout_config(x, y, residual, p)
    _check("moe_dropout_add", _lib.moe_dropout_add(
        ctypes.byref(c), x.data_ptr(), None if residual is None else residual.data_ptr(),
        _vec("rng_state", rng_state, 2, "int64"), y.data_ptr(), _stream(stream)))


def moe_dropout_backward(dy, p, rng_state, dx, stream=None):
    """dx = keep * dy / (1 - p) with the mask of moe_dropout_add for the same p and rng_state."""
    c = _dropout_config(dx, dy, None, p)
    _check("moe_dropout_backward", _lib.moe_dropout_backward(
        ctypes.byref(c), dy.data_ptr(), _vec("rng_state", rng_state, 2, "int64"), dx.data_ptr(),
        _stream(stream)))


def moe_balance_loss_workspace_size(cfg: moe_config, seq_len: int = 0) -> int:
    n = c_size_t(0)
    _check("moe_balance_loss_workspace_size", _lib.moe_balance_loss_workspace_size(
        ctypes.byref(cfg), int(seq_len), ctypes.byref(n)))
    return int(n.value)


def alloc_balance_loss_workspace(cfg: moe_config, seq_len: int = 0, device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) for moe_balance_loss."""
    import torch
    ws = torch.empty(moe_balance_loss_workspace_size(cfg, seq_len), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_balance_loss(cfg: moe_config, logits, topk_idx, token_mask, seq_len, coef_balance, coef_z,
                     grad_scale, counts, P, loss, dlogits, workspace, stream=None):
    """Balance loss and z-loss of a routed batch: loss [3] (total, balance, z), counts and P
    [sequences][N], dlogits [T][N]; each output, token_mask (uint8 or bool [T]) and
    grad_scale (fp32 [1]) may be None.  seq_len 0 takes the batch as one sequence."""
    T, N, K = cfg.T, cfg.N, cfg.K
    S = -(-T // min(int(seq_len) or T, T)) if T else 0
    mask = "bool" if token_mask is not None and token_mask.element_size() == 1 and \
        str(token_mask.dtype) == "torch.bool" else "uint8"
    _check("moe_balance_loss", _lib.moe_balance_loss(
        ctypes.byref(cfg), _vec("logits", logits, T * N), _vec("topk_idx", topk_idx, T * K, "int32"),
        _vec("token_mask", token_mask, T, mask), int(seq_len), float(coef_balance), float(coef_z),
        _vec("grad_scale", grad_scale, 1), _vec("counts", counts, S * N, "int32"),
        _vec("P", P, S * N), _vec("loss", loss, 3), _vec("dlogits", dlogits, T * N), _ptr(workspace),
        workspace.numel(), _stream(stream)))


# ---- around the block ------------------------------------------------------------------

# moe_layernorm_config and moe_embedding_config as bytes: half the time of filling a ctypes structure
_LAYERNORM = struct.Struct("@qiifiiiiqqqq")
_EMBEDDING = struct.Struct("@qqiiiifqq")
assert _LAYERNORM.size == ctypes.sizeof(moe_layernorm_config) and _EMBEDDING.size == ctypes.sizeof(moe_embedding_config)


_ID_TYPES = {}         # torch dtype of token numbers -> whether they are int64
_TORCH = []            # torch's number of the current device, and its raw stream of a device


def _torch_calls():
    import torch
    _dtypes()
    _ID_TYPES.update({torch.int32: 0, torch.int64: 1})
    _TORCH.extend((lambda: torch._C._cuda_getDevice(), lambda dev: torch._C._cuda_getCurrentRawStream(dev)))


def _device_of(name, t) -> int:
    """Device number of the first tensor of a call, which has to be the current device's."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if not _TORCH:
        _torch_calls()
    if _TORCH[0]() != dev:
        raise ValueError(f"{name}: on device {dev}, which is not the current one")
    return dev


def _rows(name, t, dev, shape):
    """(address, moe_dtype, row stride) of a matrix of this shape with contiguous rows; a row stride of 0 stands for
    dense rows."""
    dtype = _TORCH_DTYPES.get(t.dtype)
    if dtype is None:
        raise ValueError(f"{name}: fp32 or bf16 is expected, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: a tensor on device {dev} is expected, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), dtype, 0
    s0, s1 = t.stride()
    cols = shape[1]
    if (s1 != 1 and cols > 1) or s0 < cols:
        raise ValueError(f"{name}: strides {t.stride()} are not those of contiguous rows of {cols} elements with "
                         "memory of their own (an expanded or transposed tensor needs .contiguous())")
    return t.data_ptr(), dtype, s0


def _flat(name, t, dev, n, dtype):
    """Address of n contiguous values of one moe_dtype."""
    if t.get_device() != dev or t.dim() != 1 or t.numel() != n or _TORCH_DTYPES.get(t.dtype) != dtype or \
            not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous values of {'fp32' if dtype == 0 else 'bf16'} on device "
                         f"{dev}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _raw_stream(stream, dev):
    if stream is None:
        return _TORCH[1](dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(ws, dev):
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on device {dev} is expected")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def moe_layernorm_workspace_size(T: int, d: int) -> int:
    n = c_size_t(0)
    _check("moe_layernorm_workspace_size", _lib.moe_layernorm_workspace_size(int(T), int(d), ctypes.byref(n)))
    return int(n.value)


def alloc_layernorm_workspace(T: int, d: int, device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) for moe_layernorm_backward."""
    import torch
    ws = torch.empty(moe_layernorm_workspace_size(T, d), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def _norm_param(weight, bias):
    """moe_dtype of the parameters, which share one."""
    p = weight if weight is not None else bias
    return 0 if p is None else _dtype_of(p)


def moe_layernorm_forward(x, residual, weight, bias, eps, sum, y, mean, rstd, kind="layer", stream=None):
    """y = (h - mean) rstd weight + bias of rows h = x + residual, which goes to ``sum`` (then h is the sum as
    stored), or of x alone.  x, residual, sum, y: matrices [T][d], rows may be strided; residual and sum have
    one type.  weight, bias [d]; mean, rstd fp32 [T].  residual, weight, bias, sum, mean and rstd may be None;
    kind "rms" has no mean."""
    dev = _device_of("x", x)
    if x.dim() != 2:
        raise ValueError(f"x: a matrix is expected, got {tuple(x.shape)}")
    shape = x.shape
    T, d = shape
    px, xt, ldx = _rows("x", x, dev, shape)
    pr, st, ldr = (None, 0, 0) if residual is None else _rows("residual", residual, dev, shape)
    ps, s2, lds = (None, st, 0) if sum is None else _rows("sum", sum, dev, shape)
    if s2 != st and residual is not None:
        raise ValueError("sum: the type of the residual is expected")
    py, yt, ldy = _rows("y", y, dev, shape)
    wt = _norm_param(weight, bias)
    c = _LAYERNORM.pack(T, d, _enum(LAYERNORM_KINDS, kind), eps, xt, st, yt, wt, ldx, ldr, lds, ldy)
    _check("moe_layernorm_forward", _lib.moe_layernorm_forward(
        c, px, pr, None if weight is None else _flat("weight", weight, dev, d, wt),
        None if bias is None else _flat("bias", bias, dev, d, wt), ps, py,
        None if mean is None else _flat("mean", mean, dev, T, 0), None if rstd is None else _flat("rstd", rstd, dev, T, 0),
        _raw_stream(stream, dev)))


def moe_layernorm_backward(h, weight, mean, rstd, dy, dsum, dx, dweight, dbias, workspace, kind="layer",
                           stream=None):
    """dx (of x and of the residual), dweight and dbias (fp32) for the gradient dy of y and dsum of ``sum``; each
    result, weight and dsum may be None.  h is the forward call's ``sum``, or its x where it had no residual;
    dsum and dx have one type.  dx may be dsum, dy or h itself."""
    dev = _device_of("h", h)
    if h.dim() != 2:
        raise ValueError(f"h: a matrix is expected, got {tuple(h.shape)}")
    shape = h.shape
    T, d = shape
    ph, ht, ldh = _rows("h", h, dev, shape)
    py, yt, ldy = _rows("dy", dy, dev, shape)
    pr, st, ldr = (None, 0, 0) if dsum is None else _rows("dsum", dsum, dev, shape)
    px, s2, lds = (None, st, 0) if dx is None else _rows("dx", dx, dev, shape)
    if dsum is None:
        st = s2
    elif s2 != st:
        raise ValueError("dx: the type of dsum is expected")
    wt = _norm_param(weight, None)
    c = _LAYERNORM.pack(T, d, _enum(LAYERNORM_KINDS, kind), 0.0, ht, st, yt, wt, ldh, ldr, lds, ldy)
    pw, nw = _workspace(workspace, dev)
    _check("moe_layernorm_backward", _lib.moe_layernorm_backward(
        c, ph, None if weight is None else _flat("weight", weight, dev, d, wt),
        None if mean is None else _flat("mean", mean, dev, T, 0), None if rstd is None else _flat("rstd", rstd, dev, T, 0),
        py, pr, px, None if dweight is None else _flat("dweight", dweight, dev, d, 0),
        None if dbias is None else _flat("dbias", dbias, dev, d, 0), pw, nw, _raw_stream(stream, dev)))


def moe_embedding_workspace_size(T: int, V: int, d: int) -> int:
    n = c_size_t(0)
    _check("moe_embedding_workspace_size",
           _lib.moe_embedding_workspace_size(int(T), int(V), int(d), ctypes.byref(n)))
    return int(n.value)


def alloc_embedding_workspace(T: int, V: int, d: int, device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) for moe_embedding_forward and moe_embedding_backward of up to T
    tokens."""
    import torch
    ws = torch.empty(moe_embedding_workspace_size(T, V, d), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def _embedding(ids, table, out, out_name, table_name, scale):
    """(configuration, addresses of ids, table and out, device)"""
    dev = _device_of("ids", ids)
    wide = _ID_TYPES.get(ids.dtype)
    if table.dim() != 2 or wide is None or not ids.is_contiguous():
        raise ValueError("contiguous int64 or int32 token numbers and a matrix are expected, got "
                         f"{ids.dtype} of strides {ids.stride()} and {tuple(table.shape)}")
    shape = table.shape
    T, (V, d) = ids.numel(), shape
    pt, tt, ldt = _rows(table_name, table, dev, shape)
    if out.dim() > 2 and out.is_contiguous():      # token numbers of any shape
        if out.shape[:-1] != ids.shape:
            raise ValueError(f"{out_name}: expected {tuple(ids.shape)} rows of {d}, got {tuple(out.shape)}")
        out = out.view(-1, out.shape[-1])
    po, ot, ldo = _rows(out_name, out, dev, (T, d))
    return _EMBEDDING.pack(T, V, d, wide, tt, ot, scale, ldt, ldo), ids.data_ptr(), pt, po, dev


def moe_embedding_forward(ids, table, scale, out, workspace, stream=None):
    """out[t] = scale table[ids[t]], zeros where ids[t] is -1.  ids: int64 or int32, any shape; table [V][d];
    out [tokens][d], or the ids' shape and d.  Another number outside the table leaves a row of zeros and
    MOE_ERR_DEVICE_BOUNDS for moe_read_status."""
    c, pi, pt, po, dev = _embedding(ids, table, out, "out", "table", scale)
    pw, nw = _workspace(workspace, dev)
    _check("moe_embedding_forward", _lib.moe_embedding_forward(c, pi, pt, po, pw, nw,
                                                               _raw_stream(stream, dev)))


def moe_embedding_backward(ids, dout, scale, dtable, workspace, accumulate=False, stream=None):
    """dtable[v] = scale * sum of dout[t] over the tokens with ids[t] = v, zeros for the others; with
    ``accumulate`` the sums are added to what dtable holds."""
    c, pi, pt, po, dev = _embedding(ids, dtable, dout, "dout", "dtable", scale)
    pw, nw = _workspace(workspace, dev)
    _check("moe_embedding_backward", _lib.moe_embedding_backward(
        c, pi, po, pt, int(bool(accumulate)), pw, nw, _raw_stream(stream, dev)))


def alloc_grad_norm_workspace(device="cuda", stream=None):
    """A zero-status workspace (uint8 tensor) for moe_grad_norm and moe_clip_grad_norm of any list."""
    import torch
    n = c_size_t(0)
    _check("moe_grad_norm_workspace_size", _lib.moe_grad_norm_workspace_size(ctypes.byref(n)))
    ws = torch.empty(int(n.value), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def _rows_words(name, t):
    """(rows, cols, row stride) of a tensor that is not contiguous."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: contiguous tensors, or matrices of contiguous rows with memory of their own, are "
                         f"expected, got strides {t.stride()} of {tuple(t.shape)}")
    return t.shape[0], t.shape[1], t.stride(0)


def _tensor_list(tensors, dev):
    """The tensors as an array of moe_tensor, five 64-bit words each."""
    words, kind = [], _TORCH_DTYPES.get
    for t in tensors:
        dtype = kind(t.dtype)
        if dtype is None or t.get_device() != dev:
            raise ValueError(f"grads: fp32 or bf16 tensors on device {dev} are expected, got {t.dtype} on {t.device}")
        if t.is_contiguous():
            words += (t.data_ptr(), 1, t.numel(), 0, dtype)
        else:
            words += (t.data_ptr(), *_rows_words("grads", t), dtype)
    return array.array("q", words)


def _tensor_lists(tensors, outs, dev):
    """The same for two lists of equal shapes and types."""
    words, more, kind = [], [], _TORCH_DTYPES.get
    for t, o in zip(tensors, outs):
        torch_dtype = t.dtype
        dtype = kind(torch_dtype)
        if dtype is None or t.get_device() != dev:
            raise ValueError(f"grads: fp32 or bf16 tensors on device {dev} are expected, got {t.dtype} on {t.device}")
        if o.dtype is not torch_dtype or o.get_device() != dev or o.shape != t.shape:
            raise ValueError(f"out: {tuple(t.shape)} of {t.dtype} on device {dev} is expected, got {tuple(o.shape)} "
                             f"of {o.dtype} on {o.device}")
        if t.is_contiguous() and o.is_contiguous():
            n = t.numel()
            words += (t.data_ptr(), 1, n, 0, dtype)
            more += (o.data_ptr(), 1, n, 0, dtype)
        else:       # both by their rows
            words += (t.data_ptr(), *_rows_words("grads", t), dtype)
            more += (o.data_ptr(), *_rows_words("out", o), dtype)
    return array.array("q", words), array.array("q", more)


def _norm_operands(norm, workspace):
    dev = _device_of("norm", norm)
    return dev, _flat("norm", norm, dev, 2, 0), *_workspace(workspace, dev)


def moe_grad_norm(grads, norm, workspace, max_norm=float("inf"), stream=None):
    """norm (fp32 [2]) = the 2-norm over all elements of the tensors of ``grads``, and
    min(1, max_norm / (norm + 1e-6)), the factor that clips it to ``max_norm``."""
    dev, pn, pw, nw = _norm_operands(norm, workspace)
    g = _tensor_list(grads, dev)
    _check("moe_grad_norm", _lib.moe_grad_norm(g.buffer_info()[0], len(grads), max_norm, pn, pw, nw,
                                               _raw_stream(stream, dev)))


def moe_clip_grad_norm(grads, max_norm, out, norm, workspace, stream=None):
    """moe_grad_norm, then every gradient times norm[1]: into the tensors of ``out``, or in place where it is
    None."""
    dev, pn, pw, nw = _norm_operands(norm, workspace)
    if out is not None and len(out) != len(grads):
        raise ValueError(f"out: {len(grads)} tensors are expected, got {len(out)}")
    g, o = (_tensor_list(grads, dev), None) if out is None else _tensor_lists(grads, out, dev)
    _check("moe_clip_grad_norm", _lib.moe_clip_grad_norm(
        g.buffer_info()[0], None if o is None else o.buffer_info()[0], len(grads), max_norm, pn, pw, nw,
        _raw_stream(stream, dev)))
