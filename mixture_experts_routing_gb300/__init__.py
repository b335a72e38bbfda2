"""Capacity-bounded Mixture-of-Experts layer forward for NVIDIA GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/moe.h`` (``libmoe.so``,
built in-tree by ``_build.build()``). The binding only marshals arguments:
every step of the layer runs in the library's CUDA kernels. PyTorch is used
for device memory and streams. If the library is missing, every call raises;
there is no fallback path.

Typical use (all tensors on one CUDA device)::

    cfg = Config(n_tokens=N, hidden=H, n_experts=E, top_k=K, inter=I,
                 cap_num=5, cap_den=4, block_m=32)
    routes = alloc_routes(cfg, device)
    ws = alloc_workspace(cfg, device)
    pack_w13(cfg, w_gate, w_up, w13); pack_w2(cfg, w_down, w2)   # once
    route_align(cfg, x, w_router, bias, routes, ws)
    ffn_forward(cfg, routes, x, w13, w2, h, o)
    combine(cfg, routes, o, y)
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "Config", "Routes", "ACT_SWIGLU", "ACT_GEGLU", "MoEError", "lib", "library_path", "alloc_routes", "alloc_workspace",
    "alloc_buffers", "capacity", "max_slots", "max_blocks", "route_workspace_bytes",
    "route_align", "fc1_forward", "fc2_forward", "ffn_forward", "combine", "pack_w13",
    "pack_w2", "status_string", "launch_count", "device_error", "forward",
    "ffn_forward_train", "backward_workspace_bytes", "alloc_backward_workspace", "ffn_backward",
    "router_backward_workspace_bytes", "alloc_router_backward_workspace", "router_backward",
    "Ladder", "ladder_pick",
    "SharedConfig", "alloc_shared_buffers", "alloc_shared_checkpoint",
    "shared_backward_workspace_bytes", "alloc_shared_backward_workspace", "shared_forward",
    "shared_forward_train", "shared_backward",
    "W4Config", "W4Weights", "w4_quantize", "w4_workspace_bytes", "alloc_w4_workspace",
    "w4_matvec", "w4_ffn_forward",
    "FewConfig", "few_workspace_bytes", "alloc_few_workspace", "few_forward",
    "NORM_LAYER", "NORM_RMS", "NormConfig", "norm_forward", "norm_backward_workspace_bytes",
    "alloc_norm_backward_workspace", "norm_backward",
    "AdamWConfig", "AdamW",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libmoe.so")
_lib = None

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: %d (%s)" % (fn, status, status_string(status)))
        self.status = status


ACT_SWIGLU, ACT_GEGLU = 0, 1


class Config(ctypes.Structure):
    """Mirror of moe_config_t."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_tokens", "hidden", "n_experts", "top_k", "inter", "cap_num", "cap_den", "block_m",
        "renorm", "ladder_len", "ladder_den")] + [("ladder_num", ctypes.POINTER(ctypes.c_int32)),
                                                  ("activation", ctypes.c_int32),
                                                  ("prob_in_act", ctypes.c_int32),
                                                  ("n_valid", ctypes.c_void_p)]

    def __init__(self, n_tokens, hidden, n_experts, top_k, inter, cap_num=1, cap_den=1,
                 block_m=32, renorm=1, ladder=None, ladder_den=1, activation=ACT_SWIGLU,
                 prob_in_act=0):
        """cap_num=0 selects the dropless layout; ladder: rung multipliers
        (numerators over ladder_den) of the expected rows per expert;
        activation: ACT_SWIGLU or ACT_GEGLU; prob_in_act: p' multiplies the
        activation (unit-weight combine) instead of weighting the combine."""
        lad = list(ladder or [])
        self._ladder = (ctypes.c_int32 * max(len(lad), 1))(*lad)
        super().__init__(n_tokens, hidden, n_experts, top_k, inter, cap_num, cap_den, block_m,
                         renorm, len(lad), ladder_den,
                         ctypes.cast(self._ladder, ctypes.POINTER(ctypes.c_int32)), activation,
                         int(bool(prob_in_act)), None)


class SharedConfig(ctypes.Structure):
    """Mirror of moe_shared_config_t: the shared expert's shape. grad_f32: weight
    gradients in f32 instead of bf16."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "hidden", "inter", "activation",
                                              "grad_f32")]

    def __init__(self, n_tokens, hidden, inter, activation=ACT_SWIGLU, grad_f32=0):
        super().__init__(n_tokens, hidden, inter, activation, int(bool(grad_f32)))


class W4Config(ctypes.Structure):
    """Mirror of moe_w4_config_t: a decode batch through experts with 4-bit
    weights, one bf16 scale per `group` (32, 64 or 128) columns."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "hidden", "n_experts", "top_k", "inter",
                                              "group", "activation")]

    def __init__(self, n_tokens, hidden, n_experts, top_k, inter, group=128,
                 activation=ACT_SWIGLU):
        super().__init__(n_tokens, hidden, n_experts, top_k, inter, group, activation)


class FewConfig(ctypes.Structure):
    """Mirror of moe_few_config_t: the whole layer for at most 64 tokens."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "hidden", "n_experts", "top_k", "inter",
                                              "renorm", "activation")]

    def __init__(self, n_tokens, hidden, n_experts, top_k, inter, renorm=1, activation=ACT_SWIGLU):
        super().__init__(n_tokens, hidden, n_experts, top_k, inter, int(bool(renorm)), activation)


NORM_LAYER, NORM_RMS = 0, 1


class NormConfig(ctypes.Structure):
    """Mirror of moe_norm_config_t: rows of a layer norm (NORM_LAYER) or of its form
    without a mean (NORM_RMS)."""
    _fields_ = [("n_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("eps", ctypes.c_float)]

    def __init__(self, n_tokens, hidden, kind=NORM_LAYER, eps=1e-5):
        super().__init__(n_tokens, hidden, kind, eps)


class AdamWConfig(ctypes.Structure):
    """Mirror of moe_adamw_config_t."""
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("lr", ctypes.c_float),
                ("eps", ctypes.c_float), ("state_bits", ctypes.c_int32), ("seed", ctypes.c_uint32)]


class _AdamWTensorC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("first", ctypes.c_int64), ("weight_decay", ctypes.c_float),
        ("grad_bf16", ctypes.c_int32)]


class _RoutesC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_ids", "topk_p", "keep", "expert_counts", "kept_counts", "sorted_slot_ids",
        "expert_ids", "block_start", "num_tokens_post_padded", "token_routes", "gemm_sched",
        "slot_prob")]


class _LayerBufsC(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w_router", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("routes", _RoutesC),
                ("route_workspace", ctypes.c_void_p), ("route_workspace_bytes", ctypes.c_size_t),
                ("h", ctypes.c_void_p), ("o", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n_valid", ctypes.c_void_p)]


class Routes:
    """Routing metadata tensors (device), allocated to the static bounds."""
    FIELDS = _RoutesC._fields_

    def __init__(self, **tensors):
        for name, _ in self.FIELDS:
            setattr(self, name, tensors[name])

    def c(self) -> _RoutesC:
        return _RoutesC(*[getattr(self, n).data_ptr() for n, _ in self.FIELDS])


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libmoe.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libmoe.so is not built (run __graft_entry__.build() or "
                               "python -m mixture_experts_routing_gb300._build)")
        L = ctypes.CDLL(_LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        CP = ctypes.POINTER(Config)
        RP = ctypes.POINTER(_RoutesC)
        for name in ("moe_capacity", "moe_max_slots", "moe_max_blocks", "moe_route_workspace_bytes",
                     "moe_backward_workspace_bytes", "moe_router_backward_workspace_bytes"):
            getattr(L, name).argtypes = [CP]
            getattr(L, name).restype = I64
        L.moe_route_align.argtypes = [CP, P, P, P, RP, P, SZ, P]
        L.moe_fc1_forward.argtypes = [CP, RP, P, P, P, P]
        L.moe_fc2_forward.argtypes = [CP, RP, P, P, P, P]
        L.moe_ffn_forward.argtypes = [CP, RP, P, P, P, P, P, P]
        L.moe_combine.argtypes = [CP, RP, P, P, P]
        L.moe_ffn_forward_train.argtypes = [CP, RP, P, P, P, P, P, P, P]
        L.moe_ffn_backward.argtypes = [CP, RP, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_router_backward.argtypes = [CP, RP, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_route_workspace_logits.argtypes = [CP, P]
        L.moe_route_workspace_logits.restype = P
        L.moe_ladder_pick.argtypes = [P, I32, ctypes.c_int32, ctypes.c_float]
        L.moe_ladder_pick.restype = I32
        L.moe_ladder_create.argtypes = [CP, P, I32, ctypes.c_float, ctypes.POINTER(_LayerBufsC),
                                        ctypes.POINTER(ctypes.c_void_p)]
        L.moe_ladder_forward.argtypes = [P, ctypes.c_int32, P, ctypes.POINTER(ctypes.c_int)]
        L.moe_ladder_destroy.argtypes = [P]
        for name in ("moe_ladder_create", "moe_ladder_forward", "moe_ladder_destroy"):
            getattr(L, name).restype = I32
        SP, WP = ctypes.POINTER(SharedConfig), ctypes.POINTER(W4Config)
        L.moe_shared_backward_workspace_bytes.argtypes = [SP]
        L.moe_w4_workspace_bytes.argtypes = [WP]
        L.moe_shared_forward.argtypes = [SP] + [P] * 7
        L.moe_shared_forward_train.argtypes = [SP] + [P] * 9
        L.moe_shared_backward.argtypes = [SP] + [P] * 11 + [SZ, P]
        L.moe_w4_quantize.argtypes = [P, I64, I32, I32, P, P, P]
        L.moe_w4_matvec.argtypes = [P, P, P, I32, I32, I32, I32, P, P]
        L.moe_w4_ffn_forward.argtypes = [WP] + [P] * 10 + [SZ, P]
        for name in ("moe_shared_backward_workspace_bytes", "moe_w4_workspace_bytes"):
            getattr(L, name).restype = I64
        for name in ("moe_shared_forward", "moe_shared_forward_train", "moe_shared_backward",
                     "moe_w4_quantize", "moe_w4_matvec", "moe_w4_ffn_forward"):
            getattr(L, name).restype = I32
        FP, NP = ctypes.POINTER(FewConfig), ctypes.POINTER(NormConfig)
        L.moe_few_workspace_bytes.argtypes = [FP]
        L.moe_few_forward.argtypes = [FP] + [P] * 11 + [SZ, P]
        L.moe_norm_forward.argtypes = [NP] + [P] * 9
        L.moe_norm_backward_workspace_bytes.argtypes = [NP]
        L.moe_norm_backward.argtypes = [NP] + [P] * 10 + [SZ, P]
        L.moe_adamw_step.argtypes = [ctypes.POINTER(AdamWConfig), P, I32, P, P, P, P]
        for name in ("moe_few_workspace_bytes", "moe_norm_backward_workspace_bytes"):
            getattr(L, name).restype = I64
        for name in ("moe_few_forward", "moe_norm_forward", "moe_norm_backward", "moe_adamw_step"):
            getattr(L, name).restype = I32
        L.moe_pack_w13.argtypes = [CP, P, P, P, P]
        L.moe_pack_w2.argtypes = [CP, P, P, P]
        L.moe_quantize_rows_fp8.argtypes = [P, I64, P, I32, P, P, P]
        L.moe_fc1_forward_fp8.argtypes = [CP, RP, P, P, P, P, P, P]
        L.moe_fc2_forward_fp8.argtypes = [CP, RP, P, P, P, P, P, P]
        L.moe_ffn_forward_fp8.argtypes = [CP, RP, P, P, P, P, P, P, P, P, P, P, P, P]
        L.moe_quantize_mx_fp8.argtypes = [P, I64, P, I32, P, P, P]
        L.moe_quantize_mx_fp8_weights.argtypes = [P, I64, I32, P, P, P]
        L.moe_fc1_forward_mx.argtypes = [CP, RP, P, P, P, P, P, P]
        L.moe_fc2_forward_mx.argtypes = [CP, RP, P, P, P, P, P, P]
        L.moe_ffn_forward_mx.argtypes = [CP, RP, P, P, P, P, P, P, P, P, P, P, P, P]
        for name in ("moe_route_align", "moe_fc1_forward", "moe_fc2_forward", "moe_ffn_forward",
                     "moe_combine", "moe_pack_w13", "moe_pack_w2", "moe_ffn_forward_train",
                     "moe_ffn_backward", "moe_router_backward", "moe_quantize_rows_fp8",
                     "moe_fc1_forward_fp8", "moe_fc2_forward_fp8", "moe_ffn_forward_fp8",
                     "moe_quantize_mx_fp8", "moe_quantize_mx_fp8_weights", "moe_fc1_forward_mx",
                     "moe_fc2_forward_mx", "moe_ffn_forward_mx"):
            getattr(L, name).restype = I32
        L.moe_status_string.argtypes = [I32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_launch_count.argtypes = []
        L.moe_launch_count.restype = ctypes.c_uint64
        L.moe_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        L.moe_device_error.restype = I32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoEError(fn, status)


def _q(fn: str, cfg: Config) -> int:
    v = getattr(lib(), fn)(ctypes.byref(cfg))
    if v < 0:
        raise MoEError(fn, int(v))
    return int(v)


def capacity(cfg: Config) -> int:
    return _q("moe_capacity", cfg)


def max_slots(cfg: Config) -> int:
    return _q("moe_max_slots", cfg)


def max_blocks(cfg: Config) -> int:
    return _q("moe_max_blocks", cfg)


def route_workspace_bytes(cfg: Config) -> int:
    return _q("moe_route_workspace_bytes", cfg)


def backward_workspace_bytes(cfg: Config) -> int:
    return _q("moe_backward_workspace_bytes", cfg)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_current = None  # (device) -> handle of its current stream, and () -> current device


def _stream(stream) -> int:
    """The stream's handle; by default that of the current device's current
    stream, asked for without building a torch.cuda.Stream (3 us a call)."""
    global _current
    if stream is not None:
        return stream.cuda_stream
    if _current is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            raw = lambda d: torch.cuda.current_stream(d).cuda_stream  # noqa: E731
        _current = (raw, torch.cuda.current_device)
    return _current[0](_current[1]())


def alloc_routes(cfg: Config, device) -> Routes:
    import torch
    N, K, E = max(cfg.n_tokens, 1), cfg.top_k, cfg.n_experts  # >= 1 row: non-null pointers
    S, B = max_slots(cfg), max_blocks(cfg)
    i32 = dict(dtype=torch.int32, device=device)
    return Routes(
        topk_ids=torch.empty((N, K), **i32), topk_p=torch.empty((N, K), dtype=torch.float32, device=device),
        keep=torch.empty((N, K), dtype=torch.uint8, device=device),
        expert_counts=torch.empty(E, **i32), kept_counts=torch.empty(E, **i32),
        sorted_slot_ids=torch.empty(max(S, 1), **i32), expert_ids=torch.empty(max(B, 1), **i32),
        block_start=torch.empty(E, **i32), num_tokens_post_padded=torch.empty(1, **i32),
        token_routes=torch.empty((N, K), **i32), gemm_sched=torch.zeros(4, **i32),
        slot_prob=torch.empty(max(S, 1), dtype=torch.float32, device=device))


def alloc_workspace(cfg: Config, device):
    import torch
    return torch.empty(max(route_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def alloc_buffers(cfg: Config, device):
    """h [S,I], o [S,H] and y [N,H] bf16 buffers for one forward."""
    import torch
    S = max(max_slots(cfg), 1)
    bf = dict(dtype=torch.bfloat16, device=device)
    return (torch.empty((S, cfg.inter), **bf), torch.empty((S, cfg.hidden), **bf),
            torch.empty((max(cfg.n_tokens, 1), cfg.hidden), **bf))


def route_align(cfg: Config, x, w_router, bias, routes: Routes, workspace, stream=None) -> None:
    rc = lib().moe_route_align(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(bias),
                               ctypes.byref(routes.c()), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_route_align", rc)


def fc1_forward(cfg: Config, routes: Routes, x, w13, h, stream=None) -> None:
    _check("moe_fc1_forward", lib().moe_fc1_forward(ctypes.byref(cfg), ctypes.byref(routes.c()),
                                                    _ptr(x), _ptr(w13), _ptr(h), _stream(stream)))


def fc2_forward(cfg: Config, routes: Routes, h, w2, o, stream=None) -> None:
    _check("moe_fc2_forward", lib().moe_fc2_forward(ctypes.byref(cfg), ctypes.byref(routes.c()),
                                                    _ptr(h), _ptr(w2), _ptr(o), _stream(stream)))


def ffn_forward(cfg: Config, routes: Routes, x, w13, w2, h, o, stream=None) -> None:
    _check("moe_ffn_forward", lib().moe_ffn_forward(ctypes.byref(cfg), ctypes.byref(routes.c()),
                                                    _ptr(x), _ptr(w13), _ptr(w2), _ptr(h), _ptr(o),
                                                    _stream(stream)))


def ffn_forward_train(cfg: Config, routes: Routes, x, w13, w2, h, o, preact, stream=None) -> None:
    """ffn_forward that also writes FC1's pre-activations preact [S,2I] (g | u)."""
    _check("moe_ffn_forward_train",
           lib().moe_ffn_forward_train(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(x),
                                       _ptr(w13), _ptr(w2), _ptr(h), _ptr(o), _ptr(preact),
                                       _stream(stream)))


def alloc_backward_workspace(cfg: Config, device):
    import torch
    return torch.empty(max(backward_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def ffn_backward(cfg: Config, routes: Routes, x, w13, w2, preact, dy, dx, dw13, dw2, dprob,
                 workspace, stream=None) -> None:
    """Expert-path backward: dx [N,H] bf16, dw13 [E,2I,H] f32, dw2 [E,H,I] f32,
    dprob [N,K] f32 (outputs overwritten)."""
    _check("moe_ffn_backward",
           lib().moe_ffn_backward(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(x), _ptr(w13),
                                  _ptr(w2), _ptr(preact), _ptr(dy), _ptr(dx), _ptr(dw13),
                                  _ptr(dw2), _ptr(dprob), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))


def router_backward_workspace_bytes(cfg: Config) -> int:
    return _q("moe_router_backward_workspace_bytes", cfg)


def alloc_router_backward_workspace(cfg: Config, device):
    import torch
    return torch.empty(max(router_backward_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def router_backward(cfg: Config, routes: Routes, x, w_router, bias, dprob, dx, dw_router, dbias,
                    workspace, stream=None, logits=None) -> None:
    """Router backward: dx += dl . W_r^T (bf16, in place), dw_router [H,E] f32 and
    dbias [E] f32 (or None) overwritten. logits: the forward's [N,E] logits
    (route_workspace_logits), or None to recompute them."""
    _check("moe_router_backward",
           lib().moe_router_backward(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(x),
                                     _ptr(w_router), _ptr(bias), _ptr(logits), _ptr(dprob),
                                     _ptr(dx), _ptr(dw_router), _ptr(dbias), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


def route_workspace_logits(cfg: Config, workspace):
    """The [N,E] fp32 router logits moe_route_align left in its workspace, as a
    view of that workspace tensor."""
    import torch
    p = lib().moe_route_workspace_logits(ctypes.byref(cfg), _ptr(workspace))
    if not p:
        raise MoEError("moe_route_workspace_logits", MOE_ERR_INVALID_ARG)
    off = p - workspace.data_ptr()
    n = cfg.n_tokens * cfg.n_experts
    return workspace.view(-1)[off:off + 4 * n].view(torch.float32).view(cfg.n_tokens, cfg.n_experts)


def combine(cfg: Config, routes: Routes, o, y, stream=None) -> None:
    _check("moe_combine", lib().moe_combine(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(o),
                                            _ptr(y), _stream(stream)))


def pack_w13(cfg: Config, w_gate, w_up, w13, stream=None) -> None:
    _check("moe_pack_w13", lib().moe_pack_w13(ctypes.byref(cfg), _ptr(w_gate), _ptr(w_up),
                                              _ptr(w13), _stream(stream)))


def pack_w2(cfg: Config, w_down, w2, stream=None) -> None:
    _check("moe_pack_w2", lib().moe_pack_w2(ctypes.byref(cfg), _ptr(w_down), _ptr(w2),
                                            _stream(stream)))


def quantize_rows_fp8(m, q, scale, stream=None, rows_dev=None) -> None:
    """Row-wise E4M3 codes q [rows, cols] u8 and scales [rows] f32 of a bf16
    matrix m; rows_dev (a device int32 tensor) bounds the rows quantised."""
    rows, cols = m.shape
    _check("moe_quantize_rows_fp8",
           lib().moe_quantize_rows_fp8(_ptr(m), int(rows), _ptr(rows_dev), int(cols), _ptr(q),
                                       _ptr(scale), _stream(stream)))


def fc1_forward_fp8(cfg: Config, routes: Routes, xq, x_scale, w13q, w13_scale, h,
                    stream=None) -> None:
    _check("moe_fc1_forward_fp8",
           lib().moe_fc1_forward_fp8(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(xq),
                                     _ptr(x_scale), _ptr(w13q), _ptr(w13_scale), _ptr(h),
                                     _stream(stream)))


def fc2_forward_fp8(cfg: Config, routes: Routes, hq, h_scale, w2q, w2_scale, o,
                    stream=None) -> None:
    _check("moe_fc2_forward_fp8",
           lib().moe_fc2_forward_fp8(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(hq),
                                     _ptr(h_scale), _ptr(w2q), _ptr(w2_scale), _ptr(o),
                                     _stream(stream)))


class Fp8Weights:
    """w13 and w2 quantised row-wise once: codes (u8) and fp32 row scales."""

    def __init__(self, cfg: Config, w13, w2, stream=None):
        import torch
        E, H, I = cfg.n_experts, cfg.hidden, cfg.inter
        dev = w13.device
        self.w13q = torch.empty((E, 2 * I, H), dtype=torch.uint8, device=dev)
        self.w13_scale = torch.empty(E * 2 * I, dtype=torch.float32, device=dev)
        self.w2q = torch.empty((E, H, I), dtype=torch.uint8, device=dev)
        self.w2_scale = torch.empty(E * H, dtype=torch.float32, device=dev)
        quantize_rows_fp8(w13.view(E * 2 * I, H), self.w13q, self.w13_scale, stream)
        quantize_rows_fp8(w2.view(E * H, I), self.w2q, self.w2_scale, stream)


def alloc_fp8_buffers(cfg: Config, device):
    """xq [N,H] u8, x_scale [N] f32, hq [S,I] u8 and h_scale [S] f32 for ffn_forward_fp8."""
    import torch
    N, S = max(cfg.n_tokens, 1), max(max_slots(cfg), 1)
    return (torch.empty((N, cfg.hidden), dtype=torch.uint8, device=device),
            torch.empty(N, dtype=torch.float32, device=device),
            torch.empty((S, cfg.inter), dtype=torch.uint8, device=device),
            torch.empty(S, dtype=torch.float32, device=device))


def ffn_forward_fp8(cfg: Config, routes: Routes, x, wq: Fp8Weights, xq, x_scale, h, hq, h_scale, o,
                    stream=None) -> None:
    """Quantise x, FC1 on FP8, quantise h, FC2 on FP8 (one C call, four launches)."""
    _check("moe_ffn_forward_fp8",
           lib().moe_ffn_forward_fp8(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(x),
                                     _ptr(wq.w13q), _ptr(wq.w13_scale), _ptr(wq.w2q),
                                     _ptr(wq.w2_scale), _ptr(xq), _ptr(x_scale), _ptr(h), _ptr(hq),
                                     _ptr(h_scale), _ptr(o), _stream(stream)))


def quantize_mx_fp8(m, q, scale, stream=None, rows_dev=None) -> None:
    """MX (block-scaled) E4M3 codes q [rows, cols] u8 and E8M0 scale codes
    [rows, cols/32] u8 of a bf16 matrix m; rows_dev bounds the rows quantised."""
    rows, cols = m.shape
    _check("moe_quantize_mx_fp8",
           lib().moe_quantize_mx_fp8(_ptr(m), int(rows), _ptr(rows_dev), int(cols), _ptr(q),
                                     _ptr(scale), _stream(stream)))


def quantize_mx_fp8_weights(m, q, scale_atoms, stream=None) -> None:
    """MX codes of packed weight rows m [rows, cols] (multiples of 128) with
    the scale bytes in the GEMMs' 512-byte atom layout."""
    rows, cols = m.shape
    _check("moe_quantize_mx_fp8_weights",
           lib().moe_quantize_mx_fp8_weights(_ptr(m), int(rows), int(cols), _ptr(q),
                                             _ptr(scale_atoms), _stream(stream)))


def fc1_forward_mx(cfg: Config, routes: Routes, xq, x_sf, w13q, w13_sf, h, stream=None) -> None:
    _check("moe_fc1_forward_mx",
           lib().moe_fc1_forward_mx(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(xq),
                                    _ptr(x_sf), _ptr(w13q), _ptr(w13_sf), _ptr(h),
                                    _stream(stream)))


def fc2_forward_mx(cfg: Config, routes: Routes, hq, h_sf, w2q, w2_sf, o, stream=None) -> None:
    _check("moe_fc2_forward_mx",
           lib().moe_fc2_forward_mx(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(hq),
                                    _ptr(h_sf), _ptr(w2q), _ptr(w2_sf), _ptr(o), _stream(stream)))


class MxWeights:
    """w13 and w2 MX-quantised once: E4M3 codes and E8M0 block scales in the
    GEMMs' atom layout."""

    def __init__(self, cfg: Config, w13, w2, stream=None):
        import torch
        E, H, I = cfg.n_experts, cfg.hidden, cfg.inter
        dev = w13.device
        self.w13q = torch.empty((E, 2 * I, H), dtype=torch.uint8, device=dev)
        self.w13_sf = torch.empty(E * 2 * I * H // 32, dtype=torch.uint8, device=dev)
        self.w2q = torch.empty((E, H, I), dtype=torch.uint8, device=dev)
        self.w2_sf = torch.empty(E * H * I // 32, dtype=torch.uint8, device=dev)
        quantize_mx_fp8_weights(w13.view(E * 2 * I, H), self.w13q, self.w13_sf, stream)
        quantize_mx_fp8_weights(w2.view(E * H, I), self.w2q, self.w2_sf, stream)


def alloc_mx_buffers(cfg: Config, device):
    """xq [N,H] u8, x_sf [N,H/32] u8, hq [S,I] u8 and h_sf [S,I/32] u8 for ffn_forward_mx."""
    import torch
    N, S = max(cfg.n_tokens, 1), max(max_slots(cfg), 1)
    u8 = dict(dtype=torch.uint8, device=device)
    return (torch.empty((N, cfg.hidden), **u8), torch.empty((N, cfg.hidden // 32), **u8),
            torch.empty((S, cfg.inter), **u8), torch.empty((S, cfg.inter // 32), **u8))


def ffn_forward_mx(cfg: Config, routes: Routes, x, wq: MxWeights, xq, x_sf, h, hq, h_sf, o,
                   stream=None) -> None:
    """Quantise x, FC1 on MX operands, quantise h, FC2 on MX (one C call, four launches)."""
    _check("moe_ffn_forward_mx",
           lib().moe_ffn_forward_mx(ctypes.byref(cfg), ctypes.byref(routes.c()), _ptr(x),
                                    _ptr(wq.w13q), _ptr(wq.w13_sf), _ptr(wq.w2q), _ptr(wq.w2_sf),
                                    _ptr(xq), _ptr(x_sf), _ptr(h), _ptr(hq), _ptr(h_sf), _ptr(o),
                                    _stream(stream)))


def forward(cfg: Config, x, w_router, bias, w13, w2, routes: Routes, workspace, h, o, y,
            stream=None) -> None:
    """The whole layer: route_align, ffn_forward, combine (three C calls)."""
    route_align(cfg, x, w_router, bias, routes, workspace, stream)
    ffn_forward(cfg, routes, x, w13, w2, h, o, stream)
    combine(cfg, routes, o, y, stream)


# ------------------------------------------------------------------ shared expert
def _is(t, dtype, *shape) -> bool:
    """The tensor has this type and shape, its rows lie one after another and it
    is in device memory (the library is given addresses only)."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda


def _refuse(fn: str, **named) -> None:
    """Names the first argument that is not what the call needs; each keyword is
    (tensor, type, shape...)."""
    for name, (t, dtype, *shape) in named.items():
        if not _is(t, dtype, *shape):
            raise ValueError("%s: %s must be a contiguous %s CUDA tensor of shape %s, got %s %s on %s%s" % (
                fn, name, str(dtype).replace("torch.", ""), tuple(shape),
                str(t.dtype).replace("torch.", ""), tuple(t.shape), t.device,
                "" if t.is_contiguous() else ", not contiguous"))


def alloc_shared_buffers(cfg: SharedConfig, device):
    """h [N,I] and y [N,H] bf16 for shared_forward."""
    import torch
    bf = dict(dtype=torch.bfloat16, device=device)
    return (torch.empty((cfg.n_tokens, cfg.inter), **bf),
            torch.empty((cfg.n_tokens, cfg.hidden), **bf))


def alloc_shared_checkpoint(cfg: SharedConfig, device):
    """ck [N,2I] and ck_sf [N,2I/32] u8: the 8-bit pre-activations of one step."""
    import torch
    u8 = dict(dtype=torch.uint8, device=device)
    return (torch.empty((cfg.n_tokens, 2 * cfg.inter), **u8),
            torch.empty((cfg.n_tokens, cfg.inter // 16), **u8))


def shared_backward_workspace_bytes(cfg: SharedConfig) -> int:
    return _q("moe_shared_backward_workspace_bytes", cfg)


def alloc_shared_backward_workspace(cfg: SharedConfig, device):
    import torch
    return torch.empty(max(shared_backward_workspace_bytes(cfg), 256), dtype=torch.uint8,
                       device=device)


def shared_forward(cfg: SharedConfig, x, w13, w2, h, y, add=None, stream=None) -> None:
    """y = (act(x W_gate) * (x W_up)) W_down (+ add): w13 [2I,H] and w2 [H,I] bf16
    (one expert of pack_w13 / pack_w2), h [N,I] scratch; add may be y."""
    import torch
    bf, N, H, I = torch.bfloat16, cfg.n_tokens, cfg.hidden, cfg.inter
    if not (_is(x, bf, N, H) and _is(w13, bf, 2 * I, H) and _is(w2, bf, H, I) and _is(h, bf, N, I)
            and _is(y, bf, N, H) and (add is None or _is(add, bf, N, H))):
        _refuse("shared_forward", x=(x, bf, N, H), w13=(w13, bf, 2 * I, H), w2=(w2, bf, H, I),
                h=(h, bf, N, I), y=(y, bf, N, H), add=(x if add is None else add, bf, N, H))
    rc = lib().moe_shared_forward(ctypes.byref(cfg), x.data_ptr(), w13.data_ptr(), w2.data_ptr(),
                                  _ptr(add), h.data_ptr(), y.data_ptr(), _stream(stream))
    if rc:
        raise MoEError("moe_shared_forward", rc)


def shared_forward_train(cfg: SharedConfig, x, w13, w2, h, y, ck, ck_sf, add=None,
                         stream=None) -> None:
    """shared_forward that also keeps the pre-activations [g | u] in 8 bits
    (alloc_shared_checkpoint) for shared_backward."""
    import torch
    bf, u8, N, H, I = torch.bfloat16, torch.uint8, cfg.n_tokens, cfg.hidden, cfg.inter
    if not (_is(x, bf, N, H) and _is(w13, bf, 2 * I, H) and _is(w2, bf, H, I) and _is(h, bf, N, I)
            and _is(y, bf, N, H) and (add is None or _is(add, bf, N, H))
            and _is(ck, u8, N, 2 * I) and _is(ck_sf, u8, N, I // 16)):
        _refuse("shared_forward_train", x=(x, bf, N, H), w13=(w13, bf, 2 * I, H),
                w2=(w2, bf, H, I), h=(h, bf, N, I), y=(y, bf, N, H),
                add=(x if add is None else add, bf, N, H), ck=(ck, u8, N, 2 * I),
                ck_sf=(ck_sf, u8, N, I // 16))
    rc = lib().moe_shared_forward_train(ctypes.byref(cfg), x.data_ptr(), w13.data_ptr(),
                                        w2.data_ptr(), _ptr(add), h.data_ptr(), y.data_ptr(),
                                        ck.data_ptr(), ck_sf.data_ptr(), _stream(stream))
    if rc:
        raise MoEError("moe_shared_forward_train", rc)


def shared_backward(cfg: SharedConfig, x, w13, w2, ck, ck_sf, dy, dx, dw13, dw2, workspace,
                    dx_add=None, stream=None) -> None:
    """Gradients from the 8-bit checkpoint: dx [N,H] bf16 (+ dx_add, which may be
    dx), dw13 [2I,H] and dw2 [H,I] (bf16, or f32 with cfg.grad_f32; overwritten)."""
    import torch
    bf, u8, N, H, I = torch.bfloat16, torch.uint8, cfg.n_tokens, cfg.hidden, cfg.inter
    gt = torch.float32 if cfg.grad_f32 else bf
    if not (_is(x, bf, N, H) and _is(w13, bf, 2 * I, H) and _is(w2, bf, H, I)
            and _is(ck, u8, N, 2 * I) and _is(ck_sf, u8, N, I // 16) and _is(dy, bf, N, H)
            and _is(dx, bf, N, H) and (dx_add is None or _is(dx_add, bf, N, H))
            and _is(dw13, gt, 2 * I, H) and _is(dw2, gt, H, I) and workspace.is_cuda):
        _refuse("shared_backward", x=(x, bf, N, H), w13=(w13, bf, 2 * I, H), w2=(w2, bf, H, I),
                ck=(ck, u8, N, 2 * I), ck_sf=(ck_sf, u8, N, I // 16), dy=(dy, bf, N, H),
                dx=(dx, bf, N, H), dx_add=(x if dx_add is None else dx_add, bf, N, H),
                dw13=(dw13, gt, 2 * I, H), dw2=(dw2, gt, H, I),
                workspace=(workspace, workspace.dtype, *workspace.shape))
    rc = lib().moe_shared_backward(ctypes.byref(cfg), x.data_ptr(), w13.data_ptr(), w2.data_ptr(),
                                   ck.data_ptr(), ck_sf.data_ptr(), dy.data_ptr(), _ptr(dx_add),
                                   dx.data_ptr(), dw13.data_ptr(), dw2.data_ptr(),
                                   workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if rc:
        raise MoEError("moe_shared_backward", rc)


# ------------------------------------------------------------------ 4-bit weights
def w4_quantize(m, group: int, q, scale, stream=None) -> None:
    """4-bit codes q [rows, cols/2] u8 and bf16 scales [rows, cols/group] of a
    bf16 matrix m [rows, cols]."""
    import torch
    rows, cols = m.shape
    if group <= 0:
        raise MoEError("moe_w4_quantize", MOE_ERR_INVALID_ARG)
    _refuse("w4_quantize", m=(m, torch.bfloat16, rows, cols), q=(q, torch.uint8, rows, cols // 2),
            scale=(scale, torch.bfloat16, rows, cols // group))
    _check("moe_w4_quantize", lib().moe_w4_quantize(_ptr(m), int(rows), int(cols), int(group),
                                                    _ptr(q), _ptr(scale), _stream(stream)))


class W4Weights:
    """Packed expert weights w13 [E,2I,H] and w2 [E,H,I] in 4 bits, quantised once."""

    def __init__(self, w13, w2, group: int = 128, stream=None):
        import torch
        if group <= 0:
            raise MoEError("moe_w4_quantize", MOE_ERR_INVALID_ARG)
        E, I2, H = w13.shape
        I = w2.shape[2]
        dev = w13.device
        self.group = group
        self.w13q = torch.empty((E, I2, H // 2), dtype=torch.uint8, device=dev)
        self.w13_scale = torch.empty((E, I2, H // group), dtype=torch.bfloat16, device=dev)
        self.w2q = torch.empty((E, H, I // 2), dtype=torch.uint8, device=dev)
        self.w2_scale = torch.empty((E, H, I // group), dtype=torch.bfloat16, device=dev)
        w4_quantize(w13.view(E * I2, H), group, self.w13q.view(E * I2, H // 2),
                    self.w13_scale.view(E * I2, H // group), stream)
        w4_quantize(w2.view(E * H, I), group, self.w2q.view(E * H, I // 2),
                    self.w2_scale.view(E * H, I // group), stream)


def w4_workspace_bytes(cfg: W4Config) -> int:
    return _q("moe_w4_workspace_bytes", cfg)


def alloc_w4_workspace(cfg: W4Config, device):
    import torch
    return torch.empty(max(w4_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def w4_matvec(x, q, scale, y, stream=None) -> None:
    """y [n, rows] = x [n, cols] . w^T for a 4-bit matrix: q [rows, cols/2] u8,
    scale [rows, cols/group] bf16."""
    import torch
    bf, (n, cols), (rows, groups) = torch.bfloat16, x.shape, scale.shape
    group = cols // groups if groups else 0
    if not (_is(x, bf, n, cols) and _is(q, torch.uint8, rows, cols // 2)
            and _is(scale, bf, rows, groups) and _is(y, bf, n, rows)):
        _refuse("w4_matvec", x=(x, bf, n, cols), q=(q, torch.uint8, rows, cols // 2),
                scale=(scale, bf, rows, groups), y=(y, bf, n, rows))
    if group * groups != cols:
        raise ValueError("w4_matvec: %d scales a row do not divide %d columns" % (groups, cols))
    rc = lib().moe_w4_matvec(x.data_ptr(), q.data_ptr(), scale.data_ptr(), n, rows, cols, group,
                             y.data_ptr(), _stream(stream))
    if rc:
        raise MoEError("moe_w4_matvec", rc)


def w4_ffn_forward(cfg: W4Config, topk_ids, topk_p, x, w13q, w13_scale, w2q, w2_scale, y,
                   workspace, add=None, stream=None) -> None:
    """The chosen experts of a decode batch: y[t] = add[t] + sum_k p[t,k] FFN_e(x_t),
    e = topk_ids[t,k] (routes.topk_ids and routes.topk_p of route_align); an id of
    -1 is no route."""
    import torch
    N, H, E, K, I, g = cfg.n_tokens, cfg.hidden, cfg.n_experts, cfg.top_k, cfg.inter, cfg.group
    bf, u8 = torch.bfloat16, torch.uint8
    if g <= 0:
        raise MoEError("moe_w4_ffn_forward", MOE_ERR_INVALID_ARG)
    if not (_is(topk_ids, torch.int32, N, K) and _is(topk_p, torch.float32, N, K) and _is(x, bf, N, H)
            and _is(w13q, u8, E, 2 * I, H // 2) and _is(w13_scale, bf, E, 2 * I, H // g)
            and _is(w2q, u8, E, H, I // 2) and _is(w2_scale, bf, E, H, I // g) and _is(y, bf, N, H)
            and (add is None or _is(add, bf, N, H)) and workspace.is_cuda):
        _refuse("w4_ffn_forward", topk_ids=(topk_ids, torch.int32, N, K),
                topk_p=(topk_p, torch.float32, N, K), x=(x, bf, N, H),
                w13q=(w13q, u8, E, 2 * I, H // 2), w13_scale=(w13_scale, bf, E, 2 * I, H // g),
                w2q=(w2q, u8, E, H, I // 2), w2_scale=(w2_scale, bf, E, H, I // g),
                y=(y, bf, N, H), add=(x if add is None else add, bf, N, H),
                workspace=(workspace, workspace.dtype, *workspace.shape))
    rc = lib().moe_w4_ffn_forward(ctypes.byref(cfg), topk_ids.data_ptr(), topk_p.data_ptr(),
                                  x.data_ptr(), w13q.data_ptr(), w13_scale.data_ptr(),
                                  w2q.data_ptr(), w2_scale.data_ptr(), _ptr(add), y.data_ptr(),
                                  workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if rc:
        raise MoEError("moe_w4_ffn_forward", rc)


# ------------------------------------------------------------------ the layer for a few tokens
def _on(dev: int, t, dtype, *shape) -> bool:
    """_is, on this device."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def _refuse_on(fn: str, dev: int, stream, **named) -> None:
    """Names the first argument that is not what the call needs, as _refuse does; an
    argument that may be None is left out by its caller."""
    import torch
    _refuse(fn, **named)
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("%s: the tensors are on device %d, the current one is %d" % (
            fn, dev, torch.cuda.current_device()))
    for name, (t, *_) in named.items():
        if t.get_device() != dev:
            raise ValueError("%s: %s is on device %d, others on %d" % (fn, name, t.get_device(), dev))
    if stream is not None and stream.device.index != dev:
        raise ValueError("%s: the stream is of device %d, the tensors on %d" % (fn, stream.device.index, dev))


_device = None  # () -> the current device, without the checks of torch.cuda.current_device


def _here(dev: int, stream) -> bool:
    """The device is the current one, and the stream (if any) is one of its own."""
    global _device
    if _device is None:
        import torch
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return dev >= 0 and dev == _device() and (stream is None or stream.device.index == dev)


def _stream_on(dev: int, stream) -> int:
    """_stream, where the current device is known to be dev."""
    if stream is not None:
        return stream.cuda_stream
    return _current[0](dev) if _current else _stream(None)


def few_workspace_bytes(cfg: FewConfig) -> int:
    return _q("moe_few_workspace_bytes", cfg)


def alloc_few_workspace(cfg: FewConfig, device):
    import torch
    return torch.empty(max(few_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def few_forward(cfg: FewConfig, x, w_router, bias, w13, w2, y, workspace, add=None, n_valid=None,
                topk_ids=None, topk_p=None, stream=None) -> None:
    """The whole layer for up to 64 tokens: router, top-K, experts, combine (+ add). y may
    be x, or add, or both. n_valid: a device int32 tensor of one value, the live tokens; later rows
    are left as they are. topk_ids [N,K] i32 and topk_p [N,K] f32 receive the choice."""
    import torch
    N, H, E, K, I = cfg.n_tokens, cfg.hidden, cfg.n_experts, cfg.top_k, cfg.inter
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, x.get_device()
    if not (_on(dev, x, bf, N, H) and _on(dev, w_router, f32, H, E) and (bias is None or _on(dev, bias, f32, E))
            and _on(dev, w13, bf, E, 2 * I, H) and _on(dev, w2, bf, E, H, I) and _on(dev, y, bf, N, H)
            and (add is None or _on(dev, add, bf, N, H)) and (n_valid is None or _on(dev, n_valid, i32, 1))
            and (topk_ids is None or _on(dev, topk_ids, i32, N, K)) and (topk_p is None or _on(dev, topk_p, f32, N, K))
            and workspace.get_device() == dev and workspace.is_contiguous() and _here(dev, stream)):
        named = dict(x=(x, bf, N, H), w_router=(w_router, f32, H, E), bias=(bias, f32, E), w13=(w13, bf, E, 2 * I, H),
                     w2=(w2, bf, E, H, I), y=(y, bf, N, H), add=(add, bf, N, H), n_valid=(n_valid, i32, 1),
                     topk_ids=(topk_ids, i32, N, K), topk_p=(topk_p, f32, N, K),
                     workspace=(workspace, workspace.dtype, *workspace.shape))
        _refuse_on("few_forward", dev, stream, **{k: v for k, v in named.items() if v[0] is not None})
    rc = lib().moe_few_forward(ctypes.byref(cfg), x.data_ptr(), w_router.data_ptr(), _ptr(bias), w13.data_ptr(),
                               w2.data_ptr(), _ptr(add), _ptr(n_valid), y.data_ptr(), _ptr(topk_ids), _ptr(topk_p),
                               workspace.data_ptr(), workspace.nbytes, _stream_on(dev, stream))
    if rc:
        raise MoEError("moe_few_forward", rc)


# ------------------------------------------------------------------ layer norm
def norm_forward(cfg: NormConfig, x, weight, y, bias=None, add=None, sum=None, mean=None, rstd=None,
                 stream=None) -> None:
    """y = norm(x + add) * weight + bias, rows [N,H] bf16, weight and bias [H] f32. With
    add, sum receives x + add (may be x or add): the rows that norm_backward takes, with
    mean (NORM_LAYER only) and rstd [N] f32."""
    import torch
    N, H, bf, f32, dev = cfg.n_tokens, cfg.hidden, torch.bfloat16, torch.float32, x.get_device()
    if not (_on(dev, x, bf, N, H) and _on(dev, weight, f32, H) and _on(dev, y, bf, N, H)
            and (bias is None or _on(dev, bias, f32, H)) and (add is None or _on(dev, add, bf, N, H))
            and (sum is None or _on(dev, sum, bf, N, H)) and (mean is None or _on(dev, mean, f32, N))
            and (rstd is None or _on(dev, rstd, f32, N)) and _here(dev, stream)):
        named = dict(x=(x, bf, N, H), weight=(weight, f32, H), y=(y, bf, N, H), bias=(bias, f32, H), add=(add, bf, N, H),
                     sum=(sum, bf, N, H), mean=(mean, f32, N), rstd=(rstd, f32, N))
        _refuse_on("norm_forward", dev, stream, **{k: v for k, v in named.items() if v[0] is not None})
    rc = lib().moe_norm_forward(ctypes.byref(cfg), x.data_ptr(), _ptr(add), weight.data_ptr(), _ptr(bias), _ptr(sum),
                                y.data_ptr(), _ptr(mean), _ptr(rstd), _stream_on(dev, stream))
    if rc:
        raise MoEError("moe_norm_forward", rc)


def norm_backward_workspace_bytes(cfg: NormConfig) -> int:
    return _q("moe_norm_backward_workspace_bytes", cfg)


def alloc_norm_backward_workspace(cfg: NormConfig, device):
    import torch
    return torch.empty(max(norm_backward_workspace_bytes(cfg), 256), dtype=torch.uint8, device=device)


def norm_backward(cfg: NormConfig, x, weight, mean, rstd, dy, dx, dweight, workspace, dbias=None, dx_add=None,
                  stream=None) -> None:
    """Gradients of norm_forward: dx [N,H] bf16 (+ dx_add, which may be dx) of the rows x
    that were normed (sum, where there was an add), dweight and dbias [H] f32
    (overwritten). mean: None for NORM_RMS."""
    import torch
    N, H, bf, f32, dev = cfg.n_tokens, cfg.hidden, torch.bfloat16, torch.float32, x.get_device()
    if not (_on(dev, x, bf, N, H) and _on(dev, weight, f32, H) and (mean is None or _on(dev, mean, f32, N))
            and _on(dev, rstd, f32, N) and _on(dev, dy, bf, N, H) and _on(dev, dx, bf, N, H)
            and _on(dev, dweight, f32, H) and (dbias is None or _on(dev, dbias, f32, H))
            and (dx_add is None or _on(dev, dx_add, bf, N, H)) and workspace.get_device() == dev
            and workspace.is_contiguous() and _here(dev, stream)):
        named = dict(x=(x, bf, N, H), weight=(weight, f32, H), mean=(mean, f32, N), rstd=(rstd, f32, N), dy=(dy, bf, N, H),
                     dx=(dx, bf, N, H), dweight=(dweight, f32, H), dbias=(dbias, f32, H), dx_add=(dx_add, bf, N, H),
                     workspace=(workspace, workspace.dtype, *workspace.shape))
        _refuse_on("norm_backward", dev, stream, **{k: v for k, v in named.items() if v[0] is not None})
    rc = lib().moe_norm_backward(ctypes.byref(cfg), x.data_ptr(), weight.data_ptr(), _ptr(mean), rstd.data_ptr(),
                                 dy.data_ptr(), _ptr(dx_add), dx.data_ptr(), dweight.data_ptr(), _ptr(dbias),
                                 workspace.data_ptr(), workspace.nbytes, _stream_on(dev, stream))
    if rc:
        raise MoEError("moe_norm_backward", rc)


# ------------------------------------------------------------------ AdamW
class AdamW:
    """AdamW over a list of tensors and their gradient buffers, one launch a step.

    params: f32 or bf16 CUDA tensors of one device; a bf16 one gets an f32 master.
    grads: a buffer each, f32 or bf16, of the same shape (those that ffn_backward,
    router_backward, shared_backward and norm_backward write). Both are used where they
    lie at every step; a step refuses what is not 16-byte aligned, as a view may be. A
    gradient may serve several params, and overlaps none. The state is made on the current
    stream: a step on another one has to come after it. weight_decay: one number, or one a
    tensor. state_bits 32, or 8: E4M3 codes of m and sqrt(v) with one scale per 256 values,
    rounded at random (by a hash of seed, step and place).

    The state is flat, each tensor from a multiple of 256 on (offsets): m, v (f32, or u8
    codes), m_scale and v_scale (8 bits: one f32 per 256), master (of the bf16 params
    alone), and steps [2] i32 on the device (steps[0]: steps taken). Saving these and
    copying them back into another AdamW of the same list resumes it."""

    def __init__(self, params, grads, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, seed=0):
        import torch
        self.params, self.grads = list(params), list(grads)
        P = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * P
        if len(self.grads) != P or len(decay) != P or P == 0:
            raise ValueError("AdamW: %d params, %d gradients, %d weight decays" % (P, len(self.grads), len(decay)))
        if state_bits not in (8, 32):
            raise ValueError("AdamW: state_bits must be 8 or 32, got %r" % (state_bits,))
        bf, f32 = torch.bfloat16, torch.float32
        dev = self.params[0].device
        for i, (p, g) in enumerate(zip(self.params, self.grads)):
            for name, t in (("params", p), ("grads", g)):
                if t.dtype not in (bf, f32) or not t.is_contiguous() or not t.is_cuda or t.device != dev or t.shape != p.shape:
                    raise ValueError("AdamW: %s[%d] must be a contiguous float32 or bfloat16 tensor of shape %s on %s, got %s %s on %s%s" % (
                        name, i, tuple(p.shape), dev if dev.type == "cuda" else "a CUDA device", str(t.dtype).replace("torch.", ""),
                        tuple(t.shape), t.device, "" if t.is_contiguous() else ", not contiguous"))
        # in order of their places: weights, and gradients, which several weights may share
        weights_end = grads_end = 0
        for at, size, weight in sorted([(p.data_ptr(), p.nbytes, True) for p in self.params if p.numel()]
                                       + [(g.data_ptr(), g.nbytes, False) for g in self.grads if g.numel()]):
            if weight and at < weights_end:
                raise ValueError("AdamW: a tensor is in params twice, or two of them overlap")
            if at < (grads_end if weight else weights_end):
                raise ValueError("AdamW: a gradient overlaps a tensor of params")
            if weight:
                weights_end = at + size
            else:
                grads_end = max(grads_end, at + size)
        self.device, self.state_bits = dev, state_bits
        self.cfg = AdamWConfig(betas[0], betas[1], lr, eps, state_bits, seed)
        self.offsets, moffs, at, mat = [], [], 0, 0
        for p in self.params:
            blocks = -(-p.numel() // 256) * 256
            self.offsets.append(at)
            moffs.append(mat)
            at += blocks
            mat += blocks if p.dtype is bf else 0
        kind = torch.uint8 if state_bits == 8 else f32
        self.m, self.v = (torch.zeros(at, dtype=kind, device=dev) for _ in range(2))
        self.m_scale, self.v_scale = (torch.zeros(at // 256, dtype=f32, device=dev) if state_bits == 8 else None for _ in range(2))
        self.master = torch.zeros(mat, dtype=f32, device=dev) if any(p.dtype is bf for p in self.params) else None
        self.steps = torch.zeros(2, dtype=torch.int32, device=dev)
        self._table = (_AdamWTensorC * P)()
        size = 1 if state_bits == 8 else 4
        for i, (p, g) in enumerate(zip(self.params, self.grads)):
            n, a, ma = p.numel(), self.offsets[i], moffs[i]
            master = None
            if p.dtype is bf:
                self.master[ma: ma + n].copy_(p.detach().view(-1))
                master = self.master.data_ptr() + 4 * ma
            scales = [None if s is None else s.data_ptr() + 4 * (a // 256) for s in (self.m_scale, self.v_scale)]
            self._table[i] = _AdamWTensorC(p.data_ptr(), master, g.data_ptr(), self.m.data_ptr() + size * a,
                                           self.v.data_ptr() + size * a, *scales, n, a, float(decay[i]), int(g.dtype is bf))

    def step(self, grad_scale=None, lr=None, stream=None) -> None:
        """One step from the gradients as they are. grad_scale: a device f32 tensor of one
        value that multiplies them (a NaN or an infinity in it skips the step). lr: a
        number from now on, or a device f32 tensor of one value for this call."""
        import torch
        dev, before = self.steps.get_device(), self.cfg.lr
        new = before
        if lr is not None and not isinstance(lr, torch.Tensor):
            new, lr = float(lr), None
        if not ((grad_scale is None or _on(dev, grad_scale, torch.float32, 1)) and (lr is None or _on(dev, lr, torch.float32, 1))
                and _here(dev, stream)):
            named = dict(steps=(self.steps, torch.int32, 2), grad_scale=(grad_scale, torch.float32, 1), lr=(lr, torch.float32, 1))
            _refuse_on("AdamW.step", dev, stream, **{k: v for k, v in named.items() if v[0] is not None})
        self.cfg.lr = new
        rc = lib().moe_adamw_step(ctypes.byref(self.cfg), ctypes.byref(self._table), len(self._table), _ptr(lr),
                                  _ptr(grad_scale), self.steps.data_ptr(), _stream_on(dev, stream))
        if rc:
            self.cfg.lr = before
            raise MoEError("moe_adamw_step", rc)


def launch_count() -> int:
    return int(lib().moe_launch_count())


def device_error() -> int:
    v = ctypes.c_uint32(0)
    _check("moe_device_error", lib().moe_device_error(ctypes.byref(v)))
    return int(v.value)


def ladder_pick(buckets, n: int, max_pad_ratio: float = 0.0) -> int:
    """Index of the bucket a batch of n tokens replays, or -1 for eager."""
    arr = (ctypes.c_int32 * len(buckets))(*buckets)
    return int(lib().moe_ladder_pick(ctypes.cast(arr, ctypes.c_void_p), len(buckets), int(n),
                                     float(max_pad_ratio)))


class Ladder:
    """Captured forward graphs at a ladder of token-count buckets (moe_ladder_*).
    Allocates the layer's buffers for the top bucket (cfg.n_tokens must equal
    the last bucket); x, y, routes, h, o are torch tensors sized for it. A
    forward of n tokens reads x[:n] and writes y[:n]."""

    def __init__(self, cfg: Config, buckets, max_pad_ratio, w_router, bias, w13, w2, device):
        import torch
        self.cfg, self.buckets = cfg, list(buckets)
        dev = torch.device(device)
        N, H = cfg.n_tokens, cfg.hidden
        self.x = torch.zeros((max(N, 1), H), dtype=torch.bfloat16, device=dev)
        self.routes = alloc_routes(cfg, dev)
        self.ws = alloc_workspace(cfg, dev)
        self.h, self.o, self.y = alloc_buffers(cfg, dev)
        self.n_valid = torch.zeros(1, dtype=torch.int32, device=dev)
        self._keep = (w_router, bias, w13, w2)  # the graphs hold their addresses
        self._bufs = _LayerBufsC(self.x.data_ptr(), w_router.data_ptr(), _ptr(bias), w13.data_ptr(),
                                 w2.data_ptr(), self.routes.c(), self.ws.data_ptr(),
                                 self.ws.numel(), self.h.data_ptr(), self.o.data_ptr(),
                                 self.y.data_ptr(), self.n_valid.data_ptr())
        arr = (ctypes.c_int32 * len(self.buckets))(*self.buckets)
        handle = ctypes.c_void_p()
        _check("moe_ladder_create",
               lib().moe_ladder_create(ctypes.byref(cfg), ctypes.cast(arr, ctypes.c_void_p),
                                       len(self.buckets), float(max_pad_ratio),
                                       ctypes.byref(self._bufs), ctypes.byref(handle)))
        self._h = handle

    def forward(self, n: int, stream=None) -> int:
        """One forward of x[:n]; returns the bucket index replayed, -1 for eager."""
        b = ctypes.c_int(0)
        _check("moe_ladder_forward", lib().moe_ladder_forward(self._h, int(n), _stream(stream),
                                                              ctypes.byref(b)))
        return b.value

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().moe_ladder_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
