"""Thin ctypes binding of libmoe (C ABI in include/moe.h), one function per
entry point with the same name.

Arguments are torch tensors on the GPU (device memory only -- torch is used for
allocation and streams, never for the computation).  Each wrapper checks device,
dtype, contiguity and sizes before handing raw pointers to the library, so a
wrong tensor raises here instead of reaching a kernel.  Every call enqueues on
``stream`` (default: torch's current stream) and returns without synchronising.
The library is loaded on first use; if it has not been built the call fails.
"""
from __future__ import annotations

import ctypes
import os
import struct
import typing

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SILU = range(5)
_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_UNSUPPORTED",
           3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_HIP"}

_lib = None
_vp, _i, _sz, _d, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double, ctypes.c_int64
_f = ctypes.c_float

_SIGS = {
    "moe_status_string": ([_i], ctypes.c_char_p),
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_abi_version": ([], _i),
    "moe_launch_count": ([], _i64),
    "moe_signal_dh_ready": ([_vp], _i),
    "moe_router_workspace_bytes": ([_i, _i, _i], _sz),
    "moe_router_fwd": ([_i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "moe_route_topk": ([_i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "moe_router_bwd": ([_i, _i, _i, _i, _i] + [_vp] * 8 + [_i, _vp, _sz, _vp], _i),
    "moe_dispatch_workspace_bytes": ([_i, _i, _i], _sz),
    "moe_dispatch": ([_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "moe_dispatch_noalloc": ([_i, _i, _i, _i, _i] + [_vp] * 8, _i),
    "moe_dispatch_noalloc_max_workspace": ([], _sz),
    "moe_grouped_swiglu_fwd": ([_i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "moe_grouped_swiglu_fwd_gather": ([_i] * 7 + [_vp] * 10, _i),
    "moe_grouped_swiglu_recompute": ([_i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _i] + [_vp] * 5, _i),
    "moe_combine": ([_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp], _i),
    "moe_grouped_bwd_dx": ([_i, _i, _i, _i, _i, _i, _i] + [_vp] * 17, _i),
    "moe_grouped_bwd_dw": ([_i, _i, _i, _i, _i, _vp, _vp, _vp, _i] + [_vp] * 8, _i),
    "moe_quota_cap": ([_i, _i, _i, _d], _i64),
    "moe_compact_pairs": ([_i, _i, _i, _i, _i, _i, _d] + [_vp] * 16, _i),
    "moe_compact_pairs_cap": ([_i, _i, _i, _i, _i, _i, _i] + [_vp] * 16, _i),
    "moe_quota_cap_for_budget": ([_i, _i, _i, _i, _i, _i, _i, _i, _sz], _i64),
    "moe_pair_scores": ([_i, _i, _i, _i, _i] + [_vp] * 6, _i),
    "moe_quantize_weights_fp8": ([_i, _i64, _i64] + [_vp] * 6, _i),
    "moe_grouped_swiglu_fwd_fp8w": ([_i] * 5 + [_vp] * 12, _i),
    "moe_grouped_bwd_dx_fp8w": ([_i] * 6 + [_vp] * 19, _i),
    "moe_quantize_rows_fp8": ([_i, _i, _vp, _vp, _vp, _vp], _i),
    "moe_transpose_fp8": ([_i, _i, _i, _vp, _vp, _vp], _i),
    "moe_grouped_swiglu_fwd_fp8": ([_i] * 5 + [_vp] * 15, _i),
    "moe_route_scored": ([_i] * 8 + [_f] + [_vp] * 5, _i),
    "moe_route_scored_bwd": ([_i] * 5 + [_f] + [_vp] * 5, _i),
    "moe_router_bwd_dlogits": ([_i] * 4 + [_vp] * 5 + [_i, _vp, _sz, _vp], _i),
    "moe_layernorm_fwd": ([_i] * 3 + [_f] + [_vp] * 7, _i),
    "moe_layernorm_workspace_bytes": ([_i, _i], _sz),
    "moe_layernorm_bwd": ([_i] * 3 + [_vp] * 10 + [_sz, _vp], _i),
    "moe_linear_workspace_bytes": ([_i] * 4, _sz),
    "moe_linear_fwd": ([_i] * 5 + [_vp] * 8 + [_sz, _vp], _i),
    "moe_linear_bwd": ([_i] * 5 + [_vp] * 12 + [_sz, _vp], _i),
    "moe_balance_loss_workspace_bytes": ([_i] * 3, _sz),
    "moe_balance_loss_fwd": ([_i] * 5 + [_f] + [_vp] * 7 + [_sz, _vp], _i),
    "moe_balance_loss_bwd": ([_i] * 5 + [_f] + [_vp] * 7, _i),
    "moe_vocab_loss_workspace_bytes": ([_i] * 4, _sz),
    "moe_vocab_loss_fwd": ([_i] * 5 + [_vp] * 7 + [_sz, _vp], _i),
    "moe_vocab_loss_bwd": ([_i] * 5 + [_vp] * 7 + [_f] + [_vp] * 3 + [_sz, _vp], _i),
    "moe_adamw_plan_bytes": ([_i], _sz),
    "moe_adamw_plan": ([_i, _vp, _i, _i, _vp, _sz], _i),
    "moe_adamw_moments": ([_i64] + [_vp] * 7, _i),
    "moe_adamw_step": ([_vp] * 4 + [_d] * 3 + [_vp, ctypes.c_uint32, _vp], _i),
}


class MoeError(RuntimeError):
    pass


def lib():
    """Load libmoe.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(rc):
    if rc != 0:
        L = lib()
        raise MoeError(f"{L.moe_status_string(rc).decode()}: {L.moe_last_error().decode()}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dt(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return MOE_F32
    if x.dtype == torch.bfloat16:
        return MOE_BF16
    raise MoeError(f"unsupported dtype {x.dtype}")


def _ptr(t, name, dtype=None, numel=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise MoeError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise MoeError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise MoeError(f"{name} holds {t.numel()} elements, needs {numel}")
    return ctypes.c_void_p(t.data_ptr())


I32, F32 = torch.int32, torch.float32


def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_launch_count() -> int:
    """Kernel launches made so far by library calls from this thread."""
    return int(lib().moe_launch_count())


def moe_dispatch_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(lib().moe_dispatch_workspace_bytes(T, E, k))


def moe_quota_cap(T: int, E: int, k: int, rho: float) -> int:
    return int(lib().moe_quota_cap(T, E, k, float(rho)))


def moe_router_workspace_bytes(T: int, H: int, E: int) -> int:
    return int(lib().moe_router_workspace_bytes(T, H, E))


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def moe_router_fwd(x, w_r, logits, workspace=None, stream=None):
    T, H = x.shape
    E = w_r.shape[1]
    d = x.dtype
    ws, ws_bytes = _ws(workspace)
    _check(lib().moe_router_fwd(T, H, E, _dt(x), _ptr(x, "x", d, T * H), _ptr(w_r, "w_r", d, H * E),
                                _ptr(logits, "logits", F32, T * E), ws, ws_bytes, _stream(stream)))


def moe_router_bwd(x, w_r, topk_idx, topk_w, dg, dlogits, dw_r, dx, accumulate: bool, workspace=None, stream=None):
    T, H = x.shape
    E = w_r.shape[1]
    k = topk_idx.shape[1]
    d = x.dtype
    ws, ws_bytes = _ws(workspace)
    _check(lib().moe_router_bwd(T, H, E, k, _dt(x), _ptr(x, "x", d, T * H), _ptr(w_r, "w_r", d, H * E),
                                _ptr(topk_idx, "topk_idx", I32, T * k), _ptr(topk_w, "topk_w", F32, T * k),
                                _ptr(dg, "dg", F32, T * k), _ptr(dlogits, "dlogits", F32, T * E),
                                _ptr(dw_r, "dw_r", d, H * E), _ptr(dx, "dx", d, T * H), 1 if accumulate else 0,
                                ws, ws_bytes, _stream(stream)))


def moe_route_topk(logits, topk_idx, topk_w, k: int, stream=None):
    T, E = logits.shape
    _check(lib().moe_route_topk(T, E, k, _ptr(logits, "logits", F32, T * E),
                                _ptr(topk_idx, "topk_idx", I32, T * k), _ptr(topk_w, "topk_w", F32, T * k),
                                _stream(stream)))


def moe_dispatch(topk_idx, x, counts, offsets, perm, inv_perm, x_sorted, workspace, E: int, stream=None):
    T, k = topk_idx.shape
    H = x.shape[1] if x is not None else 8
    dt = _dt(x) if x is not None else MOE_BF16
    N = T * k
    ws_need = moe_dispatch_workspace_bytes(T, E, k)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().moe_dispatch(T, H, E, k, dt, _ptr(topk_idx, "topk_idx", I32, N),
                              _ptr(x, "x", None, T * H, allow_none=True), _ptr(counts, "counts", I32, E),
                              _ptr(offsets, "offsets", I32, E + 1), _ptr(perm, "perm", I32, N),
                              _ptr(inv_perm, "inv_perm", I32, N),
                              _ptr(x_sorted, "x_sorted", x.dtype if x is not None else None, N * H, allow_none=True),
                              _ptr(workspace, "workspace", None, None, allow_none=ws_need == 0), ws_bytes,
                              _stream(stream)))


def moe_dispatch_noalloc(topk_idx, x, counts, offsets, perm, inv_perm, x_sorted, E: int, stream=None):
    """moe_dispatch with the library-held workspace (no allocation anywhere)."""
    T, k = topk_idx.shape
    H = x.shape[1] if x is not None else 8
    dt = _dt(x) if x is not None else MOE_BF16
    N = T * k
    _check(lib().moe_dispatch_noalloc(T, H, E, k, dt, _ptr(topk_idx, "topk_idx", I32, N),
                                      _ptr(x, "x", None, T * H, allow_none=True), _ptr(counts, "counts", I32, E),
                                      _ptr(offsets, "offsets", I32, E + 1), _ptr(perm, "perm", I32, N),
                                      _ptr(inv_perm, "inv_perm", I32, N),
                                      _ptr(x_sorted, "x_sorted", x.dtype if x is not None else None, N * H,
                                           allow_none=True),
                                      _stream(stream)))


def moe_dispatch_noalloc_max_workspace() -> int:
    return int(lib().moe_dispatch_noalloc_max_workspace())


def moe_grouped_swiglu_fwd(offsets, x_sorted, w_gate, w_up, w_down, h_save, a_save, o_sorted, max_rows: int,
                           max_expert_rows: int | None = None, stream=None):
    E, H, F = w_gate.shape
    dt, d = _dt(w_gate), w_gate.dtype
    R = max_rows
    _check(lib().moe_grouped_swiglu_fwd(
        H, F, E, R, R if max_expert_rows is None else max_expert_rows, dt, _ptr(offsets, "offsets", I32, E + 1), _ptr(x_sorted, "x_sorted", d, R * H),
        _ptr(w_gate, "w_gate", d, E * H * F), _ptr(w_up, "w_up", d, E * H * F), _ptr(w_down, "w_down", d, E * F * H),
        _ptr(h_save, "h_save", d, R * 2 * F, allow_none=True), _ptr(a_save, "a_save", d, R * F),
        _ptr(o_sorted, "o_sorted", d, R * H), _stream(stream)))


class Fp8Weights:
    """Frozen expert weights stored once in fp8 (E4M3) by moe_quantize_weights_fp8:
    codes q_gate/q_up [E,H,F], q_down [E,F,H] (uint8) and per-expert fp32 scales
    s_gu (shared by W_gate and W_up) and s_down [E]."""

    def __init__(self, w_gate, w_up, w_down, stream=None):
        E, H, F = w_gate.shape
        if w_gate.dtype != torch.bfloat16:
            raise MoeError("fp8 storage is made from bf16 weights")
        dev = w_gate.device
        self.E, self.H, self.F = E, H, F
        self.q_gate = torch.empty(E, H, F, dtype=torch.uint8, device=dev)
        self.q_up = torch.empty(E, H, F, dtype=torch.uint8, device=dev)
        self.q_down = torch.empty(E, F, H, dtype=torch.uint8, device=dev)
        self.s_gu = torch.empty(E, dtype=F32, device=dev)
        self.s_down = torch.empty(E, dtype=F32, device=dev)
        moe_quantize_weights_fp8(w_gate, w_up, self.q_gate, self.q_up, self.s_gu, stream)
        moe_quantize_weights_fp8(w_down, None, self.q_down, None, self.s_down, stream)


class Fp8KMajorWeights:
    """fp8 (E4M3) weight codes in the K-major layout of the fp8 matrix-core
    forward (moe_grouped_swiglu_fwd_fp8): W_gate^T, W_up^T [E,F,H] and
    W_down^T [E,H,F] codes, transposed once from Fp8Weights' codes, with the
    same per-expert scales."""

    def __init__(self, wq: "Fp8Weights", stream=None):
        E, H, F = wq.E, wq.H, wq.F
        dev = wq.q_gate.device
        self.E, self.H, self.F = E, H, F
        self.t_gate = torch.empty(E, F, H, dtype=torch.uint8, device=dev)
        self.t_up = torch.empty(E, F, H, dtype=torch.uint8, device=dev)
        self.t_down = torch.empty(E, H, F, dtype=torch.uint8, device=dev)
        self.s_gu, self.s_down = wq.s_gu, wq.s_down
        moe_transpose_fp8(wq.q_gate, self.t_gate, stream)
        moe_transpose_fp8(wq.q_up, self.t_up, stream)
        moe_transpose_fp8(wq.q_down, self.t_down, stream)


def moe_transpose_fp8(q_in, q_out, stream=None):
    E, rows, cols = q_in.shape
    U8 = torch.uint8
    _check(lib().moe_transpose_fp8(E, rows, cols, _ptr(q_in, "in", U8, E * rows * cols),
                                   _ptr(q_out, "out", U8, E * rows * cols), _stream(stream)))


def moe_quantize_rows_fp8(x, q, scale, stream=None):
    rows, cols = x.shape
    _check(lib().moe_quantize_rows_fp8(rows, cols, _ptr(x, "x", torch.bfloat16, rows * cols),
                                       _ptr(q, "q", torch.uint8, rows * cols), _ptr(scale, "scale", F32, rows),
                                       _stream(stream)))


def moe_grouped_swiglu_fwd_fp8(offsets, xq, x_scale, wt: Fp8KMajorWeights, h_save, a_save, aq, a_scale, o_sorted,
                               max_rows: int, perm=None, k: int = 1, stream=None):
    """xq / x_scale: quantized rows of x_sorted, or with perm the quantized token
    rows (gathered on load)."""
    E, H, F = wt.E, wt.H, wt.F
    d, U8, R = torch.bfloat16, torch.uint8, max_rows
    nx = (R // k) if perm is not None else R
    _check(lib().moe_grouped_swiglu_fwd_fp8(
        H, F, E, k, R, _ptr(offsets, "offsets", I32, E + 1), _ptr(xq, "xq", U8, nx * H),
        _ptr(x_scale, "x_scale", F32, nx), _ptr(perm, "perm", I32, R, allow_none=True),
        _ptr(wt.t_gate, "t_gate", U8, E * F * H), _ptr(wt.t_up, "t_up", U8, E * F * H),
        _ptr(wt.t_down, "t_down", U8, E * H * F), _ptr(wt.s_gu, "s_gu", F32, E), _ptr(wt.s_down, "s_down", F32, E),
        _ptr(h_save, "h_save", d, R * 2 * F, allow_none=True), _ptr(a_save, "a_save", d, R * F),
        _ptr(aq, "aq", U8, R * F), _ptr(a_scale, "a_scale", F32, R), _ptr(o_sorted, "o_sorted", d, R * H),
        _stream(stream)))


def moe_quantize_weights_fp8(w0, w1, q0, q1, scale, stream=None):
    E = w0.shape[0]
    n0 = w0.numel() // E
    n1 = 0 if w1 is None else w1.numel() // E
    U8 = torch.uint8
    _check(lib().moe_quantize_weights_fp8(
        E, n0, n1, _ptr(w0, "w0", torch.bfloat16, E * n0), _ptr(w1, "w1", torch.bfloat16, E * n1, allow_none=True),
        _ptr(q0, "q0", U8, E * n0), _ptr(q1, "q1", U8, E * n1, allow_none=w1 is None), _ptr(scale, "scale", F32, E),
        _stream(stream)))


def moe_grouped_swiglu_fwd_fp8w(offsets, x_rows, wq: Fp8Weights, h_save, a_save, o_sorted, max_rows: int,
                                perm=None, k: int = 1, stream=None):
    """x_rows: x_sorted, or with perm the token matrix x [T, H] (rows gathered on load)."""
    E, H, F = wq.E, wq.H, wq.F
    d, U8, R = torch.bfloat16, torch.uint8, max_rows
    _check(lib().moe_grouped_swiglu_fwd_fp8w(
        H, F, E, k, R, _ptr(offsets, "offsets", I32, E + 1),
        _ptr(x_rows, "x_rows", d, (R // k) * H if perm is not None else R * H),
        _ptr(perm, "perm", I32, R, allow_none=True),
        _ptr(wq.q_gate, "q_gate", U8, E * H * F), _ptr(wq.q_up, "q_up", U8, E * H * F),
        _ptr(wq.q_down, "q_down", U8, E * F * H), _ptr(wq.s_gu, "s_gu", F32, E), _ptr(wq.s_down, "s_down", F32, E),
        _ptr(h_save, "h_save", d, R * 2 * F, allow_none=True), _ptr(a_save, "a_save", d, R * F),
        _ptr(o_sorted, "o_sorted", d, R * H), _stream(stream)))


def moe_grouped_bwd_dx_fp8w(offsets, inv, dy, topk_w, h_rows, wq: Fp8Weights, dO_rows, dh_rows, dX_rows, dx,
                            max_rows: int, inv_all=None, o_sorted=None, dg=None, stream=None, h_src=None):
    T, H = dy.shape
    E, F = wq.E, wq.F
    k = topk_w.shape[1]
    d, U8, R, N = torch.bfloat16, torch.uint8, max_rows, T * k
    _check(lib().moe_grouped_bwd_dx_fp8w(
        T, H, F, E, k, R, _ptr(offsets, "offsets", I32, E + 1), _ptr(inv, "inv", I32, N),
        _ptr(dy, "dy", d, T * H), _ptr(topk_w, "topk_w", F32, N),
        _ptr(h_rows, "h_rows", d, 2 * F if h_src is not None else R * 2 * F),
        _ptr(h_src, "h_src", I32, R, allow_none=True),
        _ptr(wq.q_gate, "q_gate", U8, E * H * F), _ptr(wq.q_up, "q_up", U8, E * H * F),
        _ptr(wq.q_down, "q_down", U8, E * F * H), _ptr(wq.s_gu, "s_gu", F32, E), _ptr(wq.s_down, "s_down", F32, E),
        _ptr(inv_all, "inv_all", I32, N, allow_none=dg is None),
        _ptr(o_sorted, "o_sorted", d, N * H, allow_none=dg is None), _ptr(dg, "dg", F32, N, allow_none=True),
        _ptr(dO_rows, "dO_rows", d, R * H), _ptr(dh_rows, "dh_rows", d, R * 2 * F), _ptr(dX_rows, "dX_rows", d, R * H),
        _ptr(dx, "dx", d, T * H), _stream(stream)))


def moe_grouped_swiglu_fwd_gather(offsets, x, perm, w_gate, w_up, w_down, h_save, a_save, o_sorted, k: int,
                                  max_rows: int, max_expert_rows: int | None = None, stream=None):
    E, H, F = w_gate.shape
    dt, d = _dt(w_gate), w_gate.dtype
    R = max_rows
    T = x.shape[0]
    _check(lib().moe_grouped_swiglu_fwd_gather(
        H, F, E, k, R, R if max_expert_rows is None else max_expert_rows, dt, _ptr(offsets, "offsets", I32, E + 1),
        _ptr(x, "x", d, T * H), _ptr(perm, "perm", I32, R), _ptr(w_gate, "w_gate", d, E * H * F),
        _ptr(w_up, "w_up", d, E * H * F), _ptr(w_down, "w_down", d, E * F * H),
        _ptr(h_save, "h_save", d, R * 2 * F, allow_none=True), _ptr(a_save, "a_save", d, R * F),
        _ptr(o_sorted, "o_sorted", d, R * H), _stream(stream)))


def moe_grouped_swiglu_recompute(offsets, x_rows, w_gate, w_up, h_rows, a_rows, max_rows: int,
                                 max_expert_rows: int | None = None, stream=None, x_src=None, x_div: int = 1):
    """x_src: row s of x is x_rows[x_src[s] / x_div] (rows gathered on load)."""
    E, H, F = w_gate.shape
    dt, d = _dt(w_gate), w_gate.dtype
    R = max_rows
    _check(lib().moe_grouped_swiglu_recompute(
        H, F, E, R, R if max_expert_rows is None else max_expert_rows, dt, _ptr(offsets, "offsets", I32, E + 1),
        _ptr(x_rows, "x_rows", d, H if x_src is not None else R * H), _ptr(x_src, "x_src", I32, R, allow_none=True),
        x_div, _ptr(w_gate, "w_gate", d, E * H * F), _ptr(w_up, "w_up", d, E * H * F),
        _ptr(h_rows, "h_rows", d, R * 2 * F), _ptr(a_rows, "a_rows", d, R * F, allow_none=True), _stream(stream)))


def moe_combine(rows, inv, topk_w, out, k: int, stream=None):
    T, H = out.shape
    d = out.dtype
    rows_needed = int(rows.shape[0])
    _check(lib().moe_combine(T, H, k, _dt(out), _ptr(rows, "rows", d, rows_needed * H), _ptr(inv, "inv", I32, T * k),
                             _ptr(topk_w, "topk_w", F32, T * k, allow_none=True), _ptr(out, "out", d, T * H),
                             _stream(stream)))


def moe_grouped_bwd_dx(offsets, inv, dy, topk_w, h_rows, w_gate, w_up, w_down, dO_rows, dh_rows, dX_rows, dx,
                       max_rows: int, inv_all=None, o_sorted=None, dg=None, stream=None, h_src=None):
    """h_src: row r's pre-activations are h_rows[h_src[r]] (e.g. h_save with kept_src)."""
    T, H = dy.shape
    E, _, F = w_gate.shape
    k = topk_w.shape[1]
    d = dy.dtype
    R = max_rows
    N = T * k
    _check(lib().moe_grouped_bwd_dx(
        T, H, F, E, k, R, _dt(dy), _ptr(offsets, "offsets", I32, E + 1), _ptr(inv, "inv", I32, N), _ptr(dy, "dy", d, T * H), _ptr(topk_w, "topk_w", F32, N),
        _ptr(h_rows, "h_rows", d, 2 * F if h_src is not None else R * 2 * F),
        _ptr(h_src, "h_src", I32, R, allow_none=True),
        _ptr(w_gate, "w_gate", d, E * H * F), _ptr(w_up, "w_up", d, E * H * F),
        _ptr(w_down, "w_down", d, E * F * H), _ptr(inv_all, "inv_all", I32, N, allow_none=dg is None),
        _ptr(o_sorted, "o_sorted", d, N * H, allow_none=dg is None), _ptr(dg, "dg", F32, N, allow_none=True),
        _ptr(dO_rows, "dO_rows", d, R * H), _ptr(dh_rows, "dh_rows", d, R * 2 * F), _ptr(dX_rows, "dX_rows", d, R * H),
        _ptr(dx, "dx", d, T * H), _stream(stream)))


def moe_signal_dh_ready(event):
    """Arm the next moe_grouped_bwd_dx* call of this thread to record `event`
    (a torch.cuda.Event, already created) once dO and dh are written."""
    _check(lib().moe_signal_dh_ready(ctypes.c_void_p(event.cuda_event if event is not None else None)))


def moe_grouped_bwd_dw(offsets, x_rows, a_rows, dO_rows, dh_rows, dw_gate, dw_up, dw_down, max_rows: int, stream=None,
                       x_src=None, x_div: int = 1, a_src=None):
    """x_src / a_src: rows gathered on load (row r of x is x_rows[x_src[r] / x_div],
    row r of a is a_rows[a_src[r]])."""
    E, H, F = dw_gate.shape
    d = dw_gate.dtype
    R = max_rows
    _check(lib().moe_grouped_bwd_dw(
        H, F, E, R, _dt(dw_gate), _ptr(offsets, "offsets", I32, E + 1),
        _ptr(x_rows, "x_rows", d, H if x_src is not None else R * H), _ptr(x_src, "x_src", I32, R, allow_none=True),
        x_div, _ptr(a_rows, "a_rows", d, F if a_src is not None else R * F),
        _ptr(a_src, "a_src", I32, R, allow_none=True),
        _ptr(dO_rows, "dO_rows", d, R * H), _ptr(dh_rows, "dh_rows", d, R * 2 * F),
        _ptr(dw_gate, "dw_gate", d, E * H * F), _ptr(dw_up, "dw_up", d, E * H * F),
        _ptr(dw_down, "dw_down", d, E * F * H), _stream(stream)))


def moe_quota_cap_for_budget(T: int, H: int, F: int, E: int, k: int, dtype, with_dw: bool, keep_graph: bool,
                             budget_bytes: int) -> int:
    dt = MOE_F32 if dtype == torch.float32 else MOE_BF16
    return int(lib().moe_quota_cap_for_budget(T, H, F, E, k, dt, int(bool(with_dw)), int(bool(keep_graph)),
                                              int(budget_bytes)))


def moe_pair_scores(inv_perm, topk_w, a_save, dy, score, stream=None):
    T, H = dy.shape
    k = topk_w.shape[1]
    F = a_save.shape[1]
    d = dy.dtype
    _check(lib().moe_pair_scores(T, H, F, k, _dt(dy), _ptr(inv_perm, "inv_perm", I32, T * k),
                                 _ptr(topk_w, "topk_w", F32, T * k), _ptr(a_save, "a_save", d, None),
                                 _ptr(dy, "dy", d, T * H), _ptr(score, "score", F32, T * k), _stream(stream)))


def moe_compact_pairs(counts, offsets, perm, score, rho, kept_counts, kept_offsets, kept_perm, kept_src,
                      kept_inv, T: int, k: int, x_sorted=None, a_save=None, h_save=None, x_kept=None, a_kept=None,
                      h_kept=None, stream=None, cap=None):
    """Quota from rho (moe_compact_pairs) or, when cap is given, that quota
    directly (moe_compact_pairs_cap; rho is then ignored)."""
    E = counts.shape[0]
    N = T * k
    ref = next((t for t in (x_sorted, a_save, h_save) if t is not None), None)
    d = ref.dtype if ref is not None else torch.bfloat16
    H = x_sorted.shape[1] if x_sorted is not None else 8
    F = a_save.shape[1] if a_save is not None else (h_save.shape[1] // 2 if h_save is not None else 8)
    q = moe_quota_cap(T, E, k, rho) if cap is None else int(cap)
    R = min(N, E * q) if q > 0 else 0
    call = lib().moe_compact_pairs if cap is None else lib().moe_compact_pairs_cap
    _check(call(
        T, H, F, E, k, MOE_F32 if d == torch.float32 else MOE_BF16, float(rho) if cap is None else q,
        _ptr(counts, "counts", I32, E),
        _ptr(offsets, "offsets", I32, E + 1), _ptr(perm, "perm", I32, N), _ptr(score, "score", F32, N),
        _ptr(kept_counts, "kept_counts", I32, E), _ptr(kept_offsets, "kept_offsets", I32, E + 1),
        _ptr(kept_perm, "kept_perm", I32, R), _ptr(kept_src, "kept_src", I32, R), _ptr(kept_inv, "kept_inv", I32, N),
        _ptr(x_sorted, "x_sorted", d, N * H, allow_none=True), _ptr(a_save, "a_save", d, N * F, allow_none=True),
        _ptr(h_save, "h_save", d, N * 2 * F, allow_none=True),
        _ptr(x_kept, "x_kept", d, R * H, allow_none=x_sorted is None),
        _ptr(a_kept, "a_kept", d, R * F, allow_none=a_save is None),
        _ptr(h_kept, "h_kept", d, R * 2 * F, allow_none=h_save is None), _stream(stream)))


# ---- the rest of a MoE block ---------------------------------------------------

def _rows(t, name):
    """The two sizes of a matrix argument."""
    if t is None:
        raise MoeError(f"{name} is required")
    shape = t.shape
    if len(shape) != 2 or 0 in shape:
        raise MoeError(f"{name} must be a matrix with at least one element, got shape {tuple(shape)}")
    if shape[0] > 0x7fffffff or shape[1] > 0x7fffffff:
        raise MoeError(f"{name} has shape {tuple(shape)}, sizes end below 2^31")
    return shape


def _addr(t, name, shape, dtype, dev):
    """The address of a contiguous tensor of exactly this shape and type on the
    current device `dev`, where the kernels run; None for None.  (A decoding
    step's calls are bound by the host: one pass of cheap tests, the message
    only where one fails.)"""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _ptr(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    raise MoeError(f"{name} is on {t.device} in a call on the current device cuda:{dev}")


def _need(t, name, shape, dtype, dev):
    p = _addr(t, name, shape, dtype, dev)
    if p is None:
        raise MoeError(f"{name} is required")
    return p


def _space(workspace, dev):
    """Address and bytes of a workspace."""
    if workspace is None:
        return None, 0
    return _addr(workspace, "workspace", workspace.shape, workspace.dtype, dev), workspace.nbytes  # any shape and type


def _device(t, name):
    """The current device, for a call whose first argument is `t`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MoeError(f"{name} must be a GPU tensor")
    return torch._C._cuda_getDevice()


def _queue(stream, dev):
    """The hipStream_t of a call on device `dev`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if stream.device_index != dev:
        raise MoeError(f"a stream of device cuda:{stream.device_index} in a call on the current device cuda:{dev}")
    return stream.cuda_stream


def moe_route_scored(logits, bias, topk_idx, topk_w, k: int, score: int = MOE_SCORE_SOFTMAX, n_groups: int = 1,
                     top_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                     stream=None):
    """Routing by scores: softmax or sigmoid, an optional selection bias [E], the
    best top_groups of n_groups groups, top-k, weights renormalised or not."""
    dev = _device(logits, "logits")
    T, E = _rows(logits, "logits")
    _check(lib().moe_route_scored(
        T, E, k, score, n_groups, top_groups, group_top, 1 if renormalize else 0, scale,
        _need(logits, "logits", (T, E), F32, dev), _addr(bias, "bias", (E,), F32, dev),
        _need(topk_idx, "topk_idx", (T, k), I32, dev), _need(topk_w, "topk_w", (T, k), F32, dev), _queue(stream, dev)))


def moe_route_scored_bwd(logits, topk_idx, dg, dlogits, score: int = MOE_SCORE_SOFTMAX, renormalize: bool = True,
                         scale: float = 1.0, stream=None):
    """dlogits from dg = dL/dtopk_w, the selection held fixed."""
    dev = _device(logits, "logits")
    T, E = _rows(logits, "logits")
    k = _rows(topk_idx, "topk_idx")[1]
    _check(lib().moe_route_scored_bwd(
        T, E, k, score, 1 if renormalize else 0, scale, _need(logits, "logits", (T, E), F32, dev),
        _need(topk_idx, "topk_idx", (T, k), I32, dev), _need(dg, "dg", (T, k), F32, dev),
        _need(dlogits, "dlogits", (T, E), F32, dev), _queue(stream, dev)))


def moe_router_bwd_dlogits(x, w_r, dlogits, dw_r, dx, accumulate: bool, workspace=None, stream=None):
    """moe_router_bwd's two products for a given dlogits."""
    dev = _device(x, "x")
    T, H = _rows(x, "x")
    E = _rows(w_r, "w_r")[1]
    d = x.dtype
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_router_bwd_dlogits(
        T, H, E, _dt(x), _need(x, "x", (T, H), d, dev), _need(w_r, "w_r", (H, E), d, dev),
        _need(dlogits, "dlogits", (T, E), F32, dev), _need(dw_r, "dw_r", (H, E), d, dev),
        _need(dx, "dx", (T, H), d, dev), 1 if accumulate else 0, ws, ws_bytes, _queue(stream, dev)))


def moe_layernorm_workspace_bytes(T: int, H: int) -> int:
    return int(lib().moe_layernorm_workspace_bytes(T, H))


def moe_layernorm_fwd(x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5, stream=None):
    """y = (x - mean) rstd gamma + beta over rows of H; beta may be None, mean and
    rstd [T] fp32 are kept for the backward when given; y may be x."""
    dev = _device(x, "x")
    T, H = rows = _rows(x, "x")
    d = x.dtype
    _check(lib().moe_layernorm_fwd(
        T, H, _dt(x), eps, _need(x, "x", rows, d, dev), _need(gamma, "gamma", (H,), d, dev),
        _addr(beta, "beta", (H,), d, dev), _need(y, "y", rows, d, dev), _addr(mean, "mean", (T,), F32, dev),
        _addr(rstd, "rstd", (T,), F32, dev), _queue(stream, dev)))


def moe_layernorm_bwd(x, gamma, mean, rstd, dy, dx, dgamma, dbeta, workspace, dx_add=None, stream=None):
    """dx [+ dx_add], dgamma and dbeta (None: not wanted); dx may be dy, x or dx_add."""
    dev = _device(x, "x")
    T, H = rows = _rows(x, "x")
    d = x.dtype
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_layernorm_bwd(
        T, H, _dt(x), _need(x, "x", rows, d, dev), _need(gamma, "gamma", (H,), d, dev),
        _need(mean, "mean", (T,), F32, dev), _need(rstd, "rstd", (T,), F32, dev), _need(dy, "dy", rows, d, dev),
        _addr(dx_add, "dx_add", rows, d, dev), _need(dx, "dx", rows, d, dev), _need(dgamma, "dgamma", (H,), d, dev),
        _addr(dbeta, "dbeta", (H,), d, dev), ws, ws_bytes, _queue(stream, dev)))


def moe_linear_workspace_bytes(T: int, I: int, O: int, dtype) -> int:  # noqa: E741
    """Bytes for moe_linear_fwd and moe_linear_bwd of these sizes (fewer rows may need more)."""
    return int(lib().moe_linear_workspace_bytes(T, I, O, MOE_F32 if dtype == torch.float32 else MOE_BF16))


def moe_linear_fwd(x, w, bias, y, act: int = MOE_ACT_NONE, mul=None, residual=None, z_save=None, workspace=None,
                   stream=None):
    """y = act(x w + bias) [* mul] [+ residual]; z_save keeps x w + bias for the
    backward.  y may be mul or residual.  workspace None: only where the reduction is not split."""
    dev = _device(x, "x")
    T, I = _rows(x, "x")  # noqa: E741
    O = _rows(w, "w")[1]  # noqa: E741
    d, out = x.dtype, (T, O)
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_linear_fwd(
        T, I, O, _dt(x), act, _need(x, "x", (T, I), d, dev), _need(w, "w", (I, O), d, dev),
        _addr(bias, "bias", (O,), d, dev), _addr(mul, "mul", out, d, dev), _addr(residual, "residual", out, d, dev),
        _addr(z_save, "z_save", out, d, dev), _need(y, "y", out, d, dev), ws, ws_bytes, _queue(stream, dev)))


def moe_linear_bwd(x, w, dy, dz, dx, dw, dbias=None, act: int = MOE_ACT_NONE, z=None, mul=None, dmul=None, dx_add=None,
                   workspace=None, stream=None):
    """Gradients of moe_linear_fwd (the residual's is dy): dx [+ dx_add], dw, dbias,
    each skipped when None, and dmul with mul.  z (the forward's z_save) and dz
    (a buffer like dy, or dy or z itself) are needed with an activation or mul."""
    dev = _device(x, "x")
    T, I = _rows(x, "x")  # noqa: E741
    O = _rows(w, "w")[1]  # noqa: E741
    d, into, out = x.dtype, (T, I), (T, O)
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_linear_bwd(
        T, I, O, _dt(x), act, _need(x, "x", into, d, dev), _need(w, "w", (I, O), d, dev), _addr(z, "z", out, d, dev),
        _addr(mul, "mul", out, d, dev), _need(dy, "dy", out, d, dev), _addr(dz, "dz", out, d, dev),
        _addr(dx_add, "dx_add", into, d, dev), _addr(dx, "dx", into, d, dev), _addr(dw, "dw", (I, O), d, dev),
        _addr(dbias, "dbias", (O,), d, dev), _addr(dmul, "dmul", out, d, dev), ws, ws_bytes, _queue(stream, dev)))


# ---- from the block's output to the next step's weights -----------------------------

def moe_balance_loss_workspace_bytes(T: int, E: int, n_seq: int = 1) -> int:
    return int(lib().moe_balance_loss_workspace_bytes(T, E, n_seq))


def moe_balance_loss_fwd(logits, topk_idx, counts, mean_p, loss, workspace=None, score: int = MOE_SCORE_SOFTMAX,
                         alpha: float = 1.0, seq_offsets=None, stream=None):
    """counts and mean_p [n_seq, E] and loss [1] of the routers' balance loss;
    seq_offsets [n_seq + 1] int32, None: one sequence of all rows."""
    dev = _device(logits, "logits")
    T, E = _rows(logits, "logits")
    k = _rows(topk_idx, "topk_idx")[1]
    S = _rows(counts, "counts")[0]
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_balance_loss_fwd(
        T, E, k, S, score, alpha, _need(logits, "logits", (T, E), F32, dev), _need(topk_idx, "topk_idx", (T, k), I32, dev),
        _addr(seq_offsets, "seq_offsets", (S + 1,), I32, dev), _need(counts, "counts", (S, E), I32, dev),
        _need(mean_p, "mean_p", (S, E), F32, dev), _need(loss, "loss", (1,), F32, dev), ws, ws_bytes, _queue(stream, dev)))


def moe_balance_loss_bwd(logits, counts, dlogits, k: int, score: int = MOE_SCORE_SOFTMAX, alpha: float = 1.0,
                         seq_offsets=None, dloss=None, dl_add=None, stream=None):
    """dlogits of the balance loss times dloss [1] (None: 1) [+ dl_add, which may be dlogits]."""
    dev = _device(logits, "logits")
    T, E = rows = _rows(logits, "logits")
    S = _rows(counts, "counts")[0]
    _check(lib().moe_balance_loss_bwd(
        T, E, k, S, score, alpha, _need(logits, "logits", rows, F32, dev), _need(counts, "counts", (S, E), I32, dev),
        _addr(seq_offsets, "seq_offsets", (S + 1,), I32, dev), _addr(dloss, "dloss", (1,), F32, dev),
        _addr(dl_add, "dl_add", rows, F32, dev), _need(dlogits, "dlogits", rows, F32, dev), _queue(stream, dev)))


def moe_vocab_loss_workspace_bytes(T: int, H: int, V: int, dtype) -> int:
    return int(lib().moe_vocab_loss_workspace_bytes(T, H, V, MOE_F32 if dtype == torch.float32 else MOE_BF16))


def moe_vocab_loss_fwd(x, w, target, loss, lse, mean, workspace, vocab: int | None = None, stream=None):
    """loss and lse [T] of the logits x w over the first `vocab` columns (None: all),
    mean = {mean loss, 1 / counted tokens}; targets outside [0, vocab) are not counted."""
    dev = _device(x, "x")
    T, H = rows = _rows(x, "x")
    V = _rows(w, "w")[1]
    d, each = x.dtype, (T,)
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_vocab_loss_fwd(
        T, H, V, V if vocab is None else vocab, _dt(x), _need(x, "x", rows, d, dev), _need(w, "w", (H, V), d, dev),
        _need(target, "target", each, I32, dev), _need(loss, "loss", each, F32, dev), _need(lse, "lse", each, F32, dev),
        _need(mean, "mean", (2,), F32, dev), ws, ws_bytes, _queue(stream, dev)))


def moe_vocab_loss_bwd(x, w, target, loss, lse, mean, dx, dw, workspace, dloss=None, scale: float = 1.0,
                       vocab: int | None = None, stream=None):
    """dx and dw (either may be None) of scale times the mean loss, or of scale times
    the sum of dloss [T] loss (mean may then be None).  A term of dx has one factor that
    is rounded to the type, one of dw two (include/moe.h)."""
    dev = _device(x, "x")
    T, H = rows = _rows(x, "x")
    V = _rows(w, "w")[1]
    d, each = x.dtype, (T,)
    ws, ws_bytes = _space(workspace, dev)
    _check(lib().moe_vocab_loss_bwd(
        T, H, V, V if vocab is None else vocab, _dt(x), _need(x, "x", rows, d, dev), _need(w, "w", (H, V), d, dev),
        _need(target, "target", each, I32, dev), _need(loss, "loss", each, F32, dev), _need(lse, "lse", each, F32, dev),
        _addr(mean, "mean", (2,), F32, dev), _addr(dloss, "dloss", each, F32, dev), scale, _addr(dx, "dx", rows, d, dev),
        _addr(dw, "dw", (H, V), d, dev), ws, ws_bytes, _queue(stream, dev)))


class AdamWTensor(typing.NamedTuple):
    """One tensor of an AdamW step: param and grad (fp32 or bf16), the moments m and
    v (fp32, or uint8 codes with their scales of one fp32 for each 256 elements),
    an fp32 master of a bf16 param, and the weight decay.  Any shapes, contiguous."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    master: torch.Tensor | None = None
    weight_decay: float = 0.0


class _AdamWEntry(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "master")] + [("numel", _i64), ("weight_decay", _d)]


class AdamWPlan:
    """A step's tensors (AdamWTensor each) laid out once for moe_adamw_step, on the
    host and on the current device.  Holds the tensors; they must stay where they are,
    the gradients too: for others it is made anew, which takes the host 2 us a tensor
    and a copy that is waited for."""

    def __init__(self, tensors):
        self.tensors = tensors = [AdamWTensor(*t) for t in tensors]
        if not tensors:
            raise MoeError("a plan needs a tensor")
        self.device_index = dev = _device(tensors[0].param, "param")
        d, small = tensors[0].param.dtype, tensors[0].m.dtype == torch.uint8
        dt, state = _dt(tensors[0].param), torch.uint8 if small else F32

        def address(x, name, dtype, numel):
            if x.dtype is dtype and x.numel() == numel and x.get_device() == dev and x.is_contiguous():
                return x.data_ptr()
            _ptr(x, name, dtype)
            if x.numel() != numel:
                raise MoeError(f"{name} holds {x.numel()} elements, needs {numel}")
            raise MoeError(f"{name} is on {x.device} in a plan on the current device cuda:{dev}")

        words = []
        for t in tensors:
            if any(not isinstance(x, torch.Tensor) for x in t[:4]):
                raise MoeError("param, grad, m and v are tensors")
            if (t.m_scale is None or t.v_scale is None) == small:
                raise MoeError("m_scale and v_scale are given with 8-bit moments, and only then")
            n = t.param.numel()
            scales = [address(x, name, F32, -(-n // 256)) if small else 0
                      for x, name in ((t.m_scale, "m_scale"), (t.v_scale, "v_scale"))]
            words += (address(t.param, "param", d, n), address(t.grad, "grad", d, n), address(t.m, "m", state, n),
                      address(t.v, "v", state, n), *scales, 0 if t.master is None else address(t.master, "master", F32, n), n,
                      float(t.weight_decay))
        entries = struct.pack("8Qd" * len(tensors), *words)  # _AdamWEntry each
        size = int(lib().moe_adamw_plan_bytes(len(tensors)))
        if size == 0:
            raise MoeError(f"a plan of {len(tensors)} tensors is too large")
        self.host = torch.zeros(size, dtype=torch.uint8)
        _check(lib().moe_adamw_plan(len(tensors), entries, dt, 8 if small else 32, self.host.data_ptr(), size))
        self.on_device = self.host.to(torch.device("cuda", dev))


def moe_adamw_step(plan: AdamWPlan, counter, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                   grad_scale=None, seed: int = 0, stream=None):
    """One step over the plan's tensors; counter [2] int32 counts the steps (zeros
    before the first), lr [1] and grad_scale [1] fp32 (None: 1) on the device."""
    dev = _device(counter, "counter")
    if plan.device_index != dev:
        raise MoeError(f"a plan of device cuda:{plan.device_index} in a call on the current device cuda:{dev}")
    _check(lib().moe_adamw_step(
        plan.host.data_ptr(), plan.on_device.data_ptr(), _need(counter, "counter", (2,), I32, dev),
        _need(lr, "lr", (1,), F32, dev), beta1, beta2, eps, _addr(grad_scale, "grad_scale", (1,), F32, dev),
        seed & 0xffffffff, _queue(stream, dev)))


def moe_adamw_moments(m, v, m_scale, v_scale, m_out, v_out, stream=None):
    """The moments that 8-bit codes stand for, in fp32 tensors of the codes' shape."""
    dev = _device(m, "m")
    n, blocks = m.numel(), (-(-m.numel() // 256),)
    _check(lib().moe_adamw_moments(
        n, _need(m, "m", m.shape, torch.uint8, dev), _need(v, "v", m.shape, torch.uint8, dev),
        _need(m_scale, "m_scale", blocks, F32, dev), _need(v_scale, "v_scale", blocks, F32, dev),
        _need(m_out, "m_out", m.shape, F32, dev), _need(v_out, "v_out", m.shape, F32, dev), _queue(stream, dev)))
