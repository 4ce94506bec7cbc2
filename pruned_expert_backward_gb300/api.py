"""Python binding of include/lrm.h: the same entry points, taking torch CUDA tensors.

Argument marshalling only (shapes, dtypes, pointers, the current stream); every step of
the pruned backward runs in liblrm.so's kernels.  There is no CPU path: a missing
library, a CPU tensor or a failed status raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
from collections import OrderedDict

import torch

from . import _lib as L


class LrmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        name = L.STATUS_NAMES.get(code, str(code))
        text = L.load().lrm_status_string(code).decode()
        super().__init__(f"{where}: {name} ({text})")


def _ok(code: int, where: str):
    if code != L.LRM_OK:
        raise LrmError(code, where)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return L.LRM_BF16
    if t.dtype == torch.float32:
        return L.LRM_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32")


def _cuda(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _opt(t, name, dtype=None):
    return None if t is None else _cuda(t, name, dtype)


def _stream() -> int:
    # the current device's current stream, without the Stream object (0.2 us instead of 2.9 us a call)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def lrm_workspace_size(T: int, k: int, E: int, H: int, I: int, dtype: torch.dtype) -> int:
    out = C.c_size_t(0)
    dt = L.LRM_BF16 if dtype == torch.bfloat16 else L.LRM_F32
    _ok(L.load().lrm_workspace_size(T, k, E, H, I, dt, C.byref(out)), "lrm_workspace_size")
    return int(out.value)


def lrm_plan_quotas(topk_idx, E, kind, num=0, den=1, cap=0, explicit=None, loads=None, quotas=None,
                    dev_status=None):
    """kind: "ratio" (num/den), "cap" (cap) or "explicit" (explicit int32 [E] tensor)."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    loads = torch.empty(E, dtype=torch.int32, device=dev) if loads is None else loads
    quotas = torch.empty(E, dtype=torch.int32, device=dev) if quotas is None else quotas
    kinds = {"ratio": L.LRM_QUOTA_RATIO, "cap": L.LRM_QUOTA_CAP, "explicit": L.LRM_QUOTA_EXPLICIT}
    _ok(L.load().lrm_plan_quotas(_cuda(topk_idx, "topk_idx", torch.int32), T, k, E, kinds[kind], num, den, cap,
                                 _opt(explicit, "explicit", torch.int32), _cuda(loads, "loads", torch.int32),
                                 _cuda(quotas, "quotas", torch.int32), _opt(dev_status, "dev_status", torch.int32),
                                 _stream()), "lrm_plan_quotas")
    return loads, quotas


def lrm_score(alpha, g, phi, scores=None, dev_status=None):
    T, H = g.shape
    k, I = phi.shape[-2], phi.shape[-1]
    if phi.numel() != T * k * I or alpha.numel() != T * k:
        raise ValueError("alpha [T,k], g [T,H], phi [T,k,I] expected")
    scores = torch.empty(T * k, dtype=torch.float32, device=g.device) if scores is None else scores
    _ok(L.load().lrm_score(_cuda(alpha, "alpha", torch.float32), _cuda(g, "g"), _cuda(phi, "phi", g.dtype), T, k,
                           H, I, _dt(g), _cuda(scores, "scores", torch.float32),
                           _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_score")
    return scores


def lrm_score_norms(alpha, g, phi_sq, scores=None, dev_status=None):
    """LRM score from the forward's ||phi_u||^2 (phi_sq fp32 [T,k] or [T*k]); phi is not read."""
    T, H = g.shape
    k = alpha.numel() // max(T, 1) if T > 0 else alpha.shape[-1]
    if phi_sq.numel() != alpha.numel():
        raise ValueError("alpha and phi_sq must both hold T*k values")
    scores = torch.empty(T * k, dtype=torch.float32, device=g.device) if scores is None else scores
    _ok(L.load().lrm_score_norms(_cuda(alpha, "alpha", torch.float32), _cuda(g, "g"),
                                 _cuda(phi_sq, "phi_sq", torch.float32), T, k, H, _dt(g),
                                 _cuda(scores, "scores", torch.float32), _opt(dev_status, "dev_status", torch.int32),
                                 _stream()), "lrm_score_norms")
    return scores


def lrm_route(logits, k, kind, num=0, den=1, cap=0, explicit=None, topk_idx=None, alpha=None, loads=None,
              quotas=None, ws=None, dev_status=None):
    """Router top-k + softmax weights + loads + quotas in one launch.  logits fp32 [T,E].
    Returns topk_idx int32 [T,k], alpha fp32 [T,k], loads int32 [E], quotas int32 [E]."""
    T, E = logits.shape
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    topk_idx = torch.empty(T, k, **i32) if topk_idx is None else topk_idx
    alpha = torch.empty(T, k, dtype=torch.float32, device=dev) if alpha is None else alpha
    loads = torch.empty(E, **i32) if loads is None else loads
    quotas = torch.empty(E, **i32) if quotas is None else quotas
    ws = torch.empty(4 * (E + 1), dtype=torch.uint8, device=dev) if ws is None else ws
    kinds = {"ratio": L.LRM_QUOTA_RATIO, "cap": L.LRM_QUOTA_CAP, "explicit": L.LRM_QUOTA_EXPLICIT}
    _ok(L.load().lrm_route(_cuda(logits, "logits", torch.float32), T, E, k, kinds[kind], num, den, cap,
                           _opt(explicit, "explicit", torch.int32), _cuda(topk_idx, "topk_idx", torch.int32),
                           _cuda(alpha, "alpha", torch.float32), _cuda(loads, "loads", torch.int32),
                           _cuda(quotas, "quotas", torch.int32), _cuda(ws, "ws"), ws.numel(),
                           _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_route")
    return topk_idx, alpha, loads, quotas


def lrm_swiglu_forward(h, phi=None, phi_sq=None, norms=True):
    """phi = SiLU(gate) * up of rows h [..., 2I] (gate first), plus ||phi||^2 per row when norms."""
    I = h.shape[-1] // 2
    P = h.numel() // (2 * I)
    phi = torch.empty(*h.shape[:-1], I, dtype=h.dtype, device=h.device) if phi is None else phi
    if norms and phi_sq is None:
        phi_sq = torch.empty(h.shape[:-1], dtype=torch.float32, device=h.device)
    _ok(L.load().lrm_swiglu_forward(_cuda(h, "h"), P, I, _dt(h), _cuda(phi, "phi", h.dtype),
                                    _opt(phi_sq if norms else None, "phi_sq", torch.float32), _stream()),
        "lrm_swiglu_forward")
    return phi, (phi_sq if norms else None)


def lrm_score_mode(alpha, g, phi, mode, scores=None, dev_status=None):
    """mode: "lrm", "grad_sq" (||g_t||^2) or "grad_abs" (||g_t||_1); phi gives k and I."""
    T, H = g.shape
    k, I = phi.shape[-2], phi.shape[-1]
    modes = {"lrm": L.LRM_SCORE_LRM, "grad_sq": L.LRM_SCORE_GRAD_SQ, "grad_abs": L.LRM_SCORE_GRAD_ABS}
    scores = torch.empty(T * k, dtype=torch.float32, device=g.device) if scores is None else scores
    _ok(L.load().lrm_score_mode(_opt(alpha, "alpha", torch.float32), _cuda(g, "g"), _opt(phi, "phi", g.dtype), T, k,
                                H, I, _dt(g), modes[mode], _cuda(scores, "scores", torch.float32),
                                _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_score_mode")
    return scores


def lrm_select(topk_idx, scores, quotas, E, cap=None, seg_offsets=None, kept_pair=None, row_of_pair=None,
               ws=None, dev_status=None):
    T, k = topk_idx.shape
    P = T * k
    dev = topk_idx.device
    cap = P if cap is None else int(cap)
    seg_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if seg_offsets is None else seg_offsets
    kept_pair = torch.empty(max(cap, 1), dtype=torch.int32, device=dev) if kept_pair is None else kept_pair
    row_of_pair = torch.empty(P, dtype=torch.int32, device=dev) if row_of_pair is None else row_of_pair
    if ws is None:
        ws = torch.empty(lrm_workspace_size(T, k, E, 8, 8, torch.float32), dtype=torch.uint8, device=dev)
    _ok(L.load().lrm_select(_cuda(topk_idx, "topk_idx", torch.int32), _cuda(scores, "scores", torch.float32),
                            _cuda(quotas, "quotas", torch.int32), T, k, E, cap,
                            _cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(kept_pair, "kept_pair", torch.int32),
                            _cuda(row_of_pair, "row_of_pair", torch.int32), _cuda(ws, "ws"), ws.numel(),
                            _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_select")
    return seg_offsets, kept_pair, row_of_pair


def lrm_compact(row_of_pair, alpha, g, x, h, phi, cap, dy_c=None, x_c=None, h_c=None, phi_c=None, dy_only=False,
                dev_status=None, x_only=False, k=None, I=None):
    """dy_only: write only dy_c (the compaction-free variant; x_c, h_c, phi_c are returned as None).
    x_only: write dy_c and x_c (h and phi may be None: the variant that recomputes them; k and I
    must then be given)."""
    T, H = g.shape
    if phi is not None:
        k, I = phi.shape[-2], phi.shape[-1]
    elif k is None or I is None:
        raise ValueError("k and I are needed when phi is not given")
    dev, dt = g.device, g.dtype
    rows = max(int(cap), 1)
    dy_c = torch.empty(rows, H, dtype=dt, device=dev) if dy_c is None else dy_c
    if dy_only:
        x_c = h_c = phi_c = None
    else:
        x_c = torch.empty(rows, H, dtype=dt, device=dev) if x_c is None else x_c
        if x_only:
            h_c = phi_c = None
        else:
            h_c = torch.empty(rows, 2 * I, dtype=dt, device=dev) if h_c is None else h_c
            phi_c = torch.empty(rows, I, dtype=dt, device=dev) if phi_c is None else phi_c
    _ok(L.load().lrm_compact(_cuda(row_of_pair, "row_of_pair", torch.int32), _cuda(alpha, "alpha", torch.float32),
                             _cuda(g, "g"), _opt(x, "x", dt), _opt(h, "h", dt), _opt(phi, "phi", dt), T, k, H, I,
                             _dt(g), int(cap), _cuda(dy_c, "dy_c", dt), _opt(x_c, "x_c", dt),
                             _opt(h_c, "h_c", dt), _opt(phi_c, "phi_c", dt),
                             _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_compact")
    return dy_c, x_c, h_c, phi_c


def lrm_grouped_backward(seg_offsets, dy_c, x_c, h_c, phi_c, w_gate_up, w_down, cap, dw_gate_up=None,
                         dw_down=None, dh_c=None, dx_c=None, ws=None, flags=L.LRM_GEMM_DEFAULT, dev_status=None,
                         row_dot=None):
    """row_dot: optional fp32 [cap] output (dphi . phi of each retained row, for lrm_router_grad)."""
    E, H, I = w_down.shape
    dev, dt = w_down.device, w_down.dtype
    rows = max(int(cap), 1)
    dw_gate_up = torch.empty(E, 2 * I, H, dtype=torch.float32, device=dev) if dw_gate_up is None else dw_gate_up
    dw_down = torch.empty(E, H, I, dtype=torch.float32, device=dev) if dw_down is None else dw_down
    dh_c = torch.empty(rows, 2 * I, dtype=dt, device=dev) if dh_c is None else dh_c
    dx_c = torch.empty(rows, H, dtype=dt, device=dev) if dx_c is None else dx_c
    if ws is None:
        ws_rows = int(cap) if row_dot is not None else 0
        ws = torch.empty(lrm_workspace_size(ws_rows, 1, E, H, I, dt), dtype=torch.uint8, device=dev)
    _ok(L.load().lrm_grouped_backward(
        _cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(dy_c, "dy_c", dt), _cuda(x_c, "x_c", dt),
        _cuda(h_c, "h_c", dt), _cuda(phi_c, "phi_c", dt), _cuda(w_gate_up, "w_gate_up", dt),
        _cuda(w_down, "w_down", dt), E, H, I, _dt(w_down), int(cap),
        _cuda(dw_gate_up, "dw_gate_up", torch.float32), _cuda(dw_down, "dw_down", torch.float32),
        _cuda(dh_c, "dh_c", dt), _cuda(dx_c, "dx_c", dt), _opt(row_dot, "row_dot", torch.float32),
        _cuda(ws, "ws"), ws.numel(), int(flags),
        _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_grouped_backward")
    return dw_gate_up, dw_down, dh_c, dx_c


def lrm_grouped_backward_gather(seg_offsets, kept_pair, k, dy_c, x, h, phi, w_gate_up, w_down, cap,
                                dw_gate_up=None, dw_down=None, dh_c=None, dx_c=None, ws=None,
                                flags=L.LRM_GEMM_DEFAULT, dev_status=None, row_dot=None):
    """Compaction-free grouped backward: x [T,H], h [T,k,2I], phi [T,k,I] read in place via kept_pair."""
    E, H, I = w_down.shape
    dev, dt = w_down.device, w_down.dtype
    rows = max(int(cap), 1)
    dw_gate_up = torch.empty(E, 2 * I, H, dtype=torch.float32, device=dev) if dw_gate_up is None else dw_gate_up
    dw_down = torch.empty(E, H, I, dtype=torch.float32, device=dev) if dw_down is None else dw_down
    dh_c = torch.empty(rows, 2 * I, dtype=dt, device=dev) if dh_c is None else dh_c
    dx_c = torch.empty(rows, H, dtype=dt, device=dev) if dx_c is None else dx_c
    if ws is None:
        ws_rows = int(cap) if row_dot is not None else 0
        ws = torch.empty(lrm_workspace_size(ws_rows, 1, E, H, I, dt), dtype=torch.uint8, device=dev)
    _ok(L.load().lrm_grouped_backward_gather(
        _cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(kept_pair, "kept_pair", torch.int32), x.shape[0], int(k),
        _cuda(dy_c, "dy_c", dt), _cuda(x, "x", dt), _cuda(h, "h", dt), _cuda(phi, "phi", dt),
        _cuda(w_gate_up, "w_gate_up", dt), _cuda(w_down, "w_down", dt), E, H, I, _dt(w_down), int(cap),
        _cuda(dw_gate_up, "dw_gate_up", torch.float32), _cuda(dw_down, "dw_down", torch.float32),
        _cuda(dh_c, "dh_c", dt), _cuda(dx_c, "dx_c", dt), _opt(row_dot, "row_dot", torch.float32),
        _cuda(ws, "ws"), ws.numel(), int(flags), _opt(dev_status, "dev_status", torch.int32), _stream()),
        "lrm_grouped_backward_gather")
    return dw_gate_up, dw_down, dh_c, dx_c


def lrm_recompute_forward(seg_offsets, x_c, w_gate_up, cap, h_c=None, phi_c=None, ws=None, flags=L.LRM_GEMM_DEFAULT,
                          dev_status=None):
    """h_c = W_gate_up[e] x_c and phi_c = SiLU(gate) * up for the retained rows (the saved forward
    state recomputed from x).  Returns (h_c [cap,2I], phi_c [cap,I])."""
    E, I2, H = w_gate_up.shape
    I = I2 // 2
    dev, dt = w_gate_up.device, w_gate_up.dtype
    rows = max(int(cap), 1)
    h_c = torch.empty(rows, 2 * I, dtype=dt, device=dev) if h_c is None else h_c
    phi_c = torch.empty(rows, I, dtype=dt, device=dev) if phi_c is None else phi_c
    if ws is None:
        ws = torch.empty(lrm_workspace_size(0, 1, E, H, I, dt), dtype=torch.uint8, device=dev)
    _ok(L.load().lrm_recompute_forward(_cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(x_c, "x_c", dt),
                                       _cuda(w_gate_up, "w_gate_up", dt), E, H, I, _dt(w_gate_up), int(cap),
                                       _cuda(h_c, "h_c", dt), _cuda(phi_c, "phi_c", dt), _cuda(ws, "ws"), ws.numel(),
                                       int(flags), _opt(dev_status, "dev_status", torch.int32), _stream()),
        "lrm_recompute_forward")
    return h_c, phi_c


def lrm_router_grad(row_of_pair, alpha, row_dot, T, k, cap, dalpha=None):
    """dL/dalpha [T*k] fp32 of the retained pairs (0 for dropped ones) from lrm_grouped_backward's row_dot."""
    dalpha = torch.empty(T * k, dtype=torch.float32, device=alpha.device) if dalpha is None else dalpha
    _ok(L.load().lrm_router_grad(_cuda(row_of_pair, "row_of_pair", torch.int32), _cuda(alpha, "alpha", torch.float32),
                                 _opt(row_dot, "row_dot", torch.float32), T, k, int(cap),
                                 _cuda(dalpha, "dalpha", torch.float32), _stream()), "lrm_router_grad")
    return dalpha


def lrm_scatter_dx(row_of_pair, dx_c, T, k, dx=None, cap=None, dev_status=None):
    """cap: rows of dx_c that row_of_pair may name (default: all of dx_c's rows)."""
    H = dx_c.shape[1]
    cap = dx_c.shape[0] if cap is None else int(cap)
    if cap > dx_c.shape[0]:
        raise ValueError(f"cap {cap} exceeds the {dx_c.shape[0]} rows of dx_c")
    dx = torch.empty(T, H, dtype=dx_c.dtype, device=dx_c.device) if dx is None else dx
    _ok(L.load().lrm_scatter_dx(_cuda(row_of_pair, "row_of_pair", torch.int32), _cuda(dx_c, "dx_c"), T, k, H,
                                _dt(dx_c), cap, _cuda(dx, "dx", dx_c.dtype),
                                _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_scatter_dx")
    return dx


@functools.lru_cache(maxsize=4096)
def _sort_ws(T, k, E):
    out = C.c_size_t(0)
    _ok(L.load().lrm_sort_workspace_size(T, k, E, C.byref(out)), "lrm_sort_workspace_size")
    return int(out.value)


def _same(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _out(t, shape, dtype, device, name):
    """An output and its address: checked if the caller gave it, else made here."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t, _cuda(t, name, dtype)


def _scratch(ws, need, device):
    """(tensor, address, bytes) of a workspace of at least `need` bytes; none is made for 0."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        return ws, ws.data_ptr(), need
    return ws, _cuda(ws, "ws"), ws.numel()


def lrm_sort_tokens(topk_idx, x, E, seg_offsets=None, pair_of_row=None, row_of_pair=None, x_s=None, ws=None,
                    dev_status=None):
    """Tokens sorted by expert.  topk_idx int32 [T,k] (-1: not routed), x [T,H] or None (indices only).
    Returns seg_offsets [E+1], pair_of_row [T*k], row_of_pair [T*k] (int32) and x_s [T*k,H].
    Its gradient is lrm_scatter_dx(row_of_pair, dx_s, T, k)."""
    T, k = topk_idx.shape
    dev, i32 = topk_idx.device, torch.int32
    idx_p = _cuda(topk_idx, "topk_idx", i32)
    seg_offsets, seg_p = _out(seg_offsets, (E + 1,), i32, dev, "seg_offsets")
    pair_of_row, pair_p = _out(pair_of_row, (T * k,), i32, dev, "pair_of_row")
    row_of_pair, row_p = _out(row_of_pair, (T * k,), i32, dev, "row_of_pair")
    if x is None:
        H, dt, x_p, x_s, xs_p = 8, L.LRM_BF16, None, None, None
    else:
        if x.dim() != 2 or x.shape[0] != T:
            raise ValueError(f"x must be [T,H] with T = {T}, got {list(x.shape)}")
        H, dt, x_p = x.shape[1], _dt(x), _cuda(x, "x")
        x_s, xs_p = _out(x_s, (T * k, H), x.dtype, dev, "x_s")
    ws, ws_p, ws_n = _scratch(ws, _sort_ws(T, k, E) if ws is None else 0, dev)
    _ok(L.load().lrm_sort_tokens(idx_p, x_p, T, k, E, H, dt, seg_p, pair_p, row_p, xs_p, ws_p, ws_n,
                                 _opt(dev_status, "dev_status", i32), _stream()), "lrm_sort_tokens")
    return seg_offsets, pair_of_row, row_of_pair, x_s


def lrm_combine(row_of_pair, alpha, y_s, residual=None, y=None, dev_status=None):
    """y [T,H] = residual + sum_j alpha[t,j] * y_s[row_of_pair[t,j]]; alpha fp32 [T,k], y_s [rows,H]."""
    T, k = alpha.shape
    rows, H = y_s.shape
    if row_of_pair.numel() != T * k:
        raise ValueError(f"row_of_pair must hold T*k = {T * k} rows, got {row_of_pair.numel()}")
    y, y_p = _out(y, (T, H), y_s.dtype, y_s.device, "y")
    _same(residual, (T, H), "residual")
    _ok(L.load().lrm_combine(_cuda(row_of_pair, "row_of_pair", torch.int32), _cuda(alpha, "alpha", torch.float32),
                             _cuda(y_s, "y_s"), _opt(residual, "residual", y_s.dtype), T, k, H, _dt(y_s), rows, y_p,
                             _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_combine")
    return y


def lrm_combine_backward(row_of_pair, alpha, dy, y_s, dy_s=None, dalpha=None, dev_status=None):
    """Gradient of lrm_combine: dy_s [rows,H] and dalpha fp32 [T,k].  y_s None: dy_s alone (it must then
    be given, it fixes the row count).  Rows that no pair names are not written: uninitialised memory in a
    dy_s made here."""
    T, k = alpha.shape
    H, dt, dev = dy.shape[1], dy.dtype, dy.device
    if y_s is None and dy_s is None:
        raise ValueError("dy_s must be given when y_s is not")
    rows = (y_s if y_s is not None else dy_s).shape[0]
    if row_of_pair.numel() != T * k:
        raise ValueError(f"row_of_pair must hold T*k = {T * k} rows, got {row_of_pair.numel()}")
    dy_s, dys_p = _out(dy_s, (rows, H), dt, dev, "dy_s")
    dalpha_p = None
    if y_s is None:
        dalpha = None
    elif dalpha is None:
        dalpha, dalpha_p = _out(None, (T, k), torch.float32, dev, "dalpha")
    else:
        if dalpha.numel() != T * k:
            raise ValueError(f"dalpha must hold T*k = {T * k} values, got {dalpha.numel()}")
        dalpha_p = _cuda(dalpha, "dalpha", torch.float32)
    _same(dy, (T, H), "dy")
    _same(y_s, (rows, H), "y_s")
    _ok(L.load().lrm_combine_backward(_cuda(row_of_pair, "row_of_pair", torch.int32),
                                      _cuda(alpha, "alpha", torch.float32), _cuda(dy, "dy"), _opt(y_s, "y_s", dt),
                                      T, k, H, _dt(dy), rows, dys_p, dalpha_p,
                                      _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_combine_backward")
    return dy_s, dalpha


_ACTS = {"none": L.LRM_ACT_NONE, "relu": L.LRM_ACT_RELU, "gelu": L.LRM_ACT_GELU, "silu": L.LRM_ACT_SILU,
         "swiglu": L.LRM_ACT_SWIGLU}


def _act_code(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _experts(w, seg_offsets, name):
    """(E, rows, columns) of a weight [rows, columns], or [E, rows, columns] with segments."""
    if seg_offsets is None:
        if w.dim() != 2:
            raise ValueError(f"{name} must be [N,K] without seg_offsets, got {list(w.shape)}")
        return (1, *w.shape)
    if w.dim() != 3:
        raise ValueError(f"{name} must be [E,N,K] with seg_offsets, got {list(w.shape)}")
    _same(seg_offsets, (w.shape[0] + 1,), "seg_offsets")
    return tuple(w.shape)


@functools.lru_cache(maxsize=4096)
def lrm_linear_workspace_size(R: int, E: int, N: int, K: int, act: str, dtype: torch.dtype,
                              uses: int = L.LRM_LINEAR_USE_ALL) -> int:
    """Scratch bytes of lrm_linear, lrm_act_backward and lrm_linear_backward (N: columns of y), or of those
    in `uses` (LRM_LINEAR_USE_* or-ed)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"unsupported dtype {dtype}: bf16 or fp32")
    out = C.c_size_t(0)
    dt = L.LRM_BF16 if dtype == torch.bfloat16 else L.LRM_F32
    _ok(L.load().lrm_linear_workspace_size_for(uses, R, E, N, K, _act_code(act), dt, C.byref(out)),
        "lrm_linear_workspace_size")
    return int(out.value)


def lrm_linear(x, w, bias=None, residual=None, act="none", seg_offsets=None, save_z=False, out_dtype=None, y=None,
               z=None, ws=None, flags=L.LRM_GEMM_DEFAULT, dev_status=None):
    """y = act(x w^T + bias) + residual; act "none", "relu", "gelu", "silu" or "swiglu" (w: gate rows, then
    up rows).  x [R,K]; w [N',K] and bias [N'], or, with seg_offsets (rows sorted by expert), w [E,N',K] and
    bias [E,N'].  save_z also returns the pre-activation z [R,N'].  out_dtype torch.float32 gives an fp32 y
    from bf16 inputs.  Rows of no segment are not written: uninitialised memory in a y or z made here.
    Returns (y, z or None)."""
    R, K = x.shape
    E, NP, Kw = _experts(w, seg_offsets, "w")
    code, dt, dev = _act_code(act), x.dtype, x.device
    x_p, dt_code = _cuda(x, "x"), _dt(x)
    if Kw != K:
        raise ValueError(f"x has {K} columns, w {Kw}")
    if act == "swiglu" and NP % 2:
        raise ValueError(f"w has {NP} rows: gate and up rows in equal number expected")
    N = NP // 2 if act == "swiglu" else NP
    if bias is not None and bias.numel() != E * NP:
        raise ValueError(f"bias must hold {E * NP} values, got {bias.numel()}")
    if y is not None and out_dtype is None:
        out_dtype = y.dtype
    y, y_p = _out(y, (R, N), dt if out_dtype is None else out_dtype, dev, "y")
    z_p = None
    if save_z or z is not None:
        z, z_p = _out(z, (R, NP), dt, dev, "z")
    _same(residual, (R, N), "residual")
    # bf16 inputs: scratch is taken where it helps (a long reduction over few rows, rows of w off the sectors)
    want = dt_code == L.LRM_F32 or (32 < R <= 1024 and K >= 2560) or (K % 16 and R >= 4096 * E)
    need = 0
    if ws is None and want:
        simt = flags == L.LRM_GEMM_FORCE_SIMT
        need = 256 if simt else lrm_linear_workspace_size(R, E, N, K, act, dt, L.LRM_LINEAR_USE_FORWARD)
    ws, ws_p, ws_n = _scratch(ws, need, dev)
    _ok(L.load().lrm_linear(_opt(seg_offsets, "seg_offsets", torch.int32), x_p, _cuda(w, "w", dt),
                            _opt(bias, "bias", dt), _opt(residual, "residual", y.dtype), R, E, N, K, code, dt_code,
                            _dt(y), y_p, z_p, ws_p, ws_n, int(flags), _opt(dev_status, "dev_status", torch.int32),
                            _stream()), "lrm_linear")
    return y, z


def lrm_act_backward(dy, z, act="none", seg_offsets=None, bias_grad=True, dz=None, db=None, ws=None,
                     dev_status=None):
    """dz = dy * act'(z) [R,N'] and db fp32 [N'] ([E,N'] with seg_offsets), the column sums of dz, unless
    bias_grad is False.  z may be None for act "none".  Rows of no segment are not written: uninitialised
    memory in a dz made here."""
    R, N = dy.shape
    code, dt, dev = _act_code(act), dy.dtype, dy.device
    NP = 2 * N if act == "swiglu" else N
    E = 1 if seg_offsets is None else seg_offsets.numel() - 1
    dy_p, dt_code = _cuda(dy, "dy"), _dt(dy)
    if act != "none" and z is None:
        raise ValueError(f"z is needed for act {act!r}")
    _same(z, (R, NP), "z")
    dz, dz_p = _out(dz, (R, NP), dt, dev, "dz")
    db_p, need = None, 0
    if not bias_grad:
        db = None
    else:
        if db is None:
            db, db_p = _out(None, (NP,) if seg_offsets is None else (E, NP), torch.float32, dev, "db")
        else:
            if db.numel() != E * NP:
                raise ValueError(f"db must hold {E * NP} values, got {db.numel()}")
            db_p = _cuda(db, "db", torch.float32)
        if ws is None:
            need = lrm_linear_workspace_size(R, E, N, 8, act, dt, L.LRM_LINEAR_USE_ACT_BACKWARD)
    ws, ws_p, ws_n = _scratch(ws, need, dev)
    _ok(L.load().lrm_act_backward(_opt(seg_offsets, "seg_offsets", torch.int32), dy_p, _opt(z, "z", dt), R, E, N, code,
                                  dt_code, dz_p, db_p, ws_p, ws_n, _opt(dev_status, "dev_status", torch.int32),
                                  _stream()), "lrm_act_backward")
    return dz, db


def lrm_linear_backward(dz, x, w, seg_offsets=None, need_dx=True, need_dw=True, dx=None, dw=None, ws=None,
                        flags=L.LRM_GEMM_DEFAULT, dev_status=None):
    """Gradients of lrm_linear's product from dz [R,N]: dx [R,K] = dz w and dw fp32 [N,K] = dz^T x ([E,N,K]
    with seg_offsets).  w may be None where dw alone is wanted and given.  Rows of no segment are not written:
    uninitialised memory in a dx made here.  Returns (dx or None, dw or None)."""
    R, N = dz.shape
    if w is None:
        if need_dx or dw is None:
            raise ValueError("w may be None only with need_dx=False and a dw that gives the sizes")
    like = dw if w is None else w
    E, Nw, K = _experts(like, seg_offsets, "w")
    dt, dev = dz.dtype, dz.device
    dz_p, dt_code = _cuda(dz, "dz"), _dt(dz)
    if Nw != N:
        raise ValueError(f"dz has {N} columns, w {Nw} rows")
    _same(x, (R, K), "x")
    dx, dx_p = _out(dx, (R, K), dt, dev, "dx") if need_dx else (None, None)
    dw, dw_p = _out(dw, tuple(like.shape), torch.float32, dev, "dw") if need_dw else (None, None)
    uses = (L.LRM_LINEAR_USE_DX if need_dx else 0) | (L.LRM_LINEAR_USE_DW if need_dw else 0)
    need = lrm_linear_workspace_size(R, E, N, K, "none", dt, uses) if ws is None and uses else 0
    ws, ws_p, ws_n = _scratch(ws, need, dev)
    _ok(L.load().lrm_linear_backward(_opt(seg_offsets, "seg_offsets", torch.int32), dz_p, _cuda(x, "x", dt),
                                     _opt(w, "w", dt), R, E, N, K, dt_code, dx_p, dw_p, ws_p, ws_n, int(flags),
                                     _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_linear_backward")
    return dx, dw


FP8 = torch.float8_e4m3fn
_QBLOCK = 128  # columns of a row, or rows and columns of a weight, that share a scale


def _qblocks(n: int) -> int:
    return -(-n // _QBLOCK)


def lrm_fp8_quantize(x, row_of_pair=None, k=1, glu=False, q=None, scale=None, dev_status=None):
    """Rows in 8 bits: q e4m3 and scale fp32, one for each 128 columns of a row.  x [T,K] bf16 or fp32.
    With row_of_pair int32 [T*k] (lrm_sort_tokens without x) each token's row goes to the rows of its k pairs: q
    [rows,K] (default T*k rows).  Rows that no pair names are not written: uninitialised memory in a q or scale made
    here.  glu: x holds SwiGLU's gate columns, then the up columns, and each half has blocks of its own.
    Returns (q [rows,K], scale [rows, blocks])."""
    T, K = x.shape
    x_p, dt, dev = _cuda(x, "x"), _dt(x), x.device
    cols, per = K, 1
    if glu:
        if row_of_pair is not None or K % 2:
            raise ValueError("glu is for a gradient [R,2N] in place")
        cols, per = K // 2, 2
    if row_of_pair is not None and row_of_pair.numel() != T * k:
        raise ValueError(f"row_of_pair must hold T*k = {T * k} rows, got {row_of_pair.numel()}")
    if row_of_pair is None and k != 1:
        raise ValueError(f"k = {k} needs row_of_pair")
    rows = q.shape[0] if q is not None else scale.shape[0] if scale is not None else T * k
    if row_of_pair is None and rows != T:
        raise ValueError(f"q and scale must have x's {T} rows")
    q, q_p = _out(q, (rows, K), FP8, dev, "q")
    scale, s_p = _out(scale, (rows, per * _qblocks(cols)), torch.float32, dev, "scale")
    _ok(L.load().lrm_fp8_quantize(x_p, _opt(row_of_pair, "row_of_pair", torch.int32), T * per, k, cols, dt, rows * per,
                                  q_p, s_p, _opt(dev_status, "dev_status", torch.int32), _stream()), "lrm_fp8_quantize")
    return q, scale


def lrm_fp8_quantize_weight(w, glu=False, q=None, scale=None):
    """Weights in 8 bits with a scale for each block of 128 x 128: w [N',K] or [E,N',K], bf16 or fp32.  glu: N'
    holds the gate rows, then the up rows, and each half has blocks of its own.  Returns (q like w, scale
    [blocks of rows, blocks of columns], or [E, ...])."""
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [N,K] or [E,N,K], got {list(w.shape)}")
    E, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    w_p, dt, per = _cuda(w, "w"), _dt(w), 2 if glu else 1
    if N % per:
        raise ValueError(f"w has {N} rows: gate and up rows in equal number expected")
    q, q_p = _out(q, tuple(w.shape), FP8, w.device, "q")
    scale, s_p = _out(scale, (*w.shape[:-2], per * _qblocks(N // per), _qblocks(K)), torch.float32, w.device, "scale")
    _ok(L.load().lrm_fp8_quantize_weight(w_p, E * per, N // per, K, dt, q_p, s_p, _stream()), "lrm_fp8_quantize_weight")
    return q, scale


@functools.lru_cache(maxsize=1024)
def _fp8_sizes(w, w_scale, per, seg_offsets, x_scale, R, columns, across):
    """(E, rows, columns) of an 8-bit weight from the operands' shapes, once they have been checked (for each set of
    shapes once: a small call is bound by the host).  The other operand has R rows of `columns`, which are w's columns
    or, across, its rows."""
    if len(w) != (2 if seg_offsets is None else 3):
        raise ValueError(f"w must be {'[N,K] without' if seg_offsets is None else '[E,N,K] with'} seg_offsets, "
                         f"got {list(w)}")
    E, NP, K = (1, *w) if seg_offsets is None else w
    if seg_offsets is not None and seg_offsets != (E + 1,):
        raise ValueError(f"seg_offsets must be {[E + 1]}, got {list(seg_offsets)}")
    if NP % per:
        raise ValueError(f"w has {NP} rows: gate and up rows in equal number expected")
    if columns != (NP if across else K):
        raise ValueError(f"{'dz' if across else 'x'} has {columns} columns, w {f'{NP} rows' if across else K}")
    blocks = per * _qblocks(NP // per)
    for name, got, want in (("w_scale", w_scale, (*w[:-2], blocks, _qblocks(K))),
                            ("dz_scale" if across else "x_scale", x_scale, (R, blocks if across else _qblocks(K)))):
        if got != want:
            raise ValueError(f"{name} must be {list(want)}, got {list(got)}")
    return E, NP, K


def lrm_fp8_linear(x, x_scale, w, w_scale, bias=None, residual=None, act="none", seg_offsets=None, save_z=False, y=None,
                   z=None, dev_status=None):
    """lrm_linear from 8-bit rows (lrm_fp8_quantize) and weights (lrm_fp8_quantize_weight): y = act(x w^T + bias) +
    residual in bf16.  x [R,K], x_scale [R,blocks]; w [N',K] and bias bf16 [N'], or, with seg_offsets (rows sorted by
    expert), w [E,N',K] and bias [E,N'].  save_z also returns the pre-activation z [R,N'].  Rows of no segment are
    not written: uninitialised memory in a y or z made here.  Returns (y, z or None)."""
    R, K = x.shape
    code, dev, b16 = _act_code(act), x.device, torch.bfloat16
    per = 2 if act == "swiglu" else 1
    E, NP, _ = _fp8_sizes(w.shape, w_scale.shape, per, None if seg_offsets is None else seg_offsets.shape,
                          x_scale.shape, R, K, False)
    N = NP // per
    if bias is not None and bias.numel() != E * NP:
        raise ValueError(f"bias must hold {E * NP} values, got {bias.numel()}")
    y, y_p = _out(y, (R, N), b16, dev, "y")
    z_p = None
    if save_z or z is not None:
        z, z_p = _out(z, (R, NP), b16, dev, "z")
    if residual is not None:
        _same(residual, (R, N), "residual")
    _ok(L.load().lrm_fp8_linear(
        None if seg_offsets is None else _cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(x, "x", FP8),
        _cuda(x_scale, "x_scale", torch.float32), _cuda(w, "w", FP8), _cuda(w_scale, "w_scale", torch.float32),
        None if bias is None else _cuda(bias, "bias", b16),
        None if residual is None else _cuda(residual, "residual", b16), R, E, N, K, code, y_p, z_p,
        None if dev_status is None else _cuda(dev_status, "dev_status", torch.int32), _stream()), "lrm_fp8_linear")
    return y, z


def lrm_fp8_linear_backward(dz, dz_scale, w, w_scale, glu=False, seg_offsets=None, dx=None, dev_status=None):
    """Gradient of lrm_fp8_linear's rows, dx [R,K] bf16 = dz w, from dz in 8 bits (lrm_fp8_quantize; glu=True for
    SwiGLU's columns) and the forward's weights.  The weights' gradient is lrm_linear_backward's, from the bf16
    rows.  Rows of no segment are not written: uninitialised memory in a dx made here."""
    R, NP = dz.shape
    per = 2 if glu else 1
    E, _, K = _fp8_sizes(w.shape, w_scale.shape, per, None if seg_offsets is None else seg_offsets.shape,
                         dz_scale.shape, R, NP, True)
    dx, dx_p = _out(dx, (R, K), torch.bfloat16, dz.device, "dx")
    _ok(L.load().lrm_fp8_linear_backward(
        None if seg_offsets is None else _cuda(seg_offsets, "seg_offsets", torch.int32), _cuda(dz, "dz", FP8),
        _cuda(dz_scale, "dz_scale", torch.float32), _cuda(w, "w", FP8), _cuda(w_scale, "w_scale", torch.float32), R, E,
        NP // per, K, per - 1, dx_p, None if dev_status is None else _cuda(dev_status, "dev_status", torch.int32),
        _stream()), "lrm_fp8_linear_backward")
    return dx


class PrunedBackward:
    """The whole pruned expert backward for one fixed problem size, with every buffer
    allocated once (device memory from torch).  `run` queues score -> select -> compact ->
    grouped backward -> scatter on the current stream; no host synchronisation.

    cap defaults to T*k, which can never overflow; a caller that knows sum(min(quota, load))
    may pass it to shrink the compacted buffers.  router_grad=True also produces dL/dalpha of
    every pair (`dalpha`, fp32 [T*k]; 0 for dropped pairs).
    compaction: "materialised" (the pages' physical compaction of dY, x, h, phi), "gather" (only dY
    is compacted; x, h, phi rows are read in place) or "recompute" (the forward kept x and
    ||phi_u||^2 only: dY and x are compacted and h, phi are recomputed for the retained rows)."""

    def __init__(self, T, k, E, H, I, dtype=torch.bfloat16, device="cuda", cap=None, flags=L.LRM_GEMM_DEFAULT,
                 router_grad=False, compaction="materialised"):
        if compaction not in ("materialised", "gather", "recompute"):
            raise ValueError("compaction: 'materialised' (the pages' physical compaction), 'gather' or 'recompute'")
        self.T, self.k, self.E, self.H, self.I = T, k, E, H, I
        self.dtype, self.flags, self.router_grad = dtype, flags, router_grad
        self.gather = compaction == "gather"
        self.recompute = compaction == "recompute"
        self.cap = T * k if cap is None else int(cap)
        dev = torch.device(device)
        rows = max(self.cap, 1)
        i32 = dict(dtype=torch.int32, device=dev)
        self.scores = torch.empty(T * k, dtype=torch.float32, device=dev)
        self.seg_offsets = torch.empty(E + 1, **i32)
        self.kept_pair = torch.empty(rows, **i32)
        self.row_of_pair = torch.empty(max(T * k, 1), **i32)
        self.dy_c = torch.empty(rows, H, dtype=dtype, device=dev)
        # the compaction-free variant keeps x, h, phi where they are
        self.x_c = None if self.gather else torch.empty(rows, H, dtype=dtype, device=dev)
        self.h_c = None if self.gather else torch.empty(rows, 2 * I, dtype=dtype, device=dev)
        self.phi_c = None if self.gather else torch.empty(rows, I, dtype=dtype, device=dev)
        self.dh_c = torch.empty(rows, 2 * I, dtype=dtype, device=dev)
        self.dx_c = torch.empty(rows, H, dtype=dtype, device=dev)
        self.dw_gate_up = torch.empty(E, 2 * I, H, dtype=torch.float32, device=dev)
        self.dw_down = torch.empty(E, H, I, dtype=torch.float32, device=dev)
        self.dx = torch.empty(T, H, dtype=dtype, device=dev)
        self.ws = torch.empty(lrm_workspace_size(T, k, E, H, I, dtype), dtype=torch.uint8, device=dev)
        self.dev_status = torch.zeros(1, **i32)
        self.row_dot = torch.empty(rows, dtype=torch.float32, device=dev) if router_grad else None
        self.dalpha = torch.empty(max(T * k, 1), dtype=torch.float32, device=dev) if router_grad else None

    def run(self, inp, quotas):
        """inp: dict with topk_idx [T,k] int32, alpha [T,k] fp32, x, g [T,H], h [T,k,2I], phi [T,k,I],
        w_gate_up [E,2I,H], w_down [E,H,I] (CUDA), and optionally phi_sq fp32 [T,k] (||phi_u||^2 from
        lrm_swiglu_forward; the score then reads it instead of phi).  quotas: int32 [E] (CUDA).
        compaction="recompute" needs phi_sq and neither h nor phi."""
        if self.recompute:
            return self._run_recompute(inp, quotas)
        if inp.get("phi_sq") is not None:  # the forward handed over ||phi_u||^2
            lrm_score_norms(inp["alpha"], inp["g"], inp["phi_sq"], scores=self.scores, dev_status=self.dev_status)
        else:
            lrm_score(inp["alpha"], inp["g"], inp["phi"], scores=self.scores, dev_status=self.dev_status)
        lrm_select(inp["topk_idx"], self.scores, quotas, self.E, cap=self.cap, seg_offsets=self.seg_offsets,
                   kept_pair=self.kept_pair, row_of_pair=self.row_of_pair, ws=self.ws, dev_status=self.dev_status)
        lrm_compact(self.row_of_pair, inp["alpha"], inp["g"], inp["x"], inp["h"], inp["phi"], self.cap,
                    dy_c=self.dy_c, x_c=self.x_c, h_c=self.h_c, phi_c=self.phi_c, dy_only=self.gather,
                    dev_status=self.dev_status)
        if self.gather:
            lrm_grouped_backward_gather(self.seg_offsets, self.kept_pair, self.k, self.dy_c, inp["x"], inp["h"],
                                        inp["phi"], inp["w_gate_up"], inp["w_down"], self.cap,
                                        dw_gate_up=self.dw_gate_up, dw_down=self.dw_down, dh_c=self.dh_c,
                                        dx_c=self.dx_c, ws=self.ws, flags=self.flags, dev_status=self.dev_status,
                                        row_dot=self.row_dot)
        else:
            lrm_grouped_backward(self.seg_offsets, self.dy_c, self.x_c, self.h_c, self.phi_c, inp["w_gate_up"],
                                 inp["w_down"], self.cap, dw_gate_up=self.dw_gate_up, dw_down=self.dw_down,
                                 dh_c=self.dh_c, dx_c=self.dx_c, ws=self.ws, flags=self.flags,
                                 dev_status=self.dev_status, row_dot=self.row_dot)
        lrm_scatter_dx(self.row_of_pair, self.dx_c, self.T, self.k, dx=self.dx, cap=self.cap,
                       dev_status=self.dev_status)
        if self.router_grad:
            lrm_router_grad(self.row_of_pair, inp["alpha"], self.row_dot, self.T, self.k, self.cap,
                            dalpha=self.dalpha)
        return self

    def _run_recompute(self, inp, quotas):
        if inp.get("phi_sq") is None:
            raise ValueError("compaction='recompute' scores from phi_sq (||phi_u||^2 of the forward)")
        lrm_score_norms(inp["alpha"], inp["g"], inp["phi_sq"], scores=self.scores, dev_status=self.dev_status)
        lrm_select(inp["topk_idx"], self.scores, quotas, self.E, cap=self.cap, seg_offsets=self.seg_offsets,
                   kept_pair=self.kept_pair, row_of_pair=self.row_of_pair, ws=self.ws, dev_status=self.dev_status)
        lrm_compact(self.row_of_pair, inp["alpha"], inp["g"], inp["x"], None, None, self.cap, dy_c=self.dy_c,
                    x_c=self.x_c, x_only=True, k=self.k, I=self.I, dev_status=self.dev_status)
        lrm_recompute_forward(self.seg_offsets, self.x_c, inp["w_gate_up"], self.cap, h_c=self.h_c, phi_c=self.phi_c,
                              ws=self.ws, flags=self.flags, dev_status=self.dev_status)
        lrm_grouped_backward(self.seg_offsets, self.dy_c, self.x_c, self.h_c, self.phi_c, inp["w_gate_up"],
                             inp["w_down"], self.cap, dw_gate_up=self.dw_gate_up, dw_down=self.dw_down,
                             dh_c=self.dh_c, dx_c=self.dx_c, ws=self.ws, flags=self.flags,
                             dev_status=self.dev_status, row_dot=self.row_dot)
        lrm_scatter_dx(self.row_of_pair, self.dx_c, self.T, self.k, dx=self.dx, cap=self.cap,
                       dev_status=self.dev_status)
        if self.router_grad:
            lrm_router_grad(self.row_of_pair, inp["alpha"], self.row_dot, self.T, self.k, self.cap,
                            dalpha=self.dalpha)
        return self

    def outputs(self):
        return {"scores": self.scores, "seg_offsets": self.seg_offsets, "kept_pair": self.kept_pair,
                "row_of_pair": self.row_of_pair, "dy_c": self.dy_c, "x_c": self.x_c, "h_c": self.h_c,
                "phi_c": self.phi_c, "dh_c": self.dh_c, "dx_c": self.dx_c, "dw_gate_up": self.dw_gate_up,
                "dw_down": self.dw_down, "dx": self.dx, "dev_status": self.dev_status,
                "row_dot": self.row_dot, "dalpha": self.dalpha}


class MoeLayer:
    """The expert layer around the routing, forward and unpruned backward, for one fixed problem size with
    every buffer allocated once.  forward: sort by expert, SwiGLU product, down product, weighted way back;
    backward: the gradients of x, alpha and both weights.  Everything is queued on the current stream; no
    host synchronisation.  train=False keeps no state for the backward (serving).
    fp8=True: the products and their rows' gradients run in 8 bits (bf16 in and out, H and I multiples of 16).  Each
    weight is then the pair that lrm_fp8_quantize_weight returns (w_gate_up with glu=True); the weights' gradients
    are taken from the bf16 rows."""

    def __init__(self, T, k, E, H, I, dtype=torch.bfloat16, device="cuda", flags=L.LRM_GEMM_DEFAULT, train=True,
                 fp8=False):
        self.T, self.k, self.E, self.H, self.I = T, k, E, H, I
        self.dtype, self.flags, self.train, self.fp8 = dtype, flags, train, fp8
        if fp8 and (dtype != torch.bfloat16 or flags != L.LRM_GEMM_DEFAULT or H % 16 or I % 16):
            raise ValueError("fp8=True is for bf16 layers with H and I multiples of 16, on the tensor cores")
        dev, P = torch.device(device), T * k
        i32 = dict(dtype=torch.int32, device=dev)
        new = dict(dtype=dtype, device=dev)
        self.seg_offsets = torch.empty(E + 1, **i32)
        self.pair_of_row = torch.empty(P, **i32)
        self.row_of_pair = torch.empty(P, **i32)
        self.x_s = torch.empty(P, H, **new) if train or not fp8 else None
        self.phi_s = torch.empty(P, I, **new)
        self.y_s, self.y = torch.empty(P, H, **new), torch.empty(T, H, **new)
        self.dev_status = torch.zeros(1, **i32)
        uses = 0 if fp8 else L.LRM_LINEAR_USE_FORWARD
        if train:
            uses |= L.LRM_LINEAR_USE_DW | (0 if fp8 else L.LRM_LINEAR_USE_DX)
        ws = _sort_ws(T, k, E)
        if uses:
            ws = max(ws, lrm_linear_workspace_size(P, E, I, H, "swiglu", dtype, uses),
                     lrm_linear_workspace_size(P, E, H, I, "none", dtype, uses))
        if fp8:
            def rows(cols, halves=1):
                return (torch.empty(P, halves * cols, dtype=FP8, device=dev),
                        torch.empty(P, halves * _qblocks(cols), dtype=torch.float32, device=dev))

            self.xq, self.phiq = rows(H), rows(I)
        if train:
            self.h_s, self.dh_s = torch.empty(P, 2 * I, **new), torch.empty(P, 2 * I, **new)
            self.dy_s, self.dphi_s = torch.empty(P, H, **new), torch.empty(P, I, **new)
            self.dx_s, self.dx = torch.empty(P, H, **new), torch.empty(T, H, **new)
            self.dalpha = torch.empty(T, k, dtype=torch.float32, device=dev)
            self.dw_gate_up = torch.empty(E, 2 * I, H, dtype=torch.float32, device=dev)
            self.dw_down = torch.empty(E, H, I, dtype=torch.float32, device=dev)
            if fp8:
                self.dyq, self.dhq = rows(H), rows(I, 2)
        self.ws = torch.empty(ws, dtype=torch.uint8, device=dev)

    def _check_weights(self, *weights):
        if any(isinstance(w, torch.Tensor) == self.fp8 for w in weights):
            raise ValueError("fp8=True takes the pairs of lrm_fp8_quantize_weight, fp8=False the weights")

    def forward(self, x, topk_idx, alpha, w_gate_up, w_down, residual=None):
        """y [T,H] = residual + sum_j alpha[t,j] * w_down[e] SwiGLU(w_gate_up[e] x_t), e = topk_idx[t,j] (-1: none)."""
        self._check_weights(w_gate_up, w_down)
        seg, st = self.seg_offsets, dict(dev_status=self.dev_status)
        # (serving in 8 bits, no row is copied in bf16: a token is rounded once, straight to its rows)
        lrm_sort_tokens(topk_idx, x if self.x_s is not None else None, self.E, seg_offsets=seg,
                        pair_of_row=self.pair_of_row, row_of_pair=self.row_of_pair, x_s=self.x_s, ws=self.ws, **st)
        z = self.h_s if self.train else None
        if self.fp8:
            xq, phiq = self.xq, self.phiq
            lrm_fp8_quantize(x, row_of_pair=self.row_of_pair, k=self.k, q=xq[0], scale=xq[1], **st)
            lrm_fp8_linear(*xq, *w_gate_up, act="swiglu", seg_offsets=seg, y=self.phi_s, z=z, **st)
            lrm_fp8_quantize(self.phi_s, q=phiq[0], scale=phiq[1], **st)
            lrm_fp8_linear(*phiq, *w_down, seg_offsets=seg, y=self.y_s, **st)
        else:
            lrm_linear(self.x_s, w_gate_up, act="swiglu", seg_offsets=seg, y=self.phi_s, z=z, ws=self.ws,
                       flags=self.flags, **st)
            lrm_linear(self.phi_s, w_down, seg_offsets=seg, y=self.y_s, ws=self.ws, flags=self.flags, **st)
        return lrm_combine(self.row_of_pair, alpha, self.y_s, residual=residual, y=self.y, **st)

    def backward(self, dy, alpha, w_gate_up, w_down):
        """Gradients of the last forward: dx [T,H], dalpha [T,k], dw_gate_up, dw_down (the residual's is dy)."""
        if not self.train:
            raise ValueError("MoeLayer(train=False) keeps no state for a backward")
        self._check_weights(w_gate_up, w_down)
        seg, st, kw = self.seg_offsets, dict(dev_status=self.dev_status), dict(ws=self.ws, dev_status=self.dev_status)
        lrm_combine_backward(self.row_of_pair, alpha, dy, self.y_s, dy_s=self.dy_s, dalpha=self.dalpha, **st)
        if self.fp8:
            dyq, dhq = self.dyq, self.dhq
            lrm_linear_backward(self.dy_s, self.phi_s, None, seg_offsets=seg, need_dx=False, dw=self.dw_down, **kw)
            lrm_fp8_quantize(self.dy_s, q=dyq[0], scale=dyq[1], **st)
            lrm_fp8_linear_backward(*dyq, *w_down, seg_offsets=seg, dx=self.dphi_s, **st)
        else:
            lrm_linear_backward(self.dy_s, self.phi_s, w_down, seg_offsets=seg, dx=self.dphi_s, dw=self.dw_down,
                                flags=self.flags, **kw)
        lrm_act_backward(self.dphi_s, self.h_s, act="swiglu", seg_offsets=seg, bias_grad=False, dz=self.dh_s, **kw)
        if self.fp8:
            lrm_linear_backward(self.dh_s, self.x_s, None, seg_offsets=seg, need_dx=False, dw=self.dw_gate_up, **kw)
            lrm_fp8_quantize(self.dh_s, glu=True, q=dhq[0], scale=dhq[1], **st)
            lrm_fp8_linear_backward(*dhq, *w_gate_up, glu=True, seg_offsets=seg, dx=self.dx_s, **st)
        else:
            lrm_linear_backward(self.dh_s, self.x_s, w_gate_up, seg_offsets=seg, dx=self.dx_s, dw=self.dw_gate_up,
                                flags=self.flags, **kw)
        lrm_scatter_dx(self.row_of_pair, self.dx_s, self.T, self.k, dx=self.dx, **st)
        return self.dx, self.dalpha, self.dw_gate_up, self.dw_down


def _on16(n, *addresses):
    """The 16-byte starts that lrm_adamw asks for, looked at before any of several launches."""
    if n and any(p is not None and p % 16 for p in addresses):
        raise LrmError(1, "lrm_adamw")


class _Frozen(dict):
    """Lists of tensors that a launch table holds by address: to be read, not assigned to.  Pickles as an ordinary
    (ordered) dict of lists."""

    def _refuse(self, *args, **kw):
        raise TypeError("AdamW's state is not assigned to: load_state() takes values into it")

    __setitem__ = __delitem__ = __ior__ = clear = pop = popitem = setdefault = update = _refuse

    def __reduce__(self):
        return OrderedDict, ([(key, list(held)) for key, held in self.items()],)


def _storages(tensors):
    return [t.untyped_storage() for t in tensors if t is not None]


class AdamW:
    """AdamW over many tensors at once (lrm_adamw): one or a few launches a step, whatever the number of tensors.

    params: bf16 or fp32 tensors, updated in place.  grads: their gradients, read at every step where they are (the
    layer's dw_gate_up and dw_down stay in place); step(grads=...) takes others.  copies: bf16 tensors that get the
    fp32 params' new values as well.  state_bits 32 keeps both moments in fp32; 8 keeps m and sqrt(v) in e4m3 with a
    scale for 256 elements, rounded at random by `seed`, the step and the element's place (lrm_adamw in lrm.h).
    weight_decay and lr_scale: one value, or one for each tensor.  max_norm: gradients are scaled so that their
    common norm is at most that; a step whose norm is not finite changes nothing and sets LRM_ERR_NONFINITE in
    dev_status (it is not counted in step_dev; in `steps` it is: the host does not learn the norm).
    state: {"m": [...], "v": [...]} and, for 8 bits, "m_scale", "v_scale" to go on from; zeros without.
    The tensors given are the ones that are used, by their addresses: params, copies, grads and state are read-only
    here, load_state takes other values, set_grads other gradients, and a step is refused where a copy, or a param
    without one, lies elsewhere since (param.data = ..., a module moved): make a new AdamW then, with state=opt.state.
    capturable: step and rate live on the device (step_dev, lr_dev), so that a captured step can be replayed."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, copies=None,
                 state_bits=32, state=None, max_norm=None, seed=0, lr_scale=1.0, capturable=False):
        n = len(params)
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        if n == 0:
            raise ValueError("AdamW needs at least one tensor")

        def each(a, name):
            a = list(a) if isinstance(a, (list, tuple)) else [a] * n
            if len(a) != n:
                raise ValueError(f"{name} must hold {n} values, got {len(a)}")
            return a

        self._params, self._copies, self._state_bits = tuple(params), tuple(each(copies, "copies")), state_bits
        self.lr, self.betas, self.eps, self.seed, self.max_norm = lr, betas, eps, seed, max_norm
        decay, scale = each(weight_decay, "weight_decay"), each(lr_scale, "lr_scale")
        dev = self.params[0].device
        for t in self.params:
            _cuda(t, "param")
            _dt(t)
        if state is None:
            kind = (torch.float32, torch.float32) if state_bits == 32 else (torch.uint8, FP8)
            state = {key: [torch.zeros(t.shape, dtype=kind[0], device=t.device).view(kind[1]) for t in self.params]
                     for key in ("m", "v")}
            if state_bits == 8:
                for key in ("m_scale", "v_scale"):
                    state[key] = [torch.zeros(-(-t.numel() // 256), dtype=torch.float32, device=t.device)
                                  for t in self.params]
        self._state = _Frozen({key: tuple(state[key]) for key in self._state_keys()})
        for key, held in self._state.items():
            if len(held) != n:
                raise ValueError(f"state {key} must hold {n} tensors, got {len(held)}")
        # the tensors by the types that share a launch, in order
        self._groups = []
        kinds = {}
        for i, t in enumerate(self.params):
            kinds.setdefault((_dt(t), self.copies[i] is not None), []).append(i)
        for (w_dt, copy), members in kinds.items():
            table = (L.AdamwTensor * len(members))()
            for j, i in enumerate(members):
                t, e = self.params[i], table[j]
                e.w, e.n, e.weight_decay, e.lr_scale, e.id = t.data_ptr(), t.numel(), decay[i], scale[i], i
                if copy:
                    if w_dt != L.LRM_F32:
                        raise TypeError("copies are of fp32 params")
                    _same(self.copies[i], t.shape, "copy")
                    e.copy = _cuda(self.copies[i], "copy", torch.bfloat16)
                for key in ("m", "v"):
                    s = self._state[key][i]
                    if s.numel() != t.numel():
                        raise ValueError(f"state {key} must hold {t.numel()} values, got {s.numel()}")
                    setattr(e, key, _cuda(s, key, torch.float32 if state_bits == 32 else FP8))
                    if state_bits == 8:
                        s = self._state[key + "_scale"][i]
                        if s.numel() != -(-t.numel() // 256):
                            raise ValueError(f"state {key}_scale must hold a value for each 256, got {s.numel()}")
                        setattr(e, key + "_scale", _cuda(s, key + "_scale", torch.float32))
            self._groups.append((w_dt, copy, members, table))
        # what a step writes: two tensors on the same bytes would race
        written = [t for own in (self.params, self.copies, *self._state.values()) for t in own if t is not None]
        spans = sorted((t.data_ptr(), t.numel() * t.element_size()) for t in written if t.numel())
        for (a, n_bytes), (b, _) in zip(spans, spans[1:]):
            if a + n_bytes > b:
                raise ValueError("params, copies and states must not share memory")
        for _, _, _, table in self._groups:
            for e in table:
                _on16(e.n, e.w, e.copy, e.m, e.v)
        # the tables hold addresses: their memory lives as long as they do, whatever becomes of the tensors, and a step
        # looks whether what a model reads, copies or else params, still lies there (54 ns a tensor)
        self._held = _storages(written)
        self._watched = [t if copy is None else copy for t, copy in zip(self.params, self.copies)]
        self._watched_at = list(map(torch.Tensor.data_ptr, self._watched))
        # one table of all tensors for the common norm
        self._all = self._groups[0][3] if len(self._groups) == 1 else (L.AdamwTensor * n)()
        if len(self._groups) > 1:
            for i, t in enumerate(self.params):
                self._all[i].n = t.numel()
        self.set_grads(grads)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.norm = self._ws = None
        if max_norm is not None:
            if not max_norm > 0:
                raise ValueError(f"max_norm must be positive, got {max_norm}")
            out = C.c_size_t(0)
            _ok(L.load().lrm_grad_norm_workspace_size(self._all, n, C.byref(out)), "lrm_grad_norm_workspace_size")
            self.norm = torch.zeros((), dtype=torch.float32, device=dev)
            self._ws = torch.empty(out.value, dtype=torch.uint8, device=dev)
        self.steps = 0
        self.step_dev = torch.zeros(1, dtype=torch.int32, device=dev) if capturable else None
        self.lr_dev = torch.full((1,), lr, dtype=torch.float32, device=dev) if capturable else None

    def set_grads(self, grads):
        """The gradients that the next steps read: one type, bf16 or fp32, for all of them."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} gradients expected, got {len(grads)}")
        g_dt = _dt(grads[0])
        at = []
        for g, t in zip(grads, self.params):
            if g.numel() != t.numel():
                raise ValueError(f"a gradient of {g.numel()} values for a param of {t.numel()}")
            at.append(_cuda(g, "gradient", grads[0].dtype))
        _on16(1, *(p for p, t in zip(at, self.params) if t.numel()))
        for _, _, members, table in self._groups:
            for j, i in enumerate(members):
                table[j].g = at[i]
        if len(self._groups) > 1:
            for i, p in enumerate(at):
                self._all[i].g = p
        self._grads, self._g_dt, self._held_grads = tuple(grads), g_dt, _storages(grads)

    def load_state(self, state):
        """Takes the values of a state like `state` (tensors on any device) into the tensors held here, where captured
        steps read them too."""
        pairs = []
        for key, held in self._state.items():
            given = list(state[key])
            if len(given) != len(held):
                raise ValueError(f"state {key} must hold {len(held)} tensors, got {len(given)}")
            for own, t in zip(held, given):
                if t.numel() != own.numel():
                    raise ValueError(f"state {key} must hold {own.numel()} values, got {t.numel()}")
                if t.dtype != own.dtype:
                    raise TypeError(f"state {key} must be {own.dtype}, got {t.dtype}")
                pairs.append((own, t))
        for own, t in pairs:
            own.copy_(t.reshape(own.shape))

    def _state_keys(self):
        return ("m", "v") if self._state_bits == 32 else ("m", "v", "m_scale", "v_scale")

    params = property(lambda self: self._params)
    copies = property(lambda self: self._copies)
    grads = property(lambda self: self._grads)
    state = property(lambda self: self._state)
    state_bits = property(lambda self: self._state_bits)

    def step(self, step=None, lr=None, grads=None):
        """One step; returns the gradients' norm (fp32 scalar on the device, the same tensor at every step: clone what
        is to be kept) with max_norm, else None.  step: its number, one more than the last by default.  lr: this step's
        rate in place of the one given at first."""
        if grads is not None:
            self.set_grads(grads)
        stream = _stream()
        if self.step_dev is not None:
            if step is not None or lr is not None:
                raise ValueError("a capturable step takes step and rate from step_dev and lr_dev")
        if list(map(torch.Tensor.data_ptr, self._watched)) != self._watched_at:
            raise ValueError("a copy, or a param without one, lies elsewhere than when AdamW was made: make another")
        number = self.steps + 1 if step is None else int(step)
        if number < 1:
            raise ValueError(f"steps count from 1, got {number}")
        h = L.AdamwHyper(self.lr if lr is None else lr, *self.betas, self.eps, number, self.seed & 0xFFFFFFFF,
                         0.0 if self.max_norm is None else self.max_norm, None, None, None)
        lib = L.load()
        if self.step_dev is not None:
            h.step_dev, h.lr_dev = self.step_dev.data_ptr(), self.lr_dev.data_ptr()
        if self.max_norm is not None:
            h.grad_norm = self.norm.data_ptr()
        # values that are refused are so before anything is launched or counted
        _ok(lib.lrm_adamw(None, 0, L.LRM_F32, self._g_dt, self.state_bits, 0, C.byref(h), stream), "lrm_adamw")
        if self.max_norm is not None:
            _ok(lib.lrm_grad_norm(self._all, len(self.params), self._g_dt, h.grad_norm, self._ws.data_ptr(),
                                  self._ws.numel(), self.dev_status.data_ptr(), stream), "lrm_grad_norm")
        if self.step_dev is not None:
            self.step_dev.add_(1 if self.max_norm is None else self.norm < math.inf)
        for w_dt, copy, members, table in self._groups:
            _ok(lib.lrm_adamw(table, len(members), w_dt, self._g_dt, self.state_bits, int(copy), C.byref(h), stream),
                "lrm_adamw")
        if self.step_dev is None:
            self.steps = number
        return self.norm


class HostPipeline:
    """The pruned backward over batches held in pinned host memory.

    Two device copies of the per-step inputs (topk_idx, alpha, x, g, h, phi and the quotas) are
    kept: while step i computes on the current stream, step i+1's inputs travel host -> device on
    a copy stream into the other copy, so transfers overlap compute.  After every step
    its result (dX and seg_offsets) is copied back to pinned host buffers and the host waits for
    it.  The weights stay on the device.  All compute runs in liblrm.so's kernels (through
    PrunedBackward); this class only orders copies with CUDA events."""

    NAMES = ("topk_idx", "alpha", "x", "g", "h", "phi")

    def __init__(self, pb: PrunedBackward, w_gate_up, w_down):
        self.pb = pb
        self.w_gate_up, self.w_down = w_gate_up, w_down
        self.copy_stream = torch.cuda.Stream(device=w_down.device)
        self.sets = [None, None]
        self.quotas = [None, None]
        self.ready = [torch.cuda.Event(), torch.cuda.Event()]
        self.free = [torch.cuda.Event(), torch.cuda.Event()]
        self.dx_host = torch.empty(pb.dx.shape, dtype=pb.dx.dtype).pin_memory()
        self.seg_host = torch.empty(pb.seg_offsets.shape, dtype=torch.int32).pin_memory()

    def _upload(self, slot, host_inp, host_quotas):
        if self.sets[slot] is None:
            self.sets[slot] = {n: torch.empty(host_inp[n].shape, dtype=host_inp[n].dtype,
                                              device=self.w_down.device) for n in self.NAMES}
            self.quotas[slot] = torch.empty(host_quotas.shape, dtype=torch.int32, device=self.w_down.device)
        with torch.cuda.stream(self.copy_stream):
            self.copy_stream.wait_event(self.free[slot])  # the step that last used this slot is done
            for n in self.NAMES:
                self.sets[slot][n].copy_(host_inp[n], non_blocking=True)
            self.quotas[slot].copy_(host_quotas, non_blocking=True)
            self.ready[slot].record(self.copy_stream)

    def run(self, batches, on_result=None):
        """batches: a list of (host_inputs dict, host_quotas int32 [E]) in pinned memory.
        Returns the retained row count of each step (read from the step's seg_offsets).
        on_result(i, dx_host, seg_offsets_host), if given, sees each step's result on the host
        (the buffers are reused by the next step)."""
        retained = []
        if not batches:
            return retained
        cur = torch.cuda.current_stream()
        self._upload(0, *batches[0])
        for i in range(len(batches)):
            slot = i & 1
            if i + 1 < len(batches):
                self._upload(slot ^ 1, *batches[i + 1])
            cur.wait_event(self.ready[slot])
            inp = dict(self.sets[slot], w_gate_up=self.w_gate_up, w_down=self.w_down)
            self.pb.run(inp, self.quotas[slot])
            self.free[slot].record(cur)
            self.dx_host.copy_(self.pb.dx, non_blocking=True)
            self.seg_host.copy_(self.pb.seg_offsets, non_blocking=True)
            cur.synchronize()
            retained.append(int(self.seg_host[-1]))
            if on_result is not None:
                on_result(i, self.dx_host, self.seg_host)
        return retained
