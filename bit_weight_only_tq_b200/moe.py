"""Mixture-of-experts calls of libtq.so (include/tq_moe.h): router, exchange of rows between
tokens and experts, and the experts' products with packed low-bit weights.

    weights, ids = tq_moe_route(logits, top_k)               # [T, E] -> [T, top_k]
    offsets, order, pos = tq_moe_sort(ids, E)                # slots sorted by expert
    h = w4g_gemm_experts(x, qweight, scales, offsets, order=order, top_k=top_k)   # [T top_k, N]
    out = tq_moe_combine(y, pos, weights)                    # [T, H]

Argument marshalling only, like the rest of the package; every tensor is contiguous, on one CUDA
device, and that device is the current one.  Each forward call of the exchange has its gradient
beside it; the products' weights are frozen and they have none.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import FMT_TERNARY, FMT_W4G128, PATH_AUTO, PATH_PREFILL, TQ_F16, TQ_F32, HEADER, _check, _i64, _int, _need, _ptr, _vp, header_functions, lib

__all__ = [
    "TQ_BF16", "tq_moe_route", "tq_moe_route_backward", "tq_moe_sort", "tq_moe_gather", "tq_moe_gather_backward",
    "tq_moe_combine", "tq_moe_combine_backward", "tq_gemm_experts", "w4g_gemm_experts", "tq_experts_path",
]

TQ_BF16 = 2
MOE_HEADER = os.path.join(os.path.dirname(HEADER), "tq_moe.h")

_SIGS = {
    "tq_moe_route": [_vp, _int, _vp, _vp, _i64, _i64, _int, _int, _vp],
    "tq_moe_route_backward": [_vp, _vp, _int, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp],
    "tq_moe_sort": [_vp, _vp, _vp, _vp, _i64, _i64, _vp],
    "tq_moe_gather": [_vp, _int, _vp, _vp, _vp, _i64, _i64, _int, _i64, _vp],
    "tq_moe_combine": [_vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp],
    "tq_moe_combine_backward": [_vp, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp],
    "tq_gemm_experts": [_vp] * 8 + [_i64] * 5 + [_int, _int, _vp],
    "w4g_gemm_experts": [_vp] * 9 + [_i64] * 5 + [_int, _int, _vp],
    "tq_experts_path": [_int, _i64, _i64, _i64, _i64, _int],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int

_DTYPES = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}


def moe_header_functions():
    """Names of the functions declared in include/tq_moe.h."""
    return header_functions(MOE_HEADER)


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return d


def _shape(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _device(first, *rest):
    """Every tensor on one device, and that device current: the call runs on the current device."""
    d = first.device
    for t in rest:
        if t is not None and t.device != d:
            raise ValueError(f"tensors on {d} and {t.device}: one device is needed")
    if d.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {d}, but the current device is cuda:{torch.cuda.current_device()}")


def _on(stream):
    """Outputs are allocated for the stream that writes them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raw(stream):
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def tq_moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, weights=None, ids=None, stream=None):
    """softmax(logits [T, E]) and the top_k per token -> (weights fp32 [T, top_k], ids int32 [T, top_k]),
    by decreasing logit, the lowest expert first among equals; renormalize: weights of a token sum to 1."""
    dt = _dtype(logits, "logits")
    _need(logits, logits.dtype, "logits", 2)
    T, E = logits.shape
    with _on(stream):
        if weights is None:
            weights = torch.empty(T, top_k, dtype=torch.float32, device=logits.device)
        if ids is None:
            ids = torch.empty(T, top_k, dtype=torch.int32, device=logits.device)
    _need(weights, torch.float32, "weights", 2)
    _need(ids, torch.int32, "ids", 2)
    _shape(weights, (T, top_k), "weights")
    _shape(ids, (T, top_k), "ids")
    _device(logits, weights, ids)
    _check(lib.tq_moe_route(logits.data_ptr(), dt, weights.data_ptr(), ids.data_ptr(), T, E, top_k, bool(renormalize),
                            _raw(stream)), "tq_moe_route")
    return weights, ids


def tq_moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, weights: torch.Tensor, ids: torch.Tensor,
                          renormalize: bool = True, dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of tq_moe_route: dweights [T, top_k] with the call's logits and results -> dlogits [T, E]."""
    dt = _dtype(logits, "logits")
    _need(logits, logits.dtype, "logits", 2)
    _need(dweights, torch.float32, "dweights", 2)
    _need(weights, torch.float32, "weights", 2)
    _need(ids, torch.int32, "ids", 2)
    T, E = logits.shape
    k = ids.shape[1]
    for t, name in ((dweights, "dweights"), (weights, "weights"), (ids, "ids")):
        _shape(t, (T, k), name)
    if dlogits is None:
        with _on(stream):
            dlogits = torch.empty_like(logits)
    _need(dlogits, logits.dtype, "dlogits", 2)
    _shape(dlogits, (T, E), "dlogits")
    _device(logits, dweights, weights, ids, dlogits)
    _check(lib.tq_moe_route_backward(dweights.data_ptr(), logits.data_ptr(), dt, weights.data_ptr(), ids.data_ptr(),
                                     dlogits.data_ptr(), T, E, k, bool(renormalize), _raw(stream)),
           "tq_moe_route_backward")
    return dlogits


def tq_moe_sort(ids: torch.Tensor, num_experts: int, stream=None):
    """Slots sorted by expert: ids int32 [T, top_k] -> (offsets int32 [E + 1], order int32 [T top_k],
    pos int32 [T, top_k]).  Slots whose id is outside [0, E) come last and have position -1."""
    _need(ids, torch.int32, "ids", 2)
    R = ids.numel()
    with _on(stream):
        offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=ids.device)
        order = torch.empty(R, dtype=torch.int32, device=ids.device)
        pos = torch.empty_like(ids)
    _device(ids)
    _check(lib.tq_moe_sort(ids.data_ptr(), offsets.data_ptr(), order.data_ptr(), pos.data_ptr(), R, num_experts,
                           _raw(stream)), "tq_moe_sort")
    return offsets, order, pos


def tq_moe_gather(x: torch.Tensor, order: torch.Tensor, offsets: torch.Tensor, top_k: int, out=None,
                  stream=None) -> torch.Tensor:
    """rows[r] = x[order[r] // top_k] for the offsets[-1] slots with an expert; later rows of `out` are
    left as they were (uninitialised when it is allocated here)."""
    dt = _dtype(x, "x")
    _need(x, x.dtype, "x", 2)
    _need(order, torch.int32, "order", 1)
    _need(offsets, torch.int32, "offsets", 1)
    T, H = x.shape
    _shape(order, (T * top_k,), "order")
    if out is None:
        with _on(stream):
            out = torch.empty(T * top_k, H, dtype=x.dtype, device=x.device)
    _need(out, x.dtype, "out", 2)
    _shape(out, (T * top_k, H), "out")
    _device(x, order, offsets, out)
    _check(lib.tq_moe_gather(x.data_ptr(), dt, order.data_ptr(), offsets.data_ptr(), out.data_ptr(), T, H, top_k,
                             offsets.shape[0] - 1, _raw(stream)), "tq_moe_gather")
    return out


def tq_moe_combine(y: torch.Tensor, pos: torch.Tensor, weights=None, out=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] y[pos[t, j]] (weights None: 1); zeros for a token without rows."""
    dt = _dtype(y, "y")
    _need(y, y.dtype, "y", 2)
    _need(pos, torch.int32, "pos", 2)
    _need(weights, torch.float32, "weights", 2)
    R, H = y.shape
    T, k = pos.shape
    _shape(weights, (T, k), "weights")
    if out is None:
        with _on(stream):
            out = torch.empty(T, H, dtype=y.dtype, device=y.device)
    _need(out, y.dtype, "out", 2)
    _shape(out, (T, H), "out")
    _device(y, pos, weights, out)
    _check(lib.tq_moe_combine(y.data_ptr(), dt, pos.data_ptr(), _ptr(weights), out.data_ptr(), T, R, H, k,
                              _raw(stream)), "tq_moe_combine")
    return out


def tq_moe_gather_backward(drows: torch.Tensor, pos: torch.Tensor, dx=None, stream=None) -> torch.Tensor:
    """Gradient of tq_moe_gather: dx[t] = sum_j drows[pos[t, j]], summed in fp32 in the order of j."""
    return tq_moe_combine(drows, pos, None, out=dx, stream=stream)


def tq_moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, dy=None,
                            dweights=None, stream=None):
    """Gradients of tq_moe_combine -> (dy like y, dweights fp32 [T, top_k]).  Rows of `dy` that no slot
    names are left as they were (uninitialised when it is allocated here)."""
    dt = _dtype(y, "y")
    _need(y, y.dtype, "y", 2)
    _need(dout, y.dtype, "dout", 2)
    _need(pos, torch.int32, "pos", 2)
    _need(weights, torch.float32, "weights", 2)
    R, H = y.shape
    T, k = pos.shape
    _shape(dout, (T, H), "dout")
    _shape(weights, (T, k), "weights")
    with _on(stream):
        if dy is None:
            dy = torch.empty_like(y)
        if dweights is None:
            dweights = torch.empty_like(weights)
    _need(dy, y.dtype, "dy", 2)
    _need(dweights, torch.float32, "dweights", 2)
    _shape(dy, (R, H), "dy")
    _shape(dweights, (T, k), "dweights")
    _device(y, dout, pos, weights, dy, dweights)
    _check(lib.tq_moe_combine_backward(dout.data_ptr(), y.data_ptr(), dt, pos.data_ptr(), weights.data_ptr(),
                                       dy.data_ptr(), dweights.data_ptr(), T, R, H, k, _raw(stream)),
           "tq_moe_combine_backward")
    return dy, dweights


def _experts(x, w, sc, zeros, offsets, order, top_k, bias, y, per_col, N, E, path, stream, rows, fmt, fn, what):
    _need(x, torch.float16, "x", 2)
    _need(bias, torch.float16, "bias", 2)
    _need(offsets, torch.int32, "offsets", 1)
    _need(order, torch.int32, "order", 1)
    X, K = x.shape
    if w.shape[2] != (K + per_col - 1) // per_col:
        raise ValueError("the weights' last dimension does not match x")
    _shape(offsets, (E + 1,), "offsets")
    _shape(bias, (E, N), "bias")
    R = X if order is None else order.shape[0]
    if y is None:
        with _on(stream):
            y = torch.empty(R, N, dtype=torch.float16, device=x.device)
    _need(y, torch.float16, "y", 2)
    _shape(y, (R, N), "y")
    if order is not None and rows is None and (
            path == PATH_PREFILL or path == PATH_AUTO and lib.tq_experts_path(fmt, R, E, N, K, 1) == PATH_PREFILL):
        with _on(stream):
            rows = torch.empty(R, K, dtype=torch.float16, device=x.device)
    _need(rows, torch.float16, "rows", 2)
    _shape(rows, (R, K), "rows")
    _device(x, w, sc, zeros, offsets, order, bias, y, rows)
    tail = (_ptr(bias), y.data_ptr(), offsets.data_ptr(), _ptr(order), _ptr(rows), X, R, E, N, K, top_k, int(path),
            _raw(stream))
    if what == "w4g_gemm_experts":
        _check(fn(x.data_ptr(), w.data_ptr(), sc.data_ptr(), _ptr(zeros), *tail), what)
    else:
        _check(fn(x.data_ptr(), w.data_ptr(), sc.data_ptr(), *tail), what)
    return y


def tq_gemm_experts(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, offsets: torch.Tensor, order=None,
                    top_k: int = 1, bias=None, y=None, path: int = PATH_AUTO, stream=None, rows=None) -> torch.Tensor:
    """Each expert's rows times its ternary weights: y[r] = x[row(r)] . What_e^T (+ bias_e) for
    offsets[e] <= r < offsets[e + 1]; row(r) = order[r] // top_k with `order` (x holds the tokens), r
    without (x holds sorted rows).  packed uint8 [E, N, ceil(K/4)], scale fp16 [E, N], bias fp16 [E, N].
    Rows from offsets[-1] on are left as they were (uninitialised when y is allocated here).
    rows: fp16 [R, K] scratch for the path that copies the rows first (allocated here when it is needed)."""
    _need(packed, torch.uint8, "packed", 3)
    _need(scale, torch.float16, "scale", 2)
    E, N = packed.shape[:2]
    _shape(scale, (E, N), "scale")
    return _experts(x, packed, scale, None, offsets, order, top_k, bias, y, 4, N, E, path, stream, rows,
                    FMT_TERNARY, lib.tq_gemm_experts, "tq_gemm_experts")


def w4g_gemm_experts(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor, zeros=None,
                     order=None, top_k: int = 1, bias=None, y=None, path: int = PATH_AUTO,
                     stream=None, rows=None) -> torch.Tensor:
    """tq_gemm_experts with W4A16 weights: qweight int32 [E, N, K/8], scales fp16 [E, N, K/128], zeros
    uint8 [E, N, K/128] or None (symmetric)."""
    _need(qweight, torch.int32, "qweight", 3)
    _need(scales, torch.float16, "scales", 3)
    _need(zeros, torch.uint8, "zeros", 3)
    E, N = qweight.shape[:2]
    _shape(scales, (E, N, x.shape[1] // 128), "scales")
    _shape(zeros, scales.shape, "zeros")
    return _experts(x, qweight, scales, zeros, offsets, order, top_k, bias, y, 8, N, E, path, stream, rows,
                    FMT_W4G128, lib.w4g_gemm_experts, "w4g_gemm_experts")


def tq_experts_path(fmt: int, R: int, E: int, N: int, K: int, aligned: bool = True) -> int:
    """The path PATH_AUTO takes for R sorted rows of E experts."""
    return int(lib.tq_experts_path(int(fmt), int(R), int(E), int(N), int(K), 1 if aligned else 0))
