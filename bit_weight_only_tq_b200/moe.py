"""Mixture-of-experts calls of libtq.so (include/tq_moe.h): router, exchange of rows between
tokens and experts, and the experts' products with packed low-bit weights.

    weights, ids = tq_moe_route(logits, top_k)               # [T, E] -> [T, top_k]
    offsets, order, pos = tq_moe_sort(ids, E)                # slots sorted by expert
    h = w4g_gemm_experts(x, qweight, scales, offsets, order=order, top_k=top_k)   # [T top_k, N]
    out = tq_moe_combine(y, pos, weights)                    # [T, H]

Argument marshalling only, like the rest of the package; every tensor is contiguous, on one CUDA
device, and that device is the current one.  Each forward call of the exchange has its gradient
beside it; the products have none yet, for x either, so that a training step takes dx of the experts'
rows from elsewhere.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import (FMT_TERNARY, FMT_W4G128, HEADER, PATH_AUTO, PATH_PREFILL, TQ_F16, TQ_F32, _check, _i64, _int, _vp,
               header_functions, lib)

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


def _refuse(t, name, dtype, shape, dev):
    """Raises what is wrong with a tensor that is not a contiguous `dtype` tensor of `shape` on cuda:dev."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _arg(t, name, dtype, shape, dev):
    """The address of a tensor argument: contiguous, of `dtype` and `shape`, on the current device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _device():
    """The current device, where every call here runs (no tensor's device before CUDA is initialised)."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _raw(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(like, shape, dtype, stream):
    """A contiguous output of one or two dims, allocated for the stream that writes it (empty_strided takes
    the host 1.6 us, new_empty 2.0)."""
    stride = (shape[1], 1) if len(shape) == 2 else (1,)
    if stream is None:
        return torch.empty_strided(shape, stride, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, stride, dtype=dtype, device=like.device)


def _shape2(t, name, ndim=2):
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t.shape


def tq_moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, weights=None, ids=None, stream=None):
    """softmax(logits [T, E]) and the top_k per token -> (weights fp32 [T, top_k], ids int32 [T, top_k]),
    by decreasing logit, the lowest expert first among equals; renormalize: weights of a token sum to 1."""
    dt, dev = _dtype(logits, "logits"), _device()
    T, E = _shape2(logits, "logits")
    pl = _arg(logits, "logits", logits.dtype, (T, E), dev)
    if weights is None:
        weights = _empty(logits, (T, top_k), torch.float32, stream)
    if ids is None:
        ids = _empty(logits, (T, top_k), torch.int32, stream)
    _check(lib.tq_moe_route(pl, dt, _arg(weights, "weights", torch.float32, (T, top_k), dev),
                            _arg(ids, "ids", torch.int32, (T, top_k), dev), T, E, top_k, 1 if renormalize else 0,
                            _raw(stream, dev)), "tq_moe_route")
    return weights, ids


def tq_moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, weights: torch.Tensor, ids: torch.Tensor,
                          renormalize: bool = True, dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of tq_moe_route: dweights [T, top_k] with the call's logits and results -> dlogits [T, E]."""
    dt, dev = _dtype(logits, "logits"), _device()
    T, E = _shape2(logits, "logits")
    k = _shape2(ids, "ids")[1]
    pl = _arg(logits, "logits", logits.dtype, (T, E), dev)
    if dlogits is None:
        dlogits = _empty(logits, (T, E), logits.dtype, stream)
    _check(lib.tq_moe_route_backward(_arg(dweights, "dweights", torch.float32, (T, k), dev), pl, dt,
                                     _arg(weights, "weights", torch.float32, (T, k), dev),
                                     _arg(ids, "ids", torch.int32, (T, k), dev),
                                     _arg(dlogits, "dlogits", logits.dtype, (T, E), dev), T, E, k,
                                     1 if renormalize else 0, _raw(stream, dev)), "tq_moe_route_backward")
    return dlogits


def tq_moe_sort(ids: torch.Tensor, num_experts: int, stream=None):
    """Slots sorted by expert: ids int32 [T, top_k] -> (offsets int32 [E + 1], order int32 [T top_k],
    pos int32 [T, top_k]).  Slots whose id is outside [0, E) come last and have position -1."""
    dev = _device()
    T, k = _shape2(ids, "ids")
    R = T * k
    p = _arg(ids, "ids", torch.int32, (T, k), dev)
    offsets = _empty(ids, (num_experts + 1,), torch.int32, stream)
    order = _empty(ids, (R,), torch.int32, stream)
    pos = _empty(ids, (T, k), torch.int32, stream)
    _check(lib.tq_moe_sort(p, offsets.data_ptr(), order.data_ptr(), pos.data_ptr(), R, num_experts, _raw(stream, dev)),
           "tq_moe_sort")
    return offsets, order, pos


def tq_moe_gather(x: torch.Tensor, order: torch.Tensor, offsets: torch.Tensor, top_k: int, out=None,
                  stream=None) -> torch.Tensor:
    """rows[r] = x[order[r] // top_k] for the offsets[-1] slots with an expert; later rows of `out` are
    left as they were (uninitialised when it is allocated here)."""
    dt, dev = _dtype(x, "x"), _device()
    T, H = _shape2(x, "x")
    E = _shape2(offsets, "offsets", 1)[0] - 1
    R = T * top_k
    px = _arg(x, "x", x.dtype, (T, H), dev)
    if out is None:
        out = _empty(x, (R, H), x.dtype, stream)
    _check(lib.tq_moe_gather(px, dt, _arg(order, "order", torch.int32, (R,), dev),
                             _arg(offsets, "offsets", torch.int32, (E + 1,), dev),
                             _arg(out, "out", x.dtype, (R, H), dev), T, H, top_k, E, _raw(stream, dev)),
           "tq_moe_gather")
    return out


def tq_moe_combine(y: torch.Tensor, pos: torch.Tensor, weights=None, out=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] y[pos[t, j]] (weights None: 1); zeros for a token without rows."""
    dt, dev = _dtype(y, "y"), _device()
    R, H = _shape2(y, "y")
    T, k = _shape2(pos, "pos")
    py = _arg(y, "y", y.dtype, (R, H), dev)
    if out is None:
        out = _empty(y, (T, H), y.dtype, stream)
    _check(lib.tq_moe_combine(py, dt, _arg(pos, "pos", torch.int32, (T, k), dev),
                              _opt(weights, "weights", torch.float32, (T, k), dev),
                              _arg(out, "out", y.dtype, (T, H), dev), T, R, H, k, _raw(stream, dev)), "tq_moe_combine")
    return out


def tq_moe_gather_backward(drows: torch.Tensor, pos: torch.Tensor, dx=None, stream=None) -> torch.Tensor:
    """Gradient of tq_moe_gather: dx[t] = sum_j drows[pos[t, j]], summed in fp32 in the order of j."""
    return tq_moe_combine(drows, pos, None, out=dx, stream=stream)


def tq_moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, dy=None,
                            dweights=None, stream=None):
    """Gradients of tq_moe_combine -> (dy like y, dweights fp32 [T, top_k]).  Rows of `dy` that no slot
    names are left as they were (uninitialised when it is allocated here)."""
    dt, dev = _dtype(y, "y"), _device()
    R, H = _shape2(y, "y")
    T, k = _shape2(pos, "pos")
    py = _arg(y, "y", y.dtype, (R, H), dev)
    pd = _arg(dout, "dout", y.dtype, (T, H), dev)
    if dy is None:
        dy = _empty(y, (R, H), y.dtype, stream)
    if dweights is None:
        dweights = _empty(y, (T, k), torch.float32, stream)
    _check(lib.tq_moe_combine_backward(pd, py, dt, _arg(pos, "pos", torch.int32, (T, k), dev),
                                       _arg(weights, "weights", torch.float32, (T, k), dev),
                                       _arg(dy, "dy", y.dtype, (R, H), dev),
                                       _arg(dweights, "dweights", torch.float32, (T, k), dev), T, R, H, k,
                                       _raw(stream, dev)), "tq_moe_combine_backward")
    return dy, dweights


def _experts(fmt, x, weights, offsets, order, top_k, bias, y, rows, E, N, path, stream, dev):
    """What the two products share: checks, the output, and the arguments after the weights."""
    X, K = _shape2(x, "x")
    R = X if order is None else _shape2(order, "order", 1)[0]
    if top_k >= 1 and R > X * top_k:  # top_k left out or too small: slots past the last token would read as zeros
        raise ValueError(f"order has {R} slots, but {X} tokens of top_k = {top_k} have {X * top_k}")
    px = _arg(x, "x", torch.float16, (X, K), dev)
    if y is None:
        y = _empty(x, (R, N), torch.float16, stream)
    if order is not None and rows is None and (
            path == PATH_PREFILL or path == PATH_AUTO and lib.tq_experts_path(fmt, R, E, N, K, 1) == PATH_PREFILL):
        rows = _empty(x, (R, K), torch.float16, stream)
    return y, (px, *weights, _opt(bias, "bias", torch.float16, (E, N), dev), _arg(y, "y", torch.float16, (R, N), dev),
               _arg(offsets, "offsets", torch.int32, (E + 1,), dev), _opt(order, "order", torch.int32, (R,), dev),
               _opt(rows, "rows", torch.float16, (R, K), dev), X, R, E, N, K, top_k, int(path), _raw(stream, dev))


def tq_gemm_experts(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, offsets: torch.Tensor, order=None,
                    top_k: int = 1, bias=None, y=None, path: int = PATH_AUTO, stream=None, rows=None) -> torch.Tensor:
    """Each expert's rows times its ternary weights: y[r] = x[row(r)] . What_e^T (+ bias_e) for
    offsets[e] <= r < offsets[e + 1]; row(r) = order[r] // top_k with `order` (x holds the tokens), r
    without (x holds sorted rows); order holds at most x.shape[0] * top_k slots.  packed uint8
    [E, N, ceil(K/4)], scale fp16 [E, N], bias fp16 [E, N].
    Rows before offsets[0] and from offsets[-1] on are left as they were (uninitialised when y is allocated
    here), so that E + 1 consecutive offsets of a sort of more experts do with the weights of those E.
    rows: fp16 [R, K] scratch for the path that copies the rows first (allocated here when it is needed)."""
    dev = _device()
    E, N, _ = _shape2(packed, "packed", 3)
    K = _shape2(x, "x")[1]
    w = (_arg(packed, "packed", torch.uint8, (E, N, (K + 3) // 4), dev), _arg(scale, "scale", torch.float16, (E, N), dev))
    y, args = _experts(FMT_TERNARY, x, w, offsets, order, top_k, bias, y, rows, E, N, path, stream, dev)
    _check(lib.tq_gemm_experts(*args), "tq_gemm_experts")
    return y


def w4g_gemm_experts(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor, zeros=None,
                     order=None, top_k: int = 1, bias=None, y=None, path: int = PATH_AUTO,
                     stream=None, rows=None) -> torch.Tensor:
    """tq_gemm_experts with W4A16 weights: qweight int32 [E, N, K/8], scales fp16 [E, N, K/128], zeros
    uint8 [E, N, K/128] or None (symmetric).  PATH_PREFILL, which PATH_AUTO takes for many rows per expert,
    rounds each weight (u - z) * s to fp16 (infinite from 65520: scales up to 4364 are safe); PATH_DECODE
    and PATH_GENERIC round no weight."""
    dev = _device()
    E, N, _ = _shape2(qweight, "qweight", 3)
    K = _shape2(x, "x")[1]
    w = (_arg(qweight, "qweight", torch.int32, (E, N, K // 8), dev),
         _arg(scales, "scales", torch.float16, (E, N, K // 128), dev),
         _opt(zeros, "zeros", torch.uint8, (E, N, K // 128), dev))
    y, args = _experts(FMT_W4G128, x, w, offsets, order, top_k, bias, y, rows, E, N, path, stream, dev)
    _check(lib.w4g_gemm_experts(*args), "w4g_gemm_experts")
    return y


def tq_experts_path(fmt: int, R: int, E: int, N: int, K: int, aligned: bool = True) -> int:
    """The path PATH_AUTO takes for R sorted rows of E experts.  A rank that holds some of the experts passes
    the number of rows that it expects and hands the result to the product, whose own R counts every slot."""
    return int(lib.tq_experts_path(int(fmt), int(R), int(E), int(N), int(K), 1 if aligned else 0))
