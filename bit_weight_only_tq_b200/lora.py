"""Low-rank adapters beside the packed projections (include/tq_lora.h): the adapters of many requests at once, their
gradients, dropout from a counter-based generator, and the packed products' gradient for x.

    offsets, order, _ = tq_moe_sort(ids.view(-1, 1), L)      # ids int32 [M]: the adapter of each row, -1 for none
    y = w4g_gemm(x, qweight, scales)                         # the frozen projection
    out = tq_lora(x, a, b, y, offsets, order=order, scaling=s, p=0.05, rng=rng, v=v)
    dx = w4g_gemm_backward(dy, qweight, scales)
    dx, da, db = tq_lora_backward(dy, x, a, b, v, dx, offsets, order=order, scaling=s, p=0.05, rng=rng)

Argument marshalling only, like the rest of the package; every tensor is contiguous, on one CUDA device, and that
device is the current one.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import HEADER, PATH_AUTO, PATH_DECODE, PATH_GENERIC, TQ_F16, _check, _i64, _int, _vp, header_functions, lib
from .moe import TQ_BF16, _arg, _device, _dtype, _empty, _opt, _raw, _shape2

__all__ = [
    "tq_lora", "tq_lora_backward", "tq_lora_path", "tq_lora_workspace_size", "tq_dropout", "tq_gemm_backward",
    "w4g_gemm_backward",
]

LORA_HEADER = os.path.join(os.path.dirname(HEADER), "tq_lora.h")

_f64 = ctypes.c_double
_SIGS = {
    "tq_lora": [_vp, _int] + [_vp] * 8 + [_f64, _vp] + [_i64] * 4 + [_int, _int, _vp],
    "tq_lora_path": [_i64] * 4 + [_int] * 3,
    "tq_lora_workspace_size": [_i64, _i64, _int],
    "tq_lora_backward": [_vp, _vp, _int] + [_vp] * 5 + [ctypes.c_size_t] + [_vp] * 6 + [_f64, _vp] + [_i64] * 4 +
    [_int, _int, _vp],
    "tq_dropout": [_vp, _int, _vp, _f64, _vp, _i64, _i64, _vp],
    "tq_gemm_backward": [_vp] * 5 + [_i64] * 3 + [_int, _vp],
    "w4g_gemm_backward": [_vp] * 6 + [_i64] * 3 + [_int, _vp],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_size_t if _name == "tq_lora_workspace_size" else ctypes.c_int

_DTYPES16 = {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}


def lora_header_functions():
    """Names of the functions declared in include/tq_lora.h."""
    return header_functions(LORA_HEADER)


def _dtype16(t, name):
    d = _DTYPES16.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return d


def _adapters(x, a, b):
    """(M, K, L, rank, N) of an adapter call."""
    M, K = _shape2(x, "x")
    L, r, _ = _shape2(a, "a", 3)
    return M, K, L, r, _shape2(b, "b", 3)[1]


def _rng(p, rng, dev):
    if p == 0.0:
        return None
    if rng is None:
        raise ValueError("p > 0 needs rng (int64 [2]: seed, offset)")
    return _arg(rng, "rng", torch.int64, (2,), dev)


def tq_lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, base, offsets: torch.Tensor, order=None, scaling=None,
            p: float = 0.0, rng=None, v=None, out=None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """out[m] = base[m] + scaling[l] (drop(x[m]) A_l^T) B_l^T, l the adapter of row m -> out [M, N].

    x [M, K], a [L, rank, K], b [L, N, rank] and base [M, N] (None: zeros) of one type, float16 or bfloat16; scaling
    fp32 [L] (None: 1).  offsets int32 [L + 1] and order int32 [M] (None: rows are sorted already) from
    tq_moe_sort(ids.view(-1, 1), L); rows whose id is outside [0, L) get base alone.
    p, rng: dropout of x; rng int64 [2] (seed, offset) on the device, read when the kernels run.
    v: fp32 [M, rank], what tq_lora_backward needs of this call (written; a scratch is allocated where a path
    needs one and none is given).  out may be base (in place).  At most 1024 adapters of rank 128: a larger rank
    takes two calls, the second on the first's out."""
    dt, dev = _dtype16(x, "x"), _device()
    M, K, L, r, N = _adapters(x, a, b)
    d = x.dtype
    px = _arg(x, "x", d, (M, K), dev)
    if out is None:
        out = _empty(x, (M, N), d, stream)
    pa, pb = _arg(a, "a", d, (L, r, K), dev), _arg(b, "b", d, (L, N, r), dev)
    pbase, po = _opt(base, "base", d, (M, N), dev), _arg(out, "out", d, (M, N), dev)
    if v is None:
        aligned = 0 if (px | pa | pb | (pbase or 0) | po) & 15 else 1
        if path != PATH_AUTO or p or lib.tq_lora_path(M, L, N, K, r, 0, aligned) != PATH_DECODE:
            v = _empty(x, (M, r), torch.float32, stream)
    _check(lib.tq_lora(px, dt, pa, pb, _opt(scaling, "scaling", torch.float32, (L,), dev), pbase, po,
                       _opt(v, "v", torch.float32, (M, r), dev), _arg(offsets, "offsets", torch.int32, (L + 1,), dev),
                       _opt(order, "order", torch.int32, (M,), dev), p, _rng(p, rng, dev), M, L, N, K, r, int(path),
                       _raw(stream, dev)), "tq_lora")
    return out


def tq_lora_backward(dy: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, v: torch.Tensor, base_dx,
                     offsets: torch.Tensor, order=None, scaling=None, p: float = 0.0, rng=None, workspace=None,
                     dx=None, da=None, db=None, need_dx: bool = True, need_ab: bool = True, path: int = PATH_AUTO,
                     stream=None):
    """Gradients of tq_lora from dy [M, N], the call's inputs and its v -> (dx [M, K], da like a, db like b), each None
    where it is not wanted.  dx is base_dx [M, K] (the projection's gradient for x; None: zeros) plus the adapters'
    part and may be base_dx; an adapter without rows gets zeros.  workspace: uint8, at least
    tq_lora_workspace_size(M, L, rank) bytes (allocated here when it is left out)."""
    dt, dev = _dtype16(x, "x"), _device()
    M, K, L, r, N = _adapters(x, a, b)
    d = x.dtype
    pd = _arg(dy, "dy", d, (M, N), dev)
    if need_dx and dx is None:
        dx = _empty(x, (M, K), d, stream)
    if need_ab and da is None:
        da = _empty3(a, stream)
    if need_ab and db is None:
        db = _empty3(b, stream)
    if workspace is None:
        workspace = _empty(x, (lib.tq_lora_workspace_size(M, L, r),), torch.uint8, stream)
    elif workspace.dim() != 1:
        raise ValueError("workspace must have 1 dims")
    _check(lib.tq_lora_backward(pd, _arg(x, "x", d, (M, K), dev), dt, _arg(a, "a", d, (L, r, K), dev),
                                _arg(b, "b", d, (L, N, r), dev), _opt(scaling, "scaling", torch.float32, (L,), dev),
                                _arg(v, "v", torch.float32, (M, r), dev),
                                _arg(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.numel(),
                                _opt(base_dx, "base_dx", d, (M, K), dev), _opt(dx, "dx", d, (M, K), dev),
                                _opt(da, "da", d, (L, r, K), dev), _opt(db, "db", d, (L, N, r), dev),
                                _arg(offsets, "offsets", torch.int32, (L + 1,), dev),
                                _opt(order, "order", torch.int32, (M,), dev), p, _rng(p, rng, dev), M, L, N, K, r,
                                int(path), _raw(stream, dev)), "tq_lora_backward")
    return dx, da, db


def _empty3(like, stream):
    if stream is None:
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        return torch.empty_like(like)


def tq_lora_path(M: int, L: int, N: int, K: int, rank: int, dropout: bool = False, aligned: bool = True) -> int:
    """The path PATH_AUTO takes for M rows of L adapters."""
    return int(lib.tq_lora_path(int(M), int(L), int(N), int(K), int(rank), 1 if dropout else 0, 1 if aligned else 0))


def tq_lora_workspace_size(M: int, L: int, rank: int) -> int:
    """Bytes of workspace that tq_lora_backward needs (0: invalid sizes)."""
    return int(lib.tq_lora_workspace_size(int(M), int(L), int(rank)))


def tq_dropout(x: torch.Tensor, p: float, rng, out=None, stream=None) -> torch.Tensor:
    """Dropout of x [M, K] (float32, float16 or bfloat16) with probability p (a multiple of 2^-16: p is rounded to one):
    zero, or x / (1 - p).  rng int64 [2] on the device: seed and offset of the generator; the same numbers drop the same
    elements, so that the gradient is this call on the gradient of out.  out may be x."""
    dt, dev = _dtype(x, "x"), _device()
    M, K = _shape2(x, "x")
    px = _arg(x, "x", x.dtype, (M, K), dev)
    if out is None:
        out = _empty(x, (M, K), x.dtype, stream)
    _check(lib.tq_dropout(px, dt, _arg(out, "out", x.dtype, (M, K), dev), p, _rng(p, rng, dev), M, K,
                          _raw(stream, dev)), "tq_dropout")
    return out


def _rows(dy, pd, M, N, K, path, rows, stream, dev):
    """The address of the scratch where the tensor-core path copies rows that it cannot read in place, or None."""
    if rows is None:
        if N % 8 == 0 and pd & 15 == 0 or K % 64 or path == PATH_GENERIC:
            return None
        rows = _empty(dy, (M, (N + 7) // 8 * 8), torch.float16, stream)
    return _arg(rows, "rows", torch.float16, (M, (N + 7) // 8 * 8), dev)


def tq_gemm_backward(dy: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, K=None, dx=None,
                     path: int = PATH_AUTO, stream=None, rows=None) -> torch.Tensor:
    """Gradient for x of tq_gemm: dx [M, K] = dy [M, N] What, fp16 (K: 4 packed.shape[1] unless given).  rows: fp16
    [M, N rounded up to a multiple of 8] scratch for rows of dy that are no whole 16-byte vectors (allocated here when
    it is needed)."""
    dev = _device()
    M, N = _shape2(dy, "dy")
    KB = _shape2(packed, "packed")[1]
    K = 4 * KB if K is None else K
    pd = _arg(dy, "dy", torch.float16, (M, N), dev)
    if dx is None:
        dx = _empty(dy, (M, K), torch.float16, stream)
    _check(lib.tq_gemm_backward(pd, _arg(packed, "packed", torch.uint8, (N, (K + 3) // 4), dev),
                                _arg(scale, "scale", torch.float16, (N,), dev),
                                _arg(dx, "dx", torch.float16, (M, K), dev),
                                _rows(dy, pd, M, N, K, path, rows, stream, dev), M, N, K, int(path),
                                _raw(stream, dev)), "tq_gemm_backward")
    return dx


def w4g_gemm_backward(dy: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros=None, dx=None,
                      path: int = PATH_AUTO, stream=None, rows=None) -> torch.Tensor:
    """Gradient for x of w4g_gemm (zeros: of w4g_gemm_zp): dx [M, K] = dy [M, N] What, fp16.  rows: as in
    tq_gemm_backward.  With weights in activation order (w4g_repack_act_order) the columns of dx are those of
    tq_permute_columns(x, perm): tq_permute_columns(dx, inverse of perm) is the gradient for x."""
    dev = _device()
    M, N = _shape2(dy, "dy")
    K = 8 * _shape2(qweight, "qweight")[1]
    pd = _arg(dy, "dy", torch.float16, (M, N), dev)
    if dx is None:
        dx = _empty(dy, (M, K), torch.float16, stream)
    _check(lib.w4g_gemm_backward(pd, _arg(qweight, "qweight", torch.int32, (N, K // 8), dev),
                                 _arg(scales, "scales", torch.float16, (N, K // 128), dev),
                                 _opt(zeros, "zeros", torch.uint8, (N, K // 128), dev),
                                 _arg(dx, "dx", torch.float16, (M, K), dev),
                                 _rows(dy, pd, M, N, K, path, rows, stream, dev), M, N, K, int(path),
                                 _raw(stream, dev)), "w4g_gemm_backward")
    return dx
