"""Experts' products at the ends of what their header allows, against the fp64 oracle.

Tolerance per element, S = sum |x w|: half an fp16 step of the result (2^-11 |y|, 2^-25 among the
subnormals); products are exact in fp32 and summed in fp32, at most K / 8 + 64 roundings of the running
sum along the longest chain of any path, each 2^-23 of at most S; where the PREFILL path is taken, and
only there, each INT4 weight rounded to fp16 (2^-11 S).
"""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import oracle as O
import tq_inputs as I
from gpu_util import bits, check_canaries, f16np, gpu, guarded_empty, need_cuda

pytestmark = gpu
FORMATS = ["ternary", "w4", "w4z"]
PATHS = [tq.PATH_AUTO, tq.PATH_GENERIC, tq.PATH_DECODE, tq.PATH_PREFILL]


def _call(fmt, x, ws, offsets, **kw):
    if fmt == "ternary":
        return tq.tq_gemm_experts(x, ws[0], ws[1], offsets, **kw)
    return tq.w4g_gemm_experts(x, ws[0], ws[1], offsets, zeros=ws[2], **kw)


def _taken(fmt, path, R, E, N, K):
    """The path that a call takes."""
    f = tq.FMT_TERNARY if fmt == "ternary" else tq.FMT_W4G128
    return tq.tq_experts_path(f, R, E, N, K) if path == tq.PATH_AUTO else path


def _what(fmt, ws, e, K, cols):
    """Rows `cols` of expert e's weights in fp64."""
    q, s = ws[0][e][cols].cpu().numpy(), bits(ws[1][e][cols])
    if fmt == "ternary":
        return O.tq_unpack(q, s, K)
    if ws[2] is None:
        return O.w4g_unpack(q, s)
    return O.w4z_unpack(q, s, ws[2][e][cols].cpu().numpy(), np.arange(K) // 128)


def _tol(fmt, taken, ref, S, K):
    rel = (K / 8 + 64) * 2.0 ** -23 + (2.0 ** -11 if fmt != "ternary" and taken == tq.PATH_PREFILL else 0.0)
    return 2.0 ** -11 * (1 + 2.0 ** -10) * np.abs(ref) + rel * S + 2.0 ** -25


def _check(fmt, path, x, ws, offsets, y, xrow, bias=None, cols=None):
    """Every row of every expert against the oracle, at the weight rows `cols`."""
    off, (R, N), K, E = offsets.cpu().numpy(), y.shape, x.shape[1], ws[0].shape[0]
    taken = _taken(fmt, path, R, E, N, K)
    cols = np.arange(N) if cols is None else cols
    xn, yn = f16np(x).astype(np.float64), f16np(y).astype(np.float64)
    for e in range(E):
        rows = np.arange(off[e], off[e + 1])
        if rows.size == 0:
            continue
        W = _what(fmt, ws, e, K, cols)
        xs = xn[xrow[rows]]
        ref, S = xs @ W.T, np.abs(xs) @ np.abs(W).T
        if bias is not None:
            b = f16np(bias)[e][cols].astype(np.float64)
            ref, S = ref + b, S + np.abs(b)
        err, tol = np.abs(yn[np.ix_(rows, cols)] - ref), _tol(fmt, taken, ref, S, K)
        assert np.all(err <= tol), (fmt, path, e, float((err - tol).max()), np.argwhere(~(err <= tol))[:4])


def _word(codes):
    """Words of eight 4-bit codes, the first in the lowest bits."""
    u = torch.as_tensor(codes, dtype=torch.int64).view(*np.shape(codes)[:-1], -1, 8)
    q = (u << torch.arange(0, 32, 4)).sum(-1)
    return torch.where(q >= 2 ** 31, q - 2 ** 32, q).to(torch.int32)


# ------------------------------------------------------------------------- INT4 weights on each path
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("path", PATHS)
def test_int4_weights_are_rounded_on_the_prefill_path_only(path, T, zeros):
    """Products that cancel exactly, (7 s)(-3) + (3 s)(7), for scales whose multiples 7 s and 3 s are no
    fp16 numbers: 0 wherever weights stay exact (every partial sum is one of integers times s, below 2^24),
    and within the rounding of the weights on the PREFILL path."""
    need_cuda()
    E, N, K = 2, 70, 256
    z = 6 if zeros else 8
    codes = np.tile(np.array([z + 7, z + 3]), (E, N, K // 2))
    ws = (_word(codes).cuda(), (0.5 + (2 * torch.arange(E * N * 2) + 1) * 2.0 ** -11).half().view(E, N, 2).cuda(),
          torch.full((E, N, 2), z, dtype=torch.uint8, device="cuda") if zeros else None)
    x = torch.tensor([-3.0, 7.0]).repeat(2 * T, K // 2).half().cuda()
    offsets = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    y = _call("w4", x, ws, offsets, path=path)
    assert tq.tq_device_status() == 0
    if _taken("w4", path, 2 * T, E, N, K) == tq.PATH_PREFILL:
        _check("w4", path, x, ws, offsets, y, np.arange(2 * T))
    else:
        assert (y == 0).all()


@pytest.mark.parametrize("path,scale", [(p, 4364.0) for p in PATHS] + [(p, s) for p in (tq.PATH_GENERIC, tq.PATH_DECODE)
                                                                       for s in (4368.0, 30000.0, 65504.0)])
def test_int4_scales_up_to_the_documented_limit(path, scale):
    """15 * 4364 = 65460 rounds to 65472, below the largest fp16, 65504; the next scale, 4368, gives 65520,
    which rounds to infinity.  The paths that round no weight take any scale."""
    need_cuda()
    E, N, K, T = 3, 67, 384, 30
    assert _taken("w4z", tq.PATH_AUTO, T, E, N, K) == tq.PATH_PREFILL
    g = torch.Generator().manual_seed(7)
    u = torch.randint(0, 16, (E, N, K), generator=g)
    u[:, :, 5] = 15
    ws = (_word(u).cuda(), torch.full((E, N, K // 128), scale, dtype=torch.float16, device="cuda"),
          torch.zeros(E, N, K // 128, dtype=torch.uint8, device="cuda"))
    # sums stay in fp16's range: K 15 scale |x| <= 384 * 15 * 65504 * 2^-14
    x = (torch.rand(T, K, generator=g) * 2.0 ** -14 * torch.where(torch.rand(T, K, generator=g) < 0.5, -1.0, 1.0)).half().cuda()
    offsets = torch.tensor([0, 11, 11, T], dtype=torch.int32, device="cuda")
    y = _call("w4z", x, ws, offsets, path=path)
    assert tq.tq_device_status() == 0 and torch.isfinite(y).all()
    _check("w4z", path, x, ws, offsets, y, np.arange(T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E", [(6, 4), (24, 3), (25, 3), (90, 2)])
def test_auto_is_as_exact_as_the_path_it_takes(T, E, fmt):
    need_cuda()
    N, K = 130, 640
    w = I.weights(E * N, K, T, device="cuda", outlier_frac=0.0 if fmt == "ternary" else 0.001)
    if fmt == "ternary":
        p, s = tq.tq_quantize_pack(w)
        ws = (p.view(E, N, -1), s.view(E, N), None)
    else:
        q, s, z, _ = tq.w4g_quantize_pack_ex(w, zero_point=fmt == "w4z")
        ws = (q.view(E, N, -1), s.view(E, N, -1), None if z is None else z.view(E, N, -1))
    ids = torch.randint(0, E, (T, 1), generator=torch.Generator().manual_seed(T)).int().cuda()
    offsets, order, _ = tq.tq_moe_sort(ids, E)
    x = I.activations(T, K, T, device="cuda", outlier_row_frac=0.02)
    y = _call(fmt, x, ws, offsets, order=order, top_k=1)
    assert tq.tq_device_status() == 0
    _check(fmt, tq.PATH_AUTO, x, ws, offsets, y, order.cpu().numpy())


# ------------------------------------------------------------------------------------ most rows there can be
def test_one_expert_with_every_row_there_can_be():
    """2^31 - 1 slots of two tokens: an expert's rows plus a chunk's, less one, are past 32 bits.  13 GB."""
    need_cuda()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    R, k, K = 2 ** 31 - 1, 2 ** 30, 64
    order = torch.arange(R, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    x = torch.tensor([[1.0], [-2.0]]).repeat(1, K).half().cuda()
    packed = torch.full((1, 1, K // 4), 0xAA, dtype=torch.uint8, device="cuda")      # every code +1
    scale = torch.tensor([[0.5]]).half().cuda()
    y = torch.full((R, 1), 7.0, dtype=torch.float16, device="cuda")
    tq.tq_gemm_experts(x, packed, scale, offsets, order=order, top_k=k, y=y, path=tq.PATH_DECODE)
    assert tq.tq_device_status() == 0
    assert (y[:k] == 32.0).all() and (y[k:] == -64.0).all()


# -------------------------------------------------------------------------- a window of a larger sort's experts
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("lo,hi", [(0, 3), (2, 5), (3, 9), (8, 9)])
@pytest.mark.parametrize("spread", [True, False])
def test_a_window_of_the_experts(lo, hi, path, fmt, spread):
    """offsets[lo:hi + 1] of a sort of nine experts with the weights of experts lo .. hi - 1: only their rows
    are written, those before the first as well as those behind the last left as they were."""
    need_cuda()
    T, k, E, N, K = 70, 2, 9, 71 + lo % 2, 256
    g = torch.Generator(device="cuda").manual_seed(lo)
    offsets, order, _ = tq.tq_moe_sort(torch.randint(0, E, (T, k), generator=g, device="cuda").int(), E)
    w = I.weights(E * N, K, 3, device="cuda", outlier_frac=0.0)
    if fmt == "ternary":
        p, s = tq.tq_quantize_pack(w)
        ws = (p.view(E, N, -1)[lo:hi], s.view(E, N)[lo:hi], None)
    else:
        q, s, z, _ = tq.w4g_quantize_pack_ex(w, zero_point=fmt == "w4z")
        ws = (q.view(E, N, -1)[lo:hi], s.view(E, N, -1)[lo:hi], None if z is None else z.view(E, N, -1)[lo:hi])
    bias = I.bias((hi - lo) * N, 4, device="cuda").view(hi - lo, N)
    x = I.activations(T, K, 5, device="cuda")
    token = (order // k).long()
    y, buf = guarded_empty(T * k, N)
    window = offsets[lo:hi + 1]
    if spread:
        _call(fmt, x, ws, window, order=order, top_k=k, bias=bias, y=y, path=path)
        _check(fmt, path, x, ws, window, y, token.cpu().numpy(), bias)
    else:
        rows = x[token].contiguous()
        _call(fmt, rows, ws, window, bias=bias, y=y, path=path)
        _check(fmt, path, rows, ws, window, y, np.arange(T * k), bias)
    assert tq.tq_device_status() == 0
    check_canaries(buf, T * k, N)
    a, b = int(window[0]), int(window[-1])
    left = y.view(torch.int16)
    assert (left[:a] == 0x7E5A).all() and (left[b:] == 0x7E5A).all()


def test_order_without_its_top_k_is_refused():
    need_cuda()
    T, k, E, N, K = 5, 3, 4, 40, 128
    offsets, order, _ = tq.tq_moe_sort(torch.zeros(T, k, dtype=torch.int32, device="cuda"), E)
    x = I.activations(T, K, 1, device="cuda")
    p, s = tq.tq_quantize_pack(I.weights(E * N, K, 1, device="cuda"))
    q, s4 = tq.w4g_quantize_pack(I.weights(E * N, K, 1, device="cuda"))
    for top_k in (1, 2):
        with pytest.raises(ValueError, match="15 slots"):
            tq.tq_gemm_experts(x, p.view(E, N, -1), s.view(E, N), offsets, order=order, top_k=top_k)
        with pytest.raises(ValueError, match="15 slots"):
            tq.w4g_gemm_experts(x, q.view(E, N, -1), s4.view(E, N, -1), offsets, order=order, top_k=top_k)
    ws = (p.view(E, N, -1), s.view(E, N), None)
    offsets = offsets.clamp(max=7)
    y = tq.tq_gemm_experts(x, *ws[:2], offsets, order=order[:7], top_k=k)           # the first slots alone
    assert tuple(y.shape) == (7, N)
    _check("ternary", tq.PATH_AUTO, x, ws, offsets, y, (order // k).cpu().numpy())


# ------------------------------------------------- one CTA per SM with more than one item (few, long items)
def _codes(fmt, E, N, K, seed):
    """Random packed weights, without quantising a matrix of that size first."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fmt == "ternary":
        c = torch.randint(0, 3, (E, N, K // 4, 4), generator=g, device="cuda", dtype=torch.uint8)
        q = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
        return q, (0.01 + 0.02 * torch.rand(E, N, generator=g, device="cuda")).half(), None
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g, device="cuda").int()
    s = (0.002 + 0.004 * torch.rand(E, N, K // 128, generator=g, device="cuda")).half()
    z = torch.randint(0, 16, (E, N, K // 128), generator=g, device="cuda", dtype=torch.uint8) if fmt == "w4z" else None
    return q, s, z


# Up to 296 items of 16 stages and more run on 148 CTAs of four consumer groups.  Stage counts (of 256 INT4 or 512
# ternary k, the last one whole or not) that are and are no multiple of the groups and of the ring; with items of
# half the rows, stages of twice the k.
@pytest.mark.parametrize("fmt,K", [("w4", 4096), ("w4z", 4352), ("w4", 4480), ("w4", 4608), ("w4z", 4864), ("w4", 5376),
                                   ("ternary", 8192), ("ternary", 8704), ("ternary", 8768), ("ternary", 9216),
                                   ("ternary", 9728), ("ternary", 10752 + 320)])
@pytest.mark.parametrize("counts,N", [([1, 1, 0, 1, 1, 1], 4001),         # 160 items, and so 315 of half the rows: 3 each
                                      ([2, 1, 1, 0, 1, 1], 5600),         # 220: 440 halves, 3 each
                                      ([1, 1, 1, 0, 1, 1], 6397),         # 250: whole items, two each
                                      ([14], 18930)])                     # 296: two chunks of one expert, 8 and 6 rows
def test_several_long_items_per_cta(counts, N, fmt, K):
    need_cuda()
    E, R = len(counts), sum(counts)
    ws = _codes(fmt, E, N, K, N + K)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    x = I.activations(R, K, N, device="cuda")
    bias = I.bias(E * N, K, device="cuda").view(E, N)
    y, buf = guarded_empty(R, N)
    _call(fmt, x, ws, offsets, bias=bias, y=y, path=tq.PATH_DECODE)
    assert tq.tq_device_status() == 0
    check_canaries(buf, R, N)
    cols = np.unique(np.concatenate([np.arange(0, N, 61), np.arange(N - 130, N)]))
    _check(fmt, tq.PATH_DECODE, x, ws, offsets, y, np.arange(R), bias, cols)
    again = _call(fmt, x, ws, offsets, bias=bias, path=tq.PATH_DECODE)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
