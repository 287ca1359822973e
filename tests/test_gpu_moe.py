"""Router, sort and row exchange of the mixture-of-experts calls against 64-bit numpy forms.

Tolerances (u = 2^-24, an fp32 rounding; h = half a step of the output type):
  weights    exp(x - m): x - m off by u |x - m|, exp by 2 ulp; sums of E terms by at most
             (E / 32 + 5) u; one division: relative (D + E / 32 + 16) u, D the spread of the scores.
  rows       sum of k products by FMA: (k + 1) u sum |w y|, plus h |out|.
  dweights   ceil(H / 128) + 9 additions in sequence at most: that many u times sum |d y|.
  dlogits    products of weights (above) and g: (D + E / 32 + 32) u (|g| + sum |g w|) w, plus h.
"""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
from gpu_util import gpu, need_cuda

pytestmark = gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DTYPES = list(HALF)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _np(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ------------------------------------------------------------------------------------------ route
def _route64(x, k, renorm):
    x = np.where(np.isnan(x), -np.inf, x)
    T, E = x.shape
    order = np.lexsort((np.broadcast_to(np.arange(E), x.shape), -x), axis=1)[:, :k]
    top = np.take_along_axis(x, order, 1)
    with np.errstate(invalid="ignore"):
        p = np.where(x == x.max(1, keepdims=True), 1.0, np.exp(x - x.max(1, keepdims=True)))
    p = np.where(x > -np.inf, p, 0.0)
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    w = np.take_along_axis(p, order, 1)
    ids = np.where(top > -np.inf, order, -1)
    w = np.where(ids >= 0, w, 0.0)
    if renorm:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return w, ids, p


def _check_route(x, k, renorm):
    T, E = x.shape
    w, ids = tq.tq_moe_route(x, k, renormalize=renorm)
    wr, ir, p = _route64(_np(x), k, renorm)
    assert np.array_equal(_np(ids), ir)
    fin = _np(x)[np.isfinite(_np(x))]
    D = float(fin.max() - fin.min()) if fin.size else 0.0
    rel = (D + E / 32 + 16) * U
    assert np.all(np.abs(_np(w) - wr) <= rel * wr + 2.0 ** -149), np.abs(_np(w) - wr).max()
    g = torch.randn(T, k, generator=_gen(E + k), device="cuda")
    dx = _np(tq.tq_moe_route_backward(g, x, w, ids, renormalize=renorm))
    gn = _np(g)
    inner = (gn * wr).sum(1, keepdims=True)
    big = (np.abs(gn) * wr).sum(1, keepdims=True)
    want, size = (np.zeros_like(p), np.zeros_like(p)) if renorm else (-p * inner, p * big)
    at, col = np.nonzero(ir >= 0)
    val = wr if renorm else np.take_along_axis(p, np.maximum(ir, 0), 1)
    np.add.at(want, (at, ir[at, col]), (val * (gn - inner if renorm else gn))[at, col])
    np.add.at(size, (at, ir[at, col]), (val * (np.abs(gn) + (big if renorm else 0)))[at, col])
    tol = (D + E / 32 + 32) * U * size + HALF[x.dtype] * np.abs(want) + TINY[x.dtype]
    assert np.all(np.abs(dx - want) <= tol), (np.abs(dx - want) - tol).max()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 32, 32), (5, 33, 4), (16, 64, 8), (7, 60, 6), (9, 127, 3),
                                   (300, 128, 8), (33, 256, 8), (4, 257, 5), (2, 512, 32), (3, 1000, 7), (2, 1024, 10)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, dtype, renorm):
    need_cuda()
    x = (2 * torch.randn(T, E, generator=_gen(T * E + k), device="cuda")).to(dtype)
    _check_route(x, k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_masks_infinities(renorm):
    need_cuda()
    inf = float("inf")
    x = torch.randn(10, 40, generator=_gen(3), device="cuda")
    x[0] = 0.0                                     # all equal: the lowest indices
    x[1] = -inf                                    # nothing to choose
    x[2, 2:] = -inf                                # fewer than top_k
    x[3] = float("nan")
    x[4, 5] = float("nan")                         # one NaN: never chosen
    x[5, 7], x[5, 30] = inf, inf                   # two share everything
    x[6] = torch.finfo(torch.float32).min          # the type's lowest value is an ordinary score
    x[7, ::2] = torch.finfo(torch.float32).min
    x[8, ::2], x[8, 1::2] = 0.0, -0.0              # equal
    x[9, 1:] = -200.0                              # weights that underflow
    for dtype in (torch.float32, torch.bfloat16):
        w, ids = tq.tq_moe_route(x.to(dtype), 4, renormalize=renorm)
        wr, ir, _ = _route64(_np(x.to(dtype)), 4, renorm)
        assert np.array_equal(_np(ids), ir)
        assert np.allclose(_np(w), wr, rtol=300 * U, atol=2.0 ** -126)
        dx = tq.tq_moe_route_backward(torch.ones_like(w), x.to(dtype), w, ids, renormalize=renorm)
        assert torch.isfinite(dx).all()
        assert (dx[1] == 0).all() and (dx[3] == 0).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    need_cuda()
    # central differences of the 64-bit formula: error h^2 / 6 |f'''| <= 1e-7 for h = 1e-4 with
    # |f'''| <= 6 sum |g|, plus 1e-16 / h; the kernel's own error is of the order of 1e-6
    x = torch.randn(2, 24, generator=_gen(11), device="cuda")
    k = 5
    w, ids = tq.tq_moe_route(x, k, renormalize=renorm)
    g = torch.randn(2, k, generator=_gen(12), device="cuda")
    dx = _np(tq.tq_moe_route_backward(g, x, w, ids, renormalize=renorm))
    xn, gn, idn = _np(x), _np(g), _np(ids)

    def loss(z):
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        c = np.take_along_axis(p, idn, 1)
        return ((c / c.sum(1, keepdims=True) if renorm else c) * gn).sum()

    for t in range(2):
        for i in range(24):
            a, b = xn.copy(), xn.copy()
            a[t, i] += 1e-4
            b[t, i] -= 1e-4
            assert abs((loss(a) - loss(b)) / 2e-4 - dx[t, i]) < 1e-5


# ------------------------------------------------------------------------------------------- sort
def _sort64(ids, E):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(E + 1))
    pos = np.empty(flat.size, np.int64)
    pos[order] = np.arange(flat.size)
    return offsets, order, np.where(key < E, pos, -1).reshape(ids.shape)


def _check_sort(ids, E):
    got = tq.tq_moe_sort(ids, E)
    for a, b in zip(got, _sort64(_np(ids), E)):
        assert np.array_equal(_np(a), b)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (13, 2, 5), (16, 8, 256), (33, 3, 1024), (127, 4, 60),
                                   (1024, 8, 128), (1025, 8, 128), (4099, 6, 60), (20000, 8, 256), (9000, 1, 1000),
                                   (300000, 2, 8)])
@pytest.mark.parametrize("low,high", [(0, 1), (-0.4, 1.4)])
def test_sort(T, k, E, low, high):
    need_cuda()
    ids = torch.randint(int(low * E), max(int(high * E), 1), (T, k), generator=_gen(T + k + E), device="cuda").int()
    _check_sort(ids, E)


@pytest.mark.parametrize("T", [1, 40, 9001])
def test_sort_extremes(T):
    need_cuda()
    for v in (0, 6, -1, 7, 2 ** 31 - 1, -2 ** 31):
        _check_sort(torch.full((T, 2), v, dtype=torch.int32, device="cuda"), 7)
    offsets, order, pos = tq.tq_moe_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 7)
    assert (offsets == 0).all() and order.numel() == 0 and pos.numel() == 0


# ------------------------------------------------------------------------------------------- rows
def _plan(T, k, E, seed, away=0.0):
    ids = torch.randint(0, int(E / (1 - away)), (T, k), generator=_gen(seed), device="cuda").int()
    return ids, tq.tq_moe_sort(ids, E)


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (1, 8, 64, 4096), (13, 8, 64, 2048), (5, 3, 7, 1), (9, 2, 4, 401),
                                     (260, 4, 60, 3584), (1001, 2, 8, 100), (40, 32, 64, 136)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("away", [0.0, 0.5])
def test_gather_and_combine(T, k, E, H, dtype, away):
    need_cuda()
    _, (offsets, order, pos) = _plan(T, k, E, T + H, away)
    total = int(offsets[-1])
    x = torch.randn(T, H, generator=_gen(H), device="cuda").to(dtype)
    mark = torch.full((T * k, H), 7.0, device="cuda").to(dtype)
    rows = tq.tq_moe_gather(x, order, offsets, k, out=mark.clone())
    want = mark.clone()
    want[:total] = x[(order[:total] // k).long()]
    assert torch.equal(rows, want)                 # copies, and the rows behind the last slot as they were
    y = torch.randn(T * k, H, generator=_gen(H + 1), device="cuda").to(dtype)
    w = torch.rand(T, k, generator=_gen(H + 2), device="cuda")
    yn, pn = _np(y), _np(pos)
    there = pn >= 0
    taken = yn[np.maximum(pn, 0)] * there[..., None]
    for wt in (w, None):
        wn = np.ones((T, k)) if wt is None else _np(wt)
        out = tq.tq_moe_combine(y, pos, wt) if wt is not None else tq.tq_moe_gather_backward(y, pos)
        ref = (taken * wn[..., None]).sum(1)
        size = (np.abs(taken) * wn[..., None]).sum(1)
        tol = HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -10) + (k + 1) * U * size + TINY[dtype]
        assert np.all(np.abs(_np(out) - ref) <= tol)
    d = torch.randn(T, H, generator=_gen(H + 3), device="cuda").to(dtype)
    dy, dw = tq.tq_moe_combine_backward(d, y, pos, w, dy=mark.clone())
    dn = _np(d)
    ref = _np(mark).copy()
    ref[pn[there]] = (_np(w)[..., None] * dn[:, None, :])[there]
    assert np.all(np.abs(_np(dy) - ref) <= HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -10) + U * np.abs(ref) + TINY[dtype])
    assert torch.equal(dy[total:], mark[total:])
    ref = (taken * dn[:, None, :]).sum(-1)
    size = (np.abs(taken) * np.abs(dn)[:, None, :]).sum(-1)
    assert np.all(np.abs(_np(dw) - ref) <= (-(-H // 128) + 9) * U * size + 2.0 ** -149)
    # one of the two gradients alone, through the C call
    dw2 = torch.empty_like(dw)
    args = (tq.moe._dtype(y, "y"), pos.data_ptr())
    st = torch.cuda.current_stream().cuda_stream
    assert tq.lib.tq_moe_combine_backward(d.data_ptr(), y.data_ptr(), *args, None, None, dw2.data_ptr(), T, T * k, H, k, st) == 0
    dy2 = mark.clone()
    assert tq.lib.tq_moe_combine_backward(d.data_ptr(), None, *args, w.data_ptr(), dy2.data_ptr(), None, T, T * k, H, k, st) == 0
    assert torch.equal(dw, dw2) and torch.equal(dy, dy2)


@pytest.mark.parametrize("shift", [1, 4])
def test_rows_at_odd_addresses(shift):
    need_cuda()
    T, k, E, H = 21, 3, 5, 64
    _, (offsets, order, pos) = _plan(T, k, E, 4)
    base = torch.randn(T * H + shift, generator=_gen(5), device="cuda").half()
    x = base[shift:].view(T, H)
    rows = tq.tq_moe_gather(x, order, offsets, k)
    assert torch.equal(rows, x[(order // k).long()])
    buf = torch.zeros(T * H + shift, dtype=torch.float16, device="cuda")
    out = tq.tq_moe_gather_backward(rows, pos, dx=buf[shift:].view(T, H))
    ref = (3 * x.double()).cpu().numpy()
    assert np.all(np.abs(_np(out) - ref) <= 2.0 ** -11 * np.abs(ref) * (1 + 2.0 ** -10) + 4 * U * np.abs(ref) + TINY[torch.float16])


def test_positions_out_of_range_and_no_rows():
    need_cuda()
    y = torch.randn(4, 16, generator=_gen(1), device="cuda")
    pos = torch.tensor([[0, 4], [-5, 9], [3, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.full((3, 2), 2.0, device="cuda")
    out = tq.tq_moe_combine(y, pos, w)
    assert torch.equal(out, torch.stack([2 * y[0], torch.zeros_like(y[0]), 2 * y[3]]))
    dy, dw = tq.tq_moe_combine_backward(torch.ones(3, 16, device="cuda"), y, pos, w, dy=torch.zeros_like(y))
    assert (dy[[1, 2]] == 0).all() and (dy[[0, 3]] == 2).all()
    assert dw[1].abs().sum() == 0 and dw[0, 1] == 0 and dw[2, 1] == 0
    out = tq.tq_moe_combine(y[:0], pos, w)
    assert (out == 0).all()


def test_another_stream_and_a_captured_graph():
    need_cuda()
    T, k, E, H = 37, 4, 16, 256
    x = torch.randn(T, H, generator=_gen(7), device="cuda").half()
    logits = torch.randn(T, E, generator=_gen(8), device="cuda")

    def step():
        w, ids = tq.tq_moe_route(logits, k)
        offsets, order, pos = tq.tq_moe_sort(ids, E)
        rows = tq.tq_moe_gather(x, order, offsets, k)
        return tq.tq_moe_combine(rows, pos, w), w, ids, offsets, order, pos

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w, ids = tq.tq_moe_route(logits, k, stream=s)
    offsets, order, pos = tq.tq_moe_sort(ids, E, stream=s)
    out = tq.tq_moe_combine(tq.tq_moe_gather(x, order, offsets, k, stream=s), pos, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip((out, w, ids, offsets, order, pos), want):
        assert torch.equal(a, b)
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    logits.copy_(torch.randn(T, E, generator=_gen(9), device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_shape_and_type_refusals():
    need_cuda()
    x = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets, order, pos = tq.tq_moe_sort(ids, 3)
    with pytest.raises(tq.TQError):
        tq.tq_moe_route(x, 9)
    with pytest.raises(ValueError):
        tq.tq_moe_route(x[:, ::2], 2)                                # strides
    with pytest.raises(ValueError):
        tq.tq_moe_sort(ids.long(), 3)
    with pytest.raises(tq.TQError):
        tq.tq_moe_sort(ids, 1025)
    with pytest.raises(ValueError):
        tq.tq_moe_gather(x, order[:-1], offsets, 2)
    with pytest.raises(ValueError):
        tq.tq_moe_gather(x, order, offsets, 2, out=torch.zeros(8, 8, device="cuda").half())
    with pytest.raises(ValueError):
        tq.tq_moe_combine(x, pos, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_moe_combine_backward(x[:3], x, pos, torch.zeros(4, 2, device="cuda"))


@pytest.mark.parametrize("H", [1, 64, 5000])
def test_gather_leaves_rows_of_no_slot(H):
    """order entries that are no slot of the tokens (negative, -1 among them, or past the last): row left as it was."""
    need_cuda()
    T, k, E = 5, 4, 3
    _, (offsets, order, pos) = _plan(T, k, E, H, 0.0)
    order = order.clone()
    bad = torch.tensor([-1, -3, -2 ** 31, T * k, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    order[[0, 4, 9, 11, 19]] = bad
    x = torch.randn(T, H, generator=_gen(H), device="cuda")
    out = tq.tq_moe_gather(x, order, offsets, k, out=torch.full((T * k, H), 7.0, device="cuda"))
    ok = (order >= 0) & (order < T * k)
    want = torch.full((T * k, H), 7.0, device="cuda")
    want[ok] = x[(order[ok] // k).long()]
    assert torch.equal(out, want)
