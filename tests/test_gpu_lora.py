"""Low-rank adapters (forward and gradients) against 64-bit host forms; the bounds are in lora_util.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from gpu_util import gpu, need_cuda

pytestmark = gpu
U, HALF, TINY, SPLIT = O.U, O.HALF, O.TINY, O.SPLIT
H, B = torch.float16, torch.bfloat16
ANY, TC, FEW = tq.PATH_GENERIC, tq.PATH_PREFILL, tq.PATH_DECODE


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _plan(M, L, seed, how):
    """ids int32 [M] and the plan of tq_moe_sort: rows spread at random, in runs, with adapters and rows left out."""
    g = _gen(seed)
    if how == "one":
        ids = torch.full((M,), L // 2, device="cuda")
    elif how == "none":
        ids = torch.full((M,), -1, device="cuda")
    else:
        ids = torch.randint(-1, L, (M,), generator=g, device="cuda")
        if how == "runs":
            ids = torch.sort(ids).values
        ids[ids == L - 1] = 0 if L > 1 else ids[ids == L - 1]       # one adapter without rows
    ids = ids.to(torch.int32)
    offsets, order, _ = tq.tq_moe_sort(ids.view(M, 1), L)
    return offsets, order


def _case(M, L, K, N, r, dtype, seed, how="spread"):
    g = _gen(seed)
    x = (torch.randn(M, K, generator=g, device="cuda") * (1 + 19 * (torch.rand(M, 1, generator=g, device="cuda") < 0.1))).to(dtype)
    a = (torch.randn(L, r, K, generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (0.2 * torch.randn(L, N, r, generator=g, device="cuda")).to(dtype)
    base = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    s = torch.rand(L, generator=g, device="cuda") * 2 + 0.5
    return (x, a, b, base, s, *_plan(M, L, seed + 1, how))


def _sum_tol(n):
    return (2 * n + 16) * U


def _forward64(x, a, b, base, s, offsets, order, p=0.0, seed=0, offset=0):
    M, K = x.shape
    segs = list(O.segments(offsets, order, M))
    keep, f = O.kept(M, K, p, seed, offset), O.factor(p)
    sc = np.ones(a.shape[0]) if s is None else O.f64(s)
    out, v, vs, mag, spread = O.forward(O.f64(x), O.f64(a), O.f64(b), O.f64(base), sc, segs, keep, f)
    dt, r = x.dtype, a.shape[1]
    tv = _sum_tol(K) * vs
    tol = _sum_tol(K) * spread + (SPLIT[dt] + _sum_tol(2 * r)) * (mag + spread * _sum_tol(K))
    tol = tol + HALF[dt] * (np.abs(out) + tol) + TINY[dt]
    return out, tol, v, tv, segs


def _check_v(v, want, tol, segs):
    for _, rows, at in segs:
        O.check(O.f64(v)[at], want[rows], tol[rows] + 2.0 ** -149, "v")


SHAPES = [(1, 1, 8, 8, 1), (1, 3, 64, 24, 16), (7, 2, 136, 8, 8), (8, 8, 512, 72, 16), (9, 4, 1000, 200, 32),
          (33, 5, 72, 264, 64), (61, 32, 256, 1032, 24), (130, 1, 264, 136, 128), (129, 3, 2048, 40, 4), (300, 7, 520, 520, 40),
          (1, 2, 8200, 16, 128), (257, 2, 128, 4096, 100)]
ODD = [(5, 2, 7, 3, 5), (19, 3, 101, 67, 12), (70, 2, 33, 129, 33), (3, 1, 1, 1, 1), (300, 4, 1001, 264, 16), (260, 2, 128, 515, 64),
       (140, 3, 650, 1026, 128)]


def _paths(M, p=0.0):
    return [ANY, TC] + ([FEW] if not p else [])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("how", ["spread", "runs"])
def test_forward(shape, dtype, how):
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, M * 7 + K, how)
    want, tol, v64, tv, segs = _forward64(x, a, b, base, s, offsets, order)
    for path in _paths(M):
        v = torch.full((M, r), float("nan"), device="cuda")
        out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, v=v, path=path)
        O.check(out, want, tol, f"path {path}")
        _check_v(v, v64, tv, segs)
        again = base.clone()                                         # in place, without a v from the caller
        assert tq.tq_lora(x, a, b, again, offsets, order=order, scaling=s, out=again, path=path) is again
        assert torch.equal(again, out)
    O.check(tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s), want, tol, "auto")
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("shape", ODD, ids=str)
@pytest.mark.parametrize("dtype", [H, B])
def test_forward_odd_sizes(shape, dtype):
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, M)
    want, tol, v64, tv, segs = _forward64(x, a, b, base, s, offsets, order)
    for path in (tq.PATH_AUTO, ANY, TC):
        v = torch.empty(M, r, device="cuda")
        O.check(tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, v=v, path=path), want, tol)
        _check_v(v, v64, tv, segs)
        again = base.clone()
        assert torch.equal(tq.tq_lora(x, a, b, again, offsets, order=order, scaling=s, out=again, path=path),
                           tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path))
    with pytest.raises(tq.TQError):
        tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=FEW)


@pytest.mark.parametrize("path", [ANY, TC, FEW])
def test_forward_without_base_scaling_or_order(path):
    """NULL arguments; sorted rows with rows of no adapter before the first and after the last one."""
    need_cuda()
    M, L, K, N, r = 45, 3, 128, 96, 16
    x, a, b, base, s, _, _ = _case(M, L, K, N, r, H, 5)
    offsets = torch.tensor([4, 4, 21, 39], dtype=torch.int32, device="cuda")
    want, tol, *_ = _forward64(x, a, b, None, None, offsets, None)
    out = tq.tq_lora(x, a, b, None, offsets, path=path)
    O.check(out, want, tol)
    assert not out[:4].any() and not out[39:].any()
    want, tol, *_ = _forward64(x, a, b, base, s, offsets, None)
    out = tq.tq_lora(x, a, b, base, offsets, scaling=s, path=path)
    O.check(out, want, tol)
    assert torch.equal(out[:4], base[:4]) and torch.equal(out[39:], base[39:])


@pytest.mark.parametrize("path", [ANY, TC, FEW])
@pytest.mark.parametrize("how", ["none", "one"])
def test_forward_no_adapter_and_one_adapter(path, how):
    need_cuda()
    M, L, K, N, r = 150, 6, 192, 320, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, B, 8, how)
    want, tol, *_ = _forward64(x, a, b, base, s, offsets, order)
    out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path)
    O.check(out, want, tol)
    if how == "none":
        assert torch.equal(out, base)


@pytest.mark.parametrize("path", [ANY, TC, FEW])
def test_an_order_with_foreign_rows(path):
    """Entries of order outside [0, M) name no row: nothing is read or written for them, the others are right."""
    need_cuda()
    M, L, K, N, r = 20, 2, 64, 40, 8
    x, a, b, base, s, _, _ = _case(M, L, K, N, r, H, 4)
    order = torch.arange(M, dtype=torch.int32, device="cuda").flip(0).contiguous()
    order[3], order[11], order[19] = -1, M, 2 ** 31 - 1
    offsets = torch.tensor([1, 9, 18], dtype=torch.int32, device="cuda")
    named = [i for i in order.tolist() if 0 <= i < M]
    out = torch.full_like(base, 7.0)
    tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, out=out, path=path)
    o = order.clone()
    o[(o < 0) | (o >= M)] = 0
    segs = [(l, rows[np.isin(rows, named)], at) for l, rows, at in O.segments(offsets, order, M)]
    want, _, _, mag, spread = O.forward(O.f64(x), O.f64(a), O.f64(b), O.f64(base), O.f64(s), segs, np.ones((M, K), bool), 1.0)
    O.check(O.f64(out)[named], want[named], (1e-3 * (mag + spread) + HALF[H] * np.abs(want) + 2.0 ** -25)[named])
    left = sorted(set(range(M)) - set(named))
    assert (out[left] == 7.0).all()


@pytest.mark.parametrize("path", [ANY, TC, FEW])
def test_infinities_stay_in_their_row(path):
    need_cuda()
    M, L, K, N, r = 40, 2, 256, 128, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, 12)
    clean = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path)
    rows = [int(order[int(offsets[0])]), int(order[int(offsets[1]) - 1])]
    x[rows[0], 3], x[rows[1], 200] = float("inf"), float("nan")
    out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path)
    others = [m for m in range(M) if m not in rows]
    assert torch.equal(out[others], clean[others])
    assert not torch.isfinite(out[rows]).any()


@pytest.mark.parametrize("path", [ANY, TC, FEW])
@pytest.mark.parametrize("scale", [1e-6, 3e3])
def test_inner_rows_outside_the_half_range(path, scale):
    """v far below and above what fp16 holds: it is kept in fp32, and split with a power of two per row."""
    need_cuda()
    M, L, K, N, r = 24, 2, 512, 64, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, 3)
    x = (x.float().clamp(-4, 4) * scale).half() if scale > 1 else (x.float() * 1e-3).half()
    a = (a.float() * (8 if scale > 1 else 1e-3)).half()
    b = (b.float() * (1e-4 if scale > 1 else 1e3)).half()
    want, tol, *_ = _forward64(x, a, b, None, s, offsets, order)
    O.check(tq.tq_lora(x, a, b, None, offsets, order=order, scaling=s, path=path), want, tol)


def test_bad_sizes_are_refused_on_the_gpu_too():
    need_cuda()
    x, a, b, base, s, offsets, order = _case(8, 2, 64, 64, 8, H, 2)
    with pytest.raises(tq.TQError):
        tq.tq_lora(x, a.repeat(1, 17, 1), b.repeat(1, 1, 17), base, offsets)           # rank 136
    with pytest.raises(ValueError, match="order"):
        tq.tq_lora(x, a, b, base, offsets, order=order[:4])
    with pytest.raises(ValueError, match="contiguous"):
        tq.tq_lora(x.t().contiguous().t(), a, b, base, offsets)
    with pytest.raises(ValueError, match="base"):
        tq.tq_lora(x, a, b, base.bfloat16(), offsets)
    with pytest.raises(ValueError, match="scaling"):
        tq.tq_lora(x, a, b, base, offsets, scaling=s.half())


# ------------------------------------------------------------------------------------------ gradients
def _backward64(dy, x, a, b, v, base_dx, s, offsets, order, p, seed, offset):
    """Gradients and their bounds, v taken as the forward call left it."""
    x64, a64, b64, dy64, v64 = O.f64(x), O.f64(a), O.f64(b), O.f64(dy), O.f64(v)
    M, K = x.shape
    L, r, N, dt = a.shape[0], a.shape[1], b.shape[1], x.dtype
    keep, f = O.kept(M, K, p, seed, offset), O.factor(p)
    sc = np.ones(L) if s is None else O.f64(s)
    xd = x64 * keep * f
    dx = np.zeros((M, K)) if base_dx is None else O.f64(base_dx)
    tx = np.zeros((M, K))
    da, ta, db, tb = np.zeros(a.shape), np.zeros(a.shape), np.zeros(b.shape), np.zeros(b.shape)
    for l, rows, at in O.segments(offsets, order, M):
        if not len(rows):
            continue
        n = len(rows)
        d, ds = sc[l] * (dy64[rows] @ b64[l]), sc[l] * (np.abs(dy64[rows]) @ np.abs(b64[l]))
        td = _sum_tol(N) * ds                                        # bound of dv
        dx[rows] += f * keep[rows] * (d @ a64[l])
        tx[rows] = f * keep[rows] * ((td + (SPLIT[dt] + _sum_tol(2 * r)) * (np.abs(d) + td)) @ np.abs(a64[l]))
        da[l] = d.T @ xd[rows]
        # wgrad's common power of two: what is below 2^-24 of the adapter's largest value counts as zero or keeps an error of
        # 2^-39 of that value
        ta[l] = (td + (SPLIT[dt] + _sum_tol(2 * n)) * (np.abs(d) + td) + 2.0 ** -36 * np.abs(d).max()).T @ np.abs(xd[rows])
        db[l] = sc[l] * dy64[rows].T @ v64[at]
        tb[l] = sc[l] * np.abs(dy64[rows]).T @ ((SPLIT[dt] + _sum_tol(2 * n)) * np.abs(v64[at]) + 2.0 ** -36 * np.abs(v64[at]).max())
    done = []
    for want, t in ((dx, tx), (da, ta), (db, tb)):
        done.append((want, t + HALF[dt] * (np.abs(want) + t) + TINY[dt]))
    return done


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward(shape, dtype, p):
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, M * 11 + N, "runs" if M % 2 else "spread")
    dy = (0.1 * torch.randn(M, N, generator=_gen(9), device="cuda")).to(dtype)
    base_dx = (0.1 * torch.randn(M, K, generator=_gen(10), device="cuda")).to(dtype)
    rng = torch.tensor([2 ** 63 - 5, -7], dtype=torch.int64, device="cuda")
    v64, tol, _, _, _ = _forward64(x, a, b, base, s, offsets, order, p, 2 ** 63 - 5, -7)
    for path in (ANY, TC):
        v = torch.zeros(M, r, device="cuda")
        out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, p=p, rng=rng, v=v, path=path)
        O.check(out, v64, tol, f"forward, path {path}")
        want = _backward64(dy, x, a, b, v, base_dx, s, offsets, order, p, 2 ** 63 - 5, -7)
        kw = dict(order=order, scaling=s, p=p, rng=rng, path=path)
        got = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, **kw)
        for g, (w, t), name in zip(got, want, ("dx", "da", "db")):
            O.check(g, w, t, f"{name}, path {path}")
        again = base_dx.clone()
        more = tq.tq_lora_backward(dy, x, a, b, v, again, offsets, dx=again, **kw)
        assert more[0] is again and all(torch.equal(g, h) for g, h in zip(got, more))
        only = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, need_ab=False, **kw)
        assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
        only = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, need_dx=False, **kw)
        assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("shape", ODD, ids=str)
def test_backward_odd_sizes(shape):
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, M)
    dy = (0.1 * torch.randn(M, N, generator=_gen(9), device="cuda")).half()
    rng = torch.tensor([11, 12], dtype=torch.int64, device="cuda")
    for path in (ANY, TC):
        v = torch.zeros(M, r, device="cuda")
        tq.tq_lora(x, a, b, None, offsets, order=order, scaling=s, p=0.25, rng=rng, v=v, path=path)
        want = _backward64(dy, x, a, b, v, None, s, offsets, order, 0.25, 11, 12)
        got = tq.tq_lora_backward(dy, x, a, b, v, None, offsets, order=order, scaling=s, p=0.25, rng=rng, path=path)
        for g, (w, t), name in zip(got, want, ("dx", "da", "db")):
            O.check(g, w, t, f"{name}, path {path}")


@pytest.mark.parametrize("path", [ANY, TC])
def test_backward_of_no_rows(path):
    """Adapters without rows get zeros, rows without an adapter the base, a batch without rows zeros."""
    need_cuda()
    M, L, K, N, r = 20, 3, 64, 72, 8
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, B, 8, "none")
    v = torch.full((M, r), float("nan"), device="cuda")
    dx, da, db = tq.tq_lora_backward(base, x, a, b, v, x, offsets, order=order, scaling=s, path=path)
    assert torch.equal(dx, x) and not da.any() and not db.any()
    e = torch.zeros(L + 1, dtype=torch.int32, device="cuda")
    dx, da, db = tq.tq_lora_backward(base[:0], x[:0], a, b, v[:0], None, e, path=path)
    assert dx.shape == (0, K) and not da.any() and not db.any()


@pytest.mark.parametrize("path", [ANY, TC])
@pytest.mark.parametrize("dtype", [H, B])
def test_no_output_columns(path, dtype):
    """N = 0: nothing to write forward, the projection's part alone backward."""
    need_cuda()
    M, L, K, r = 20, 2, 64, 8
    x, a, b, base, s, offsets, order = _case(M, L, K, 8, r, dtype, 8)
    b, base = b[:, :0].contiguous(), base[:, :0].contiguous()
    assert tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path).shape == (M, 0)
    v = torch.zeros(M, r, device="cuda")
    dx, da, db = tq.tq_lora_backward(base, x, a, b, v, x, offsets, order=order, scaling=s, path=path)
    assert torch.equal(dx, x) and not da.any() and db.shape == b.shape


@pytest.mark.parametrize("path", [ANY, TC])
def test_small_and_large_gradients(path):
    """dv far outside the range of fp16: it is scaled by powers of two where it enters a tensor-core product."""
    need_cuda()
    M, L, K, N, r = 140, 2, 128, 256, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, 21)
    for size, more in ((2.0 ** -18, 2.0 ** -4), (1000.0, 30.0)):
        dy = (size * torch.randn(M, N, generator=_gen(2), device="cuda")).half()
        bb = (b.float() * more).half()
        aa = (a.float() / more).half()
        v = torch.zeros(M, r, device="cuda")
        tq.tq_lora(x, aa, bb, None, offsets, order=order, scaling=s, v=v, path=path)
        want = _backward64(dy, x, aa, bb, v, None, s, offsets, order, 0.0, 0, 0)
        got = tq.tq_lora_backward(dy, x, aa, bb, v, None, offsets, order=order, scaling=s, path=path)
        for g, (w, t), name in zip(got, want, ("dx", "da", "db")):
            fits = np.abs(w) < 60000
            O.check(np.where(fits, O.f64(g), 0), np.where(fits, w, 0), t, name)


def _shifted(t):
    """The same values two bytes past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = buf[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def test_misaligned_tensors():
    """Rows that are no aligned vectors are read and written element by element: the same results."""
    need_cuda()
    M, L, K, N, r = 150, 3, 136, 264, 24
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, B, 77)
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    dy, base_dx = (base * 0.1), (x * 0.1)
    v = torch.zeros(M, r, device="cuda")
    kw = dict(order=order, scaling=s, p=0.2, rng=rng, path=TC)
    out = tq.tq_lora(x, a, b, base, offsets, v=v, **kw)
    grads = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, **kw)
    w = torch.zeros(M, r, device="cuda")
    dest = _shifted(torch.zeros_like(base))
    got = tq.tq_lora(_shifted(x), _shifted(a), _shifted(b), _shifted(base), offsets, v=w, out=dest, **kw)
    assert got is dest and torch.equal(got, out) and torch.equal(v, w)
    more = tq.tq_lora_backward(_shifted(dy), _shifted(x), _shifted(a), _shifted(b), w, _shifted(base_dx), offsets,
                               dx=_shifted(x), da=_shifted(a), db=_shifted(b), **kw)
    assert all(torch.equal(g, h) for g, h in zip(more, grads))
    plain = tq.tq_lora(_shifted(x), a, b, base, offsets, order=order, scaling=s)
    want, tol, *_ = _forward64(x, a, b, base, s, offsets, order)
    O.check(plain, want, tol)
    with pytest.raises(tq.TQError):
        tq.tq_lora(_shifted(x), a, b, base, offsets, order=order, scaling=s, path=FEW)


def test_two_streams_at_once_and_two_captured_graphs():
    """Calls with scratch of their own may run at once, eager and replayed."""
    need_cuda()
    cases = [_case(400, 4, 512, 768, 32, H, 90 + i) for i in range(2)]
    dys = [(c[3] * 0.1) for c in cases]
    vs = [torch.zeros(400, 32, device="cuda") for _ in cases]
    ws = [torch.empty(tq.tq_lora_workspace_size(400, 4, 32), dtype=torch.uint8, device="cuda") for _ in cases]

    def step(i):
        x, a, b, base, s, offsets, order = cases[i]
        out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, v=vs[i], path=TC)
        few = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=FEW)
        return (out, few, *tq.tq_lora_backward(dys[i], x, a, b, vs[i], None, offsets, order=order, scaling=s, workspace=ws[i]))

    want = [tuple(t.clone() for t in step(i)) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(step(i))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, w in zip(got, want) for p, q in zip(g, w))
    graphs, outs = [], []
    for i, st in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(step(i))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, w in zip(outs, want) for p, q in zip(g, w))
    assert tq.tq_device_status() == 0


def test_a_captured_graph_serves_any_plan():
    need_cuda()
    M, L, K, N, r = 96, 5, 256, 320, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, 50)
    ids = torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step(path):
        o, w, _ = tq.tq_moe_sort(ids, L)
        return tq.tq_lora(x, a, b, base, o, order=w, scaling=s, path=path)

    with torch.cuda.stream(st):
        step(TC), step(FEW)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        outs = [step(TC), step(FEW)]
    for seed, how in ((1, "spread"), (2, "none"), (3, "one"), (4, "runs")):
        offsets, order = _plan(M, L, seed, how)
        new = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        for l in range(L):
            new[order[offsets[l]:offsets[l + 1]].long()] = l
        ids.copy_(new.view(M, 1))
        g.replay()
        torch.cuda.synchronize()
        want, tol, *_ = _forward64(x, a, b, base, s, offsets, order)
        for out in outs:
            O.check(out, want, tol, how)


def test_many_adapters_and_highest_rank():
    """1024 adapters, most without rows, of rank 128."""
    need_cuda()
    M, L, K, N, r = 40, 1024, 64, 72, 128
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, B, 60)
    want, tol, *_ = _forward64(x, a, b, base, s, offsets, order)
    for path in (ANY, TC, FEW):
        O.check(tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=path), want, tol, f"path {path}")
    v = torch.zeros(M, r, device="cuda")
    tq.tq_lora(x, a, b, None, offsets, order=order, scaling=s, v=v, path=TC)
    w = _backward64(base, x, a, b, v, None, s, offsets, order, 0.0, 0, 0)
    for g, (want, tol), name in zip(tq.tq_lora_backward(base, x, a, b, v, None, offsets, order=order, scaling=s), w, ("dx", "da", "db")):
        O.check(g, want, tol, name)


def test_rows_past_two_to_the_31_elements():
    """Offsets of rows in x and base past 2^31 elements, on the tensor cores and element offsets of dropout with them."""
    need_cuda()
    M, L, K, N, r = 140000, 2, 16384, 16, 8
    x = torch.zeros(M, K, dtype=H, device="cuda")
    last = torch.randn(64, K, generator=_gen(1), device="cuda").half()
    x[-64:] = last
    _, a, b, base, s, _, _ = _case(64, L, K, N, r, H, 1)
    offsets = torch.tensor([0, M - 30, M], dtype=torch.int32, device="cuda")
    small = torch.tensor([0, 34, 64], dtype=torch.int32, device="cuda")
    out = tq.tq_lora(x, a, b, None, offsets, scaling=s)
    want, tol, *_ = _forward64(last, a, b, None, s, small, None)
    O.check(out[-64:], want, tol)
    assert not out[:-64].any()
    rng = torch.tensor([4, 4], dtype=torch.int64, device="cuda")
    y = tq.tq_dropout(x, 0.5, rng)
    tail = O.kept_rows(M, K, 0.5, 4, 4, M - 64)
    assert np.array_equal(O.f64(y[-64:]) != 0, tail & (O.f64(last) != 0))
    v = torch.zeros(M, r, device="cuda")
    tq.tq_lora(x, a, b, None, offsets, scaling=s, p=0.5, rng=rng, v=v, path=TC)
    xd = O.f64(last) * tail * 2.0
    for l, lo, hi in ((0, 0, 34), (1, 34, 64)):
        w = xd[lo:hi] @ O.f64(a[l]).T
        mag = np.abs(xd[lo:hi]) @ np.abs(O.f64(a[l])).T
        O.check(O.f64(v[-64:])[lo:hi], w, _sum_tol(K) * mag + 2.0 ** -149, "v")


def test_same_results_on_every_run():
    need_cuda()
    M, L, K, N, r = 700, 5, 512, 640, 32
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, 31)
    dy = base * 0.1
    first = None
    for _ in range(3):
        v = torch.zeros(M, r, device="cuda")
        out = tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, v=v)
        now = (out, v, *tq.tq_lora_backward(dy, x, a, b, v, None, offsets, order=order, scaling=s))
        first = first or now
        assert all(torch.equal(p, q) for p, q in zip(first, now))
