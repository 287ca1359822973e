"""Adapters: sums long enough to hide what is left out of them, both weight gradients in one launch at any widths and
alignments, plans with foreign rows in the gradients.

Bounds here (closer than lora_util.py's for long sums, whose terms' magnitudes all add up there).  An fp32 sum of n products
in steps of 16 is off by at most one unit in the last place (2^-23 of it) of each step's partial sum, once for the sum itself and
again where the products of a step are aligned with it: n / 16 steps, and 32 more for parts added across warps and CTAs.  A partial
sum of products with random signs is taken to stay below 6 sqrt(sum p^2), six standard deviations of it.  So
  E(n, p) = (n / 16 + 32) 2 2^-23 6 sqrt(sum p^2).
One rounding per product instead of per step, as in the plain kernels, 2^-24 of a partial sum over 1/32 of the products, is
below that."""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from gpu_util import gpu, need_cuda
from test_gpu_lora import _case, _gen, _shifted
from test_gpu_lora_more import _backward as _products_backward, _weights

pytestmark = gpu
HALF, TINY, SPLIT = O.HALF, O.TINY, O.SPLIT
H, B = torch.float16, torch.bfloat16
ANY, TC, FEW = tq.PATH_GENERIC, tq.PATH_PREFILL, tq.PATH_DECODE


def _e(n, squares):
    return (n / 16 + 32) * 2.0 ** -22 * 6 * np.sqrt(squares)


def _rounded(want, tol, dt):
    """The bound after the one rounding to dt, and before it the fp32 roundings of factor and base (two units each)."""
    tol = tol + 2.0 ** -21 * np.abs(want)
    return tol + HALF[dt] * (np.abs(want) + tol) + TINY[dt]


def _segments(offsets, order, M):
    """O.segments without the entries of order that name no row."""
    for l, rows, at in O.segments(offsets, order, M):
        there = (rows >= 0) & (rows < M)
        yield l, rows[there], at[there]


def _forward(x, a, b, base, s, segs, keep, f, dt):
    """(out, its bound, v by row, its bound)."""
    M, r, N = x.shape[0], a.shape[1], b.shape[1]
    out = np.zeros((M, N)) if base is None else base.copy()
    tol, v, tv = np.zeros((M, N)), np.zeros((M, r)), np.zeros((M, r))
    for l, rows, _ in segs:
        if not len(rows):
            continue
        xd = (x * keep * f)[rows]
        v[rows], tv[rows] = xd @ a[l].T, _e(x.shape[1], xd ** 2 @ (a[l] ** 2).T)
        out[rows] += s[l] * (v[rows] @ b[l].T)
        tol[rows] = abs(s[l]) * ((tv[rows] + SPLIT[dt] * np.abs(v[rows])) @ np.abs(b[l]).T + _e(2 * r, v[rows] ** 2 @ (b[l] ** 2).T))
    return out, _rounded(out, tol, dt), v, tv


def _backward(dy, x, a, b, v, base_dx, s, segs, keep, f, dt):
    """(dx, da, db), each with its bound; v by sorted position, as the forward call left it."""
    xd = x * keep * f
    dx = np.zeros(x.shape) if base_dx is None else base_dx.copy()
    tx, da, ta, db, tb = np.zeros(x.shape), np.zeros(a.shape), np.zeros(a.shape), np.zeros(b.shape), np.zeros(b.shape)
    for l, rows, at in segs:
        if not len(rows):
            continue
        n, y, vl = len(rows), dy[rows], v[at]
        d = s[l] * (y @ b[l])
        td = abs(s[l]) * _e(b.shape[1], y ** 2 @ b[l] ** 2)
        m = f * keep[rows]
        dx[rows] += m * (d @ a[l])
        tx[rows] = m * ((td + SPLIT[dt] * np.abs(d)) @ np.abs(a[l]) + _e(2 * a.shape[1], d ** 2 @ a[l] ** 2))
        # a power of two per adapter: what the two parts leave out is 2^-39 of the adapter's largest number at least
        da[l] = d.T @ xd[rows]
        ta[l] = (td + SPLIT[dt] * np.abs(d) + 2.0 ** -39 * np.abs(d).max()).T @ np.abs(xd[rows]) + _e(2 * n, (d ** 2).T @ xd[rows] ** 2)
        db[l] = s[l] * y.T @ vl
        tb[l] = abs(s[l]) * (np.abs(y).T @ (SPLIT[dt] * np.abs(vl) + 2.0 ** -39 * np.abs(vl).max()) + _e(2 * n, (y ** 2).T @ vl ** 2))
    return [(w, _rounded(w, t, dt)) for w, t in ((dx, tx), (da, ta), (db, tb))]


def _check(got, want, tol, rough, label):
    """got is within tol of want, and something of the same size is not: `rough`, want with one chunk left out of the sums."""
    O.check(got, want, tol, label)
    assert (np.abs(rough - want) > tol).any(), f"{label}: the bound would not notice"


# ------------------------------------------------------------------------------------------ long sums
LONG = [(1, 2, 8200, 16, 128), (3, 1, 65536, 24, 16), (140, 2, 16384, 40, 64), (200, 1, 40008, 16, 8), (40, 1, 12345, 9, 33)]


@pytest.mark.parametrize("shape", LONG, ids=str)
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_long_rows(shape, dtype, p):
    """v and out, and dx's other direction (dv of long rows of dy): a chunk of eight columns left out would be noticed."""
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, K, "one")
    rng = torch.tensor([17, 1], dtype=torch.int64, device="cuda")
    x64, a64, b64, y64, s64 = (O.f64(t) for t in (x, a, b, base, s))
    segs, keep, f = list(_segments(offsets, order, M)), O.kept(M, K, p, 17, 1), O.factor(p)
    want, tol, v64, tv = _forward(x64, a64, b64, None, s64, segs, keep, f, dtype)
    cut = x64.copy()
    cut[:, K - 8:] = 0
    out_c, _, v_c, _ = _forward(cut, a64, b64, None, s64, segs, keep, f, dtype)
    rows, at = next((rows, at) for _, rows, at in segs if len(rows))
    for path in [ANY, TC] + ([FEW] if not p and K % 8 == 0 and N % 8 == 0 else []):
        v = torch.zeros(M, r, device="cuda")
        out = tq.tq_lora(x, a, b, None, offsets, order=order, scaling=s, p=p, rng=rng, v=v, path=path)
        _check(out, want, tol, out_c, f"out, path {path}")
        _check(O.f64(v)[at], v64[rows], tv[rows] + 2.0 ** -22 * np.abs(v64[rows]) + 2.0 ** -149, v_c[rows], f"v, path {path}")
    # the other way round: rows of K columns as dy, of N as x
    a2, b2 = b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous()
    keep, f = O.kept(M, N, p, 17, 1), O.factor(p)
    for path in (ANY, TC):
        v = torch.zeros(M, r, device="cuda")
        kw = dict(order=order, scaling=s, p=p, rng=rng, path=path)
        tq.tq_lora(base, a2, b2, None, offsets, v=v, **kw)
        got = tq.tq_lora_backward(x, base, a2, b2, v, None, offsets, **kw)
        args = (y64, O.f64(a2), O.f64(b2), O.f64(v), None, s64, segs, keep, f, dtype)
        for name, g, (w, t), (c, _) in zip(("dx", "da"), got, _backward(x64, *args), _backward(cut, *args)):
            _check(g, w, t, c, f"{name}, path {path}")
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("M,K,N,r", [(20000, 64, 72, 16), (50001, 40, 16, 8), (9000, 33, 24, 100)])
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_weight_gradients_of_many_rows(M, K, N, r, dtype, p):
    """Sums over all rows of one adapter: a chunk of 16 rows left out would be noticed."""
    need_cuda()
    x, a, b, base, s, offsets, order = _case(M, 1, K, N, r, dtype, M, "one")
    dy = (base.float() * 0.1).to(dtype)
    rng = torch.tensor([18, 2], dtype=torch.int64, device="cuda")
    segs, keep, f = list(_segments(offsets, order, M)), O.kept(M, K, p, 18, 2), O.factor(p)
    left = [(l, rows[:-16], at[:-16]) for l, rows, at in segs]
    for path in (ANY, TC):
        v = torch.zeros(M, r, device="cuda")
        kw = dict(order=order, scaling=s, p=p, rng=rng, path=path)
        tq.tq_lora(x, a, b, None, offsets, v=v, **kw)
        got = tq.tq_lora_backward(dy, x, a, b, v, None, offsets, **kw)
        args = [O.f64(t) for t in (dy, x, a, b, v)] + [None, O.f64(s)]
        whole, part = _backward(*args, segs, keep, f, dtype), _backward(*args, left, keep, f, dtype)
        O.check(got[0], *whole[0], f"dx, path {path}")
        for i, name in ((1, "da"), (2, "db")):
            _check(got[i], *whole[i], part[i][0], f"{name}, path {path}")
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(5, 14336, 256), (70, 30000, 128), (300, 14341, 384)])
@pytest.mark.parametrize("fmt", ["ternary", "w4", "w4z"])
def test_gradient_for_x_of_many_weight_rows(M, N, K, fmt):
    """A chunk of eight weight rows left out would be noticed.  An INT4 weight of the tensor-core path is rounded to fp16: half a
    step, 2^-11 of it, with a random sign."""
    need_cuda()
    t, w64 = _weights(N, K, M, fmt)
    dy = torch.randn(M, N, generator=_gen(K), device="cuda").half()
    d = O.f64(dy)
    want, squares = d @ w64, d ** 2 @ w64 ** 2
    rough = want - d[:, N - 8:] @ w64[N - 8:]
    for path in (ANY, TC):
        rounding = 6 * 2.0 ** -11 * np.sqrt(squares) if fmt != "ternary" and path == TC else 0.0
        _check(_products_backward(dy, t, fmt, K, path=path), want, _rounded(want, _e(N, squares) + rounding, H), rough, f"path {path}")
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("zero_point", [False, True])
def test_gradient_through_activation_order(zero_point):
    need_cuda()
    M, N, K = 70, 200, 384
    w = 0.05 * torch.randn(N, K, generator=_gen(1), device="cuda")
    perm = torch.randperm(K, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    q, sc, z, _ = tq.w4g_quantize_pack_ex(w, zero_point=zero_point, perm=perm)
    q = tq.w4g_repack_act_order(q, perm)
    dy = torch.randn(M, N, generator=_gen(3), device="cuda").half()
    inverse = torch.empty_like(perm)
    inverse[perm.long()] = torch.arange(K, dtype=torch.int32, device="cuda")
    dx = tq.tq_permute_columns(tq.w4g_gemm_backward(dy, q, sc, zeros=z), inverse)
    w64, d = np.empty((N, K)), O.f64(dy)
    w64[:, perm.cpu().numpy()] = O.w4_values(q, sc, z)           # in the order of x
    assert np.abs(w64 - O.f64(w)).max() < 0.05                   # the matrix that was packed
    squares = d ** 2 @ w64 ** 2
    O.check(dx, d @ w64, _rounded(d @ w64, _e(N, squares) + 6 * 2.0 ** -11 * np.sqrt(squares), H))


# ------------------------------------------------------------------------------------------ one launch for dA and dB
@pytest.mark.parametrize("shape", [(5, 2, 7, 3, 5), (70, 2, 33, 128, 33), (70, 2, 136, 67, 16), (300, 4, 1001, 264, 16),
                                   (260, 2, 128, 515, 64), (140, 3, 650, 1026, 128), (130, 2, 264, 129, 8)], ids=str)
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_gradients_of_widths_of_two_kinds(shape, dtype, p):
    """K and N that are whole vectors and that are not, in one launch (p = 0) and in two."""
    need_cuda()
    M, L, K, N, r = shape
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, M + N)
    dy, base_dx = (base.float() * 0.1).to(dtype), (x.float() * 0.1).to(dtype)
    rng = torch.tensor([19, 3], dtype=torch.int64, device="cuda")
    segs, keep, f = list(_segments(offsets, order, M)), O.kept(M, K, p, 19, 3), O.factor(p)
    for path in (ANY, TC):
        v = torch.zeros(M, r, device="cuda")
        kw = dict(order=order, scaling=s, p=p, rng=rng, path=path)
        tq.tq_lora(x, a, b, None, offsets, v=v, **kw)
        got = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, **kw)
        want = _backward(*(O.f64(t) for t in (dy, x, a, b, v, base_dx, s)), segs, keep, f, dtype)
        for name, g, (w, t) in zip(("dx", "da", "db"), got, want):
            O.check(g, w, t, f"{name}, path {path}")
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("moved", ["x", "dy", "da", "db", "x dy da db"])
@pytest.mark.parametrize("dtype", [H, B])
def test_one_launch_with_misaligned_operands(moved, dtype):
    need_cuda()
    M, L, K, N, r = 150, 3, 136, 264, 24
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, 78)
    dy = (base.float() * 0.1).to(dtype)
    v = torch.zeros(M, r, device="cuda")
    kw = dict(order=order, scaling=s, path=TC)
    tq.tq_lora(x, a, b, None, offsets, v=v, **kw)
    want = tq.tq_lora_backward(dy, x, a, b, v, None, offsets, **kw)
    to = lambda name, t: _shifted(t) if name in moved.split() else t
    got = tq.tq_lora_backward(to("dy", dy), to("x", x), a, b, v, None, offsets, da=to("da", torch.empty_like(a)),
                              db=to("db", torch.empty_like(b)), **kw)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


# ------------------------------------------------------------------------------------------ plans
@pytest.mark.parametrize("path", [ANY, TC])
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("K", [136, 101])
def test_gradients_of_a_plan_with_foreign_rows(path, dtype, p, K):
    """Rows before offsets[0], behind offsets[L] and entries of order outside [0, M): only named rows of dx are written, those
    without an adapter with the projection's part, and the weight gradients are sums over the named rows of an adapter."""
    need_cuda()
    M, L, N, r = 200, 4, 72, 16
    x, a, b, base, s, _, _ = _case(M, L, K, N, r, dtype, 9)
    dy, base_dx = (base.float() * 0.1).to(dtype), (x.float() * 0.1).to(dtype)
    order = torch.randperm(M, generator=_gen(9), device="cuda").to(torch.int32)
    gone = [0, 5, 64, 65, 140, 198]                              # positions that name no row
    named = sorted(set(range(M)) - set(order[gone].tolist()))
    order[gone] = torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31, M + 1, -7], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([3, 70, 70, 186, 192], dtype=torch.int32, device="cuda")
    rng = torch.tensor([20, 4], dtype=torch.int64, device="cuda")
    segs, keep, f = list(_segments(offsets, order, M)), O.kept(M, K, p, 20, 4), O.factor(p)
    v = torch.full((M, r), float("nan"), device="cuda")
    kw = dict(order=order, scaling=s, p=p, rng=rng, path=path)
    tq.tq_lora(x, a, b, None, offsets, v=v, **kw)
    dx = torch.full_like(x, 7.0)
    dx, da, db = tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, dx=dx, **kw)
    want = _backward(*(O.f64(t) for t in (dy, x, a, b, v, base_dx, s)), segs, keep, f, dtype)
    O.check(O.f64(dx)[named], want[0][0][named], want[0][1][named], "dx")
    left = sorted(set(range(M)) - set(named))
    assert (dx[left] == 7.0).all()
    without = sorted(set(named) - {int(m) for _, rows, _ in segs for m in rows})
    assert without and torch.equal(dx[without], base_dx[without])
    for g, (w, t), name in ((da, want[1], "da"), (db, want[2], "db")):
        O.check(g, w, t, name)
    assert not da[1].any() and not db[1].any()


# ------------------------------------------------------------------------------------------ non-finite rows
@pytest.mark.parametrize("path", [ANY, TC])
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["x", "dy", "b"])
def test_what_is_not_finite_stays_where_it_belongs(path, dtype, bad, where):
    """Elements that are finite by the formula are as before; those that are not are not finite (an infinity may come as NaN)."""
    need_cuda()
    M, L, K, N, r = 150, 2, 136, 72, 16
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, 10)
    dy = (base.float() * 0.1).to(dtype)
    kw = dict(order=order, scaling=s, path=path)

    def step(x, b, dy):
        v = torch.zeros(M, r, device="cuda")
        out = tq.tq_lora(x, a, b, base, offsets, v=v, **kw)
        return [out, v, *tq.tq_lora_backward(dy, x, a, b, v, None, offsets, **kw)]

    clean = step(x, b, dy)
    x, b, dy = x.clone(), b.clone(), dy.clone()
    pos = int(offsets[1]) - 1
    m = int(order[pos])                                          # a row of adapter 0
    if where == "x":
        x[m, 5] = bad
    elif where == "dy":
        dy[m, 5] = bad
    else:
        b[0, 5, 3] = bad
    got = step(x, b, dy)
    hit = [torch.zeros_like(t, dtype=torch.bool) for t in got]
    out, v, dx, da, db = hit
    mine = order[int(offsets[0]):pos + 1].long()
    if where == "x":
        out[m], v[pos], da[0, :, 5], db[0] = True, True, True, True
    elif where == "dy":
        dx[m], da[0], db[0, 5] = True, True, True
    else:
        out[mine, 5], dx[mine], da[0, 3] = True, True, True
    for g, w, h, name in zip(got, clean, hit, ("out", "v", "dx", "da", "db")):
        assert torch.equal(torch.where(h, 0, g), torch.where(h, 0, w)), name
        assert not torch.isfinite(g[h]).any(), name
