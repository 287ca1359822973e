"""Dropout, the packed products' gradient for x, and a training step of an adapter beside a packed projection, against 64-bit
host forms; the bounds are in lora_util.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from gpu_util import check_canaries, gpu, guarded_empty, need_cuda

pytestmark = gpu
U, HALF, TINY = O.U, O.HALF, O.TINY


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------------------ dropout
@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 7), (5, 64), (33, 1001), (130, 4096), (2, 9)])
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("p,seed,offset", [(0.0, 0, 0), (0.1, 1234567890123456789, 5), (0.5, -1, 2 ** 40 + 1), (0.9999, 7, -3)])
def test_dropout(M, K, dtype, p, seed, offset):
    need_cuda()
    x = torch.randn(M, K, generator=_gen(M + K), device="cuda").to(dtype)
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    out = tq.tq_dropout(x, p, rng)
    want = O.f64(x) * O.kept(M, K, p, seed, offset) * O.factor(p)
    # one multiplication in fp32 by a factor rounded to fp32, one rounding of the result
    tol = (3 * U + HALF[dtype]) * np.abs(want) + TINY[dtype]
    fits = np.abs(want) < (6e4 if dtype == torch.float16 else 1e30)
    O.check(np.where(fits, O.f64(out), 0), np.where(fits, want, 0), tol)
    assert np.array_equal(O.f64(out) == 0, want == 0)
    again = x.clone()
    assert tq.tq_dropout(again, p, rng, out=again) is again and torch.equal(again, out)


def test_dropped_elements_are_zero_whatever_they_hold():
    need_cuda()
    x = torch.full((16, 40), float("nan"), device="cuda")
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    out = tq.tq_dropout(x, 0.5, rng)
    keep = O.kept(16, 40, 0.5, 3, 4)
    assert np.array_equal(np.isnan(O.f64(out)), keep) and not out[torch.from_numpy(~keep).cuda()].any()


def test_dropout_of_misaligned_rows_and_empty_ones():
    need_cuda()
    buf = torch.randn(1 + 6 * 16, generator=_gen(1), device="cuda").half()
    rng = torch.tensor([9, 9], dtype=torch.int64, device="cuda")
    a, b = tq.tq_dropout(buf[1:].view(6, 16), 0.3, rng), tq.tq_dropout(buf[1:].clone().view(6, 16), 0.3, rng)
    assert torch.equal(a, b)
    assert tq.tq_dropout(buf[:0].view(0, 8), 0.3, rng).shape == (0, 8)
    assert tq.tq_dropout(buf[:0].view(3, 0), 0.3, rng).shape == (3, 0)


def test_share_of_dropped_elements():
    """Of 2^20 elements a share p is dropped, to five standard deviations; neighbours and offsets are independent."""
    need_cuda()
    M, K, p = 256, 4096, 0.25
    x = torch.ones(M, K, device="cuda")
    r = [tq.tq_dropout(x, p, torch.tensor([1, o], dtype=torch.int64, device="cuda")) == 0 for o in (0, 1)]
    n = M * K
    dev = 5 * (p * (1 - p) / n) ** 0.5
    assert all(abs(float(t.float().mean()) - p) < dev for t in r)
    assert abs(float((r[0] & r[1]).float().mean()) - p * p) < 5 * (p * p / n) ** 0.5
    assert abs(float((r[0][:, 1:] & r[0][:, :-1]).float().mean()) - p * p) < 5 * (2 * p * p / n) ** 0.5


def test_a_replayed_graph_reads_the_generators_state():
    need_cuda()
    x = torch.randn(64, 256, generator=_gen(2), device="cuda").half()
    rng = torch.tensor([5, 0], dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = tq.tq_dropout(x, 0.4, rng)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.tq_dropout(x, 0.4, rng, out=out)
        rng[1] += 1
    rng[1] = 0
    seen = []
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        seen.append(out.clone())
        assert np.array_equal(O.f64(out) != 0, O.kept(64, 256, 0.4, 5, i) & (O.f64(x) != 0))
    assert not torch.equal(seen[0], seen[1])


# ------------------------------------------------------------------------------------------ gradient for x
def _weights(N, K, seed, fmt):
    w = 0.05 * torch.randn(N, K, generator=_gen(seed), device="cuda")
    if fmt == "ternary":
        packed, scale = tq.tq_quantize_pack(w)
        return (packed, scale), O.ternary_values(packed, scale, K)
    if fmt == "w4":
        q, s = tq.w4g_quantize_pack(w)
        return (q, s, None), O.w4_values(q, s, None)
    q, s, z, _ = tq.w4g_quantize_pack_ex(w + 0.03, zero_point=True)
    return (q, s, z), O.w4_values(q, s, z)


def _backward(dy, t, fmt, K, **kw):
    if fmt == "ternary":
        return tq.tq_gemm_backward(dy, t[0], t[1], K=K, **kw)
    return tq.w4g_gemm_backward(dy, t[0], t[1], zeros=t[2], **kw)


def _dx_check(dy, w64, out, rounded):
    """A sum of N products of fp16 dy and weights in fp32; rounded: each weight rounded to fp16 before (2^-11)."""
    d = O.f64(dy)
    want, mag = d @ w64, np.abs(d) @ np.abs(w64)
    N = d.shape[1]
    tol = ((2 * N + 20) * U + (2.0 ** -11 if rounded else 0.0)) * mag
    O.check(out, want, tol + HALF[torch.float16] * (np.abs(want) + tol) + 2.0 ** -25)


@pytest.mark.parametrize("M,N,K", [(1, 8, 128), (7, 72, 128), (61, 1024, 256), (64, 128, 384), (129, 200, 640), (130, 520, 1152),
                                   (257, 1000, 512), (300, 64, 2304), (5, 4096, 128), (520, 264, 128),
                                   (2816, 1024, 1792)])  # 154 tiles: the last six in a launch of their own
@pytest.mark.parametrize("fmt", ["ternary", "w4", "w4z"])
def test_gradient_for_x(M, N, K, fmt):
    need_cuda()
    t, w64 = _weights(N, K, M + N, fmt)
    dy = torch.randn(M, N, generator=_gen(K), device="cuda").half()
    for path in (tq.PATH_AUTO, tq.PATH_GENERIC, tq.PATH_PREFILL):
        dx, buf = guarded_empty(M, K)
        _backward(dy, t, fmt, K, dx=dx, path=path)
        _dx_check(dy, w64, dx, fmt != "ternary" and path != tq.PATH_GENERIC)
        check_canaries(buf, M, K)
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(3, 5, 7), (9, 33, 130), (17, 100, 64), (1, 1, 1), (40, 9, 192), (40, 16, 192),
                                   (300, 72, 64)])
def test_gradient_for_x_ternary_odd_sizes(M, N, K):
    need_cuda()
    t, w64 = _weights(N, K, M + N, "ternary")
    dy = torch.randn(M, N, generator=_gen(K), device="cuda").half()
    for path in (tq.PATH_AUTO, tq.PATH_GENERIC, tq.PATH_PREFILL):
        if K % 64 and path == tq.PATH_PREFILL:
            with pytest.raises(tq.TQError):
                _backward(dy, t, "ternary", K, path=path)
            continue
        dx, buf = guarded_empty(M, K)
        _dx_check(dy, w64, _backward(dy, t, "ternary", K, dx=dx, path=path), False)
        check_canaries(buf, M, K)


@pytest.mark.parametrize("fmt", ["ternary", "w4"])
def test_gradient_for_x_of_misaligned_rows(fmt):
    need_cuda()
    M, N, K = 6, 64, 256
    t, w64 = _weights(N, K, 1, fmt)
    buf = torch.randn(M * N + 1, generator=_gen(1), device="cuda").half()
    dy = buf[1:].view(M, N)
    _dx_check(dy, w64, _backward(dy, t, fmt, K, path=tq.PATH_GENERIC), False)
    for path in (tq.PATH_AUTO, tq.PATH_PREFILL):
        _dx_check(dy, w64, _backward(dy, t, fmt, K, path=path), fmt != "ternary")


@pytest.mark.parametrize("fmt", ["w4", "w4z"])
@pytest.mark.parametrize("M,N,K", [(70, 101, 256), (300, 1003, 384), (1, 9, 128)])
def test_gradient_for_x_int4_odd_rows(fmt, M, N, K):
    need_cuda()
    t, w64 = _weights(N, K, M, fmt)
    dy = torch.randn(M, N, generator=_gen(1), device="cuda").half()
    rows = torch.full((M, (N + 7) // 8 * 8), float("nan"), dtype=torch.float16, device="cuda")
    _dx_check(dy, w64, _backward(dy, t, fmt, K, path=tq.PATH_PREFILL, rows=rows), True)
    with pytest.raises(ValueError, match="rows"):
        _backward(dy, t, fmt, K, rows=rows[:, :-1].contiguous())


def test_gradient_for_x_of_nothing():
    need_cuda()
    t, _ = _weights(16, 128, 1, "ternary")
    assert _backward(torch.zeros(0, 16, device="cuda").half(), t, "ternary", 128).shape == (0, 128)


@pytest.mark.parametrize("fmt", ["ternary", "w4z"])
def test_infinities_of_dy_stay_in_their_row(fmt):
    need_cuda()
    M, N, K = 140, 264, 256
    t, w64 = _weights(N, K, 4, fmt)
    dy = torch.randn(M, N, generator=_gen(K), device="cuda").half()
    clean = _backward(dy, t, fmt, K)
    dy[77, 130] = float("nan")
    out = _backward(dy, t, fmt, K)
    rows = [m for m in range(M) if m != 77]
    assert torch.equal(out[rows], clean[rows]) and torch.isnan(out[77]).all()


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt", ["ternary", "w4z"])
@pytest.mark.parametrize("graph", [False, True])
def test_training_step_of_adapters_beside_a_packed_projection(fmt, graph):
    """Projection, adapters with dropout, and all gradients, as a step uses them: against 64 bits, and captured and replayed."""
    need_cuda()
    M, L, K, N, r, p = 200, 3, 256, 384, 16, 0.2
    t, w64 = _weights(N, K, 6, fmt)
    g = _gen(17)
    x = torch.randn(M, K, generator=g, device="cuda").half()
    a = (torch.randn(L, r, K, generator=g, device="cuda") / 16).half()
    b = (0.1 * torch.randn(L, N, r, generator=g, device="cuda")).half()
    s = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    dy = (0.1 * torch.randn(M, N, generator=g, device="cuda")).half()
    ids = torch.randint(-1, L, (M, 1), generator=g, device="cuda").to(torch.int32)
    rng = torch.tensor([8, 21], dtype=torch.int64, device="cuda")
    v = torch.zeros(M, r, device="cuda")

    def step():
        offsets, order, _ = tq.tq_moe_sort(ids, L)
        y = tq.tq_gemm(x, t[0], t[1]) if fmt == "ternary" else tq.w4g_gemm_zp(x, t[0], t[1], t[2])
        out = tq.tq_lora(x, a, b, y, offsets, order=order, scaling=s, p=p, rng=rng, v=v)
        base = _backward(dy, t, fmt, K)
        dx, da, db = tq.tq_lora_backward(dy, x, a, b, v, base, offsets, order=order, scaling=s, p=p, rng=rng, dx=base)
        return out, dx, da, db

    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=st):
            got = step()
        for _ in range(2):
            for o in got:
                o.zero_()
            cg.replay()
            torch.cuda.synchronize()
    else:
        got = step()
    X, A, Bm, D, S, ID = O.f64(x), O.f64(a), O.f64(b), O.f64(dy), O.f64(s), ids.view(-1).cpu().numpy()
    m = O.kept(M, K, p, 8, 21) * O.factor(p)
    out, dx, da, db = X @ w64.T, D @ w64, np.zeros(a.shape), np.zeros(b.shape)
    for l in range(L):
        i = np.nonzero(ID == l)[0]
        out[i] += S[l] * ((X * m)[i] @ A[l].T @ Bm[l].T)
        dv = S[l] * (D[i] @ Bm[l])
        dx[i] += m[i] * (dv @ A[l])
        da[l] = dv.T @ (X * m)[i]
        db[l] = S[l] * D[i].T @ ((X * m)[i] @ A[l].T)
    # the projection's rows and gradient are fp16 in between: two half steps each (2^-11), each sum's fp32 errors far below; weights
    # of the INT4 tensor-core path rounded once; against the 2-norm of each result, with a factor of two for what sums share
    for name, g_, w in zip(("out", "dx", "da", "db"), got, (out, dx, da, db)):
        err = np.linalg.norm(O.f64(g_) - w) / np.linalg.norm(w)
        assert err < 2 * 3 * 2.0 ** -11, (name, err)
