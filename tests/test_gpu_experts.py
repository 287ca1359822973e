"""Experts' products (tq_gemm_experts, w4g_gemm_experts) against the fp64 oracle, per path.

Tolerance per element, S = sum |x w|: half an fp16 step of the result (2^-11 |y|, 2^-25 among the
subnormals); on the PREFILL path of INT4 each weight (u - z) s rounded to fp16 (2^-11 S); products
are exact in fp32 and summed in fp32: at most K / 8 + 64 roundings of the running sum along the
longest chain of any path (tensor-core steps of 16 products, splits, 32 lanes), each 2^-23 of at
most S (the tensor cores truncate).
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _bits16(t):
    return t.view(torch.int16)


def _weights(fmt, E, N, K, seed):
    w = I.weights(E * N, K, seed, device="cuda", outlier_frac=0.0 if fmt == "ternary" else 0.001)
    if fmt == "ternary":
        p, s = tq.tq_quantize_pack(w)
        return p.view(E, N, -1), s.view(E, N), None
    q, s, z, _ = tq.w4g_quantize_pack_ex(w, zero_point=fmt == "w4z")
    return q.view(E, N, -1), s.view(E, N, -1), None if z is None else z.view(E, N, -1)


def _what(fmt, ws, e, K):
    q, s, z = ws
    q, s = q[e].cpu().numpy(), bits(s[e])
    if fmt == "ternary":
        return O.tq_unpack(q, s, K)
    if fmt == "w4":
        return O.w4g_unpack(q, s)
    return O.w4z_unpack(q, s, z[e].cpu().numpy(), np.arange(K) // 128)


def _call(fmt, x, ws, offsets, **kw):
    if fmt == "ternary":
        return tq.tq_gemm_experts(x, ws[0], ws[1], offsets, **kw)
    return tq.w4g_gemm_experts(x, ws[0], ws[1], offsets, zeros=ws[2], **kw)


def _check(fmt, path, x, ws, bias, offsets, y, xrow, K, N, cols=None, most=48):
    """Every expert's rows (at most `most` of each, spread over them) against the oracle."""
    off = offsets.cpu().numpy()
    xn, yn = f16np(x).astype(np.float64), f16np(y)
    cols = np.arange(N) if cols is None else cols
    for e in range(len(off) - 1):
        rows = np.arange(off[e], off[e + 1])
        if rows.size == 0:
            continue
        rows = np.unique(rows[np.linspace(0, rows.size - 1, min(most, rows.size)).astype(int)])
        W = _what(fmt, ws, e, K)[cols]
        src = xrow[rows]
        xs = np.where((src >= 0)[:, None], xn[np.maximum(src, 0)], 0.0)
        ref = xs @ W.T
        S = np.abs(xs) @ np.abs(W).T
        if bias is not None:
            b = f16np(bias)[e][cols].astype(np.float64)
            ref, S = ref + b, S + np.abs(b)
        rel = (K / 8 + 64) * 2.0 ** -23 + (2.0 ** -11 if fmt != "ternary" and path in (tq.PATH_AUTO, tq.PATH_PREFILL) else 0)
        tol = 2.0 ** -11 * (1 + 2.0 ** -10) * np.abs(ref) + rel * S + 2.0 ** -25
        err = np.abs(yn[np.ix_(rows, cols)].astype(np.float64) - ref)
        assert np.all(err <= tol), (fmt, path, e, float((err - tol).max()), np.argwhere(err > tol)[:4])


def _problem(fmt, T, k, E, N, K, seed, spread, bias, away=0.0, ids=None):
    if ids is None:
        ids = torch.randint(0, int(E / (1 - away)), (T, k), generator=_gen(seed), device="cuda").int()
    offsets, order, pos = tq.tq_moe_sort(ids, E)
    x = I.activations(T, K, seed, device="cuda", outlier_row_frac=0.02)
    b = I.bias(E * N, seed, device="cuda").view(E, N) if bias else None
    token = (order // k).long()
    xrow = token.cpu().numpy() if spread else np.arange(T * k)
    return x if spread else x[token].contiguous(), offsets, order if spread else None, b, xrow


def _run(fmt, path, T, k, E, N, K, seed, spread=True, bias=False, away=0.0, ids=None, cols=None):
    x, offsets, order, b, xrow = _problem(fmt, T, k, E, N, K, seed, spread, bias, away, ids)
    ws = _weights(fmt, E, N, K, seed)
    y, buf = guarded_empty(T * k, N)
    _call(fmt, x, ws, offsets, order=order, top_k=k, bias=b, y=y, path=path)
    assert tq.tq_device_status() == 0
    check_canaries(buf, T * k, N)
    total = int(offsets[-1])
    assert (y.view(torch.int16)[total:] == 0x7E5A).all()      # rows behind the last expert's as they were
    _check(fmt, path, x, ws, b, offsets, y, xrow, K, N, cols)


# (T, k, E, N, K): one token, few, ragged; N below, at and past the tile sizes; K of one and many stages
SMALL = [(1, 1, 1, 1, 128), (1, 2, 4, 128, 128), (1, 8, 64, 300, 256), (3, 2, 5, 129, 640), (13, 4, 6, 257, 1152),
         (40, 2, 3, 96, 384), (150, 2, 4, 200, 512), (300, 1, 2, 130, 256)]


@pytest.mark.parametrize("T,k,E,N,K", SMALL)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("spread", [True, False])
def test_products(T, k, E, N, K, fmt, path, spread):
    need_cuda()
    _run(fmt, path, T, k, E, N, K, T * N + K, spread, bias=(T + k) % 2 == 1, away=0.3 if T % 3 == 0 else 0.0)


@pytest.mark.parametrize("K", [1, 63, 64, 100, 192, 1088])
@pytest.mark.parametrize("T", [2, 70])
def test_ternary_any_k(K, T):
    need_cuda()
    _run("ternary", tq.PATH_AUTO, T, 2, 3, 70, K, K + T, True, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", PATHS)
def test_uneven_rows(fmt, path):
    need_cuda()
    T, k, E = 331, 2, 9
    for name in ("all to one", "one expert empty in the middle", "none here", "last only"):
        ids = torch.randint(0, E, (T, k), generator=_gen(17), device="cuda").int()
        if name == "all to one":
            ids[:] = 4
        elif name == "one expert empty in the middle":
            ids[ids == 4] = 5
        elif name == "none here":
            ids[:] = E
        else:
            ids[:] = -1
            ids[7, 1] = E - 1
        _run(fmt, path, T, k, E, 136, 256, 23, True, ids=ids)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", PATHS)
def test_rows_out_of_range_read_as_zeros(fmt, path):
    need_cuda()
    T, k, E, N, K = 6, 2, 3, 64, 256
    x, offsets, order, b, xrow = _problem(fmt, T, k, E, N, K, 5, True, True)
    order = order.clone()
    order[3], order[7] = -40, 10 ** 6
    xrow = (order // k).cpu().numpy()
    xrow[[3, 7]] = -1
    ws = _weights(fmt, E, N, K, 5)
    y = _call(fmt, x, ws, offsets, order=order, top_k=k, bias=b, path=path)
    _check(fmt, path, x, ws, b, offsets, y, xrow, K, N)


def test_misaligned_takes_the_generic_path():
    need_cuda()
    x, offsets, order, b, xrow = _problem("w4", 9, 2, 3, 65, 256, 5, True, False)
    buf = torch.empty(x.numel() + 1, dtype=torch.float16, device="cuda")
    xm = buf[1:].view(x.shape)
    xm.copy_(x)
    ws = _weights("w4", 3, 65, 256, 5)
    y = _call("w4", xm, ws, offsets, order=order, top_k=2)
    _check("w4", tq.PATH_GENERIC, xm, ws, b, offsets, y, xrow, 256, 65)
    with pytest.raises(tq.TQError):
        _call("w4", xm, ws, offsets, order=order, top_k=2, path=tq.PATH_DECODE)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [3, 200])
def test_whole_layer_captured_and_on_another_stream(fmt, T):
    """route -> sort -> product -> second product -> combine, as one graph replayed on new inputs."""
    need_cuda()
    k, E, K, N = 2, 8, 256, 384
    w1, w2 = _weights(fmt, E, N, K, 1), _weights(fmt, E, K, 128 * 3, 2)
    x = I.activations(T, K, 3, device="cuda")
    logits = torch.randn(T, E, generator=_gen(4), device="cuda")

    def layer():
        wt, ids = tq.tq_moe_route(logits, k)
        offsets, order, pos = tq.tq_moe_sort(ids, E)
        h = torch.relu(_call(fmt, x, w1, offsets, order=order, top_k=k))
        y = _call(fmt, h, w2, offsets)
        return tq.tq_moe_combine(y, pos, wt), wt, ids

    layer()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, wt, ids = layer()
    x.copy_(I.activations(T, K, 5, device="cuda"))
    logits.copy_(torch.randn(T, E, generator=_gen(6), device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    first = out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)                            # the same bits on every run
    eager = layer()
    assert torch.equal(eager[0], out) and torch.equal(eager[2], ids)
    # and against 64 bits: h rounded to fp16 (2^-11 of each, S1 its sum of sizes), then the second product
    W1 = [_what(fmt, w1, e, K) for e in range(E)]
    W2 = [_what(fmt, w2, e, N) for e in range(E)]
    xn, idn, wn, on = f16np(x).astype(np.float64), ids.cpu().numpy(), wt.double().cpu().numpy(), f16np(out)
    for t in range(0, T, max(1, T // 8)):
        ref, tol = np.zeros(K), np.full(K, 2.0 ** -24)
        for j in range(k):
            A, B = W1[idn[t, j]], W2[idn[t, j]]
            h = np.maximum(A @ xn[t], 0)
            eh = 2.0 ** -11 * h + (2.0 ** -11 + (K / 8 + 64) * 2.0 ** -23) * (np.abs(A) @ np.abs(xn[t]))
            v, S = B @ h, np.abs(B) @ h
            ev = 2.0 ** -10 * np.abs(v) + (2.0 ** -11 + (N / 8 + 64) * 2.0 ** -23) * S + 1.01 * np.abs(B) @ eh
            ref, tol = ref + wn[t, j] * v, tol + 1.01 * wn[t, j] * ev
        tol += 2.0 ** -11 * np.abs(ref)
        assert np.all(np.abs(on[t].astype(np.float64) - ref) <= tol)


def test_refusals():
    need_cuda()
    x, offsets, order, b, _ = _problem("w4", 4, 2, 3, 64, 256, 5, True, True)
    q, s, _ = _weights("w4", 3, 64, 256, 5)
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x[:, :128].contiguous(), q, s, offsets, order=order, top_k=2)
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x, q, s, offsets[:-1], order=order, top_k=2)
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x, q, s[:, :, :1], offsets, order=order, top_k=2)
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x.float(), q, s, offsets, order=order, top_k=2)
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x, q, s, offsets, order=order, top_k=2, bias=b[:, :8])
    with pytest.raises(ValueError):
        tq.w4g_gemm_experts(x, q, s, offsets, order=order, top_k=2, y=torch.zeros(8, 63, device="cuda").half())
    with pytest.raises(tq.TQError):
        tq.w4g_gemm_experts(x, q, s, offsets, order=order, top_k=0)
    y = tq.w4g_gemm_experts(x, q, s, offsets, order=order[:0], top_k=2)      # no rows
    assert tuple(y.shape) == (0, 64)


# more items than CTAs, with numbers of stages that do not divide by the groups and rings of any path
@pytest.mark.parametrize("T,k,E,N,K", [(96, 2, 5, 7001, 384), (40, 3, 12, 4160, 640), (700, 4, 24, 2311, 896),
                                       (1500, 1, 4, 5000, 1152)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", [tq.PATH_DECODE, tq.PATH_PREFILL])
@pytest.mark.parametrize("spread", [True, False])
def test_many_items_per_cta(T, k, E, N, K, fmt, path, spread):
    need_cuda()
    cols = np.unique(np.concatenate([np.arange(0, N, 97), np.arange(N - 130, N)]))
    _run(fmt, path, T, k, E, N, K, T + N, spread, bias=k == 3, cols=cols)


@pytest.mark.parametrize("K", [64, 320, 448, 704])
def test_ternary_many_items_of_odd_stage_counts(K):
    need_cuda()
    for path in (tq.PATH_DECODE, tq.PATH_PREFILL):
        _run("ternary", path, 333, 2, 6, 4500, K, K, True, bias=True, cols=np.arange(0, 4500, 53))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("path", PATHS)
def test_every_negative_slot_reads_as_zeros(fmt, path):
    """-1 is no slot of token 0, whatever a division that truncates makes of it."""
    need_cuda()
    T, k, E, N, K = 9, 4, 3, 70, 256
    x, offsets, order, b, xrow = _problem(fmt, T, k, E, N, K, 6, True, True)
    order = order.clone()
    order[[0, 5, 6, 20]] = torch.tensor([-1, -3, -4, -2 ** 31], dtype=torch.int32, device="cuda")
    xrow[[0, 5, 6, 20]] = -1
    ws = _weights(fmt, E, N, K, 6)
    y = _call(fmt, x, ws, offsets, order=order, top_k=k, bias=b, path=path)
    _check(fmt, path, x, ws, b, offsets, y, xrow, K, N)


# many rows per expert, beside experts with none or a few: items of 256 weight rows and up to 128 rows of x.  N
# ending inside an item's first 128 rows, at its middle, inside its second half, odd; K of one stage and of many
@pytest.mark.parametrize("N,K", [(2056, 128), (2176, 384), (2311, 640), (2424, 896), (2304, 1152)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[0, 1, 33, 700, 257, 513, 256], [1500, 0, 0, 0, 0, 0, 3, 30], [255, 161, 225]])
def test_many_rows_per_expert(N, K, fmt, counts):
    need_cuda()
    ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(N))].view(-1, 1).cuda()
    cols = np.unique(np.concatenate([np.arange(0, N, 61), np.arange(N - 140, N)]))
    _run(fmt, tq.PATH_PREFILL, ids.shape[0], 1, len(counts), N, K, N + K, True, bias=K == 640, ids=ids, cols=cols)


@pytest.mark.parametrize("K", [64, 448, 704, 1344])
def test_ternary_many_rows_per_expert_of_half_stages(K):
    need_cuda()
    cols = np.arange(0, 4096, 61)
    _run("ternary", tq.PATH_PREFILL, 900, 2, 5, 4096, K, K, True, cols=cols)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K", [(2, 1024), (300, 1024), (900, 512)])
def test_wait_runs_out_then_recovers(T, K, fmt):
    """Activation loads switched off and a wait limit of about a millisecond: every wait of the product
    kernels runs out, the call reports it once, and the next one is as before."""
    need_cuda()
    k, E, N = 2, 4, 384 if T < 900 else 4096
    x, offsets, order, b, _ = _problem(fmt, T, k, E, N, K, 8, True, True)
    ws = _weights(fmt, E, N, K, 8)
    run = lambda: _call(fmt, x, ws, offsets, order=order, top_k=k, bias=b)
    ref = run()
    assert tq.tq_device_status() == 0
    assert tq.lib.tq_debug_set_wait_limit(2_000_000) == 0
    assert tq.lib.tq_debug_skip_activation_loads(1) == 0
    try:
        run()
        assert tq.tq_device_status() == -6
    finally:
        assert tq.lib.tq_debug_skip_activation_loads(0) == 0
        assert tq.lib.tq_debug_set_wait_limit(0) == 0
    assert tq.tq_device_status() == 0
    assert torch.equal(_bits16(ref), _bits16(run()))
    assert tq.tq_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_at_once(fmt):
    """Calls of both kernels on two streams, interleaved: no state is shared between them."""
    need_cuda()
    k, E, N, K = 2, 6, 2200, 1024
    cases = []
    for T in (3, 500):
        x, offsets, order, b, _ = _problem(fmt, T, k, E, N, K, T, True, True)
        ws = _weights(fmt, E, N, K, T)
        cases.append((lambda s, y=None, x=x, ws=ws, offsets=offsets, order=order, b=b:
                      _call(fmt, x, ws, offsets, order=order, top_k=k, bias=b, y=y, stream=s)))
    ref = [c(None) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[torch.empty_like(r) for r in ref for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(12):
        for j, s in enumerate(streams):
            c = (i + j) % 2
            cases[c](s, out[j][6 * c + i // 2])
    torch.cuda.synchronize()
    assert tq.tq_device_status() == 0
    for o in out:
        for i, y in enumerate(o):
            assert torch.equal(_bits16(y), _bits16(ref[i // 6]))


# few items: 64 weight rows each, in stages of twice the k.  N around multiples of 64 and 128; K that ends in the
# first half of such a stage, in its second half, and at either's end
@pytest.mark.parametrize("N", [1, 63, 64, 65, 127, 191, 4033])
@pytest.mark.parametrize("fmt,K", [("w4", 128), ("w4z", 384), ("w4", 640), ("w4z", 896), ("w4", 2176), ("ternary", 64),
                                   ("ternary", 512), ("ternary", 576), ("ternary", 1536), ("ternary", 1600),
                                   ("ternary", 4160)])
def test_few_items(N, fmt, K):
    need_cuda()
    cols = None if N < 1000 else np.unique(np.concatenate([np.arange(0, N, 53), np.arange(N - 70, N)]))
    _run(fmt, tq.PATH_DECODE, 2, 2, 3, N, K, N + K, True, bias=N % 2 == 1, cols=cols)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("E,N", [(1024, 96), (700, 257)])
def test_many_experts(E, N, fmt):
    """A token each for most experts, several for a few, none for the rest."""
    need_cuda()
    for path in (tq.PATH_DECODE, tq.PATH_PREFILL):
        _run(fmt, path, 300, 4, E, N, 256, E, True)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [512, 640])
def test_scales_and_zeros_of_least_alignment(path, fmt, K):
    """Scales, zero-points and bias may start at any element: only x, weights and y are 16-byte aligned."""
    need_cuda()
    T, k, E, N = 20, 2, 4, 333
    x, offsets, order, b, xrow = _problem(fmt, T, k, E, N, K, K, True, True)

    def shifted(t):
        return None if t is None else torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)

    ws = _weights(fmt, E, N, K, K)
    off = (ws[0], shifted(ws[1]), shifted(ws[2]))
    assert off[1].data_ptr() % 4 == 2 and (off[2] is None or off[2].data_ptr() % 2 == 1)
    y = _call(fmt, x, off, offsets, order=order, top_k=k, bias=shifted(b), path=path)
    assert tq.tq_device_status() == 0
    _check(fmt, path, x, ws, b, offsets, y, xrow, K, N)
