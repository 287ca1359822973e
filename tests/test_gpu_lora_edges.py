"""The adapters' calls and the products' gradient for x at the edges of what they allow: operands of different alignment in one
call, bounded waits that run out, non-finite numbers.  The bounds are in lora_util.py."""
import contextlib

import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from gpu_util import gpu, need_cuda
from test_gpu_lora import _backward64, _case, _gen, _shifted
from test_gpu_lora_more import _backward, _weights

pytestmark = gpu
H, B = torch.float16, torch.bfloat16
ANY, TC, FEW = tq.PATH_GENERIC, tq.PATH_PREFILL, tq.PATH_DECODE


# ------------------------------------------------------------------------------------------ alignment
@pytest.mark.parametrize("moved", ["x", "dy", "x dy", "a", "b", "x a", "dy b", "base", "out"])
@pytest.mark.parametrize("M,L,K,N,r", [(150, 3, 136, 264, 24),      # a rank padded to 32: copies that are all zeros
                                       (77, 2, 72, 200, 100),       # columns and rows that end inside a stage
                                       (3, 2, 8, 16, 8)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_some_operands_misaligned(moved, M, L, K, N, r, p):
    """Each tensor is copied by its own alignment: two bytes past a 16-byte boundary beside aligned ones, the same results."""
    need_cuda()
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, M + r)
    dy, base_dx = base * 0.1, x * 0.1
    rng = torch.tensor([3, 5], dtype=torch.int64, device="cuda")
    kw = dict(order=order, scaling=s, p=p, rng=rng, path=TC)

    def step(x, a, b, base, dy, base_dx, out, dx):
        v = torch.zeros(M, r, device="cuda")
        tq.tq_lora(x, a, b, base, offsets, v=v, out=out, **kw)
        return (out, v, *tq.tq_lora_backward(dy, x, a, b, v, base_dx, offsets, dx=dx, **kw))

    want = step(x, a, b, base, dy, base_dx, torch.empty_like(base), torch.empty_like(x))
    m = moved.split()
    to = lambda name, t: _shifted(t) if name in m else t
    got = step(to("x", x), to("a", a), to("b", b), to("base", base), to("dy", dy), to("base", base_dx),
               to("out", torch.empty_like(base)), to("out", torch.empty_like(x)))
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert tq.tq_device_status() == 0


# ------------------------------------------------------------------------------------------ waits
@contextlib.contextmanager
def _waits_run_out():
    """The failure-path hooks: the adapters' kernels issue no products (few rows: no block of B is requested; the products'
    gradient: no tile of dy is), so that every wait that depends on them gives up, after about a millisecond each.  No copy is
    left in flight."""
    assert tq.lib.tq_debug_set_wait_limit(2_000_000) == 0
    assert tq.lib.tq_debug_skip_activation_loads(1) == 0
    try:
        yield
    finally:
        assert tq.lib.tq_debug_skip_activation_loads(0) == 0
        assert tq.lib.tq_debug_set_wait_limit(0) == 0


def _runs_out_then_recovers(run):
    ref = [t.clone() for t in run()]
    assert tq.tq_device_status() == 0
    with _waits_run_out():
        run()
        assert tq.tq_device_status() == -6
    assert tq.tq_device_status() == 0
    assert all(torch.equal(g, w) for g, w in zip(run(), ref))
    assert tq.tq_device_status() == 0


# tiles of several sets of row indices (wgrad) and of several runs per CTA (expand); clusters of one and of several CTAs
@pytest.mark.parametrize("M,L,K,N,r", [(40, 2, 4096, 512, 16), (5000, 3, 128, 384, 64), (3000, 1, 1000, 8200, 128),
                                       (20000, 5, 1288, 264, 8)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_waits_of_the_adapters_kernels_run_out(M, L, K, N, r, p):
    """Warps whose waits ran out still come to every barrier: the call ends, says so once, and the next one is as before."""
    need_cuda()
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, M)
    dy = 0.1 * base
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    v = torch.zeros(M, r, device="cuda")
    kw = dict(order=order, scaling=s, p=p, rng=rng, path=TC)

    def forward():
        return (tq.tq_lora(x, a, b, base, offsets, v=v, **kw), v)

    def backward():
        return tq.tq_lora_backward(dy, x, a, b, w, None, offsets, **kw)

    _runs_out_then_recovers(forward)
    w = v.clone()
    _runs_out_then_recovers(backward)


@pytest.mark.parametrize("M,L,K,N,r", [(1, 2, 512, 4096, 16), (24, 5, 256, 8200, 64), (3, 1, 64, 8, 128)])
def test_waits_of_the_kernel_for_few_rows_run_out(M, L, K, N, r):
    need_cuda()
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, H, M, "one")
    _runs_out_then_recovers(lambda: (tq.tq_lora(x, a, b, base, offsets, order=order, scaling=s, path=FEW),))


@pytest.mark.parametrize("fmt", ["ternary", "w4z"])
@pytest.mark.parametrize("M,N,K", [(200, 1024, 384), (64, 4096, 256), (9, 72, 128), (2816, 1024, 1792)])
def test_waits_of_the_gradient_for_x_run_out(fmt, M, N, K):
    need_cuda()
    w, _ = _weights(N, K, 3, fmt)
    dy = torch.randn(M, N, generator=_gen(5), device="cuda").half()
    _runs_out_then_recovers(lambda: (_backward(dy, w, fmt, K, path=TC),))


@pytest.mark.parametrize("M,K,N,p", [(128, 1 << 22, 4096, 0.0), (1 << 22, 128, 64, 0.25)])
def test_waits_do_not_count_the_kernels_ahead(M, K, N, p):
    """Kernels of a call start before the ones ahead of them end: the limit of their waits (here 0.2 ms) is for their own
    stages, however long the others take (here, with eight CTAs at work, more than a millisecond)."""
    need_cuda()
    r = 1
    x = torch.zeros(M, K, dtype=H, device="cuda")
    x[:, :128] = torch.randn(M, 128, generator=_gen(1), device="cuda").half()
    a, b = torch.randn(1, r, K, generator=_gen(2), device="cuda").half(), torch.randn(1, N, r, generator=_gen(3), device="cuda").half()
    dy = torch.randn(M, N, generator=_gen(4), device="cuda").half() * 0.01
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    v = torch.zeros(M, r, device="cuda")

    def run():
        out = tq.tq_lora(x, a, b, None, offsets, p=p, rng=rng, v=v, path=TC)
        return (out, *tq.tq_lora_backward(dy, x, a, b, v, None, offsets, p=p, rng=rng, need_dx=False, path=TC)[1:])

    want = run()
    assert tq.tq_device_status() == 0
    assert tq.lib.tq_debug_set_wait_limit(400_000) == 0
    try:
        got = run()
        assert tq.tq_device_status() == 0
    finally:
        assert tq.lib.tq_debug_set_wait_limit(0) == 0
    assert all(torch.equal(g, w) for g, w in zip(got, want))


# ------------------------------------------------------------------------------------------ non-finite numbers
@pytest.mark.parametrize("path", [ANY, TC])
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("xs,as_,ds,bs", [(14, 3, -9, -8),       # v about 1e5
                                          (-9, 0, 7, 11),        # dv about 4e5
                                          (-13, -10, 6, 0),      # v about 1e-7
                                          (0, 0, -13, -8)])      # dv about 1e-6
def test_a_non_finite_inner_column_leaves_the_others_right(path, dtype, xs, as_, ds, bs):
    """An infinity in one row of A (one column of B) makes one inner column of v (of dv) non-finite in all of an adapter's rows.
    The other columns of dB (rows of dA), made of numbers that fp16 holds only with a power of two of their own, are as if it
    were not there."""
    need_cuda()
    M, L, K, N, r, bad = 200, 2, 128, 72, 8, 3
    x, a, b, base, s, offsets, order = _case(M, L, K, N, r, dtype, 44)
    to = lambda t, e: (t.float().clamp(-3, 3) * 2.0 ** e).to(dtype)
    x, a, b, dy = to(x, xs), to(a, as_), to(b, bs), to(base, ds)
    assert all(torch.isfinite(t).all() for t in (x, a, b, dy))
    rest = [j for j in range(r) if j != bad]
    v = torch.zeros(M, r, device="cuda")
    kw = dict(order=order, scaling=s, path=path)
    for hit in ("none", "a", "b"):
        a_, b_ = a.clone(), b.clone()
        if hit == "a":
            a_[0, bad, 5] = float("inf")
        if hit == "b":
            b_[0, 7, bad] = float("-inf")
        tq.tq_lora(x, a_, b_, None, offsets, v=v, **kw)
        _, da, db = tq.tq_lora_backward(dy, x, a_, b_, v, None, offsets, need_dx=False, **kw)
        if hit == "none":
            want = _backward64(dy, x, a, b, v, None, s, offsets, order, 0.0, 0, 0)
            assert all(np.abs(w).max() < 60000 for w, _ in want[1:])
        if hit == "a":
            assert not torch.isfinite(db[0, :, bad]).any()
        if hit == "b":
            assert not torch.isfinite(da[0, bad]).any()
        for l in range(L):
            ja, jb = rest if (hit, l) == ("b", 0) else range(r), rest if (hit, l) == ("a", 0) else range(r)
            for got, (w, t), at in ((da, want[1], (l, list(ja))), (db, want[2], (l, slice(None), list(jb)))):
                O.check(O.f64(got)[at], w[at], t[at], f"{hit}, adapter {l}")
