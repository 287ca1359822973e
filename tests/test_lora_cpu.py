"""Host-side checks of the adapters' calls (include/tq_lora.h) that need no GPU: exports, argument errors before anything is
launched, the dispatch rule, refusal of host tensors; the 64-bit forms against published values and differences."""
import ctypes

import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from bit_weight_only_tq_b200 import lora

P = ctypes.c_void_p(4096)
Q = ctypes.c_void_p(4098)


def test_library_exports_every_lora_header_function():
    assert sorted(lora._SIGS) == lora.lora_header_functions()
    for n in lora._SIGS:
        assert hasattr(tq.lib, n), n
    for n in lora.__all__:
        assert hasattr(tq, n) and n in tq.__all__


def _fwd(x=P, dtype=1, a=P, b=P, scaling=None, base=P, out=P, v=P, off=P, order=None, p=0.0, rng=None, M=4, L=2, N=64, K=64,
         rank=8, path=0):
    return tq.lib.tq_lora(x, dtype, a, b, scaling, base, out, v, off, order, p, rng, M, L, N, K, rank, path, None)


def _bwd(dy=P, x=P, dtype=1, a=P, b=P, scaling=None, v=P, ws=P, ws_bytes=1 << 30, base_dx=P, dx=P, da=P, db=P, off=P, order=None, p=0.0, rng=None,
         M=4, L=2, N=64, K=64, rank=8, path=0):
    return tq.lib.tq_lora_backward(dy, x, dtype, a, b, scaling, v, ws, ws_bytes, base_dx, dx, da, db, off, order, p, rng, M, L, N,
                                   K, rank, path, None)


@pytest.mark.parametrize("f", [_fwd, _bwd])
def test_adapter_argument_errors(f):
    assert f(dtype=0) == -4 and f(dtype=3) == -4                    # float32 rows, no dtype
    for bad in (dict(M=-1), dict(M=2 ** 31), dict(L=0), dict(L=1025), dict(N=-1), dict(N=2 ** 24 + 1), dict(K=0), dict(K=2 ** 24 + 1),
                dict(rank=0), dict(rank=129), dict(p=-0.1), dict(p=1.0), dict(p=0.999999), dict(p=float("nan"))):
        assert f(**bad) == -2, bad
    assert f(path=4) == -8 and f(path=-1) == -8
    assert f(off=None) == -1 and f(p=0.5) == -1                     # dropout without a generator's state


def test_forward_argument_errors():
    for name in ("x", "a", "b", "out"):
        assert _fwd(**{name: None}) == -1, name
    assert _fwd(M=0, x=None, out=None, off=None) == 0 and _fwd(N=0, out=None) == 0
    assert _fwd(v=None, path=tq.PATH_GENERIC) == -1 and _fwd(v=None, path=tq.PATH_PREFILL) == -1
    assert _fwd(K=63, path=tq.PATH_DECODE) == -8 and _fwd(N=62, path=tq.PATH_DECODE) == -8
    assert _fwd(M=65536, path=tq.PATH_DECODE) == -8 and _fwd(path=tq.PATH_DECODE, p=0.5, rng=P) == -8
    for name in ("x", "a", "b", "base", "out", "v"):
        assert _fwd(**{name: Q}, path=tq.PATH_DECODE) == -3, name
    assert _fwd(v=Q, path=tq.PATH_PREFILL) == -3


def test_backward_argument_errors():
    for name in ("dy", "x", "b", "ws", "v", "a"):
        assert _bwd(**{name: None}) == -1, name
    assert _bwd(dx=None, da=None, db=None, off=None) == 0           # nothing wanted
    assert _bwd(path=tq.PATH_DECODE) == -8
    assert _bwd(v=Q, path=tq.PATH_PREFILL) == -3 and _bwd(ws=Q) == -3
    need = tq.tq_lora_workspace_size(4, 2, 8)
    assert need >= 4 * 4 * 8 and _bwd(ws_bytes=need - 1) == -2
    for M, L, r in ((-1, 2, 8), (4, 0, 8), (4, 1025, 8), (4, 2, 0), (4, 2, 129), (2 ** 31, 2, 8)):
        assert tq.tq_lora_workspace_size(M, L, r) == 0


def test_path_rule():
    for M, L, N, K, r in ((1, 1, 4096, 4096, 16), (250, 1, 4096, 4096, 64), (61, 32, 14336, 4096, 64), (1024, 64, 4096, 4096, 16),
                          (190, 4, 512, 512, 128)):
        assert tq.tq_lora_path(M, L, N, K, r) == tq.PATH_DECODE
        assert tq.tq_lora_path(M, L, N, K, r, dropout=True) == tq.PATH_PREFILL
        assert tq.tq_lora_path(M, L, N, K, r, aligned=False) == tq.PATH_PREFILL
        assert tq.tq_lora_path(M, L, N + 1, K, r) == tq.PATH_PREFILL and tq.tq_lora_path(M, L, N, K + 4, r) == tq.PATH_PREFILL
    for M, L, r in ((1024, 1, 16), (512, 1, 64), (2048, 64, 64), (256, 64, 128), (100000, 1024, 1)):
        assert tq.tq_lora_path(M, L, 4096, 4096, r) == tq.PATH_PREFILL
    assert tq.tq_lora_path(0, 1, 64, 64, 8) == tq.PATH_GENERIC and tq.tq_lora_path(-1, 1, 64, 64, 8) == -2


def test_dropout_argument_errors():
    f = tq.lib.tq_dropout
    assert f(P, 3, P, 0.5, P, 4, 8, None) == -4
    for p, M, K in ((-0.1, 4, 8), (1.0, 4, 8), (0.5, -1, 8), (0.5, 2 ** 31, 8), (0.5, 4, -1), (0.5, 4, 2 ** 28 + 1)):
        assert f(P, 1, P, p, P, M, K, None) == -2
    assert f(None, 1, P, 0.5, P, 4, 8, None) == -1 and f(P, 1, None, 0.5, P, 4, 8, None) == -1
    assert f(P, 1, P, 0.5, None, 4, 8, None) == -1
    assert f(None, 1, None, 0.5, None, 0, 8, None) == 0 and f(None, 1, None, 0.5, None, 4, 0, None) == 0


def test_gemm_backward_argument_errors():
    def tern(dy=P, w=P, s=P, dx=P, rows=None, M=4, N=64, K=64, path=0):
        return tq.lib.tq_gemm_backward(dy, w, s, dx, rows, M, N, K, path, None)

    def int4(dy=P, w=P, s=P, z=None, dx=P, rows=None, M=4, N=64, K=128, path=0):
        return tq.lib.w4g_gemm_backward(dy, w, s, z, dx, rows, M, N, K, path, None)

    for f in (tern, int4):
        for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(M=2 ** 31 + 1), dict(N=2 ** 31 + 1), dict(K=2 ** 28 + 128)):
            assert f(**bad) == -2, bad
        for name in ("dy", "w", "s", "dx"):
            assert f(**{name: None}) == -1, name
        assert f(M=0, dy=None, dx=None) == 0
        assert f(path=4) == -8 and f(path=tq.PATH_DECODE) == -8
        assert f(N=60, path=tq.PATH_PREFILL) == -1 and f(dy=Q, path=tq.PATH_PREFILL) == -1      # no room for copies
        assert f(N=60, rows=Q, path=tq.PATH_PREFILL) == -3
        for name in ("w", "dx"):
            assert f(**{name: Q}, path=tq.PATH_PREFILL) == -3, name
    assert int4(K=192) == -2 and tern(K=100, path=tq.PATH_PREFILL) == -8


def test_host_tensors_wrong_types_and_shapes_are_refused():
    x, a, b = torch.zeros(4, 16).half(), torch.zeros(2, 8, 16).half(), torch.zeros(2, 24, 8).half()
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tq.tq_lora(x, a, b, None, off)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        tq.tq_lora(x.float(), a, b, None, off)
    with pytest.raises(ValueError, match="dims"):
        tq.tq_lora(x, a[0], b, None, off)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tq.tq_lora_backward(torch.zeros(4, 24).half(), x, a, b, torch.zeros(4, 8), None, off)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        tq.tq_dropout(x.double(), 0.5, off)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tq.tq_dropout(x, 0.5, off)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tq.tq_gemm_backward(x, torch.zeros(16, 4, dtype=torch.uint8), torch.zeros(16).half())
    with pytest.raises(ValueError, match="CUDA tensor"):
        tq.w4g_gemm_backward(x, torch.zeros(16, 16, dtype=torch.int32), torch.zeros(16, 1).half())
    with pytest.raises(ValueError, match="needs rng"):
        lora._rng(0.5, None, 0)


def test_philox_gives_the_published_values():
    """The known answers that the method's authors publish for ten rounds on four 32-bit words."""
    ff = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((ff, ff, ff, ff), (ff, ff), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in O.philox(counter, key)) == want


def test_formulas_against_differences():
    """The gradients that the tests check the kernels against are those of the forward form, by central differences."""
    rs = np.random.RandomState(3)
    M, L, K, N, r, p = 5, 2, 12, 6, 3, 0.4
    x, a, b, base = rs.randn(M, K), rs.randn(L, r, K), rs.randn(L, N, r), rs.randn(M, N)
    s, dy = rs.rand(L) + 0.5, rs.randn(M, N)
    keep, f = O.kept(M, K, p, 99, 7), O.factor(p)
    assert 0 < keep.sum() < keep.size
    segs = list(O.segments([1, 3, 4], torch.tensor([4, 0, 2, 1, 3]), M))

    def loss(x, a, b):
        return float((O.forward(x, a, b, base, s, segs, keep, f)[0] * dy).sum())

    dx, da, db = np.zeros_like(x), np.zeros_like(a), np.zeros_like(b)
    for l, rows, _ in segs:
        v, dv = (x * keep * f)[rows] @ a[l].T, s[l] * dy[rows] @ b[l]
        dx[rows] += keep[rows] * f * (dv @ a[l])
        da[l], db[l] = dv.T @ (x * keep * f)[rows], s[l] * dy[rows].T @ v
    for arg, grad in ((0, dx), (1, da), (2, db)):
        for i in np.ndindex(*grad.shape):
            vals = []
            for e in (1e-5, -1e-5):
                t = [x.copy(), a.copy(), b.copy()]
                t[arg][i] += e
                vals.append(loss(*t))
            assert abs((vals[0] - vals[1]) / 2e-5 - grad[i]) < 1e-6 * (1 + abs(grad[i]))
