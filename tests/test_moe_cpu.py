"""Host-side checks of the mixture-of-experts calls (include/tq_moe.h) that need no GPU: exports,
argument errors before anything is launched, the dispatch rule, refusal of host tensors."""
import ctypes

import pytest
import torch

import bit_weight_only_tq_b200 as tq
from bit_weight_only_tq_b200 import moe

P = ctypes.c_void_p(4096)
Q = ctypes.c_void_p(4098)


def test_library_exports_every_moe_header_function():
    names = moe.moe_header_functions()
    assert sorted(moe._SIGS) == names
    for n in names:
        assert hasattr(tq.lib, n), n
    for n in moe.__all__:
        assert hasattr(tq, n) and n in tq.__all__


def test_route_argument_errors():
    f = tq.lib.tq_moe_route
    assert f(P, 7, P, P, 4, 8, 2, 1, None) == -4
    for T, E, k in ((-1, 8, 2), (4, 0, 1), (4, 1025, 2), (4, 8, 0), (4, 8, 9), (4, 64, 33), (2 ** 31, 8, 1)):
        assert f(P, 0, P, P, T, E, k, 1, None) == -2, (T, E, k)
    assert f(None, 0, P, P, 4, 8, 2, 1, None) == -1
    assert f(P, 0, None, P, 4, 8, 2, 1, None) == -1
    assert f(None, 0, None, None, 0, 8, 2, 1, None) == 0            # no token: nothing to do
    b = tq.lib.tq_moe_route_backward
    assert b(P, P, 3, P, P, P, 4, 8, 2, 1, None) == -4
    assert b(P, P, 2, P, P, P, 4, 8, 9, 1, None) == -2
    assert b(P, P, 2, P, P, None, 4, 8, 2, 1, None) == -1
    assert b(None, None, 2, None, None, None, 0, 8, 2, 1, None) == 0


def test_sort_argument_errors():
    f = tq.lib.tq_moe_sort
    for R, E in ((-1, 8), (2 ** 31, 8), (16, 0), (16, 1025)):
        assert f(P, P, P, P, R, E, None) == -2
    assert f(None, P, P, P, 16, 8, None) == -1
    assert f(P, None, P, P, 16, 8, None) == -1
    assert f(P, P, P, None, 16, 8, None) == -1


def test_row_argument_errors():
    g = tq.lib.tq_moe_gather
    assert g(P, 9, P, P, P, 4, 8, 2, 8, None) == -4
    for T, H, k, E in ((-1, 8, 2, 8), (4, 0, 2, 8), (4, 2 ** 25, 2, 8), (4, 8, 33, 8), (4, 8, 2, 0), (2 ** 30, 8, 2, 8)):
        assert g(P, 1, P, P, P, T, H, k, E, None) == -2
    assert g(P, 1, None, P, P, 4, 8, 2, 8, None) == -1
    assert g(None, 1, None, None, None, 0, 8, 2, 8, None) == 0
    c = tq.lib.tq_moe_combine
    assert c(P, 9, P, P, P, 4, 8, 8, 2, None) == -4
    assert c(P, 1, P, P, P, 4, -1, 8, 2, None) == -2
    assert c(P, 1, P, P, P, 4, 8, 0, 2, None) == -2
    assert c(None, 1, P, P, P, 4, 8, 8, 2, None) == -1
    assert c(P, 1, P, None, None, 4, 8, 8, 2, None) == -1
    assert c(None, 1, None, None, None, 0, 0, 8, 2, None) == 0
    b = tq.lib.tq_moe_combine_backward
    assert b(P, P, 9, P, P, P, P, 4, 8, 8, 2, None) == -4
    assert b(P, P, 1, P, P, P, P, 4, 8, 8, 0, None) == -2
    assert b(P, P, 1, P, None, P, P, 4, 8, 8, 2, None) == -1        # dy needs the weights
    assert b(P, None, 1, P, P, P, P, 4, 8, 8, 2, None) == -1        # dweights needs y
    assert b(None, P, 1, P, P, P, P, 4, 8, 8, 2, None) == -1
    assert b(P, P, 1, P, P, None, None, 4, 8, 8, 2, None) == 0      # nothing wanted


def test_experts_argument_errors():
    t, w = tq.lib.tq_gemm_experts, tq.lib.w4g_gemm_experts

    def tern(x=P, p=P, s=P, y=P, off=P, X=4, R=8, E=4, N=16, K=64, k=2, path=0, order=None, rows=None):
        return t(x, p, s, None, y, off, order, rows, X, R, E, N, K, k, path, None)

    def int4(K=128, **kw):
        return w(P, P, P, None, None, P, P, None, None, kw.get("X", 4), kw.get("R", 8), 4, 16, K, 2, kw.get("path", 0), None)

    for bad in (dict(X=-1), dict(R=-1), dict(R=2 ** 31), dict(E=0), dict(E=1025), dict(N=-1), dict(N=2 ** 30), dict(K=0),
                dict(K=2 ** 28 + 1), dict(k=0)):
        assert tern(**bad) == -2, bad
    assert int4(K=192) == -2
    assert tern(path=4) == -8 and tern(path=-1) == -8
    assert tern(x=None) == -1 and tern(p=None) == -1 and tern(s=None) == -1 and tern(y=None) == -1 and tern(off=None) == -1
    assert tern(R=0, x=None, y=None) == 0 and tern(N=0, p=None) == 0
    for path in (tq.PATH_DECODE, tq.PATH_PREFILL):
        assert tern(K=100, path=path) == -8                         # K % 64
        assert tern(x=Q, path=path) == -3 and tern(p=Q, path=path) == -3 and tern(y=Q, path=path) == -3


    # PREFILL through `order` copies the rows first: it needs the scratch, aligned
    assert tern(path=tq.PATH_PREFILL, order=P) == -1
    assert tern(path=tq.PATH_PREFILL, order=P, rows=Q) == -3


def test_experts_path_rule():
    T, W = tq.FMT_TERNARY, tq.FMT_W4G128
    assert tq.tq_experts_path(T, 8, 4, 64, 100) == tq.PATH_GENERIC
    assert tq.tq_experts_path(T, 8, 4, 64, 64, aligned=False) == tq.PATH_GENERIC
    assert tq.tq_experts_path(W, 8, 4, 64, 192) == -2
    for f in (T, W):
        for R, E in ((1, 1), (8, 1), (8, 8), (64, 8), (512, 64)):
            assert tq.tq_experts_path(f, R, E, 1000, 1024) == tq.PATH_DECODE
        for R, E in ((9, 1), (65, 8), (513, 64), (16384, 8)):
            assert tq.tq_experts_path(f, R, E, 1000, 1024) == tq.PATH_PREFILL
    assert tq.tq_experts_path(5, 8, 4, 64, 128) == -8
    assert tq.tq_experts_path(T, -1, 4, 64, 128) == -2


def test_host_tensors_and_wrong_types_are_refused():
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.tq_moe_route(x, 2)
    with pytest.raises(ValueError):
        tq.tq_moe_route(torch.zeros(4, 8, dtype=torch.int64), 2)
    with pytest.raises(ValueError):
        tq.tq_moe_sort(ids, 4)
    with pytest.raises(ValueError):
        tq.tq_moe_gather(x, ids.view(-1), ids.view(-1), 2)
    with pytest.raises(ValueError):
        tq.tq_moe_combine(x, ids)
    with pytest.raises(ValueError):
        tq.tq_gemm_experts(x.half(), torch.zeros(2, 4, 2, dtype=torch.uint8), torch.zeros(2, 4).half(), ids.view(-1))


def test_an_order_of_more_slots_than_the_tokens_have_is_refused():
    """top_k left out: the slots past the last token would all read as zeros."""
    x, order = torch.zeros(4, 64).half(), torch.zeros(8, dtype=torch.int32)
    for top_k, X in ((1, 4), (3, 2), (2, 0)):
        with pytest.raises(ValueError, match="8 slots"):
            moe._experts(tq.FMT_TERNARY, x[:X], (), order, order, top_k, None, None, None, 7, 16, tq.PATH_AUTO, None, 0)
    for top_k, X in ((2, 4), (8, 1), (3, 4)):                        # refused for being on the host, and no earlier
        with pytest.raises(ValueError, match="CUDA tensor"):
            moe._experts(tq.FMT_TERNARY, x[:X], (), order, order, top_k, None, None, None, 7, 16, tq.PATH_AUTO, None, 0)
