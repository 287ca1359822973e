"""Router, sort and row exchange at the ends of what their header allows."""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
from gpu_util import gpu, need_cuda

pytestmark = gpu


def _sorted(ids, E):
    flat = ids.reshape(-1).cpu().numpy()
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    pos = np.empty(flat.size, np.int64)
    pos[order] = np.arange(flat.size)
    return np.searchsorted(key[order], np.arange(E + 1)), order, np.where(key < E, pos, -1)


def _same(got, ids, E):
    for a, b in zip(got, _sorted(ids, E)):
        assert np.array_equal(a.cpu().numpy().reshape(-1), b)


# From 8193 slots on the sort is one cluster of eight CTAs, and thread 0 of each reads the earlier ones' numbers
# of slots without an expert while the rest of its warp waits at the cluster's barrier.  8193 slots leave the last
# CTA's warps without any; E below, at and past the number of threads.
@pytest.mark.parametrize("R", [8192, 8193, 16385, 65537])
@pytest.mark.parametrize("E", [1, 7, 256, 1023, 1024])
def test_sort_of_a_cluster_with_slots_of_no_expert(R, E):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(R + E)
    ids = torch.randint(-E, 2 * E, (R, 1), generator=g, device="cuda").int()
    _same(tq.tq_moe_sort(ids, E), ids, E)


def test_sort_of_a_cluster_captured_and_back_to_back():
    """As a graph on new ids, and many launches in a row whose prologues overlap."""
    need_cuda()
    R, E, k = 40000, 60, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda: torch.randint(-20, 80, (R // k, k), generator=g, device="cuda").int()
    ids = new()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tq.tq_moe_sort(ids, E)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = tq.tq_moe_sort(ids, E)
    for _ in range(3):
        ids.copy_(new())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _same(got, ids, E)
    many = [new() for _ in range(20)]
    outs = [tq.tq_moe_sort(i, E) for i in many]
    for i, o in zip(many, outs):
        _same(o, i, E)
