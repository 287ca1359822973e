"""Adapters' calls at the edges of what they allow: operands of different alignment in one call, bounded waits that run out,
non-finite numbers in the gradients, plans with foreign rows, long sums.  The bounds are in lora_util.py."""
import numpy as np
import pytest
import torch

import bit_weight_only_tq_b200 as tq
import lora_util as O
from gpu_util import gpu, need_cuda
from test_gpu_lora import _backward64, _case, _forward64, _gen, _shifted

pytestmark = gpu
U, HALF, TINY, SPLIT = O.U, O.HALF, O.TINY, O.SPLIT
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
