"""64-bit forms of the adapters' calls, dropout and the packed products' gradient for x, on the host, and the bounds that
the tests hold the kernels to.

Bounds (u = 2^-24, an fp32 rounding; h = half a step of the output type; q = what the two 16-bit parts of a number leave
out of it, 2^-22 of it in fp16 and 2^-16 in bf16):
  a sum of n products of 16-bit numbers, each exact in fp32, in any order, each addition off by at most one unit in the last
  place (2u; a tensor core may cut off instead of rounding): (2 n + 16) u times the sum of the magnitudes.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
SPLIT = {torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def philox(counter, key):
    """Philox4x32-10 on arrays: counter four and key two uint64 arrays of 32-bit words."""
    low = np.uint64(0xFFFFFFFF)
    c, k = [np.asarray(v, dtype=np.uint64) for v in counter], [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def factor(p):
    return 65536.0 / (65536 - threshold(p))


def kept(M, K, p, seed, offset):
    """The elements of [M, K] that dropout keeps."""
    return kept_rows(M, K, p, seed, offset, 0)


def kept_rows(M, K, p, seed, offset, first):
    """Rows first .. M - 1 of the same."""
    if threshold(p) == 0:
        return np.ones((M - first, K), dtype=bool)
    low = 0xFFFFFFFF
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    G = -(-K // 8)
    i = np.arange(first * G, M * G, dtype=np.uint64)
    w = philox([i & np.uint64(low), i >> np.uint64(32), np.full_like(i, offset & low), np.full_like(i, offset >> 32)],
               [seed & low, seed >> 32])
    e = np.stack([w[j // 2] >> np.uint64(16) if j % 2 else w[j // 2] & np.uint64(0xFFFF) for j in range(8)], -1)
    return (e >= threshold(p)).reshape(M - first, G * 8)[:, :K]


def segments(offsets, order, M):
    """(adapter, rows, sorted positions) of each adapter; rows outside [0, M) are left out."""
    o = f64(offsets).astype(np.int64) if torch.is_tensor(offsets) else np.asarray(offsets)
    rows = np.arange(M) if order is None else f64(order).astype(np.int64)
    for l in range(len(o) - 1):
        at = np.arange(o[l], o[l + 1])
        yield l, rows[at], at


def forward(x, a, b, base, scaling, segs, keep, f):
    """(out, v by row, bound sums): out [M, N], v [M, r], and for the bounds sum |x a| [M, r] and sum |v b| s [M, N]."""
    M, r, N = x.shape[0], a.shape[1], b.shape[1]
    out = np.zeros((M, N)) if base is None else base.copy()
    v, vs, mag, spread = np.zeros((M, r)), np.zeros((M, r)), np.zeros((M, N)), np.zeros((M, N))
    xd = x * keep * f
    for l, rows, _ in segs:
        if not len(rows):
            continue
        v[rows] = xd[rows] @ a[l].T
        vs[rows] = np.abs(xd[rows]) @ np.abs(a[l]).T
        out[rows] += scaling[l] * (v[rows] @ b[l].T)
        mag[rows] = abs(scaling[l]) * (np.abs(v[rows]) @ np.abs(b[l]).T)
        spread[rows] = abs(scaling[l]) * (vs[rows] @ np.abs(b[l]).T)
    return out, v, vs, mag, spread


def check(got, want, tol, label=""):
    got = f64(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, label
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (label, int(bad.sum()), got[bad][:4], want[bad][:4], np.broadcast_to(tol, want.shape)[bad][:4])


def ternary_values(packed, scale, K):
    """The weights [N, K] that ternary bytes stand for."""
    p = packed.cpu().numpy()
    c = np.stack([(p >> (2 * i)) & 3 for i in range(4)], -1).reshape(p.shape[0], -1)[:, :K]
    return (c.astype(np.float64) - 1) * f64(scale)[:, None]


def w4_values(q, s, z):
    """The weights [N, K] that INT4 words stand for."""
    w = q.cpu().numpy().view(np.uint32)
    u = np.stack([(w >> np.uint32(4 * i)) & np.uint32(15) for i in range(8)], -1).reshape(w.shape[0], -1).astype(np.float64)
    zz = 8.0 if z is None else np.repeat(f64(z), 128, 1)
    return (u - zz) * np.repeat(f64(s), 128, 1)
