"""What training and serving low-rank adapters beside packed projections computes, in plain torch, with the calls that
replace it.

A projection with packed low-bit weights stays frozen and is shared by all requests; each adapter l adds
s_l (x A_l^T) B_l^T to the rows that are its own.  Four operators:

  lora             out = base + s_l (x A_l^T) B_l^T, every row with its own adapter or none (serving)
  lora_train       the same with dropout on the adapters' input, then the gradients of x, A and B
  dropout          dropout from a counter-based generator (no mask is stored; its gradient is the same call)
  w4_backward      the gradient for x of a product with INT4 weights, dx = dy What (group 128 along K)
  ternary_backward the same with ternary weights (one fp16 scale per output row)

A case is a dict of plain values.  `own` selects between the plain form (False) and the package's calls (True); both
take the same state.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_GROUP = 128


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one request's decode step with its adapter, beside a square projection
        dict(name="lora_token", op="lora", rows=1, adapters=8, width=4096, out=4096, rank=16, type="f16", away=0.0,
             runs=False),
        # a decode batch of many requests: most rows have an adapter of their own, some have none
        dict(name="lora_batch", op="lora", rows=61, adapters=32, width=4096, out=14336, rank=64, type="f16", away=0.1,
             runs=False),
        # a larger decode batch of short-rank adapters, down to a narrow projection
        dict(name="lora_many", op="lora", rows=250, adapters=100, width=3584, out=512, rank=8, type="bf16", away=0.0,
             runs=False),
        # prompts of several requests together, each a run of rows with one adapter
        dict(name="lora_prompts", op="lora", rows=4096, adapters=6, width=3584, out=18944, rank=32, type="bf16",
             away=0.05, runs=True),
        # a training step of one adapter with dropout
        dict(name="train_one", op="lora_train", rows=8192, adapters=1, width=4096, out=4096, rank=64, type="bf16",
             away=0.0, runs=True, p=0.05),
        # a training step of three adapters at once, an odd number of tokens, no dropout, the widest input
        dict(name="train_three", op="lora_train", rows=3001, adapters=3, width=14336, out=4096, rank=16, type="f16",
             away=0.0, runs=True, p=0.0),
        # activations of a training step
        dict(name="dropout_step", op="dropout", rows=16384, width=4096, type="bf16", p=0.1),
        # a small matrix of odd sizes
        dict(name="dropout_small", op="dropout", rows=37, width=1001, type="f32", p=0.5),
        # a training step's gradient through the widest ternary projection
        dict(name="ternary_step", op="ternary_backward", rows=8192, width=4096, out=14336),
        # the same through a small batch of odd length
        dict(name="ternary_small", op="ternary_backward", rows=333, width=3584, out=3584),
        # a micro-batch through asymmetric INT4 weights
        dict(name="w4_step", op="w4_backward", rows=4096, width=14336, out=4096, zeros=True),
        # a short sequence through a narrow INT4 projection
        dict(name="w4_small", op="w4_backward", rows=61, width=4096, out=1024, zeros=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_train", "dropout", "w4_backward", "ternary_backward"])
    if op in ("lora", "lora_train"):
        train = op == "lora_train"
        # rows of whole 16-byte vectors mostly, any width now and then
        width, out = (_log(rng, 100, 8192) if rng.random() < 0.1 else 8 * _log(rng, 16, 1024) for _ in range(2))
        c = dict(op=op, rows=_log(rng, 64 if train else 1, 8192), adapters=_log(rng, 1, 8 if train else 64), width=width,
                 out=out, rank=rng.choice([4, 8, 16, 16, 32, 64, 128]), type=rng.choice(["f16", "bf16"]),
                 away=rng.choice([0.0, 0.0, 0.2]), runs=train or rng.random() < 0.5)
        if train:
            c["p"] = rng.choice([0.0, 0.05, 0.3])
        return c
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 16384), width=_log(rng, 60, 4096), type=rng.choice(["f32", "f16", "bf16"]),
                    p=rng.choice([0.05, 0.1, 0.5]))
    c = dict(op=op, rows=_log(rng, 8, 8192), width=128 * _log(rng, 2, 48), out=8 * _log(rng, 16, 1024))
    if op == "w4_backward":
        c["zeros"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------------------ inputs
def _rows(n, width, dtype, g):
    """Activations ~ N(0, 1), one row in a hundred scaled up (outlier tokens)."""
    x = torch.randn(n, width, generator=g, device="cuda")
    return (x * (1 + 19 * (torch.rand(n, 1, generator=g, device="cuda") < 0.01))).to(dtype)


def _adapter_ids(case, g):
    """The adapter of each row; -1 for rows without one.  runs: requests one after the other, ragged."""
    M, L = case["rows"], case["adapters"]
    if case["runs"]:
        cuts = torch.sort(torch.rand(max(L, 1) - 1, generator=g, device="cuda")).values * M
        ids = torch.searchsorted(cuts.contiguous(), torch.arange(M, device="cuda") + 0.5)
        ids = torch.randperm(L, generator=g, device="cuda")[ids]
        gone = torch.arange(M, device="cuda") >= M - int(case["away"] * M)
    else:
        ids = torch.randint(0, L, (M,), generator=g, device="cuda")
        gone = torch.rand(M, generator=g, device="cuda") < case["away"]
    return torch.where(gone, torch.full_like(ids, -1), ids).to(torch.int32)


def _w4_pack(w, zeros):
    """INT4, group 128 along K: words of 8 codes, fp16 scales, zero-points or None."""
    N, K = w.shape
    wg = w.view(N, K // _GROUP, _GROUP)
    if zeros:
        lo, hi = wg.amin(-1).clamp(max=0), wg.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).half()
        z = torch.clamp(torch.round(-lo / s.float()), 0, 15)
    else:
        s, z = (wg.abs().amax(-1) / 7).half(), None
    u = torch.round(wg / s.float()[..., None]) + (8 if z is None else z[..., None])
    u = u.clamp_(0, 15).to(torch.int32).view(N, K // 8, 8)
    shift = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    q = torch.bitwise_left_shift(u, shift).sum(-1, dtype=torch.int32)
    return q, s, None if z is None else z.to(torch.uint8)


def _ternary_pack(w):
    """Codes 0, 1, 2 for -1, 0, +1 (threshold 0.7 mean |w|), four per byte; one fp16 scale per row."""
    N, K = w.shape
    a = w.abs()
    keep = a > 0.7 * a.mean(-1, keepdim=True)
    scale = ((a * keep).sum(-1) / keep.sum(-1).clamp(min=1)).half()
    c = (1 + torch.sign(w) * keep).to(torch.uint8).view(N, K // 4, 4)
    return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, s = case, dict(case)
    M, K = c["rows"], c["width"]
    if c["op"] == "dropout":
        s["x"] = _rows(M, K, _TYPES[c["type"]], g)
        s["rng"] = torch.tensor([int(seed) * 7919 + 13, 3], dtype=torch.int64, device="cuda")
        return s
    N = c["out"]
    if c["op"] in ("lora", "lora_train"):
        dtype, L, r = _TYPES[c["type"]], c["adapters"], c["rank"]
        s["x"] = _rows(M, K, dtype, g)
        s["a"] = (torch.randn(L, r, K, generator=g, device="cuda") / math.sqrt(K)).to(dtype)
        s["b"] = (0.1 * torch.randn(L, N, r, generator=g, device="cuda")).to(dtype)
        s["scaling"] = 2.0 * torch.rand(L, generator=g, device="cuda") + 0.5
        s["base"] = torch.randn(M, N, generator=g, device="cuda").to(dtype)  # the shared projection's rows
        ids = _adapter_ids(c, g)
        # the plan of a step, which all of its layers share: rows sorted by adapter, rows without one last
        key = torch.where(ids < 0, torch.full_like(ids, L), ids).long()
        order = torch.argsort(key, stable=True)
        offsets = torch.searchsorted(key[order].contiguous(), torch.arange(L + 1, device="cuda"))
        s["order"], s["offsets"] = order.to(torch.int32), offsets.to(torch.int32)
        s["bounds"] = offsets.tolist()  # the same numbers on the host, for the plain form's slices
        if c["op"] == "lora_train":
            s["rng"] = torch.tensor([int(seed) * 104729 + 5, 11], dtype=torch.int64, device="cuda")
            s["dy"] = (0.01 * torch.randn(M, N, generator=g, device="cuda")).to(dtype)
            s["base_dx"] = (0.01 * torch.randn(M, K, generator=g, device="cuda")).to(dtype)  # the projection's part
        return s
    w = 0.02 * torch.randn(N, K, generator=g, device="cuda")
    if c["op"] == "w4_backward":
        s["q"], s["s"], s["z"] = _w4_pack(w, c["zeros"])
    else:
        s["q"], s["s"] = _ternary_pack(w)
    s["dy"] = (0.01 * torch.randn(M, N, generator=g, device="cuda")).half()
    return s


# ----------------------------------------------------------------------------------------- plain forms
def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _philox_round(c, k):
    """One round of Philox4x32 (Salmon et al., Parallel random numbers: as easy as 1, 2, 3, 2011) on 32-bit words held
    in 64-bit integers; a product's high word comes out right because 64-bit products wrap."""
    low = 0xFFFFFFFF
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return (((p1 >> 32) & low) ^ c[1] ^ k[0], p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k[1], p0 & low)


def _kept(rows, width, p, rng):
    """The truth value of each element of a [rows, width] matrix: element e of the group of eight consecutive columns
    with number i = row ceil(width / 8) + column / 8 takes 16 bits of the block with counter (i, offset)."""
    low = 0xFFFFFFFF
    groups = -(-width // 8)
    i = torch.arange(rows * groups, device=rng.device, dtype=torch.int64)
    k0, k1, o0, o1 = rng[0] & low, (rng[0] >> 32) & low, rng[1] & low, (rng[1] >> 32) & low
    c = (i & low, i >> 32, o0.expand_as(i), o1.expand_as(i))
    c = _philox_round(c, (k0, k1))
    c = _philox_round(c, ((k0 + 1 * 0x9E3779B9) & low, (k1 + 1 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 2 * 0x9E3779B9) & low, (k1 + 2 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 3 * 0x9E3779B9) & low, (k1 + 3 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 4 * 0x9E3779B9) & low, (k1 + 4 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 5 * 0x9E3779B9) & low, (k1 + 5 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 6 * 0x9E3779B9) & low, (k1 + 6 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 7 * 0x9E3779B9) & low, (k1 + 7 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 8 * 0x9E3779B9) & low, (k1 + 8 * 0xBB67AE85) & low))
    c = _philox_round(c, ((k0 + 9 * 0x9E3779B9) & low, (k1 + 9 * 0xBB67AE85) & low))
    t = _threshold(p)
    word = torch.stack(c, -1)
    half = torch.stack([word & 0xFFFF, word >> 16], -1) >= t
    return half.reshape(rows, groups * 8)[:, :width]


def _scale(p):
    return 65536.0 / (65536 - _threshold(p))


def _plain_lora(s):
    b, order = s["bounds"], s["order"].long()
    x = s["x"].float()
    if s.get("p"):
        keep = _kept(s["rows"], s["width"], s["p"], s["rng"])
        x = x * keep * _scale(s["p"])
    out = s["base"].float()
    some = [l for l in range(s["adapters"]) if b[l + 1] > b[l]]
    at = [order[b[l]:b[l + 1]] for l in some]
    v = [x[i] @ s["a"][l].float().t() for l, i in zip(some, at)]
    if some:
        there = torch.cat(at)
        out[there] += torch.cat([(h @ s["b"][l].float().t()) * s["scaling"][l] for l, h in zip(some, v)])
    out = out.to(s["base"].dtype)
    if s["op"] == "lora":
        return out
    dy, dx = s["dy"].float(), torch.zeros_like(x)
    da = torch.zeros(s["a"].shape, device=x.device)
    db = torch.zeros(s["b"].shape, device=x.device)
    if some:
        dv = [(dy[i] @ s["b"][l].float()) * s["scaling"][l] for l, i in zip(some, at)]
        dx[there] = torch.cat([d @ s["a"][l].float() for l, d in zip(some, dv)])
        da[some] = torch.stack([d.t() @ x[i] for d, i in zip(dv, at)])
        db[some] = torch.stack([(dy[i].t() @ h) * s["scaling"][l] for l, i, h in zip(some, at, v)])
    if s["p"]:
        dx = dx * keep * _scale(s["p"])
    return out, (s["base_dx"].float() + dx).to(out.dtype), da.to(out.dtype), db.to(out.dtype)


def _w4_values(q, s, z, to):
    """The weights that the words stand for."""
    u = torch.bitwise_and(torch.bitwise_right_shift(q[..., None], torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)), 15)
    u = u.reshape(s.shape[0], s.shape[1], _GROUP).to(to)
    return ((u - (8 if z is None else z.to(to)[..., None])) * s.to(to)[..., None]).reshape(s.shape[0], -1)


def _ternary_values(q, s, to):
    c = torch.stack([q & 3, (q >> 2) & 3, (q >> 4) & 3, q >> 6], -1).reshape(q.shape[0], -1)
    return (c.to(to) - 1) * s.to(to)[:, None]


# -------------------------------------------------------------------------------------- the package's calls
def _own(s):
    import bit_weight_only_tq_b200 as tq

    op = s["op"]
    if op == "dropout":
        return tq.tq_dropout(s["x"], s["p"], s["rng"])
    if op == "w4_backward":
        return tq.w4g_gemm_backward(s["dy"], s["q"], s["s"], zeros=s["z"])
    if op == "ternary_backward":
        return tq.tq_gemm_backward(s["dy"], s["q"], s["s"])
    if op == "lora":
        return tq.tq_lora(s["x"], s["a"], s["b"], s["base"], s["offsets"], order=s["order"], scaling=s["scaling"])
    # the adapters' inner rows are kept from the forward pass for the backward one
    v = torch.empty(s["rows"], s["rank"], dtype=torch.float32, device="cuda")
    out = tq.tq_lora(s["x"], s["a"], s["b"], s["base"], s["offsets"], order=s["order"], scaling=s["scaling"], p=s["p"],
                     rng=s["rng"], v=v)
    dx, da, db = tq.tq_lora_backward(s["dy"], s["x"], s["a"], s["b"], v, s["base_dx"], s["offsets"], order=s["order"],
                                     scaling=s["scaling"], p=s["p"], rng=s["rng"])
    return out, dx, da, db


def run(state):
    if own:
        return _own(state)
    s = state
    if s["op"] == "dropout":
        keep = _kept(s["rows"], s["width"], s["p"], s["rng"])
        return torch.where(keep, s["x"].float() * _scale(s["p"]), 0.0).to(s["x"].dtype)
    if s["op"] == "w4_backward":
        return (s["dy"].float() @ _w4_values(s["q"], s["s"], s["z"], torch.float32)).half()
    if s["op"] == "ternary_backward":
        return (s["dy"].float() @ _ternary_values(s["q"], s["s"], torch.float32)).half()
    return _plain_lora(s)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    M, K = c["rows"], c["width"]
    if c["op"] == "dropout":
        return {"bytes": 2 * M * K * _SIZE[c["type"]], "flops": M * K}
    N = c["out"]
    if c["op"] == "w4_backward":
        n = N * K // 2 + N * (K // _GROUP) * (3 if c["zeros"] else 2)
        return {"bytes": n + 2 * M * (N + K), "flops": 2 * M * N * K}
    if c["op"] == "ternary_backward":
        return {"bytes": N * K // 4 + 2 * N + 2 * M * (N + K), "flops": 2 * M * N * K}
    e, r, L = _SIZE[c["type"]], c["rank"], c["adapters"]
    R = M - int(c["away"] * M)                                       # rows with an adapter, on average
    met = L if c["runs"] else L * (1.0 - (1.0 - 1.0 / L) ** R)       # adapters with rows, on average
    n = int(e * (R * K + 2 * M * N + met * r * (K + N)))             # x, base and out, the adapters met
    f = 2 * R * r * (K + N)
    if c["op"] == "lora_train":  # dy, base and gradient of x, both gradients of the weights; x and the adapters again
        n += int(e * (R * N + R * K + 2 * M * K + 2 * L * r * (K + N)))
        f *= 3
    return {"bytes": n, "flops": f}


# ------------------------------------------------------------------------------------------- 64 bits
def _kept64(rows, width, p, rng):
    """Philox4x32-10 in numpy's unsigned integers."""
    low = np.uint64(0xFFFFFFFF)
    seed, offset = (np.uint64(int(v) & 0xFFFFFFFFFFFFFFFF) for v in rng.tolist())
    groups = (width + 7) // 8
    i = np.arange(rows * groups, dtype=np.uint64)
    c = [i & low, i >> np.uint64(32), np.full_like(i, offset & low), np.full_like(i, offset >> np.uint64(32))]
    key = [int(seed) & 0xFFFFFFFF, int(seed) >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(key[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.empty((rows * groups, 8), dtype=np.uint16)
    for j in range(4):
        bits[:, 2 * j] = c[j] & np.uint64(0xFFFF)
        bits[:, 2 * j + 1] = c[j] >> np.uint64(16)
    keep = bits.reshape(rows, groups * 8)[:, :width] >= int(p * 65536 + 0.5)
    return torch.from_numpy(keep).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "dropout":
        keep = _kept64(c["rows"], c["width"], c["p"], s["rng"])
        return s["x"].double() / (1.0 - int(c["p"] * 65536 + 0.5) / 65536.0) * keep
    N, K = c["out"], c["width"]
    if c["op"] == "w4_backward":
        k = torch.arange(K, device="cuda")
        u = ((s["q"][:, k // 8].long() >> (4 * (k % 8))) & 15).double()
        z = 8.0 if s["z"] is None else s["z"].double()[:, k // _GROUP]
        return s["dy"].double() @ ((u - z) * s["s"].double()[:, k // _GROUP])
    if c["op"] == "ternary_backward":
        k = torch.arange(K, device="cuda")
        u = ((s["q"][:, k // 4].long() >> (2 * (k % 4))) & 3).double()
        return (s["dy"].double() * s["s"].double()) @ (u - 1.0)
    M, L = c["rows"], c["adapters"]
    row_of = s["order"].tolist()
    first = s["offsets"].tolist()
    y, x = s["base"].double(), s["x"].double()
    train = c["op"] == "lora_train"
    mask = None
    if train:
        mask = torch.ones(M, K, dtype=torch.float64, device="cuda")
        if c["p"]:
            mask = _kept64(M, K, c["p"], s["rng"]).double() / (1.0 - int(c["p"] * 65536 + 0.5) / 65536.0)
        x = x * mask
        dx, dy = s["base_dx"].double(), s["dy"].double()
        da, db = s["a"].double() * 0, s["b"].double() * 0
    for l in range(L):
        mine = torch.tensor(row_of[first[l]:first[l + 1]], dtype=torch.int64, device="cuda")
        if not len(mine):
            continue
        w = s["scaling"][l].double() * (s["b"][l].double() @ s["a"][l].double())  # [N, K]
        y.index_add_(0, mine, x[mine] @ w.t())
        if train:
            g = dy[mine].t() @ x[mine]                                            # gradient of w without its scaling
            da[l] = s["scaling"][l].double() * (s["b"][l].double().t() @ g)
            db[l] = s["scaling"][l].double() * (g @ s["a"][l].double().t())
            dx.index_add_(0, mine, (dy[mine] @ w) * mask[mine])
    return (y, dx, da, db) if train else y
