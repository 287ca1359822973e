"""What the mixture-of-experts operators compute, in plain torch, with the calls that replace it.

A mixture-of-experts layer with packed low-bit expert weights runs: router scores -> top-k experts
and their weights per token -> slots (token, choice) sorted by expert -> each expert's product with
its rows -> the rows brought back to their tokens, weighted and summed.  Six operators:

  route            softmax over the experts, top-k, optionally renormalised (and its gradient)
  dispatch         slots sorted by expert (offsets, order, positions) and the rows gathered
  dispatch_grad    the gradient of the gather: each token's rows summed
  combine          rows weighted and summed per token (and its gradients)
  w4_experts       rows of each expert times its INT4 weights (group 128 along K, fp16 scales)
  ternary_experts  rows of each expert times its ternary weights (one fp16 scale per output row)

A case is a dict of plain values.  `own` selects between the plain form (False) and the package's
calls (True); both take the same state.
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
        # one decode step of a small batch: router scores in fp32, weights renormalised
        dict(name="route_decode", op="route", tokens=16, experts=64, top_k=8, type="f32", renorm=True, grad=False),
        # a training step over many experts: probabilities kept as they are, scores in bf16
        dict(name="route_train", op="route", tokens=8192, experts=256, top_k=8, type="bf16", renorm=False, grad=True),
        # a decode step: a handful of tokens to the experts of one rank, some slots routed elsewhere
        dict(name="dispatch_decode", op="dispatch", tokens=13, experts=64, top_k=8, width=2048, type="f16", away=0.25),
        # a prefill chunk: every row copied top_k times
        dict(name="dispatch_prefill", op="dispatch", tokens=4096, experts=128, top_k=8, width=4096, type="f16", away=0.0),
        # its gradient in a training step with an odd number of tokens
        dict(name="dispatch_grad", op="dispatch_grad", tokens=4099, experts=60, top_k=4, width=3584, type="bf16", away=0.1),
        # one token's experts added up
        dict(name="combine_token", op="combine", tokens=1, experts=64, top_k=8, width=4096, type="f16", away=0.0,
             grad=False),
        # a training step: the weighted sum, and the gradients of rows and weights
        dict(name="combine_train", op="combine", tokens=8192, experts=8, top_k=2, width=4096, type="bf16", away=0.0,
             grad=True),
        # one token through its experts' first product (fine-grained experts, asymmetric weights)
        dict(name="w4_token", op="w4_experts", tokens=1, experts=64, top_k=8, width=2048, out=2816, zeros=True,
             spread=True, bias=False),
        # a decode batch: most experts see a few tokens each, rows read through the sorted order
        dict(name="w4_batch", op="w4_experts", tokens=61, experts=32, top_k=4, width=4096, out=2048, zeros=False,
             spread=True, bias=True),
        # a prefill chunk through eight wide experts, rows already gathered
        dict(name="w4_prefill", op="w4_experts", tokens=8192, experts=8, top_k=2, width=4096, out=14336, zeros=False,
             spread=False, bias=False),
        # a small decode batch through eight wide ternary experts' last product
        dict(name="ternary_token", op="ternary_experts", tokens=4, experts=8, top_k=2, width=14336, out=4096, zeros=False,
             spread=False, bias=False),
        # a prefill chunk through many ternary experts, ragged numbers of rows, an odd output width
        dict(name="ternary_prefill", op="ternary_experts", tokens=2500, experts=24, top_k=4, width=3584, out=4607,
             zeros=False, spread=True, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "dispatch_grad", "combine", "w4_experts", "ternary_experts"])
    experts = _log(rng, 4, 256)
    top_k = min(experts, rng.randint(1, 8))
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=_log(rng, 9, 512), top_k=top_k,
                    type=rng.choice(["f32", "f16", "bf16"]), renorm=rng.random() < 0.5, grad=rng.random() < 0.5)
    if op in ("dispatch", "dispatch_grad", "combine"):
        c = dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, top_k=top_k,
                 width=rng.choice([1, 8]) * _log(rng, 60, 500), type=rng.choice(["f32", "f16", "bf16"]),
                 away=rng.choice([0.0, 0.0, 0.3]))
        if op == "combine":
            c["grad"] = rng.random() < 0.5
        return c
    ternary = op == "ternary_experts"
    unit = 64 if ternary else _GROUP
    width = unit * _log(rng, 2, 8192 // unit)
    out = _log(rng, 100, 8192)
    experts = max(2, min(_log(rng, 2, 64), (1 << 28) // (width * out)))
    return dict(op=op, tokens=_log(rng, 1, 4096), experts=experts, top_k=min(experts, rng.randint(1, 8)), width=width,
                out=out, zeros=not ternary and rng.random() < 0.3, spread=rng.random() < 0.5, bias=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------ inputs
def _routing(case, g):
    """Expert ids [T, k] (distinct per token, uneven loads); ids >= experts are other ranks' experts."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    total = int(round(E / (1.0 - case.get("away", 0.0))))
    score = torch.randn(T, total, generator=g, device="cuda") + 0.5 * torch.randn(total, generator=g, device="cuda")
    ids = torch.topk(score, k, dim=1).indices
    # the local experts lie among the others in no order
    return torch.randperm(total, generator=g, device="cuda")[ids].to(torch.int32)


def _sorted(ids, E):
    """Offsets [E+1], order [T k] (slots sorted by expert, in slot order within one; other ranks' last)
    and the position of each slot (-1: another rank's), for the plain forms and as a plan in hand."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    bounds = torch.arange(E + 1, device=key.device)
    offsets = (key[None, :] < bounds[:, None]).sum(1) if E * key.numel() <= 1 << 22 else torch.searchsorted(key[order], bounds)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(key < E, pos, torch.full_like(pos, -1))
    return offsets.to(torch.int32), order.to(torch.int32), pos.to(torch.int32).reshape(ids.shape)


def _rows(n, width, dtype, g):
    """Activations ~ N(0, 1), one row in a hundred scaled up (outlier tokens)."""
    x = torch.randn(n, width, generator=g, device="cuda")
    return (x * (1 + 19 * (torch.rand(n, 1, generator=g, device="cuda") < 0.01))).to(dtype)


def _w4_pack(w, zeros):
    """INT4, group 128 along K: words of 8 codes, fp16 scales, zero-points or None."""
    E, N, K = w.shape
    wg = w.view(E, N, K // _GROUP, _GROUP)
    if zeros:
        lo, hi = wg.amin(-1).clamp(max=0), wg.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).half()
        z = torch.clamp(torch.round(-lo / s.float()), 0, 15)
    else:
        s, z = (wg.abs().amax(-1) / 7).half(), None
    u = torch.round(wg / s.float()[..., None]) + (8 if z is None else z[..., None])
    u = u.clamp_(0, 15).to(torch.int32).view(E, N, K // 8, 8)
    shift = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    q = torch.bitwise_left_shift(u, shift).sum(-1, dtype=torch.int32)
    return q, s, None if z is None else z.to(torch.uint8)


def _ternary_pack(w):
    """Codes 0, 1, 2 for -1, 0, +1 (threshold 0.7 mean |w|), four per byte; one fp16 scale per row."""
    E, N, K = w.shape
    a = w.abs()
    keep = a > 0.7 * a.mean(-1, keepdim=True)
    scale = ((a * keep).sum(-1) / keep.sum(-1).clamp(min=1)).half()
    c = (1 + torch.sign(w) * keep).to(torch.uint8).view(E, N, K // 4, 4)
    return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, s = case, dict(case)
    if c["op"] == "route":
        s["logits"] = (1.5 * torch.randn(c["tokens"], c["experts"], generator=g, device="cuda")).to(_TYPES[c["type"]])
        if c["grad"]:
            s["dweights"] = torch.randn(c["tokens"], c["top_k"], generator=g, device="cuda")
        return s
    ids = _routing(c, g)
    offsets, order, pos = _sorted(ids, c["experts"])
    T, R, E = c["tokens"], c["tokens"] * c["top_k"], c["experts"]
    if c["op"] == "dispatch":
        dtype = _TYPES[c["type"]]
        # rows past the last local slot stay as the program left them (zeros here)
        return dict(s, ids=ids, x=_rows(T, c["width"], dtype, g),
                    rows=torch.zeros(R, c["width"], dtype=dtype, device="cuda"))
    if c["op"] == "dispatch_grad":
        return dict(s, pos=pos, drows=_rows(R, c["width"], _TYPES[c["type"]], g))
    if c["op"] == "combine":
        dtype = _TYPES[c["type"]]
        s.update(pos=pos, y=_rows(R, c["width"], dtype, g))
        s["weights"] = torch.softmax(1.5 * torch.randn(T, c["top_k"], generator=g, device="cuda"), 1)
        if c["grad"]:
            s["dout"] = torch.randn(T, c["width"], generator=g, device="cuda").to(dtype)
            s["dy"] = torch.zeros_like(s["y"])  # rows of no local slot stay as they are
        return s
    K, N = c["width"], c["out"]
    w = 0.02 * torch.randn(E, N, K, generator=g, device="cuda")
    if c["op"] == "w4_experts":
        s["q"], s["s"], s["z"] = _w4_pack(w, c["zeros"])
    else:
        s["q"], s["s"] = _ternary_pack(w)
    del w
    s["b"] = (0.01 * torch.randn(E, N, generator=g, device="cuda")).half() if c["bias"] else None
    x = _rows(T, K, torch.float16, g)
    # `spread`: x holds the tokens and the product reads them through the order; else x is gathered
    s.update(offsets=offsets, order=order if c["spread"] else None,
             x=x if c["spread"] else x[(order // c["top_k"]).long()].contiguous())
    s["bounds"] = offsets.tolist()  # the same numbers on the host, for the plain form's slices
    return s


# ----------------------------------------------------------------------------------------- plain forms
def _plain_route(s):
    x = s["logits"].float()
    k = s["top_k"]
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]  # ties: the lowest index
    e = torch.exp(x - x.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    w = torch.gather(p, 1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if not s["grad"]:
        return w, ids.to(torch.int32)
    dw = s["dweights"]
    inner = (dw * w).sum(1, keepdim=True)
    if s["renorm"]:  # a softmax over the chosen ones
        dx = torch.zeros_like(x).scatter(1, ids, w * (dw - inner))
    else:
        dx = p * (torch.zeros_like(x).scatter(1, ids, dw) - inner)
    return w, ids.to(torch.int32), dx.to(s["logits"].dtype)


def _plain_dispatch(s):
    offsets, order, pos = _sorted(s["ids"], s["experts"])
    rows = s["x"][(order // s["top_k"]).long()]
    there = torch.arange(rows.shape[0], device=rows.device) < offsets[-1]
    return offsets, order, pos, torch.where(there[:, None], rows, torch.zeros_like(rows))


def _taken(y, pos):
    """[T, k, H] in 32 bits: each slot's row, zeros for slots of other ranks."""
    return y.float()[pos.clamp(min=0).long()] * (pos >= 0)[..., None]


def _plain_combine(s):
    rows = _taken(s["y"], s["pos"])
    out = (rows * s["weights"][..., None]).sum(1).to(s["y"].dtype)
    if not s["grad"]:
        return out
    d = s["dout"].float()
    dw = (rows * d[:, None, :]).sum(-1)
    there = s["pos"].reshape(-1) >= 0
    at = torch.where(there, s["pos"].reshape(-1), s["y"].shape[0]).long()  # other ranks' slots: a row past the end
    dy = torch.zeros(s["y"].shape[0] + 1, s["y"].shape[1], device=d.device)
    dy[at] = (s["weights"][..., None] * d[:, None, :]).reshape(-1, d.shape[1])
    return out, dy[:-1].to(s["y"].dtype), dw


def _w4_values(q, s, z, to):
    """The weights that the words of one expert stand for."""
    u = torch.bitwise_and(torch.bitwise_right_shift(q[..., None], torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)), 15)
    u = u.reshape(s.shape[0], s.shape[1], _GROUP).to(to)
    return ((u - (8 if z is None else z.to(to)[..., None])) * s.to(to)[..., None]).reshape(s.shape[0], -1)


def _ternary_values(q, s, to):
    c = torch.stack([q & 3, (q >> 2) & 3, (q >> 4) & 3, q >> 6], -1).reshape(q.shape[0], -1)
    return (c.to(to) - 1) * s.to(to)[:, None]


def _values(s, e, to):
    if s["op"] == "w4_experts":
        return _w4_values(s["q"][e], s["s"][e], None if s["z"] is None else s["z"][e], to)
    return _ternary_values(s["q"][e], s["s"][e], to)


def _plain_experts(s):
    x = s["x"] if s["order"] is None else s["x"][(s["order"] // s["top_k"]).long()]
    b = s["bounds"]

    def product(e):
        y = x[b[e]:b[e + 1]].float() @ _values(s, e, torch.float32).t()
        return (y if s["b"] is None else y + s["b"][e].float()).half()

    return torch.cat([product(e) for e in range(s["experts"]) if b[e + 1] > b[e]])


# -------------------------------------------------------------------------------------- the package's calls
def _own(s):
    import bit_weight_only_tq_b200 as tq

    op = s["op"]
    if op == "route":
        w, ids = tq.tq_moe_route(s["logits"], s["top_k"], renormalize=s["renorm"])
        if not s["grad"]:
            return w, ids
        return w, ids, tq.tq_moe_route_backward(s["dweights"], s["logits"], w, ids, renormalize=s["renorm"])
    if op == "dispatch":
        offsets, order, pos = tq.tq_moe_sort(s["ids"], s["experts"])
        return offsets, order, pos, tq.tq_moe_gather(s["x"], order, offsets, s["top_k"], out=s["rows"])
    if op == "dispatch_grad":
        return tq.tq_moe_gather_backward(s["drows"], s["pos"])
    if op == "combine":
        out = tq.tq_moe_combine(s["y"], s["pos"], s["weights"])
        if not s["grad"]:
            return out
        dy, dw = tq.tq_moe_combine_backward(s["dout"], s["y"], s["pos"], s["weights"], dy=s["dy"])
        return out, dy, dw
    if op == "w4_experts":
        return tq.w4g_gemm_experts(s["x"], s["q"], s["s"], s["offsets"], zeros=s["z"], bias=s["b"], order=s["order"],
                                   top_k=s["top_k"])
    return tq.tq_gemm_experts(s["x"], s["q"], s["s"], s["offsets"], bias=s["b"], order=s["order"], top_k=s["top_k"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "route":
        return _plain_route(state)
    if op == "dispatch":
        return _plain_dispatch(state)
    if op == "dispatch_grad":
        return _taken(state["drows"], state["pos"]).sum(1).to(state["drows"].dtype)
    if op == "combine":
        return _plain_combine(state)
    return _plain_experts(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    R = T * k
    if c["op"] == "route":
        n, f = T * E * _SIZE[c["type"]] + R * 8, 4 * T * E
        if c["grad"]:  # weights' gradient, weights, ids; the scores again unless renormalised; the scores' gradient
            n += R * 12 + T * E * _SIZE[c["type"]] * (1 if c["renorm"] else 2)
            f += 3 * T * E
        return {"bytes": n, "flops": f}
    if c["op"] in ("dispatch", "dispatch_grad", "combine"):
        there = int(R * (1.0 - c["away"]))  # slots of this rank's experts, on average
        row = c["width"] * _SIZE[c["type"]]
        if c["op"] == "dispatch":
            return {"bytes": 4 * (3 * R + E + 1) + (T + there) * row, "flops": 0}
        if c["op"] == "dispatch_grad":
            return {"bytes": 4 * R + (T + there) * row, "flops": there * c["width"]}
        n, f = 8 * R + (T + there) * row, 2 * there * c["width"]
        if c["grad"]:
            n += 12 * R + (T + 2 * there) * row
            f += 3 * there * c["width"]
        return {"bytes": n, "flops": f}
    N, K = c["out"], c["width"]
    weights = N * K // 4 + 2 * N if c["op"] == "ternary_experts" else N * (K // 2 + K // _GROUP * (3 if c["zeros"] else 2))
    active = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token takes, on average
    n = active * (weights + (2 * N if c["bias"] else 0)) + 2 * (T if c["spread"] else R) * K + 2 * R * N
    return {"bytes": int(n) + 4 * (E + 1) + (4 * R if c["spread"] else 0), "flops": 2 * R * N * K}


# ----------------------------------------------------------------------------------------------- 64 bits
def _exact_route(s):
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    k = s["top_k"]
    ids = np.lexsort((np.broadcast_to(np.arange(E), x.shape), -x), axis=1)[:, :k]
    at = np.arange(T)[:, None]
    top = x[at, ids]
    if s["renorm"]:
        w = np.exp(top - top[:, :1])
        w /= w.sum(1, keepdims=True)
    else:
        lse = x.max(1, keepdims=True) + np.log(np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True))
        w = np.exp(top - lse)
    if not s["grad"]:
        return w, ids.astype(np.int32)
    dw = s["dweights"].double().cpu().numpy()
    mean = (w * dw).sum(1, keepdims=True)
    dx = np.zeros_like(x) if s["renorm"] else -np.exp(x - lse) * mean
    dx[at, ids] += w * (dw - mean) if s["renorm"] else w * dw
    return w, ids.astype(np.int32), dx


def _exact_experts(s):
    b, k = s["bounds"], s["top_k"]
    y = torch.empty(b[-1], s["out"], dtype=torch.float64, device="cuda")
    for e in range(s["experts"]):
        if b[e] == b[e + 1]:
            continue
        if s["order"] is None:
            x = s["x"][b[e]:b[e + 1]].double()
        else:
            x = s["x"].double()[torch.div(s["order"][b[e]:b[e + 1]], k, rounding_mode="floor").long()]
        q, sc = s["q"][e], s["s"][e].double()
        out = torch.zeros(x.shape[0], s["out"], dtype=torch.float64, device="cuda")
        if s["op"] == "w4_experts":  # one digit of the words at a time: codes of columns i, i + 8, ...
            zero = torch.full_like(sc, 8.0) if s["z"] is None else s["z"][e].double()
            sc, zero = (t.repeat_interleave(_GROUP // 8, 1) for t in (sc, zero))
            for i in range(8):
                out += x[:, i::8] @ (sc * (((q >> (4 * i)) & 15).double() - zero)).t()
        else:
            for i in range(4):
                out += x[:, i::4] @ (((q >> (2 * i)) & 3).double() - 1).t()
            out *= sc
        y[b[e]:b[e + 1]] = out if s["b"] is None else out + s["b"][e].double()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        return _exact_route(s)
    if op in ("w4_experts", "ternary_experts"):
        return _exact_experts(s)
    if op == "dispatch":
        ids = s["ids"].cpu().numpy().reshape(-1)
        key = np.where((ids >= 0) & (ids < s["experts"]), ids, s["experts"])
        order = np.lexsort((np.arange(key.size), key))
        offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=s["experts"] + 1)[:-1])])
        pos = np.empty(key.size, np.int64)
        pos[order] = np.arange(key.size)
        rows = torch.zeros(key.size, s["width"], dtype=torch.float64, device="cuda")
        n = int(offsets[-1])
        rows[:n] = s["x"].double()[torch.from_numpy(order[:n] // s["top_k"]).cuda()]
        return (offsets.astype(np.int32), order.astype(np.int32),
                np.where(key < s["experts"], pos, -1).astype(np.int32).reshape(s["ids"].shape), rows)
    pos = s["pos"].long()
    src = s["drows"] if op == "dispatch_grad" else s["y"]
    out = torch.zeros(s["tokens"], s["width"], dtype=torch.float64, device="cuda")
    for j in range(s["top_k"]):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        w = 1.0 if op == "dispatch_grad" else s["weights"][t, j].double()[:, None]
        out[t] += w * src[pos[t, j]].double()
    if op == "dispatch_grad" or not s["grad"]:
        return out
    dy = torch.zeros(src.shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(pos.shape, dtype=torch.float64, device="cuda")
    for j in range(s["top_k"]):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        dy[pos[t, j]] = s["weights"][t, j].double()[:, None] * s["dout"][t].double()
        dw[t, j] = (s["dout"][t].double() * src[pos[t, j]].double()).sum(1)
    return out, dy, dw
