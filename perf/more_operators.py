"""Measured cases of the router and of the 4-bit operators: the choice of experts from a router's
logits, its gradient, the MXFP4 quantizer, and the routed product of MXFP4 activations with MXFP4
experts.

MXFP4 holds E2M1 codes (two a byte, the even element in the low nibble) and one E8M0 scale byte
per 32 consecutive elements of a row. An expert layer holds E units back to back, each its codes
[out][in / 2] followed by its scales [out][in / 32].

With ``own`` false, ``run`` computes an operator by elementary torch operations (the plain form);
with ``own`` true it calls the package. Both take what ``prepare`` made; with ``own`` true that
also holds what a serving program keeps: the layer in its read order and a workspace.
"""

import math

import torch

own = False

# The largest listed cases, which drawn ones do not exceed.
MAX_ROUTE = 8192 * 384
MAX_ELEMENTS = 49152 * 5120
MAX_FLOPS = 2 * 65536 * 1536 * 5120
MAX_UNITS = 384 * 1536 * 5120  # weights of a layer


def listed():
    """384 experts of 128 x 5,120 units, top-8 routing, 64-token decode batches and 8,192-token
    chunks are the repository's own workloads, 1,536 outputs its fused gate and up projections of
    768 channels; the others are generic."""
    return [
        # one token of a served sequence: latency
        {"name": "route one token", "op": "route", "T": 1, "E": 384, "topk": 8, "score": "softmax",
         "dtype": "bf16", "bias": False, "groups": 1, "group_topk": 1, "group_top": 1,
         "renorm": True, "scale": 1.0},
        # a decode batch with experts chosen inside the best groups
        {"name": "route grouped batch", "op": "route", "T": 64, "E": 256, "topk": 8,
         "score": "sigmoid", "dtype": "f32", "bias": True, "groups": 8, "group_topk": 4,
         "group_top": 2, "renorm": True, "scale": 2.5},
        # a prefill chunk under a balancing bias
        {"name": "route chunk", "op": "route", "T": 8192, "E": 384, "topk": 8, "score": "sigmoid",
         "dtype": "f32", "bias": True, "groups": 1, "group_topk": 1, "group_top": 1,
         "renorm": True, "scale": 1.0},
        # the router's gradient in a training step of an odd batch
        {"name": "route backward odd", "op": "route_backward", "T": 1001, "E": 100, "topk": 6,
         "score": "sigmoid", "dtype": "f32", "bias": True, "groups": 1, "group_topk": 1,
         "group_top": 1, "renorm": True, "scale": 1.0},
        # the router's gradient over a chunk: every logit has one
        {"name": "route backward chunk", "op": "route_backward", "T": 8192, "E": 384, "topk": 8,
         "score": "softmax", "dtype": "bf16", "bias": False, "groups": 1, "group_topk": 1,
         "group_top": 1, "renorm": False, "scale": 1.0},
        # activations of a decode batch, quantized and read back
        {"name": "quantize decode", "op": "quantize", "rows": 64, "n": 5120},
        # a layer's weights brought to the store's values (an encoding and its check)
        {"name": "quantize layer", "op": "quantize", "rows": 49152, "n": 5120},
        # one token through its eight experts' gate and up projections: latency
        {"name": "experts one token", "op": "experts", "T": 1, "topk": 8, "E": 384, "out": 1536,
         "in": 5120, "combine": False, "skew": 0.0},
        # a decode batch over the repository's expert layer, each slot weighted
        {"name": "experts decode batch", "op": "experts", "T": 64, "topk": 8, "E": 384, "out": 128,
         "in": 5120, "combine": False, "skew": 0.0},
        # an odd batch with padded tokens, the slots of a token added up
        {"name": "experts ragged", "op": "experts", "T": 333, "topk": 6, "E": 60, "out": 1424,
         "in": 2560, "combine": True, "skew": 0.0},
        # a prefill chunk over the repository's expert layer, popular experts far ahead
        {"name": "experts chunk", "op": "experts", "T": 8192, "topk": 8, "E": 384, "out": 128,
         "in": 5120, "combine": False, "skew": 1.1},
        # a prefill chunk through 32 experts' gate and up projections: the matrix cores' rate
        {"name": "experts wide chunk", "op": "experts", "T": 8192, "topk": 8, "E": 32, "out": 1536,
         "in": 5120, "combine": False, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    """Tokens 1 .. 8,192, experts 4 .. 512 for the router and 8 .. 384 for the product, widths
    512 .. 7,168 and outputs 16 .. 1,536, over their logarithms."""
    op = rng.choice(["route", "route", "route_backward", "quantize", "experts", "experts", "experts"])
    T = max(1, round(_log(rng, 1, 8192)))
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, round(_log(rng, 4, 512) / groups))
        group_topk = rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": max(1, min(T, MAX_ROUTE // E)), "E": E,
                "topk": rng.randint(1, min(16, E // groups * group_topk)), "score": score,
                "dtype": rng.choice(["bf16", "f32"]), "bias": rng.random() < 0.5,
                "groups": groups, "group_topk": group_topk, "group_top": rng.choice([1, 2]),
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    if op == "quantize":
        n = 32 * round(_log(rng, 1, 640))
        return {"op": op, "rows": max(1, min(round(_log(rng, 1, 65536)), MAX_ELEMENTS // n)), "n": n}
    E = max(8, round(_log(rng, 8, 384)))
    topk = rng.randint(1, 8)
    out, n = 16 * round(_log(rng, 1, 96)), 512 * rng.randint(1, 14)
    out = max(16, min(out, MAX_UNITS // (E * n) // 16 * 16))
    return {"op": op, "T": max(1, min(T, MAX_FLOPS // (2 * topk * out * n))), "topk": topk, "E": E,
            "out": out, "in": n, "combine": rng.random() < 0.4, "skew": rng.choice([0.0, 0.5, 1.1])}


# ---- inputs ------------------------------------------------------------------------------
def _logits(gen, c):
    """A router's logits: unit normal values of a token on top of each expert's popularity, one
    expert out of service, and padded tokens (no expert at all) at the end of a longer batch."""
    T, E = c["T"], c["E"]
    x = torch.randn((T, E), generator=gen, device="cuda")
    x += 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    if E > 2 * c["topk"]:
        x[:, E // 3] = -math.inf
    if T > 16:
        x[T - T // 16:] = -math.inf
    return x.bfloat16() if c["dtype"] == "bf16" else x


def _choices(gen, T, topk, E, skew):
    """Routes of T tokens: distinct experts, the expert of rank r drawn with weight (r + 1)^-skew,
    a few empty slots, and padded tokens at the end of a longer batch."""
    weight = -skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    weight = weight[torch.randperm(E, generator=gen, device="cuda")]
    u = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)
    ids = torch.sort(weight - torch.log(-torch.log(u)), dim=1, descending=True).indices[:, :topk].int()
    if T > 16:
        ids[T - T // 16:] = -1
        ids[:: 50, topk - 1] = -1
    return ids.contiguous()


def _units(gen, c):
    """An expert layer's units: E2M1 codes as normal weights have them, and scales about 2^-6."""
    low = torch.tensor([14, 13, 12, 12, 11, 10, 9, 8, 0, 1, 2, 3, 4, 4, 5, 6], device="cuda")
    high = torch.tensor([15, 13, 12, 12, 11, 10, 9, 8, 0, 1, 2, 3, 4, 4, 5, 7], device="cuda")
    pair = (high[:, None] << 4 | low[None]).byte().reshape(256)
    E, out, n = c["E"], c["out"], c["in"]
    units = torch.empty((E, out * n // 2 + out * n // 32), dtype=torch.uint8, device="cuda")
    for part in units.split(max(1, (1 << 28) // units.shape[1])):
        part[:] = pair[torch.randint(0, 256, part.shape, generator=gen, device="cuda", dtype=torch.int32)]
        part[:, out * n // 2:] = torch.randint(119, 123, (part.shape[0], out * n // 32), generator=gen,
                                               device="cuda", dtype=torch.uint8)
    return units


def _activations(gen, T, n):
    """bf16 rows of hidden states: unit normal values, a few channels far larger than the rest,
    tokens of different norms, and a zero row (a padded token) where there are several."""
    x = torch.randn((T, n), generator=gen, device="cuda")
    x[:, :: 97] *= 12.0
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device="cuda"))
    if T > 8:
        x[T // 2] = 0
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _activations(gen, case["rows"], case["n"])
        return s
    if case["op"] == "experts":
        T, topk, E, out, n = (case[k] for k in ("T", "topk", "E", "out", "in"))
        s["x"] = _activations(gen, T, n)
        s["ids"] = _choices(gen, T, topk, E, case["skew"])
        s["w"] = torch.rand((T, topk), generator=gen, device="cuda") + 0.1
        s["units"] = _units(gen, case)
        if own:
            from trellis_quantized_moe_amd import ops
            s["layer"] = ops.Mxfp4Layer(E, out, n, s["units"].view(-1)).repacked()
            s["flags"] = ops.TQ_FP4 | (ops.TQ_COMBINE if case["combine"] else 0)
            s["ws"] = ops.workspace(T, topk, E, out, n, s["flags"])
        return s
    s["logits"] = _logits(gen, case)
    # a balancing bias moves by a fixed step per training step
    b = 0.001 * torch.round(20 * torch.randn(case["E"], generator=gen, device="cuda"))
    s["b"] = b if case["bias"] else None
    if case["op"] == "route_backward":
        s["ids"] = _route(s)[0]
        s["dw"] = torch.randn(s["ids"].shape, generator=gen, device="cuda")
    if own:
        from trellis_quantized_moe_amd import ops
        s["router"] = ops.Router(case["E"], case["topk"], score=case["score"], bias=s["b"],
                                 groups=case["groups"], group_topk=case["group_topk"],
                                 group_top=case["group_top"], renorm=case["renorm"],
                                 scale=case["scale"])
    return s


# ---- the operators in their plain form -----------------------------------------------------
def _scores(s):
    """Softmax or sigmoid scores in 64 bits; a row without experts has only zeros."""
    x = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _route(s):
    """(ids, weights): the values next to a border decide, so the scores are in 64 bits."""
    x, p = s["logits"].double(), _scores(s)
    T, E = x.shape
    key = p + s["b"].double() if s["b"] is not None else p
    open_ = x > -math.inf
    if s["groups"] > 1:
        size = E // s["groups"]
        g = torch.where(open_, key, torch.full_like(key, -math.inf)).view(T, s["groups"], size)
        best = torch.sort(g, dim=2, descending=True).values[:, :, :s["group_top"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        total = torch.where(some, total, torch.full_like(total, -math.inf))
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :s["group_topk"]]
        kept = torch.zeros((T, s["groups"]), dtype=torch.bool, device=x.device)
        kept.scatter_(1, order, True)
        open_ = open_ & kept[:, :, None].expand(T, s["groups"], size).reshape(T, E)
    # without a bias a score grows with its logit, which orders where scores round together
    key = torch.where(open_, key if s["b"] is not None else x, torch.full_like(key, -math.inf))
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids, some = ids[:, :s["topk"]], top[:, :s["topk"]] > -math.inf
    w = torch.where(some, torch.gather(p, 1, ids), torch.zeros_like(p[:, :1]))
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    ids = torch.where(some, ids, torch.full_like(ids, -1)).int()
    return ids, (s["scale"] * w).float()


def _route_backward(s):
    p, dw = _scores(s), s["dw"].double()
    some = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    zero = torch.zeros_like(dw)
    c = torch.where(some, torch.gather(p, 1, ids), zero)
    g = torch.where(some, dw, zero)
    if s["renorm"]:
        total = c.sum(1, keepdim=True).clamp(min=1e-300)
        g = torch.where(some, (g - (c * g).sum(1, keepdim=True) / total) / total, zero)
    g = torch.zeros_like(p).scatter_add_(1, ids, s["scale"] * g)
    if s["score"] == "sigmoid":
        d = g * p * (1 - p)
    else:
        d = p * (g - (p * g).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _quantized(x):
    """The MXFP4 values of bf16 rows in fp32: per 32 the smallest power of two 2^k, k >= -127, with
    max|x| <= 7 * 2^k, and each element's nearest E2M1 multiple of it, ties to the even code."""
    v = x.float().view(x.shape[0], -1, 32)
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    k = torch.where(m <= 0.875, e - 3, e - 2).clamp(min=-127)
    k = torch.where(m > 0, k, torch.zeros_like(k)).int()
    r = v * ((127 - k) << 23).view(torch.float32)
    a = r.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6)
    return (torch.copysign(q, r) * torch.exp2(k.float())).view(x.shape)


def _decoded(units, out, n):
    """fp32 weights [units][out][in] of MXFP4 units."""
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=units.device)
    value = torch.cat([value, -value])
    pair = torch.stack([value.repeat(16), value.repeat_interleave(16)], 1)
    w = pair[units[:, :out * n // 2].int()].view(-1, out, n // 32, 32)
    scale = (units[:, out * n // 2:].int() << 23).view(torch.float32)
    return (w * scale.view(-1, out, n // 32, 1)).view(-1, out, n)


def _experts(s):
    """The slots sorted by expert, cut into blocks of rows of one expert each, one product a block."""
    T, topk, E, out, n = s["T"], s["topk"], s["E"], s["out"], s["in"]
    ids, N = s["ids"].reshape(-1).long(), T * topk
    rows = 128 if N > 16 * E else 16
    items = (N + rows - 1) // rows + min(E, N)
    which, slots = torch.sort(torch.where(ids < 0, torch.full_like(ids, E), ids), stable=True)
    first = torch.searchsorted(which, torch.arange(E + 1, device=ids.device))
    blocks = (first[1:] - first[:-1] + rows - 1) // rows
    ends = torch.cumsum(blocks, 0)
    item = torch.arange(items, device=ids.device)
    e = torch.searchsorted(ends, item, right=True)
    real, e = e < E, e.clamp(max=E - 1)
    at = first[e] + (item - ends[e] + blocks[e]) * rows
    at = at[:, None] + torch.arange(rows, device=ids.device)
    real = real[:, None] & (at < first[e + 1][:, None])
    slot = slots[at.clamp(0, N - 1)]
    x = _quantized(s["x"])[slot // topk]
    if E <= items:
        w = _decoded(s["units"], out, n).transpose(1, 2).contiguous()[e]
    else:
        w = _decoded(s["units"][e], out, n).transpose(1, 2).contiguous()
    y = torch.zeros((N + 1, out), device=ids.device)
    y[torch.where(real, slot, torch.full_like(slot, N)).view(-1)] = torch.bmm(x, w).view(-1, out)
    y = torch.where((ids >= 0)[:, None], y[:N], torch.zeros_like(y[:N]))
    y = y.view(T, topk, out) * s["w"][:, :, None]
    return y.sum(1) if s["combine"] else y


def _run_own(s):
    from trellis_quantized_moe_amd import ops
    if s["op"] == "route":
        ids, w = ops.expert_route(s["router"], s["logits"])
        return {"ids": ids, "w": w}
    if s["op"] == "route_backward":
        return {"dlogits": ops.expert_route_backward(s["router"], s["logits"], s["ids"], s["dw"])}
    if s["op"] == "experts":
        return {"y": ops.mxfp4_expert_gemm(s["layer"], s["x"], s["ids"], s["w"], flags=s["flags"],
                                           ws=s["ws"])}
    rows, n = s["x"].shape
    unit = torch.empty(rows * n // 2 + rows * n // 32, dtype=torch.uint8, device="cuda")
    ops.mxfp4_quantize(s["x"], codes=unit[:rows * n // 2].view(rows, n // 2),
                       scales=unit[rows * n // 2:].view(rows, n // 32))
    return {"values": ops.mxfp4_decode(unit, rows, n).view(torch.bfloat16)}


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "route":
        ids, w = _route(s)
        return {"ids": ids, "w": w}
    if s["op"] == "route_backward":
        return {"dlogits": _route_backward(s)}
    if s["op"] == "quantize":
        return {"values": _quantized(s["x"]).bfloat16()}
    return {"y": _experts(s)}


# ---- bounds ------------------------------------------------------------------------------
def work(case):
    if case["op"] == "quantize":  # read, written in 4 bits, and written as what those stand for
        size = case["rows"] * case["n"]
        return {"bytes": 4 * size + size // 2 + size // 32, "flops": 3 * size}
    T, topk, E = case["T"], case["topk"], case["E"]
    if case["op"] == "experts":
        out, n = case["out"], case["in"]
        touched = E * (1 - (1 - topk / E) ** T)
        y = 4 * T * out * (1 if case["combine"] else topk)
        return {"bytes": 2 * T * n + 8 * T * topk + touched * (out * n // 2 + out * n // 32) + y,
                "flops": 2 * T * topk * out * n}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        return {"bytes": size * T * E + 8 * T * topk, "flops": 4 * T * E}
    read = E if case["score"] == "softmax" and not case["renorm"] else topk
    return {"bytes": size * T * (E + read) + 8 * T * topk, "flops": 4 * T * E}


# ---- the definitions in 64 bits ------------------------------------------------------------
def _before(key):
    """How many entries of its row go before each: larger ones, and equal ones further left."""
    n = key.shape[1]
    left = torch.arange(n, device=key.device)
    left = left[None, :] < left[:, None]
    found = []
    for part in key.split(max(1, (1 << 27) // (n * n))):
        a, b = part[:, :, None], part[:, None, :]
        found.append(((b > a) | ((b == a) & left)).sum(2))
    return torch.cat(found)


def _exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    out_of_service = torch.isinf(x)
    if s["score"] == "sigmoid":
        score = torch.sigmoid(x)
    else:
        score = torch.softmax(x.masked_fill(out_of_service.all(1, keepdim=True), 0.0), 1)
    score = score.masked_fill(out_of_service, 0.0)
    choice = score if s["b"] is None else score + s["b"].double()
    choice = choice.masked_fill(out_of_service, -math.inf)
    if s["groups"] > 1:
        per = choice.view(T, s["groups"], -1)
        if s["group_top"] == 1 or per.shape[2] == 1:
            of_group = per.amax(2)
        else:
            first, second = per.topk(2, dim=2).values.unbind(2)
            of_group = first + torch.where(torch.isinf(second), torch.zeros_like(second), second)
        lost = _before(of_group) >= s["group_topk"]
        out_of_service = out_of_service | lost.repeat_interleave(E // s["groups"], 1)
    key = x if s["b"] is None else choice
    rank = _before(key.masked_fill(out_of_service, -math.inf))
    ids = torch.full((T, s["topk"]), -1, dtype=torch.int32, device=x.device)
    weight = torch.zeros((T, s["topk"]), dtype=torch.float64, device=x.device)
    for k in range(s["topk"]):
        here = (rank == k) & ~out_of_service
        expert = here.int().argmax(1)
        chosen = here.any(1)
        ids[:, k] = torch.where(chosen, expert, torch.full_like(expert, -1)).int()
        weight[:, k] = (score * here).sum(1)
    if s["renorm"]:
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids, "w": s["scale"] * weight}


def _exact_route_backward(s):
    """By automatic differentiation of the weights, the choice held fixed."""
    x = s["logits"].double()
    padded = torch.isinf(x).all(1, keepdim=True)
    leaf = x.masked_fill(padded, 0.0).requires_grad_()
    score = torch.sigmoid(leaf) if s["score"] == "sigmoid" else torch.softmax(leaf, 1)
    chosen = s["ids"] >= 0
    weight = torch.gather(score, 1, s["ids"].clamp(min=0).long()) * chosen
    if s["renorm"]:
        weight = weight / (weight.sum(1, keepdim=True) + padded)
    total = (s["scale"] * weight * s["dw"].double() * chosen).sum()
    return {"dlogits": torch.autograd.grad(total, leaf)[0].masked_fill(padded, 0.0)}


def _exact_values(x):
    """The nearest of the 15 values at the block's scale, by the borders between them."""
    rows, n = x.shape
    v = x.double().reshape(-1, 32)
    top = v.abs().max(1, keepdim=True).values
    k = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 7.0)) / 7))
    k = torch.where(top > 7 * torch.exp2(k), k + 1, k)
    k = torch.where((top > 0) & (top <= 7 * torch.exp2(k - 1)), k - 1, k).clamp(min=-127)
    size = v.abs() / torch.exp2(k)
    q = torch.zeros_like(v)
    last = 0.0
    for border, value, even in ((0.25, 0.5, 0), (0.75, 1.0, 1), (1.25, 1.5, 0), (1.75, 2.0, 1),
                                (2.5, 3.0, 0), (3.5, 4.0, 1), (5.0, 6.0, 0)):
        q += ((size > border) | ((size == border) & bool(even))) * (value - last)
        last = value
    return (q * torch.sign(v) * torch.exp2(k)).view(rows, n)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "route_backward":
        return _exact_route_backward(s)
    x = _exact_values(s["x"])
    if s["op"] == "quantize":
        return {"values": x}
    T, topk, out, n = s["T"], s["topk"], s["out"], s["in"]
    flat = s["ids"].reshape(-1)
    y = torch.zeros((T * topk, out), dtype=torch.float64, device="cuda")
    size = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    for e in torch.unique(flat[flat >= 0]).tolist():
        codes = s["units"][e, :out * n // 2].view(out, n // 2)
        nibble = torch.stack([codes & 15, codes >> 4], 2).reshape(out, n)
        w = size[(nibble & 7).long()] * (1 - 2 * (nibble >> 3).double())
        power = s["units"][e, out * n // 2:].view(out, n // 32).double() - 127
        w = w * torch.exp2(power).repeat_interleave(32, 1)
        slot = torch.nonzero(flat == e).view(-1)
        y[slot] = torch.matmul(x[slot // topk], w.t())
    y = y.view(T, topk, out) * s["w"].double()[:, :, None]
    return {"y": y.sum(1) if s["combine"] else y}
