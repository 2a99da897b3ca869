"""Measured cases of the 4-bit base layers and the router.

Three operators, each in two forms: elementary torch operations (``own``
false), and the calls a user makes of this package (``own`` true).

  w4       y[t] = W x[t], W held as 4-bit codes with a scale (and a zero point) per group of inputs
  experts  the same product with a matrix per expert: row (t, j) takes the matrix ids[t, j] names;
           the rows themselves, or a token's rows summed with the router's weights
  route    the router: scores of a token's experts, the chosen ids and their weights
"""
import math

import torch

own = False

#: The work (in bytes, or flops / 100 where that is more) that no drawn case exceeds.
_LARGEST = 9.7e9


def listed():
    return [
        # One decode token through the smallest projection of the fleet's model (its k or v): latency.
        dict(name="w4-one-token-kv", op="w4", T=1, d_in=3584, d_out=512, group=128, zeros=False, scales="bf16", dtype="bf16"),
        # One decode token through its gate or up projection: a stream of codes.
        dict(name="w4-one-token-gate", op="w4", T=1, d_in=3584, d_out=18944, group=128, zeros=True, scales="bf16", dtype="bf16"),
        # A decode batch of odd size through its down projection, finer groups.
        dict(name="w4-batch-down", op="w4", T=23, d_in=18944, d_out=3584, group=64, zeros=True, scales="bf16", dtype="bf16"),
        # Float32 activations over a checkpoint with fine groups.
        dict(name="w4-float32", op="w4", T=5, d_in=4096, d_out=4096, group=32, zeros=False, scales="f32", dtype="f32"),
        # A prefill step, the MLP up projection of the prefill workload.
        dict(name="w4-prefill", op="w4", T=8192, d_in=4096, d_out=14336, group=128, zeros=False, scales="bf16", dtype="bf16"),
        # One decode token's eight experts of 64, gate and up together.
        dict(name="experts-one-token", op="experts", T=1, k=8, E=64, d_in=2048, d_out=2816, group=128, zeros=False, scales="bf16",
             dtype="bf16", combine=False, padded=False),
        # A decode batch's down projections, summed with the router's weights; the batch is padded.
        dict(name="experts-batch-down", op="experts", T=45, k=4, E=32, d_in=1408, d_out=2048, group=32, zeros=True, scales="bf16",
             dtype="bf16", combine=True, padded=True),
        # A prefill step's gate and up.
        dict(name="experts-prefill", op="experts", T=4096, k=4, E=32, d_in=2048, d_out=2816, group=128, zeros=False, scales="bf16",
             dtype="bf16", combine=False, padded=False),
        # A prefill step's down, summed with the weights.
        dict(name="experts-prefill-down", op="experts", T=2047, k=8, E=64, d_in=1408, d_out=2048, group=128, zeros=True, scales="bf16",
             dtype="bf16", combine=True, padded=False),
        # One decode token, softmax scores.
        dict(name="route-one-token", op="route", T=1, E=64, k=8, score="softmax", groups=1, top_groups=1, bias=False, dtype="bf16"),
        # A decode batch, sigmoid scores with a bias for balance and groups of experts.
        dict(name="route-batch-groups", op="route", T=250, E=256, k=8, score="sigmoid", groups=8, top_groups=4, bias=True, dtype="f32"),
        # A prefill step, softmax scores.
        dict(name="route-prefill", op="route", T=8192, E=128, k=8, score="softmax", groups=1, top_groups=1, bias=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["w4", "w4", "experts", "experts", "route"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, _log(rng, 8, 512) // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top_groups))
        bias = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                    top_groups=top_groups, bias=bias, dtype=rng.choice(["bf16", "f32"]))
    group = rng.choice([32, 64, 128])
    dtype, scales = rng.choice([("bf16", "bf16")] * 4 + [("bf16", "f32"), ("f32", "f32")])
    zeros = rng.random() < 0.5
    if op == "w4":
        return dict(op=op, T=_log(rng, 1, 8192 if dtype == "bf16" else 512), d_in=8 * _log(rng, 32, 2368), d_out=8 * _log(rng, 8, 2368),
                    group=group, zeros=zeros, scales=scales, dtype=dtype)
    E = _log(rng, 4, 160)
    k = rng.randint(1, min(8, E))
    combine = rng.random() < 0.5
    return dict(op=op, T=_log(rng, 1, 4096 if dtype == "bf16" else 128), k=k, E=E, d_in=8 * _log(rng, 32, 512), d_out=8 * _log(rng, 16, 512),
                group=group, zeros=zeros, scales=scales, dtype=dtype, combine=combine, padded=rng.random() < 0.3)


def draw(rng):
    c = _draw(rng)
    while max(work(c)["bytes"], work(c)["flops"] / 100) > _LARGEST or (c["op"] == "experts" and c["E"] * c["d_in"] * c["d_out"] > 6e8):
        c = _draw(rng)
    return c


def _groups(c):
    return -(-c["d_in"] // c["group"])


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    T = c["T"]
    if c["op"] == "route":
        # scores, the bias, then ids (int32) and weights (float32); a few operations per score
        return {"bytes": T * c["E"] * e + 4 * c["E"] * c["bias"] + 8 * T * c["k"], "flops": 4 * T * c["E"]}
    matrix = c["d_out"] * c["d_in"] // 2 + c["d_out"] * _groups(c) * ((2 if c["scales"] == "bf16" else 4) + c["zeros"])
    if c["op"] == "w4":
        return {"bytes": matrix + T * (c["d_in"] + c["d_out"]) * e, "flops": 2 * T * c["d_in"] * c["d_out"]}
    real = T - T // 8 if c["padded"] else T  # tokens that are routed
    rows = real * c["k"]
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** real)  # experts with a row, with even routing
    x_rows, y_rows = (rows, T) if c["combine"] else (real, T * c["k"])
    return {"bytes": int(used * matrix) + (x_rows * c["d_in"] + y_rows * c["d_out"]) * e + T * c["k"] * (8 if c["combine"] else 4),
            "flops": 2 * rows * c["d_in"] * c["d_out"]}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    T, dt = c["T"], _TYPES[c["dtype"]]
    if c["op"] == "route":
        # Router logits of a trained layer: a spread of a few units, some experts liked more than others.
        logits = (1.5 * normal(T, c["E"]) + 0.5 * normal(1, c["E"])).to(dt)
        return dict(case=c, logits=logits, bias=0.05 * normal(c["E"]) if c["bias"] else None)
    n = c["E"] if c["op"] == "experts" else 1
    q = torch.randint(0, 256, (n, c["d_out"], c["d_in"] // 2), device="cuda", generator=g, dtype=torch.uint8)
    shape = (n, c["d_out"], _groups(c))
    scales = ((0.25 * normal(*shape)).exp() / (4.6 * math.sqrt(c["d_in"]))).to(_TYPES[c["scales"]])
    zeros = torch.randint(5, 12, shape, device="cuda", generator=g, dtype=torch.uint8) if c["zeros"] else None
    s = dict(case=c, q=q, scales=scales, zeros=zeros)
    if c["op"] == "experts":
        ids = torch.rand(T, c["E"], device="cuda", generator=g).argsort(1)[:, : c["k"]].to(torch.int32)
        if c["padded"]:  # rows behind the batch's last token name no expert
            ids[T - T // 8:] = -1
        s["ids"] = ids.contiguous()
        s["weights"] = torch.softmax(normal(T, c["k"]), 1) if c["combine"] else None
        s["x"] = normal(T * c["k"] if c["combine"] else T, c["d_in"]).to(dt)
    else:
        s["x"] = normal(T, c["d_in"]).to(dt)
    if own:  # the model's weights, laid out once when it is loaded
        import rank_specialized_amd as rs
        s["store"] = rs.lora_w4_pack(q, scales, zeros, group=c["group"])
    return s


def _dequantize(q, scales, zeros, group):
    """Codes [..., d_out, d_in / 2] (the lower four bits first) as float32 matrices."""
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float()
    d_in = v.shape[-1]
    s = scales.float().repeat_interleave(group, -1)[..., :d_in]
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(group, -1)[..., :d_in]
    return (v - z) * s


def _plain_experts(s):
    c, ids = s["case"], s["ids"].long().flatten()
    k, dt = c["k"], s["x"].dtype
    rows = s["x"] if c["combine"] else s["x"].repeat_interleave(k, 0)
    none = ids < 0
    if ids.numel() <= c["E"]:  # few rows: each with its own matrix
        e = ids.clamp(min=0)
        w = _dequantize(s["q"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e], c["group"])
        v = torch.bmm(w, rows.float().unsqueeze(2)).squeeze(2)
    else:  # rows sorted by expert, every expert's rows padded to the largest count, one batched product
        e = torch.where(none, c["E"], ids)
        counts = torch.bincount(e, minlength=c["E"] + 1)
        order = torch.argsort(e, stable=True)
        first = torch.cumsum(counts, 0) - counts
        place = torch.empty_like(e)
        place[order] = torch.arange(e.numel(), device=e.device) - first[e[order]]
        cap = int(counts[: c["E"]].max())
        w = _dequantize(s["q"], s["scales"], s["zeros"], c["group"])
        slot = torch.where(none, c["E"] * cap, e * cap + place)
        x = torch.zeros(c["E"] * cap + 1, c["d_in"], device=rows.device)
        x[slot] = rows.float()
        v = torch.bmm(x[: c["E"] * cap].view(c["E"], cap, -1), w.transpose(1, 2).contiguous()).flatten(0, 1)
        v = v[slot.clamp(max=c["E"] * cap - 1)]
    v = torch.where(none.unsqueeze(1), 0.0, v)
    if c["combine"]:
        v = (v.view(c["T"], k, -1) * s["weights"].unsqueeze(2)).sum(1)
    return v.to(dt)


def _plain_route(s):
    """In 64 bits: a choice is a comparison of scores that may be close."""
    c = s["case"]
    l = s["logits"].double()
    score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        by = choice.view(c["T"], c["groups"], -1)
        top = by.sort(dim=2, descending=True).values
        of_group = top[:, :, 0] if c["score"] == "softmax" else top[:, :, :2].sum(2)
        best = of_group.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, best, True)
        choice = torch.where(keep.unsqueeze(2), by, -math.inf).flatten(1)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(1, ids)
    return ids.int(), (w / w.sum(1, keepdim=True)).float()


def run(state):
    s, c = state, state["case"]
    if own:
        import rank_specialized_amd as rs
        if c["op"] == "w4":
            return rs.lora_w4_apply(s["store"], s["x"])
        if c["op"] == "experts":
            return rs.lora_w4_apply_experts(s["store"], s["x"], s["ids"], s["weights"])
        return rs.lora_route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"])
    if c["op"] == "w4":
        w = _dequantize(s["q"][0], s["scales"][0], None if s["zeros"] is None else s["zeros"][0], c["group"])
        return (s["x"].float() @ w.t()).to(s["x"].dtype)
    return _plain_experts(s) if c["op"] == "experts" else _plain_route(s)


def _exact_rows(q, s, z, group, x):
    """sum over groups of s (sum of q x - z sum of x), in float64."""
    d_out, half = q.shape
    d_in = 2 * half
    y = torch.zeros(x.shape[0], d_out, dtype=torch.float64, device=x.device)
    lo, hi = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
    s = s.double()
    w = torch.empty(d_out, d_in, dtype=torch.float64, device=x.device)
    w[:, 0::2], w[:, 1::2] = lo, hi
    for g in range(s.shape[1]):
        at = slice(g * group, min(d_in, (g + 1) * group))
        w[:, at] -= 8 if z is None else z[:, g: g + 1].double()
        w[:, at] *= s[:, g: g + 1]
    step = max(1, (1 << 28) // d_out)
    for a in range(0, x.shape[0], step):
        y[a: a + step] = x[a: a + step].double() @ w.t()
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "w4":
        return _exact_rows(s["q"][0], s["scales"][0], None if s["zeros"] is None else s["zeros"][0], c["group"], s["x"])
    if c["op"] == "experts":
        ids = s["ids"].long()
        y = torch.zeros(c["T"], c["k"], c["d_out"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                x = s["x"][t * c["k"] + j] if c["combine"] else s["x"][t]
                y[t, j] = _exact_rows(s["q"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e], c["group"], x)
        if c["combine"]:
            return (y * s["weights"].double().unsqueeze(2)).sum(1)
        return y.flatten(0, 1)
    l = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    b = p if s["bias"] is None else p + s["bias"].double()
    T, E, n = c["T"], c["E"], c["E"] // c["groups"]
    left = b.clone()
    if c["groups"] > 1:
        far = torch.full((T, 1), -math.inf, dtype=torch.float64, device="cuda")
        size = []
        for g in range(c["groups"]):
            part = b[:, g * n: (g + 1) * n]
            size.append(part.amax(1) if c["score"] == "softmax" else part.topk(2, 1).values.sum(1))
        size = torch.stack(size, 1)
        allowed = torch.zeros(T, c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            at = size.max(1, keepdim=True)
            first = (size == at.values).int().argmax(1, keepdim=True)
            allowed.scatter_(1, first, True)
            size.scatter_(1, first, far)
        left[~allowed.repeat_interleave(n, 1)] = -math.inf
    ids, w = [], []
    for _ in range(c["k"]):
        best = left.amax(1, keepdim=True)
        first = (left == best).int().argmax(1, keepdim=True)
        ids.append(first)
        w.append(p.gather(1, first))
        left.scatter_(1, first, -math.inf)
    w = torch.cat(w, 1)
    return torch.cat(ids, 1).int(), w / w.sum(1, keepdim=True)
