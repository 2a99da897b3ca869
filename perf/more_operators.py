"""Measured cases of the 8-bit base layers and of the mixture-of-experts layer.

Three operators, each in two forms: elementary torch operations (``own``
false), and the calls a user makes of this package (``own`` true).

  w8        y[t] = W x[t], W held as 8-bit integers with a scale per output, x[t] rounded to 8-bit
            integers with a scale of its own within the call
  w8-shared several such layers of one input (q, k and v; gate and up): the rows are rounded once
            and every layer takes the integers
  moe       a mixture-of-experts layer for a few tokens, its matrices held as 4-bit codes:
            y[t] = sum_j w[t, j] D_e (act(G_e x[t]) * (U_e x[t])), e = ids[t, j]
"""
import math

import torch

own = False

#: The work (in bytes, or flops / 100 where that is more) that no drawn case exceeds.
_LARGEST = 9.7e9
#: Values of the experts' matrices that no drawn case exceeds (each is a float32 in the plain form).
_MATRICES = 1.9e8


def listed():
    return [
        # One decode token through the smallest projection of the fleet's model (its k or v): latency.
        dict(name="w8-one-token-kv", op="w8", T=1, d_in=3584, d_out=512, d_out_2=0, layers=1, scales="f32", dtype="bf16"),
        # One decode token through its gate or up projection: a stream of codes.
        dict(name="w8-one-token-gate", op="w8", T=1, d_in=3584, d_out=18944, d_out_2=0, layers=1, scales="f32", dtype="bf16"),
        # A decode batch of odd size through its down projection.
        dict(name="w8-batch-down", op="w8", T=23, d_in=18944, d_out=3584, d_out_2=0, layers=1, scales="bf16", dtype="bf16"),
        # Float32 activations.
        dict(name="w8-float32", op="w8", T=5, d_in=4096, d_out=4096, d_out_2=0, layers=1, scales="f32", dtype="f32"),
        # A prefill step, the MLP up projection of the prefill workload.
        dict(name="w8-prefill", op="w8", T=8192, d_in=4096, d_out=14336, d_out_2=0, layers=1, scales="f32", dtype="bf16"),
        # A full decode batch through q, k and v.
        dict(name="w8-shared-batch", op="w8-shared", T=256, d_in=3584, d_out=3584, d_out_2=512, layers=3, scales="bf16", dtype="bf16"),
        # A prompt of odd length through gate and up.
        dict(name="w8-shared-prompt", op="w8-shared", T=1999, d_in=3584, d_out=18944, d_out_2=18944, layers=2, scales="f32", dtype="bf16"),
        # One decode token, eight experts of 64: latency.
        dict(name="moe-one-token", op="moe", T=1, k=8, E=64, d=2048, ffn=1408, group=128, zeros=False, scales="bf16", dtype="bf16",
             act="silu", padded=False),
        # A few float32 tokens of a layer with few, larger experts.
        dict(name="moe-float32", op="moe", T=3, k=2, E=8, d=4096, ffn=1368, group=64, zeros=False, scales="f32", dtype="f32",
             act="gelu_tanh", padded=False),
        # A small batch: most chosen experts have one row.
        dict(name="moe-small-batch", op="moe", T=7, k=4, E=32, d=2048, ffn=1408, group=32, zeros=True, scales="bf16", dtype="bf16",
             act="silu", padded=False),
        # A padded decode batch: every expert has some rows.
        dict(name="moe-batch", op="moe", T=64, k=8, E=64, d=2048, ffn=1408, group=128, zeros=True, scales="bf16", dtype="bf16",
             act="silu", padded=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["w8", "w8", "w8-shared", "moe", "moe", "moe"])
    if op != "moe":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        layers = 1 if op == "w8" else rng.randint(2, 3)
        return dict(op=op, T=_log(rng, 1, 8192), d_in=8 * _log(rng, 8, 2368), d_out=8 * _log(rng, 8, 2368),
                    d_out_2=8 * _log(rng, 8, 2368) if layers > 1 else 0, layers=layers, scales=rng.choice(["f32", "bf16"]), dtype=dtype)
    dtype, scales = rng.choice([("bf16", "bf16")] * 4 + [("bf16", "f32"), ("f32", "f32")])
    E = _log(rng, 4, 160)
    return dict(op=op, T=_log(rng, 1, 64), k=rng.randint(1, min(8, E)), E=E, d=8 * _log(rng, 32, 512), ffn=8 * _log(rng, 16, 512),
                group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, scales=scales, dtype=dtype,
                act=rng.choice(["silu", "gelu_tanh"]), padded=rng.random() < 0.3)


def draw(rng):
    c = _draw(rng)
    while max(work(c)["bytes"], work(c)["flops"] / 100) > _LARGEST or (c["op"] == "moe" and c["E"] * c["d"] * c["ffn"] > _MATRICES):
        c = _draw(rng)
    return c


def _widths(c):
    """Outputs of each of the layers that share an input: the first, and the others."""
    return [c["d_out"]] + [c["d_out_2"]] * (c["layers"] - 1)


def _real(c):
    """Tokens that are routed."""
    return c["T"] - c["T"] // 8 if c["padded"] else c["T"]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    T = c["T"]
    if c["op"] != "moe":
        n = sum(_widths(c))
        return {"bytes": n * c["d_in"] + n * (4 if c["scales"] == "f32" else 2) + T * (c["d_in"] + n) * e, "flops": 2 * T * c["d_in"] * n}
    per = (2 if c["scales"] == "bf16" else 4) + c["zeros"]  # bytes of a group's scale and zero point
    groups = 2 * c["ffn"] * -(-c["d"] // c["group"]) + c["d"] * -(-c["ffn"] // c["group"])
    expert = 3 * c["ffn"] * c["d"] // 2 + groups * per
    used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** _real(c))  # experts with a row, with even routing
    return {"bytes": int(used * expert) + (_real(c) + T) * c["d"] * e + 8 * T * c["k"], "flops": 6 * _real(c) * c["k"] * c["d"] * c["ffn"]}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _w4(g, c, d_in, d_out):
    """Random 4-bit matrices, one per expert, whose products with values of size one are of size one."""
    E = c["E"]
    shape = (E, d_out, -(-d_in // c["group"]))
    q = torch.randint(0, 256, (E, d_out, d_in // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = ((0.25 * _normal(g, *shape)).exp() / (4.6 * math.sqrt(d_in))).to(_TYPES[c["scales"]])
    zeros = torch.randint(5, 12, shape, device="cuda", generator=g, dtype=torch.uint8) if c["zeros"] else None
    return dict(q=q, scales=scales, zeros=zeros)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    T, dt = c["T"], _TYPES[c["dtype"]]
    if c["op"] != "moe":
        s = dict(case=c, layers=[])
        for n in _widths(c):
            # Weights as rounded from a trained layer: a bell of integers, the largest of each output near 127.
            q = (36 * _normal(g, n, c["d_in"])).round_().clamp_(-127, 127).to(torch.int8)
            scales = ((0.25 * _normal(g, n)).exp() / (36 * math.sqrt(c["d_in"]))).to(_TYPES[c["scales"]])
            s["layers"].append(dict(q=q, scales=scales))
        # Activations: a few channels are much larger than the others.
        size = 1 + 12 * (torch.rand(c["d_in"], device="cuda", generator=g) < 0.002).float()
        s["x"] = (_normal(g, T, c["d_in"]) * size).to(dt)
        if own:  # the model's weights, laid out once when it is loaded
            import rank_specialized_amd as rs
            s["stores"] = [rs.lora_w8_pack(w["q"], w["scales"]) for w in s["layers"]]
        return s
    s = dict(case=c, gate=_w4(g, c, c["d"], c["ffn"]), up=_w4(g, c, c["d"], c["ffn"]), down=_w4(g, c, c["ffn"], c["d"]))
    ids = torch.rand(T, c["E"], device="cuda", generator=g).argsort(1)[:, : c["k"]].to(torch.int32)
    ids[_real(c):] = -1  # rows behind the batch's last token name no expert
    s["ids"] = ids.contiguous()
    s["weights"] = torch.softmax(_normal(g, T, c["k"]), 1)
    s["x"] = (1.5 * _normal(g, T, c["d"])).to(dt)
    if own:
        import rank_specialized_amd as rs
        s["stores"] = [rs.lora_w4_pack(m["q"], m["scales"], m["zeros"], group=c["group"]) for m in (s["gate"], s["up"], s["down"])]
    return s


def _plain_w8(s):
    # A row's integers are rounded in 64 bits: a value may lie on the border between two.
    x = s["x"].double()
    top = x.abs().amax(1, keepdim=True)
    codes = torch.round(x * 127 / torch.where(top > 0, top, 1.0)).float()
    sx = (top / 127).float()
    return [((codes @ w["q"].float().t()) * sx * w["scales"].float()).to(s["x"].dtype) for w in s["layers"]]


def _dequantize(m, group, at=slice(None)):
    """Matrices of 4-bit codes [.., d_out, d_in / 2] (the lower four bits first) in float32."""
    q, scales = m["q"][at], m["scales"][at]
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float()
    d_in = v.shape[-1]
    z = 8.0 if m["zeros"] is None else m["zeros"][at].float().repeat_interleave(group, -1)[..., :d_in]
    return (v - z) * scales.float().repeat_interleave(group, -1)[..., :d_in]


def _act(kind, g):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_moe(s):
    c, ids = s["case"], s["ids"].long().flatten()
    group, E, k = c["group"], c["E"], c["k"]
    rows = s["x"].float().repeat_interleave(k, 0)
    none = (ids < 0).unsqueeze(1)
    if ids.numel() <= E:  # few rows: each with its own matrices
        e = ids.clamp(min=0)
        product = lambda m, v: torch.bmm(_dequantize(m, group, e), v.unsqueeze(2)).squeeze(2)  # noqa: E731
        h = _act(c["act"], product(s["gate"], rows)) * product(s["up"], rows)
        v = product(s["down"], h)
    else:  # rows sorted by expert, every expert's rows padded to the largest count, batched products
        e = torch.where(ids < 0, E, ids)
        counts = torch.bincount(e, minlength=E + 1)
        order = torch.argsort(e, stable=True)
        first = torch.cumsum(counts, 0) - counts
        place = torch.empty_like(e)
        place[order] = torch.arange(e.numel(), device=e.device) - first[e[order]]
        cap = int(counts[:E].max())
        slot = torch.where(ids < 0, E * cap, e * cap + place)
        x = torch.zeros(E * cap + 1, c["d"], device=rows.device)
        x[slot] = rows
        x = x[: E * cap].view(E, cap, -1)
        product = lambda m, v: torch.bmm(v, _dequantize(m, group).transpose(1, 2).contiguous())  # noqa: E731
        h = _act(c["act"], product(s["gate"], x)) * product(s["up"], x)
        v = product(s["down"], h).flatten(0, 1)[slot.clamp(max=E * cap - 1)]
    v = torch.where(none, 0.0, v)
    return (v.view(c["T"], k, -1) * s["weights"].unsqueeze(2)).sum(1).to(s["x"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_moe(s) if c["op"] == "moe" else _plain_w8(s)
    import rank_specialized_amd as rs
    if c["op"] == "w8":
        return [rs.lora_w8_apply(s["stores"][0], s["x"])]
    if c["op"] == "w8-shared":
        q, scales = rs.lora_w8_quantize(s["x"])
        return [rs.lora_w8_apply_quantized(w, q, scales, dtype=s["x"].dtype) for w in s["stores"]]
    gate, up, down = s["stores"]
    return rs.lora_w4_moe(gate, up, down, s["x"], s["ids"], s["weights"], act=c["act"])


def _exact_rows(m, e, group, x):
    """x times the transpose of matrix e, in float64, a group of inputs at a time."""
    q, scales = m["q"][e].long(), m["scales"][e].double()
    codes = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    codes[:, 0::2], codes[:, 1::2] = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
    y = torch.zeros(x.shape[0], q.shape[0], dtype=torch.float64, device=x.device)
    for i in range(scales.shape[1]):
        at = slice(i * group, (i + 1) * group)
        zero = 8.0 if m["zeros"] is None else m["zeros"][e][:, i: i + 1].double()
        y += (x[:, at] @ (codes[:, at] - zero).t()) * scales[:, i]
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    x = s["x"].double()
    if c["op"] != "moe":
        top = x.abs().max(dim=1).values
        step = top / 127
        # x / step, from products that 64 bits hold (254 x has 32 bits): the nearest integer, the even one of two.
        twice = 254 * x
        low = torch.floor(127 * x / torch.where(top > 0, top, 1.0)[:, None])
        over = twice - (2 * low + 1) * top[:, None]
        odd = (low % 2).abs() == 1
        codes = low + ((over > 0) | ((over == 0) & odd)).double()
        codes = torch.where(top[:, None] > 0, codes, 0.0)
        return [(codes @ w["q"].double().t()) * step[:, None] * w["scales"].double() for w in s["layers"]]
    ids = s["ids"].long()
    y = torch.zeros(c["T"], c["k"], c["d"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g, u = _exact_rows(s["gate"], e, c["group"], x[t]), _exact_rows(s["up"], e, c["group"], x[t])
        if c["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:  # tanh(v) = 1 - 2 / (exp(2 v) + 1)
            a = g - g / (torch.exp(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) + 1)
        y[t, j] = _exact_rows(s["down"], e, c["group"], a * u)
    return (y * s["weights"].double().unsqueeze(2)).sum(1)
