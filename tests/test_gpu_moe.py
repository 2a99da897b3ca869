"""The mixture-of-experts layer on the GPU against the float64 oracle, whose
bound (oracle/moe_ref.py) covers the float32 sums, the activation, and for bf16
rows h held to 16 bits; y then rounds once, half a step: 2^-8 (bf16) or 2^-24
(float32) of the value."""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, hbits, note
from oracle import apply_ref
from oracle.moe_ref import act_ref, moe_ref
from oracle.w4_ref import route_ref
from oracle.w8_ref import w8_apply_ref
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def experts(seed, n, d_out, d_in, group, zeros, scales):
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (n, d_out, d_in // 2), dtype=np.uint8)
    shape = (n, d_out, -(-d_in // group))
    s = (np.exp(0.3 * rng.normal(size=shape)) / (4.6 * np.sqrt(d_in))).astype(np.float32)
    s = round_to_bf16(s) if scales == "bf16" else s
    return packed, np.asarray(s, np.float32), rng.integers(0, 16, shape).astype(np.uint8) if zeros else None


def pack(m, group, scales, dev):
    packed, s, z = m
    return rs.lora_w4_pack(torch.from_numpy(packed).to(dev), torch.from_numpy(s).to(dev).to(DT[scales]),
                           None if z is None else torch.from_numpy(z).to(dev), group=group)


class Layer:
    def __init__(self, E, d, ffn, group=64, zeros=True, scales="bf16", d_out=None, down=None, seed=1):
        self.group, self.down_kind = group, down or (group, zeros, scales)
        g2, z2, s2 = self.down_kind
        self.gate, self.up = (experts(seed + i, E, ffn, d, group, zeros, scales) for i in (0, 1))
        self.down = experts(seed + 2, E, d_out or d, ffn, g2, z2, s2)
        dev = device()
        self.stores = [pack(self.gate, group, scales, dev), pack(self.up, group, scales, dev), pack(self.down, g2, s2, dev)]

    def __call__(self, x, ids, w, dtype, **kw):
        dev = device()
        return rs.lora_w4_moe(*self.stores, torch.from_numpy(x).to(dev).to(DT[dtype]), torch.from_numpy(ids).to(dev),
                              torch.from_numpy(w).to(dev), **kw)

    def ref(self, x, ids, w, dtype, act="silu"):
        return moe_ref(self.gate, self.up, self.down, self.group, self.down_kind[0], x, ids, w, act, 16 if dtype == "bf16" else None)


def inputs(seed, T, k, E, d, dtype, dup=False):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, d)).astype(np.float32)
    if dup:
        ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    else:
        ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    return (round_to_bf16(x) if dtype == "bf16" else x), np.ascontiguousarray(ids), w


def check(y, ref, bound, dtype):
    y = y.float().cpu().numpy().astype(np.float64)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = half * np.abs(ref) * (1 + 2.0 ** -8) + bound + 1e-30
    worst = float((np.abs(y - ref) / tol).max()) if y.size else 0.0
    assert np.isfinite(y).all() and worst <= 1.0, f"{worst:.3g} of the tolerance"


# T, k, E, d, ffn, group, zeros, scales, dtype, act
CASES = [
    (1, 1, 1, 8, 8, 32, False, "bf16", "bf16", "silu"),
    (1, 8, 16, 264, 136, 128, False, "bf16", "bf16", "silu"),
    (1, 2, 4, 2048, 1408, 128, False, "bf16", "bf16", "silu"),
    (2, 3, 8, 136, 24, 32, True, "bf16", "bf16", "gelu_tanh"),
    (3, 2, 8, 520, 152, 64, True, "f32", "bf16", "silu"),
    (4, 4, 32, 128, 128, 128, True, "bf16", "bf16", "silu"),
    (7, 4, 12, 1032, 200, 32, True, "bf16", "bf16", "silu"),
    (9, 8, 9, 72, 264, 96, False, "f32", "bf16", "gelu_tanh"),
    (16, 2, 3, 136, 72, 64, False, "bf16", "bf16", "silu"),
    (17, 1, 40, 200, 40, 32, False, "bf16", "bf16", "gelu_tanh"),
    (33, 5, 6, 264, 136, 128, True, "bf16", "bf16", "silu"),
    (64, 4, 5, 136, 72, 32, True, "f32", "bf16", "silu"),
    (64, 8, 64, 64, 40, 64, False, "bf16", "bf16", "silu"),
    (64, 32, 33, 40, 24, 32, True, "bf16", "bf16", "silu"),
    (33, 8, 64, 136, 1032, 128, True, "bf16", "bf16", "silu"),
    (2, 2, 5, 136, 2056, 32, True, "f32", "bf16", "silu"),
    (1, 1, 3, 72, 2048, 128, False, "bf16", "bf16", "gelu_tanh"),
    (1, 1, 1, 8, 8, 32, True, "f32", "f32", "gelu_tanh"),
    (1, 4, 8, 520, 136, 64, False, "f32", "f32", "silu"),
    (3, 2, 8, 1032, 344, 64, False, "f32", "f32", "gelu_tanh"),
    (12, 3, 4, 264, 72, 32, True, "bf16", "f32", "silu"),
    (16, 2, 32, 136, 520, 128, False, "f32", "f32", "silu"),
    (3, 1, 4, 72, 2000, 64, True, "bf16", "f32", "silu"),
    (40, 2, 3, 136, 200, 128, True, "bf16", "f32", "silu"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_layer(case):
    T, k, E, d, ffn, group, zeros, scales, dtype, act = case
    note(f"moe {case}")
    layer = Layer(E, d, ffn, group, zeros, scales)
    a = inputs(3, T, k, E, d, dtype)
    check(layer(*a, dtype, act=act), *layer.ref(*a, dtype, act), dtype)


@pytest.mark.parametrize("T,k,E", [(5, 4, 3), (33, 6, 4), (64, 32, 2), (3, 8, 300)])
def test_repeated_and_absent_experts(T, k, E):
    """An expert twice in a token, ids outside the range, tokens without any."""
    layer = Layer(E, 136, 40)
    x, ids, w = inputs(4, T, k, E, 136, "bf16", dup=True)
    ids[0] = [-1, E, 2**31 - 1, -(2**31)][: min(k, 4)] + [-5] * max(0, k - 4)
    w[0, 0] = np.nan  # of no expert: not read into the sum
    y = layer(x, ids, w, "bf16")
    assert (y[0] == 0).all()
    w[0, 0] = 0
    check(y, *layer.ref(x, ids, w, "bf16"), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_tokens_on_one_expert(dtype):
    layer = Layer(7, 264, 72)
    x, _, w = inputs(5, 64, 1, 7, 264, dtype)
    ids = np.full((64, 1), 5, np.int32)
    check(layer(x, ids, w, dtype), *layer.ref(x, ids, w, dtype), dtype)


# The largest rows of x that LDS does not hold at once, and of h that it does.
@pytest.mark.parametrize("T,d,ffn,dtype", [(64, 8200, 24, "f32"), (16, 8200, 24, "bf16"), (64, 24, 16384, "f32"), (64, 24, 16376, "bf16"),
                                           (2, 24, 8200, "f32")])
def test_long_rows(T, d, ffn, dtype):
    layer = Layer(2, d, ffn, 128, False)
    a = inputs(6, T, 2, 2, d, dtype)
    check(layer(*a, dtype), *layer.ref(*a, dtype), dtype)


def test_down_of_another_kind_and_width():
    layer = Layer(4, 200, 104, 32, True, "f32", d_out=72, down=(128, False, "bf16"))
    a = inputs(7, 6, 3, 4, 200, "bf16")
    y = layer(*a, "bf16")
    assert y.shape == (6, 72)
    check(y, *layer.ref(*a, "bf16"), "bf16")


def test_float32_rows_are_taken_in_whole():
    """One input and one feature matter: y is w D act(G x) (U x) with x's last
    bits in it."""
    dev = device()
    packed = np.full((1, 8, 4), 0x88, np.uint8)  # all codes 8: zeros
    one = packed.copy()
    one[0, 0, 0] = 0x89  # W[0, 0] = 1
    s = np.ones((1, 8, 1), np.float32)
    stores = [pack((one, s, None), 32, "f32", dev) for _ in range(3)]
    x = np.zeros((5, 8), np.float32)
    x[:, 0] = np.array([1 + 2.0 ** -23, 3 - 2.0 ** -22, 1e-3, 7.7777777, -2.3456789], np.float32)
    y = rs.lora_w4_moe(*stores, torch.from_numpy(x).to(dev), torch.zeros(5, 1, dtype=torch.int32, device=dev),
                       torch.ones(5, 1, device=dev)).cpu().numpy()
    v = x[:, 0].astype(np.float64)
    want = act_ref("silu", v) * v
    # act: exp (2 steps of 2^-24 by its error bound, and its argument is exact), 1 + exp, the quotient, times u: 6 in all
    assert (np.abs(y[:, 0] - want) <= 6 * 2.0 ** -24 * np.abs(want)).all()
    assert not y[:, 1:].any()


@pytest.mark.parametrize("T", [1, 20])
def test_strides_and_neighbours(T):
    dev = device()
    layer = Layer(4, 200, 72, d_out=136)
    x, ids, w = inputs(8, T, 2, 4, 200, "bf16")
    base = layer(x, ids, w, "bf16")
    wide = torch.full((T, 224), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 16: 216] = torch.from_numpy(x).to(dev).to(torch.bfloat16)
    yb = torch.full((T + 2, 160), 7.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w4_moe(*layer.stores, wide[:, 16: 216], torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), yb[:T, 8: 144])
    assert np.array_equal(hbits(yb[:T, 8: 144].contiguous()), hbits(base))
    yb[:T, 8: 144] = 7.0
    assert (yb == 7.0).all()


@pytest.mark.parametrize("T", [2, 24])
def test_values_that_are_no_numbers(T):
    """An infinity or a NaN in a row of x, or as a weight, reaches its own row
    alone; a token without experts is zeros whatever x holds."""
    layer = Layer(3, 136, 72)
    x, ids, w = inputs(9, T, 2, 3, 136, "bf16")
    ids[T - 1] = -1
    base = layer(x, ids, w, "bf16")
    assert (base[T - 1] == 0).all()
    for bad in (np.inf, -np.inf, np.nan):
        z = x.copy()
        z[0, 7] = bad
        z[T - 1, 3] = bad
        y = layer(z, ids, w, "bf16")
        assert not torch.isfinite(y[0]).any()
        assert np.array_equal(hbits(y[1:]), hbits(base[1:]))
        v = w.copy()
        v[0, 1] = bad
        y = layer(x, ids, v, "bf16")
        assert not torch.isfinite(y[0]).any()
        assert np.array_equal(hbits(y[1:]), hbits(base[1:]))


def test_no_tokens():
    dev = device()
    layer = Layer(2, 40, 24)
    for dt in DT.values():
        y = rs.lora_w4_moe(*layer.stores, torch.empty(0, 40, dtype=dt, device=dev),
                           torch.empty(0, 2, dtype=torch.int32, device=dev), torch.empty(0, 2, device=dev))
        assert y.shape == (0, 40)


def test_repeats_bit_for_bit():
    layer = Layer(8, 520, 264, 32)
    a = inputs(10, 30, 4, 8, 520, "bf16")
    first = hbits(layer(*a, "bf16"))
    for _ in range(5):
        assert np.array_equal(hbits(layer(*a, "bf16")), first)


@pytest.mark.parametrize("T", [1, 40])
def test_graph_replays(T):
    """A captured layer, replayed with new tokens and choices among eager calls."""
    dev = device()
    E, d, k = 6, 264, 3
    layer = Layer(E, d, 136)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=dev)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device=dev), torch.zeros(T, k, device=dev)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        rs.lora_w4_moe(*layer.stores, x, ids, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = rs.lora_w4_moe(*layer.stores, x, ids, w)
    for i in range(5):
        a = inputs(20 + i, T, k, E, d, "bf16", dup=i % 2 == 1)
        for dst, src in zip((x, ids, w), a):
            dst.copy_(torch.from_numpy(src))
        g.replay()
        eager = rs.lora_w4_moe(*layer.stores, x, ids, w)
        torch.cuda.synchronize()
        assert np.array_equal(hbits(y), hbits(eager))
        check(y, *layer.ref(*a, "bf16"), "bf16")


def test_streams_at_once():
    dev = device()
    layer = Layer(8, 264, 136)
    cases = [inputs(30 + i, T, 3, 8, 264, "bf16") for i, T in enumerate((1, 9, 64))]
    args = [[torch.from_numpy(x).to(dev).to(torch.bfloat16), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev)]
            for x, ids, w in cases]
    torch.cuda.synchronize()
    out = {}
    for _ in range(3):
        for i, a in enumerate(args):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                out[i] = rs.lora_w4_moe(*layer.stores, *a)
            for t in a:
                t.record_stream(s)
    torch.cuda.synchronize()
    for i, a in enumerate(cases):
        check(out[i], *layer.ref(*a, "bf16"), "bf16")


def test_workspace_checked_and_reused():
    dev = device()
    layer = Layer(8, 264, 136)
    need = rs.lora_w4_moe_workspace_bytes(*layer.stores, torch.bfloat16, 33, 3)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    for T in (33, 1, 20, 33):
        a = inputs(40 + T, T, 3, 8, 264, "bf16", dup=True)
        check(layer(*a, "bf16", ws=ws), *layer.ref(*a, "bf16"), "bf16")
    with pytest.raises(rs.LoraError):
        layer(*inputs(1, 33, 3, 8, 264, "bf16"), "bf16", ws=ws[:-16])


@pytest.mark.parametrize("T", [1, 19])
def test_a_block_of_a_decode_step(T):
    """As they are used in turn: an 8-bit projection with its adapters' branch,
    the router on what it gives, and the experts' layer, each checked on what
    the one before has left."""
    dev = device()
    rng = np.random.default_rng(50)
    d, E, k, ranks = 264, 8, 3, [5, 16]
    w8 = rng.integers(-127, 128, (d, d)).astype(np.int8)
    sw = (rng.uniform(0.5, 2, d) / (74 * np.sqrt(d))).astype(np.float32)
    A = [round_to_bf16((rng.normal(size=(r, d)) / 16).astype(np.float32)) for r in ranks]
    B = [round_to_bf16((rng.normal(size=(d, r)) / 4).astype(np.float32)) for r in ranks]
    ids = rng.integers(-1, 2, T).astype(np.int32)
    router = (rng.normal(size=(E, d)) / 8).astype(np.float32)
    x = round_to_bf16(rng.normal(size=(T, d)).astype(np.float32))
    layer = Layer(E, d, 136)

    def put(a, dt=torch.bfloat16):
        return torch.from_numpy(a).to(dev).to(dt)

    adapters = rs.lora_pack_retained([put(a) for a in A], [put(b) for b in B], [0.5, 1.5])
    h = rs.lora_w8_apply(rs.lora_w8_pack(put(w8, torch.int8), put(sw, torch.float32)), put(x))
    rs.lora_apply_batched(adapters, put(x), h, ids=put(ids, torch.int32))
    logits = h.float() @ put(router, torch.float32).t()
    chosen, weights = rs.lora_route(logits, k)
    y = rs.lora_w4_moe(*layer.stores, h, chosen, weights)

    hh = h.float().cpu().numpy()
    ref = w8_apply_ref(x, w8, sw) + apply_ref(x, ids, A, B, [0.5, 1.5])
    # the base rounds, and the sum with the branch does: half a step each, of values up to the largest of both
    big = np.abs(w8_apply_ref(x, w8, sw)) + np.abs(ref)
    assert (np.abs(hh - ref) <= 2.0 ** -8 * big * 1.01 + 1e-4).all()
    ri, rw = route_ref(logits.cpu().numpy(), k)
    assert np.array_equal(chosen.cpu().numpy(), ri) and np.allclose(weights.cpu().numpy(), rw, rtol=1e-5)
    check(y, *layer.ref(hh, chosen.cpu().numpy(), weights.cpu().numpy(), "bf16"), "bf16")


def test_two_graphs_share_a_workspace():
    """Layers of different sizes captured over one workspace and replayed in turn,
    with eager calls over it in between."""
    dev = device()
    k, layers = 2, [Layer(5, 200, 136), Layer(4, 72, 2056, 128, False, seed=9)]
    sizes = [(20, 200), (2, 72)]
    args = []
    for i, ((T, d), layer) in enumerate(zip(sizes, layers)):
        x, ids, w = inputs(60 + i, T, k, 4, d, "bf16")
        args.append((torch.from_numpy(x).to(dev).to(torch.bfloat16), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev)))
    need = max(rs.lora_w4_moe_workspace_bytes(*layer.stores, torch.bfloat16, a[0].shape[0], k) for layer, a in zip(layers, args))
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=dev)
    want = [hbits(rs.lora_w4_moe(*layer.stores, *a)) for layer, a in zip(layers, args)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for layer, a in zip(layers, args):
            rs.lora_w4_moe(*layer.stores, *a, ws=ws)
    torch.cuda.synchronize()
    graphs, ys = [], []
    for layer, a in zip(layers, args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(rs.lora_w4_moe(*layer.stores, *a, ws=ws))
        graphs.append(g)
    for turn in range(4):
        for i in (turn % 2, 1 - turn % 2, turn % 2):
            ys[i].fill_(7.0)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert np.array_equal(hbits(ys[i]), want[i])
            assert np.array_equal(hbits(rs.lora_w4_moe(*layers[1 - i].stores, *args[1 - i], ws=ws)), want[1 - i])
