"""The 8-bit base products on the GPU against the oracle.

Codes have to be the oracle's.  A product's sum is an exact integer, and what
follows it is one float32 conversion, two float32 products and y's rounding,
which numpy's float32 does the same way: y has to have the oracle's bits.
"""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, hbits, note
from oracle import apply_ref
from oracle.w8_ref import w8_product_ref, w8_quantize_ref
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def acts(seed, rows, d, dtype):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, d)) * np.where(rng.random(d) < 0.02, 15, 1)
    x = x.astype(np.float32)
    return round_to_bf16(x) if dtype == "bf16" else x


def weights(seed, d_out, d_in):
    rng = np.random.default_rng(seed)
    return (rng.integers(-128, 128, (d_out, d_in)).astype(np.int8),
            (np.exp(0.3 * rng.normal(size=d_out)) / (70 * np.sqrt(d_in))).astype(np.float32))


def pack(w, sw, dev):
    return rs.lora_w8_pack(torch.from_numpy(w).to(dev), torch.from_numpy(sw).to(dev))


def up(x, dtype, dev):
    return torch.from_numpy(x).to(dev).to(DT[dtype])


def want(q, s, w, sw, dtype):
    """The float32 steps behind the exact sum, as a tensor of `dtype`."""
    total = (q.astype(np.float64) @ w.astype(np.float64).T).astype(np.float32)  # below 2^53: exact before it rounds
    with np.errstate(invalid="ignore", over="ignore"):
        y = total * np.asarray(s, np.float32)[:, None] * sw[None, :]
    assert y.dtype == np.float32
    return torch.from_numpy(y).to(DT[dtype])


def want_of(x, w, sw, dtype):
    q, s = w8_quantize_ref(x)
    return want(q, s, w, sw, dtype)


def same(y, ref):
    a, b = hbits(y), hbits(ref)
    assert a.shape == b.shape
    assert np.array_equal(a, b), f"{int((a != b).sum())} of {a.size} differ"


# ------------------------------------------------------------ rounding
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (5, 1000), (1, 18944), (2, 40008), (1100, 520), (1030, 4104), (9, 512)])
def test_quantize(T, d, dtype):
    dev = device()
    note(f"w8 quantize {T} {d} {dtype}")
    x = acts(1, T, d, dtype)
    q, s = rs.lora_w8_quantize(up(x, dtype, dev))
    rq, rs_ = w8_quantize_ref(x)
    assert q.shape == (T, d) and np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs_.astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_borders(dtype):
    """Values on the border between two codes, next to it, and rows of the
    smallest and largest numbers."""
    dev = device()
    rows = [np.arange(-256, 256) / 2.0, (np.arange(512) % 255 - 127.0) / 2.0, np.zeros(512), np.full(512, -0.0)]
    rows[0][0] = 254.0
    rows[1][0] = 127.0 * 0.9921875  # the row's largest; borders at odd multiples of 127 / 256
    rng = np.random.default_rng(2)
    for a in (1e-45, 3e-39, 1.2e-38, 1e-30, 3e38):
        rows.append(a * rng.uniform(-1, 1, 512))
    rows.append(np.where(rng.random(512) < 0.5, 1.0, -1.0))
    for _ in range(6):  # borders (k + 1/2) a / 127 rounded to float32, and the float32 on each side
        a = np.float32(rng.uniform(0.5, 2))
        b = ((np.arange(127) + 0.5) * float(a) / 127).astype(np.float32)
        r = np.concatenate([b, np.nextafter(b, np.float32(9)), np.nextafter(b, np.float32(0)), -b, [a, -a, 0, a / 2]])
        rows.append(np.resize(r, 512))
    x = np.array(rows).astype(np.float32)
    if dtype == "bf16":
        x = round_to_bf16(x)
    q, s = rs.lora_w8_quantize(up(x, dtype, dev))
    rq, rs_ = w8_quantize_ref(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs_.astype(np.float32))
    # the few rows of a decode step are rounded by another kernel: through the identity, y is s q
    w, one = np.eye(512, dtype=np.int8), np.ones(512, np.float32)
    st = pack(w, one, dev)
    for t in range(x.shape[0]):
        same(rs.lora_w8_apply(st, up(x[t: t + 1], dtype, dev)), want(rq[t: t + 1], rs_[t: t + 1], w, one, dtype))


def test_quantize_outputs_and_neighbours():
    """Rows of a wider buffer whose other columns are NaN; codes into a slice
    of a larger tensor: what is around them keeps its values."""
    dev = device()
    T, d = 37, 104
    x = acts(3, T, d, "bf16")
    wide = torch.full((T, d + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8: 8 + d] = up(x, "bf16", dev)
    big = torch.full((T + 2, 160), 99, dtype=torch.int8, device=dev)
    s = torch.full((T,), -5.0, device=dev)
    q, s2 = rs.lora_w8_quantize(wide[:, 8: 8 + d], big[1: T + 1, 16: 16 + d], s)
    assert s2 is s and np.array_equal(q.cpu().numpy(), w8_quantize_ref(x)[0])
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[1: T + 1, 16: 16 + d] = False
    assert (big[keep] == 99).all()


# ------------------------------------------------------------ products
# T, d_in, d_out: every form of the kernels, ends inside tiles, blocks and stages
SIZES = [
    (1, 8, 8), (1, 64, 64), (1, 72, 40), (1, 3584, 512), (1, 20480, 72), (1, 20488, 24), (1, 1032, 12296), (1, 264, 40008),
    (2, 1000, 136), (3, 2056, 4104), (4, 512, 264), (4, 5120, 64), (4, 5128, 64), (5, 136, 520), (8, 1000, 136), (16, 520, 72), (12, 1032, 8264), (11, 1024, 33000), (13, 4104, 72),
    (16, 648, 8200), (16, 1000, 33000), (16, 1544, 33000), (17, 1032, 200), (30, 3000, 8264), (32, 520, 33000), (33, 776, 136), (64, 2056, 328), (40, 264, 4104), (256, 264, 3592), (200, 520, 3592), (90, 520, 4104), (120, 200, 8200), (70, 72, 1096), (200, 1152, 520),
    (256, 136, 264), (256, 200, 14344), (257, 64, 64), (600, 72, 7176), (700, 264, 16392), (300, 200, 328), (513, 1000, 264), (700, 2056, 72), (1030, 128, 1032),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_in,d_out", SIZES)
def test_apply(T, d_in, d_out, dtype):
    dev = device()
    note(f"w8 apply {T} {d_in} {d_out} {dtype}")
    w, sw = weights(4, d_out, d_in)
    st = pack(w, sw, dev)
    x = acts(5, T, d_in, dtype)
    y = rs.lora_w8_apply(st, up(x, dtype, dev))
    q, s = w8_quantize_ref(x)
    ref = want(q, s, w, sw, dtype)
    same(y, ref)
    # the oracle's own value: four float32 roundings and y's
    exact = w8_product_ref(q, s, w, sw)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert (np.abs(y.float().cpu().numpy() - exact) <= (half + 4.01 * 2.0 ** -24) * np.abs(exact)).all()
    dq, ds = rs.lora_w8_quantize(up(x, dtype, dev))
    same(rs.lora_w8_apply_quantized(st, dq, ds, dtype=DT[dtype]), ref)


@pytest.mark.parametrize("T", [1, 3, 20, 90, 270])
def test_largest_sums(T):
    """Codes of -128 on both sides at the largest d_in: sums up to 2^31 - 2^17."""
    dev = device()
    d_in, d_out = 131064, 16
    w, sw = np.full((d_out, d_in), -128, np.int8), np.full(d_out, 2.0 ** -20, np.float32)
    w[1] = 127
    w[2, ::2] = 127
    q = np.full((T, d_in), -128, np.int8)
    q[-1, 1::3] = 127
    buf = torch.zeros(T, d_in + 8, dtype=torch.int8, device=dev)
    buf[:, :d_in] = torch.from_numpy(q).to(dev)
    s = np.full(T, 0.5, np.float32)
    y = rs.lora_w8_apply_quantized(pack(w, sw, dev), buf[:, :d_in], torch.from_numpy(s).to(dev), dtype=torch.float32)
    same(y, want(q, s, w, sw, "f32"))


@pytest.mark.parametrize("T", [1, 4, 20, 100, 300])
def test_strides_and_neighbours(T):
    """x, q and y as slices of wider buffers; x's other columns are NaN, the
    codes behind d_in anything; y's other columns and the rows behind the last
    one keep their values."""
    dev = device()
    d_in, d_out = 1000, 264
    w, sw = weights(6, d_out, d_in)
    st = pack(w, sw, dev)
    x = acts(7, T, d_in, "bf16")
    ref = want_of(x, w, sw, "bf16")
    wide = torch.full((T, d_in + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8: 8 + d_in] = up(x, "bf16", dev)
    yb = torch.full((T + 3, d_out + 32), 7.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w8_apply(st, wide[:, 8: 8 + d_in], yb[:T, 16: 16 + d_out])
    same(yb[:T, 16: 16 + d_out].contiguous(), ref)
    q = torch.full((T, 1040), 77, dtype=torch.int8, device=dev)
    _, s = rs.lora_w8_quantize(up(x, "bf16", dev), q[:, 16: 16 + d_in])
    y2 = torch.full_like(yb, 7.0)
    rs.lora_w8_apply_quantized(st, q[:, 16: 16 + d_in], s, y2[:T, 16: 16 + d_out])
    same(y2, yb)
    yb[:T, 16: 16 + d_out] = 7.0
    assert (yb == 7.0).all()


@pytest.mark.parametrize("T", [2, 12, 48, 300])
def test_rows_without_numbers(T):
    """An infinity or a NaN makes its own row's outputs NaN, a row of zeros
    gives zeros, and the others do not change."""
    dev = device()
    d_in, d_out = 520, 136
    w, sw = weights(8, d_out, d_in)
    st = pack(w, sw, dev)
    x = acts(9, T, d_in, "bf16")
    x[-1] = 0
    base = rs.lora_w8_apply(st, up(x, "bf16", dev))
    assert (base[-1] == 0).all() and torch.isfinite(base).all()
    for bad in (np.inf, -np.inf, np.nan):
        z = x.copy()
        z[0, 515] = bad
        y = rs.lora_w8_apply(st, up(z, "bf16", dev))
        assert torch.isnan(y[0]).all()
        same(y[1:], base[1:])
        q, s = rs.lora_w8_quantize(up(z, "bf16", dev))
        assert torch.isnan(s[0]) and (q[0] == 0).all()
        assert torch.isnan(rs.lora_w8_apply_quantized(st, q, s)[0]).all()


def test_bf16_scales_and_a_store_of_rounded_weights():
    """lora_w8_quantize also makes a store: a matrix's rows are its outputs."""
    dev = device()
    W = acts(10, 200, 328, "f32") / 20
    q, s = rs.lora_w8_quantize(torch.from_numpy(W).to(dev))
    sb = s.to(torch.bfloat16)
    st = rs.lora_w8_pack(q, sb)
    x = acts(11, 6, 328, "bf16")
    same(rs.lora_w8_apply(st, up(x, "bf16", dev)), want_of(x, w8_quantize_ref(W)[0], sb.float().cpu().numpy(), "bf16"))


def hbits_t(t):
    return t.contiguous().view(torch.int16)


def test_offsets_past_31_bits():
    """The last rows of a call with 2^31 bytes of codes of x, and the last
    outputs of a store of as many, are those of small calls."""
    dev = device()
    g = torch.Generator(device=dev).manual_seed(11)
    d_in, T = 4096, (1 << 19) + 300
    w = rs.lora_w8_pack(torch.randint(-127, 128, (264, d_in), dtype=torch.int8, device=dev, generator=g), torch.rand(264, device=dev, generator=g))
    x = torch.empty(T, d_in, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    y = rs.lora_w8_apply(w, x)
    assert torch.equal(hbits_t(y[-300:]), hbits_t(rs.lora_w8_apply(w, x[-300:])))
    assert torch.equal(hbits_t(y[-9:]), hbits_t(rs.lora_w8_apply(w, x[-9:])))
    del x, y
    d_in, d_out = 65536, 32768 + 200
    q, s = torch.randint(-127, 128, (d_out, d_in), dtype=torch.int8, device=dev, generator=g), torch.rand(d_out, device=dev, generator=g)
    whole, last = rs.lora_w8_pack(q, s), rs.lora_w8_pack(q[-200:], s[-200:])
    for rows in (1, 9, 300):
        x = torch.empty(rows, d_in, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        assert torch.equal(hbits_t(rs.lora_w8_apply(whole, x)[:, -200:]), hbits_t(rs.lora_w8_apply(last, x)))


def test_no_rows():
    dev = device()
    st = pack(*weights(12, 24, 40), dev)
    for dt in DT.values():
        x = torch.empty(0, 40, dtype=dt, device=dev)
        assert rs.lora_w8_apply(st, x).shape == (0, 24)
        q, s = rs.lora_w8_quantize(x)
        assert q.shape == (0, 40) and rs.lora_w8_apply_quantized(st, q, s, dtype=dt).dtype == dt


@pytest.mark.parametrize("T", [1, 16, 64, 300])
def test_graph_replays(T):
    """A captured call, replayed with new inputs among eager work."""
    dev = device()
    d_in, d_out = 1032, 520
    w, sw = weights(13, d_out, d_in)
    st = pack(w, sw, dev)
    x = torch.zeros(T, d_in, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        rs.lora_w8_apply(st, x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = rs.lora_w8_apply(st, x)
        q, s = rs.lora_w8_quantize(x)
        y2 = rs.lora_w8_apply_quantized(st, q, s)
    for i in range(4):
        v = acts(20 + i, T, d_in, "bf16")
        x.copy_(up(v, "bf16", dev))
        g.replay()
        eager = rs.lora_w8_apply(st, x)
        torch.cuda.synchronize()
        same(y, eager)
        same(y2, eager)
        same(eager, want_of(v, w, sw, "bf16"))


def test_streams_at_once():
    """Calls in flight together on two streams, each with its own workspace."""
    dev = device()
    w, sw = weights(14, 776, 2056)
    st = pack(w, sw, dev)
    xs = [acts(30 + i, T, 2056, "bf16") for i, T in enumerate((1, 40, 300, 16))]
    dx = [up(x, "bf16", dev) for x in xs]
    torch.cuda.synchronize()
    out = {}
    for rep in range(3):
        for i, x in enumerate(dx):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                out[i] = rs.lora_w8_apply(st, x)
            x.record_stream(s)
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        same(out[i], want_of(x, w, sw, "bf16"))


def test_workspace_checked_and_reused():
    dev = device()
    w, sw = weights(15, 136, 520)
    st = pack(w, sw, dev)
    need = rs.lora_w8_workspace_bytes(st, 300)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    for T in (300, 20, 300):
        x = acts(16, T, 520, "bf16")
        same(rs.lora_w8_apply(st, up(x, "bf16", dev), ws=ws), want_of(x, w, sw, "bf16"))
    with pytest.raises(rs.LoraError):
        rs.lora_w8_apply(st, torch.zeros(300, 520, dtype=torch.bfloat16, device=dev), ws=ws[:-16])


def test_with_adapters():
    """The base layer, then the adapters' branch on top of it."""
    dev = device()
    rng = np.random.default_rng(17)
    T, d_in, d_out, ranks = 21, 256, 136, [4, 0, 9]
    w, sw = weights(18, d_out, d_in)
    x = acts(19, T, d_in, "f32")
    A = [(rng.normal(size=(r, d_in)) / 16).astype(np.float32) for r in ranks]
    B = [rng.normal(size=(d_out, r)).astype(np.float32) for r in ranks]
    ids = rng.integers(-1, 3, T).astype(np.int32)
    store = rs.lora_pack_retained([up(a, "f32", dev) for a in A], [up(b, "f32", dev) for b in B], [0.5, 1.0, 2.0])
    y = rs.lora_w8_apply(pack(w, sw, dev), up(x, "f32", dev))
    base = y.cpu().numpy().astype(np.float64)
    rs.lora_apply_batched(store, up(x, "f32", dev), y, ids=torch.from_numpy(ids).to(dev))
    ref = base + apply_ref(x, ids, A, B, [0.5, 1.0, 2.0])
    assert np.abs(y.cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()
