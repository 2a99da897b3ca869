"""The 4-bit base products on the GPU against the float64 oracle.

Tolerance of a value.  Every product (32 + q) x or (q - z) x is exact in
float32 (a bf16 value, or a bf16 part of a float32 one, times an integer below
64).  A product then passes through at most `gran` + 2 additions inside its
group of `gran` <= 128 inputs, one scaling, and the additions of the groups
and of the waves: gran + groups + 32 roundings in all, each at most 2^-23 of
the magnitudes added up (a matrix core may truncate).  Those are bounded by
sum |s| (32 + q + 32 + z) |x| (the products and the correction, in absolute
value).  A weighted sum multiplies each of its rows' bounds by the weight and
adds k + 2 roundings.  y then rounds once: half a step, 2^-8 (bf16) or 2^-24
(float32) of the value.  The f16 form holds x to 2^-25 of its row's largest
value: x of below 2^-14 of that is rounded by at most 2^-39 of it; d_in of
those, at |s| 15 each, are inside the same bound (2^-23 of the largest alone).
"""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, hbits, note
from oracle.w4_ref import experts_ref, w4_apply_ref, w4_magnitude_ref
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, n, d_out, d_in, group, zeros, scales):
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (n, d_out, d_in // 2), dtype=np.uint8)
    shape = (n, d_out, -(-d_in // group))
    s = np.exp(0.3 * rng.normal(size=shape)) / (4.6 * np.sqrt(d_in))
    s = round_to_bf16(s.astype(np.float32)) if scales == "bf16" else s.astype(np.float32)
    z = rng.integers(0, 16, shape).astype(np.uint8) if zeros else None
    return packed, np.asarray(s, np.float32), z


def pack(packed, s, z, group, scales, dev):
    return rs.lora_w4_pack(torch.from_numpy(packed).to(dev), torch.from_numpy(s).to(dev).to(DT[scales]),
                           None if z is None else torch.from_numpy(z).to(dev), group=group)


def acts(seed, rows, d, dtype):
    x = np.random.default_rng(seed).normal(size=(rows, d)).astype(np.float32)
    return round_to_bf16(x) if dtype == "bf16" else x


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def tolerance(ref, mag, d_in, group, dtype, k=0):
    gran = min(128, group)
    steps = gran + -(-d_in // gran) + 32 + (k + 2 if k else 0)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return half * np.abs(ref) * (1 + 2.0 ** -8) + steps * 2.0 ** -23 * mag + 1e-30


def assert_close(y, ref, mag, *a, **kw):
    err, tol = np.abs(host(y) - ref), tolerance(ref, mag, *a, **kw)
    worst = float((err / tol).max()) if err.size else 0.0
    assert np.isfinite(host(y)).all() and worst <= 1.0, f"{worst:.3g} of the tolerance"


# T, d_in, d_out, group, zeros, scales, dtype
DENSE = [
    (1, 128, 16, 128, False, "bf16", "bf16"),
    (1, 8, 8, 32, False, "bf16", "bf16"),
    (1, 136, 24, 64, True, "bf16", "bf16"),
    (1, 3584, 512, 128, False, "bf16", "bf16"),
    (2, 264, 40, 32, True, "f32", "bf16"),
    (3, 1000, 72, 96, True, "bf16", "bf16"),
    (15, 1032, 200, 128, False, "f32", "bf16"),
    (16, 512, 128, 64, False, "bf16", "bf16"),
    (17, 520, 136, 64, True, "bf16", "bf16"),
    (33, 768, 264, 256, True, "bf16", "bf16"),
    (70, 2056, 248, 32, False, "bf16", "bf16"),
    (127, 384, 520, 128, True, "bf16", "bf16"),
    (200, 1152, 1032, 128, False, "bf16", "bf16"),
    (513, 776, 328, 64, True, "bf16", "bf16"),
    (1030, 512, 776, 32, True, "f32", "bf16"),
    (2049, 264, 1096, 128, False, "bf16", "bf16"),
    (16, 2056, 136, 64, True, "bf16", "bf16"),
    (13, 4104, 72, 32, True, "bf16", "bf16"),
    (16, 4096, 40, 128, False, "f32", "bf16"),
    (30, 4104, 136, 64, True, "bf16", "bf16"),
    (64, 3000, 72, 128, False, "bf16", "bf16"),
    (800, 1032, 64, 32, True, "bf16", "bf16"),
    (5, 2056, 40, 64, True, "f32", "f32"),
    (9, 2056, 136, 128, False, "bf16", "f32"),
    (40, 1032, 24, 32, True, "f32", "f32"),
    (1, 8, 8, 32, True, "f32", "f32"),
    (1, 1040, 136, 128, False, "f32", "f32"),
    (5, 520, 72, 32, True, "bf16", "f32"),
    (19, 904, 200, 64, False, "bf16", "f32"),
    (150, 512, 136, 128, True, "f32", "f32"),
]


@pytest.mark.parametrize("case", DENSE, ids=lambda c: "-".join(map(str, c)))
def test_dense(case):
    T, d_in, d_out, group, zeros, scales, dtype = case
    dev = device()
    note(f"w4 dense {case}")
    packed, s, z = make(1, 1, d_out, d_in, group, zeros, scales)
    st = pack(packed, s, z, group, scales, dev)
    x = acts(2, T, d_in, dtype)
    y = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).to(DT[dtype]))
    a = (packed[0], s[0], None if z is None else z[0], group, x)
    assert_close(y, w4_apply_ref(*a), w4_magnitude_ref(*a), d_in, group, dtype)


@pytest.mark.parametrize("T", [1, 9, 40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_integers_are_exact(T, dtype):
    """Integer x, scales of powers of two: every sum is exact, so y is the
    oracle's value rounded once, bit for bit."""
    dev = device()
    rng = np.random.default_rng(3)
    d_in, d_out, group = 648, 328, 32
    packed, s, z = make(4, 1, d_out, d_in, group, True, "bf16")
    s = np.exp2(rng.integers(-2, 2, s.shape)).astype(np.float32)
    x = rng.integers(-4, 5, (T, d_in)).astype(np.float32)
    y = rs.lora_w4_apply(pack(packed, s, z, group, "bf16", dev), torch.from_numpy(x).to(dev).to(DT[dtype]))
    want = torch.from_numpy(w4_apply_ref(packed[0], s[0], z[0], group, x)).to(DT[dtype])
    assert np.array_equal(hbits(y), hbits(want))


@pytest.mark.parametrize("T", [1, 20, 260])
def test_strides_and_neighbours(T):
    """x and y as column slices of wider buffers, x's other columns NaN; y's
    other columns and the rows behind the last one keep their values."""
    dev = device()
    d_in, d_out, group = 1000, 264, 64
    packed, s, z = make(5, 1, d_out, d_in, group, False, "bf16")
    st = pack(packed, s, z, group, "bf16", dev)
    x = acts(6, T, d_in, "bf16")
    wide = torch.full((T, d_in + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8: 8 + d_in] = torch.from_numpy(x).to(dev)
    out = torch.full((T + 3, d_out + 32), 7.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w4_apply(st, wide[:, 8: 8 + d_in], out[:T, 16: 16 + d_out])
    plain = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).bfloat16())
    assert np.array_equal(hbits(out[:T, 16: 16 + d_out].contiguous()), hbits(plain))
    out[:T, 16: 16 + d_out] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("T", [4, 40, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_alone(T, bad):
    dev = device()
    d_in, d_out, group = 264, 72, 32
    packed, s, z = make(7, 1, d_out, d_in, group, True, "bf16")
    st = pack(packed, s, z, group, "bf16", dev)
    x = torch.from_numpy(acts(8, T, d_in, "bf16")).to(dev).bfloat16()
    good = rs.lora_w4_apply(st, x)
    x[1, 17] = bad
    y = rs.lora_w4_apply(st, x)
    keep = [t for t in range(T) if t != 1]
    assert np.array_equal(hbits(y[keep]), hbits(good[keep]))
    assert not bool(torch.isfinite(y[1]).any())


def test_large_and_small_values():
    """Rows of very different size in one call: each keeps its own precision."""
    dev = device()
    d_in, d_out, group = 520, 136, 64
    packed, s, z = make(9, 1, d_out, d_in, group, True, "bf16")
    st = pack(packed, s, z, group, "bf16", dev)
    for T in (6, 300):
        x = acts(10, T, d_in, "bf16") * np.exp2(np.linspace(-90, 90, T).round())[:, None].astype(np.float32)
        x[2] = 0
        y = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).bfloat16())
        a = (packed[0], s[0], z[0], group, x)
        assert_close(y, w4_apply_ref(*a), w4_magnitude_ref(*a), d_in, group, "bf16")


def test_no_rows():
    dev = device()
    packed, s, z = make(11, 1, 16, 64, 32, False, "bf16")
    st = pack(packed, s, z, 32, "bf16", dev)
    assert rs.lora_w4_apply(st, torch.empty(0, 64, dtype=torch.bfloat16, device=dev)).shape == (0, 16)
    ids = torch.empty(0, 2, dtype=torch.int32, device=dev)
    assert rs.lora_w4_apply_experts(st, torch.empty(0, 64, dtype=torch.bfloat16, device=dev), ids).shape == (0, 16)


# T, k, E, d_in, d_out, group, zeros, scales, dtype, per choice, combine
EXPERTS = [
    (1, 1, 1, 64, 16, 32, False, "bf16", "bf16", False, False),
    (1, 8, 12, 264, 72, 64, True, "bf16", "bf16", False, False),
    (1, 8, 12, 264, 72, 64, True, "bf16", "bf16", True, True),
    (3, 2, 5, 136, 40, 32, True, "f32", "f32", True, True),
    (7, 3, 4, 520, 104, 128, False, "bf16", "bf16", False, True),
    (30, 4, 9, 392, 136, 32, True, "bf16", "bf16", True, True),
    (64, 2, 3, 512, 264, 128, True, "bf16", "bf16", False, False),
    (50, 3, 200, 136, 40, 64, False, "f32", "bf16", False, True),
    (300, 4, 6, 264, 200, 64, True, "bf16", "bf16", True, True),
    (700, 2, 5, 384, 328, 128, False, "bf16", "bf16", False, False),
    (1500, 3, 17, 136, 72, 32, True, "f32", "bf16", True, False),
    (120, 4, 8, 264, 72, 64, True, "bf16", "f32", False, True),
    (3, 8, 20, 4104, 40, 128, True, "bf16", "bf16", True, True),
    (1, 9, 9, 1032, 24, 64, False, "f32", "f32", True, True),
    (30, 1, 1, 1032, 64, 32, True, "bf16", "bf16", False, False),
    (40, 2, 2, 776, 72, 64, False, "bf16", "bf16", True, True),
    (3000, 2, 300, 136, 24, 64, True, "bf16", "bf16", False, False),
    (60, 1, 1, 1032, 64, 32, True, "bf16", "bf16", False, False),
    (110, 2, 4, 1544, 72, 64, False, "bf16", "bf16", True, True),
    (90, 3, 2, 1032, 136, 128, False, "f32", "bf16", False, True),
    (260, 3, 12, 520, 264, 128, True, "bf16", "bf16", False, False),
]


def experts_case(case, seed, dev, hole=True):
    T, k, E, d_in, d_out, group, zeros, scales, dtype, per, combine = case
    rng = np.random.default_rng(seed)
    packed, s, z = make(seed + 1, E, d_out, d_in, group, zeros, scales)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if hole and T > 2:
        ids[1] = -1
        ids[T - 1, 0], ids[T - 1, k - 1] = E, -5
        ids[2, :] = ids[2, 0]  # the same expert for every choice
    w = rng.random((T, k)).astype(np.float32) if combine else None
    x = acts(seed + 2, T * k if per else T, d_in, dtype)
    return packed, s, z, x, ids, w


@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_experts(case):
    T, k, E, d_in, d_out, group, zeros, scales, dtype, per, combine = case
    dev = device()
    note(f"w4 experts {case}")
    packed, s, z, x, ids, w = experts_case(case, 20, dev)
    st = pack(packed, s, z, group, scales, dev)
    xd = torch.from_numpy(x).to(dev).to(DT[dtype])
    # rows that no choice with an expert reads hold NaN
    if per:
        xd[torch.from_numpy(((ids < 0) | (ids >= E)).reshape(-1)).to(dev)] = float("nan")
    elif T > 2:
        xd[1] = float("nan")
    wd = None
    if combine:
        wd = torch.from_numpy(w).to(dev)
        wd[torch.from_numpy((ids < 0) | (ids >= E)).to(dev)] = float("nan")  # whatever its weight
    y = rs.lora_w4_apply_experts(st, xd, torch.from_numpy(ids).to(dev), wd)
    ref = experts_ref(packed, s, z, group, x, ids, w)
    mag = experts_ref(packed, s, z, group, x, ids, w, product=w4_magnitude_ref)
    assert_close(y, ref, mag, d_in, group, dtype, k=k if combine else 0)
    if T > 2:
        empty = y[1:2] if combine else y[k: 2 * k]
        assert bool((empty == 0).all())


def test_one_expert_for_all():
    """Every row names the same expert (and, once, none at all)."""
    dev = device()
    case = (600, 2, 7, 264, 136, 64, True, "bf16", "bf16", False, False)
    packed, s, z, x, ids, _ = experts_case(case, 30, dev)
    st, one = pack(packed, s, z, 64, "bf16", dev), pack(packed[3:4], s[3:4], z[3:4], 64, "bf16", dev)
    xd = torch.from_numpy(x).to(dev).bfloat16()
    y = rs.lora_w4_apply_experts(st, xd, torch.full((600, 2), 3, dtype=torch.int32, device=dev))
    want = rs.lora_w4_apply(one, xd.repeat_interleave(2, 0))
    # The two calls may be different kernels, whose float32 sums run in another
    # order: float32 addition is not associative, so the same bits do not
    # follow.  Each is within the bound of any order of the sum (tolerance()).
    a = (packed[3], s[3], z[3], 64, np.repeat(x, 2, 0))
    ref, mag = w4_apply_ref(*a), w4_magnitude_ref(*a)
    assert_close(y, ref, mag, 264, 64, "bf16")
    assert_close(want, ref, mag, 264, 64, "bf16")
    none = torch.full((600, 2), -1, dtype=torch.int32, device=dev)
    out = torch.full((1200, 136), 5.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w4_apply_experts(st, xd, none, None, out)
    assert bool((out == 0).all())
    out = torch.full((600, 136), 5.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w4_apply_experts(st, xd, none, torch.ones(600, 2, device=dev), out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("case", [EXPERTS[2], EXPERTS[5], EXPERTS[8], EXPERTS[9]], ids=lambda c: "-".join(map(str, c)))
def test_repeated_and_captured(case):
    """The same call twice is equal bit for bit; so is every replay of a
    captured one, on new inputs, with eager work on the same store between."""
    T, k, E, d_in, d_out, group, zeros, scales, dtype, per, combine = case
    dev = device()
    packed, s, z, x, ids, w = experts_case(case, 40, dev, hole=False)
    st = pack(packed, s, z, group, scales, dev)
    xd = torch.from_numpy(x).to(dev).to(DT[dtype])
    idd = torch.from_numpy(ids).to(dev)
    wd = torch.from_numpy(w).to(dev) if combine else None
    first = rs.lora_w4_apply_experts(st, xd, idd, wd)
    assert np.array_equal(hbits(first), hbits(rs.lora_w4_apply_experts(st, xd, idd, wd)))
    out = torch.empty_like(first)
    nb = rs.lora_w4_workspace_bytes(st, DT[dtype], T, k, combine)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rs.lora_w4_apply_experts(st, xd, idd, wd, out, ws=ws)
    for i in range(4):
        if i:
            xd.copy_(torch.from_numpy(acts(50 + i, x.shape[0], d_in, dtype)).to(dev))
            idd.copy_(torch.roll(idd, 1, 0))
        ws.fill_(255)  # scratch needs no initial value
        out.fill_(3.0)
        graph.replay()
        want = rs.lora_w4_apply_experts(st, xd, idd, wd)
        torch.cuda.synchronize()
        assert np.array_equal(hbits(out), hbits(want)), i


@pytest.mark.parametrize("T", [1, 24, 400])
def test_dense_captured_and_on_two_streams(T):
    dev = device()
    d_in, d_out, group = 776, 328, 64
    packed, s, z = make(60, 1, d_out, d_in, group, True, "bf16")
    st = pack(packed, s, z, group, "bf16", dev)
    xs = [torch.from_numpy(acts(61 + i, T, d_in, "bf16")).to(dev).bfloat16() for i in range(2)]
    want = [rs.lora_w4_apply(st, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            got[i] = [rs.lora_w4_apply(st, xs[i]) for _ in range(5)]
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert np.array_equal(hbits(y), hbits(want[i]))
    out = torch.empty_like(want[0])
    x = xs[0].clone()
    ws = torch.empty(max(rs.lora_w4_workspace_bytes(st, torch.bfloat16, T), 16), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.lora_w4_apply(st, x, out, ws=ws)
    for i in (0, 1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(hbits(out), hbits(want[i]))


# T, d_in, d_out: sizes that the many-rows kernel takes, with its small tiles,
# its large ones, splits of the inputs, many of them, and a last split shorter.
MANY = [(300, 1032, 8200), (1000, 1032, 4104), (300, 4104, 4104), (100, 2056, 16392), (1100, 2056, 2056)]


@pytest.mark.parametrize("group,zeros,scales", [(32, True, "bf16"), (64, False, "f32"), (128, True, "bf16"), (128, False, "bf16")])
@pytest.mark.parametrize("T,d_in,d_out", MANY)
def test_many_rows(T, d_in, d_out, group, zeros, scales):
    """As test_dense, and with rows of very different size."""
    dev = device()
    packed, s, z = make(100, 1, d_out, d_in, group, zeros, scales)
    st = pack(packed, s, z, group, scales, dev)
    x = acts(101, T, d_in, "bf16")
    x[3] *= 2.0 ** 60
    x[5] *= 2.0 ** -60
    x[7] = 0.0
    note(f"w4 {T} {d_in} {d_out} {group}")
    y = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).bfloat16())
    some = sorted({0, 1, 2, 3, 5, 7, 63, 64, 95, 96, T // 2, T - 2, T - 1})
    a = (packed[0], s[0], None if z is None else z[0], group, x[some])
    assert_close(y[some], w4_apply_ref(*a), w4_magnitude_ref(*a), d_in, group, "bf16")
    assert bool(torch.isfinite(y).all())
    again = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).bfloat16())
    assert np.array_equal(hbits(y), hbits(again))


@pytest.mark.parametrize("T,d_in,d_out", MANY[:3])
def test_many_rows_strided_and_bad(T, d_in, d_out):
    """Column slices of wider buffers with NaN beside x; then a row with a NaN,
    one with an infinity: the others keep their bits, and what is beside y its
    values."""
    dev = device()
    packed, s, z = make(102, 1, d_out, d_in, 64, True, "bf16")
    st = pack(packed, s, z, 64, "bf16", dev)
    x = torch.from_numpy(acts(103, T, d_in, "bf16")).to(dev).bfloat16()
    plain = rs.lora_w4_apply(st, x)
    wide = torch.full((T, d_in + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8: 8 + d_in] = x
    out = torch.full((T + 3, d_out + 32), 7.0, dtype=torch.bfloat16, device=dev)
    rs.lora_w4_apply(st, wide[:, 8: 8 + d_in], out[:T, 16: 16 + d_out])
    assert np.array_equal(hbits(out[:T, 16: 16 + d_out].contiguous()), hbits(plain))
    out[:T, 16: 16 + d_out] = 7.0
    assert bool((out == 7.0).all())
    x[1, d_in - 1], x[T - 1, 0] = float("nan"), float("inf")
    y = rs.lora_w4_apply(st, x)
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert np.array_equal(hbits(y[keep]), hbits(plain[keep]))
    assert not bool(torch.isfinite(y[[1, T - 1]]).any())


@pytest.mark.parametrize("T,d_in,d_out", MANY[:3])
def test_many_rows_captured_and_on_two_streams(T, d_in, d_out):
    dev = device()
    packed, s, z = make(104, 1, d_out, d_in, 128, True, "bf16")
    st = pack(packed, s, z, 128, "bf16", dev)
    xs = [torch.from_numpy(acts(105 + i, T, d_in, "bf16")).to(dev).bfloat16() for i in range(2)]
    want = [rs.lora_w4_apply(st, x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            got[i] = [rs.lora_w4_apply(st, xs[i]) for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert np.array_equal(hbits(y), hbits(want[i]))
    out, x = torch.empty_like(want[0]), xs[0].clone()
    ws = torch.empty(rs.lora_w4_workspace_bytes(st, torch.bfloat16, T), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.lora_w4_apply(st, x, out, ws=ws)
    for i in (0, 1, 0, 1):
        x.copy_(xs[i])
        ws.fill_(255)  # scratch needs no initial value
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(hbits(out), hbits(want[i]))


def test_calls_of_several_threads():
    """Four host threads, a stream and a size each, at once: the results of
    calls made alone."""
    import threading

    dev = device()
    sizes = [(1, 3592, 136), (40, 3592, 136), (16, 3592, 136), (300, 4104, 4104)]
    jobs = []
    for i, (T, d_in, d_out) in enumerate(sizes):
        packed, s, z = make(110 + i, 1, d_out, d_in, 64, True, "bf16")
        st = pack(packed, s, z, 64, "bf16", dev)
        x = torch.from_numpy(acts(120 + i, T, d_in, "bf16")).to(dev).bfloat16()
        jobs.append((st, x, rs.lora_w4_apply(st, x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got, failed = [[] for _ in jobs], []

    def work(i):
        try:
            st, x, _, stream = jobs[i]
            with torch.cuda.stream(stream):
                got[i] = [rs.lora_w4_apply(st, x) for _ in range(20)]
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for (_, _, want, _), ys in zip(jobs, got):
        assert len(ys) == 20 and all(np.array_equal(hbits(y), hbits(want)) for y in ys)


def test_routed_layer():
    """A layer as it is served: the base projection with the adapters' branch
    on it, the router, the experts' up product, and their weighted down
    product, against the oracle fed with the same intermediate values."""
    from oracle import apply_ref
    from workloads import make_random_workload

    dev = device()
    T, d, E, k, inner = 37, 264, 6, 2, 136
    base = make(70, 1, d, d, 64, False, "bf16")
    wl = make_random_workload(71, T, 5, d, d, [1, 3, 8, 0, 16], dtype="bf16")
    st = pack(*base, 64, "bf16", dev)
    A = [torch.from_numpy(a).to(dev).bfloat16() for a in wl.module.A]
    B = [torch.from_numpy(b).to(dev).bfloat16() for b in wl.module.B]
    store = rs.lora_pack_retained(A, B, wl.module.scales)
    x = torch.from_numpy(wl.x).to(dev).bfloat16()
    y = rs.lora_w4_apply(st, x)
    y0 = host(y)
    rs.lora_apply_batched(store, x, y, ids=torch.from_numpy(wl.ids.astype(np.int32)).to(dev))
    ref = apply_ref(host(x), wl.ids, wl.module.A, wl.module.B, wl.module.scales, y0=y0)
    assert np.abs(host(y) - ref).max() <= 2e-2 * np.abs(ref).max()

    gate = torch.from_numpy(acts(72, E, d, "bf16")).to(dev)
    logits = (y.float() @ gate.t()) / d ** 0.5
    ids, w = rs.lora_route(logits, k, score="sigmoid", bias=torch.linspace(-0.1, 0.1, E, device=dev))
    up, down = make(73, E, inner, d, 32, True, "bf16"), make(74, E, d, inner, 32, True, "bf16")
    u = rs.lora_w4_apply_experts(pack(*up, 32, "bf16", dev), y, ids)
    idh, wh = ids.cpu().numpy(), w.cpu().numpy()
    a = (*up, 32, host(y), idh)
    assert_close(u, experts_ref(*a), experts_ref(*a, product=w4_magnitude_ref), d, 32, "bf16")
    act = torch.nn.functional.silu(u)
    out = rs.lora_w4_apply_experts(pack(*down, 32, "bf16", dev), act, ids, w)
    a = (*down, 32, host(act), idh, wh)
    assert_close(out, experts_ref(*a), experts_ref(*a, product=w4_magnitude_ref), inner, 32, "bf16", k=k)
    # experts' ids also group rows for adapters of the experts
    seg = rs.lora_segment(ids.flatten(), E)
    assert int(seg.seg_off[E]) == T * k and int(seg.n_invalid[0]) == 0


def test_rows_beyond_32_bits():
    """y, then x, of more than 2^32 bytes: the last rows are those of a call
    of their own, the rows before them are written."""
    dev = device()
    T = 1 << 20
    packed, s, z = make(90, 1, 2304, 64, 32, True, "bf16")
    st = pack(packed, s, z, 32, "bf16", dev)
    x = torch.randn(T, 64, device=dev).bfloat16()
    note("w4 y of 4.8 GB")
    y = rs.lora_w4_apply(st, x)
    for at in (0, 777777, T - 4):
        xs = x[at: at + 4].float().cpu().numpy()
        a = (packed[0], s[0], z[0], 32, xs)
        assert_close(y[at: at + 4], w4_apply_ref(*a), w4_magnitude_ref(*a), 64, 32, "bf16")
    del x, y
    packed, s, z = make(91, 1, 16, 2304, 64, True, "bf16")
    st = pack(packed, s, z, 64, "bf16", dev)
    note("w4 x of 4.8 GB")
    x = torch.randn(T, 2304, device=dev, dtype=torch.bfloat16)
    y = rs.lora_w4_apply(st, x)
    for at in (0, 931234, T - 4):
        xs = x[at: at + 4].float().cpu().numpy()
        a = (packed[0], s[0], z[0], 64, xs)
        assert_close(y[at: at + 4], w4_apply_ref(*a), w4_magnitude_ref(*a), 2304, 64, "bf16")
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [2, 40, 300])
def test_scales_and_zeros_that_are_special(T):
    """Scales of zero, negative and very small; codes equal to their zero
    point in whole groups; a group's last inputs missing."""
    dev = device()
    d_in, d_out, group = 200, 40, 64
    packed, s, z = make(92, 1, d_out, d_in, group, True, "f32")
    s[0, 0] = 0.0
    s[0, 1] *= -1
    s[0, 2] = 1e-30
    s[0, 3, 1] = 0.0
    packed[0, 4], z[0, 4] = 0xBB, 11
    packed[0, 5], z[0, 5] = 0x00, 15
    st = pack(packed, s, z, group, "f32", dev)
    x = acts(93, T, d_in, "bf16")
    y = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).bfloat16())
    a = (packed[0], s[0], z[0], group, x)
    assert_close(y, w4_apply_ref(*a), w4_magnitude_ref(*a), d_in, group, "bf16")
    assert bool((y[:, 0] == 0).all())


def test_weights_that_are_special():
    """A weight of zero drops a finite row; negative weights; every weight zero."""
    dev = device()
    for T in (2, 60, 200):
        case = (T, 3, 4, 136, 40, 32, True, "bf16", "bf16", False, True)
        packed, s, z, x, ids, w = experts_case(case, 94, dev, hole=False)
        w[0], w[1, 0] = 0.0, -2.5
        st = pack(packed, s, z, 32, "bf16", dev)
        y = rs.lora_w4_apply_experts(st, torch.from_numpy(x).to(dev).bfloat16(), torch.from_numpy(ids).to(dev),
                                     torch.from_numpy(w).to(dev))
        ref = experts_ref(packed, s, z, 32, x, ids, w)
        mag = experts_ref(packed, s, z, 32, x, ids, np.abs(w), product=w4_magnitude_ref)
        assert_close(y, ref, mag, 136, 32, "bf16", k=3)
        assert bool((y[0] == 0).all())


def test_refused_on_the_gpu():
    dev = device()
    packed, s, z = make(80, 2, 16, 64, 32, False, "bf16")
    st = pack(packed, s, z, 32, "bf16", dev)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(rs.LoraError):
        rs.lora_w4_apply(st, x)  # two matrices
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="GPU|cpu"):
        rs.lora_w4_apply_experts(st, x.cpu(), ids)
    with pytest.raises(ValueError, match="ids"):
        rs.lora_w4_apply_experts(st, x, ids.long())
    with pytest.raises(ValueError, match="x must"):
        rs.lora_w4_apply_experts(st, x[:3], ids)
    with pytest.raises(ValueError, match="weights"):
        rs.lora_w4_apply_experts(st, x, ids, torch.ones(4, 2, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError, match="y must"):
        rs.lora_w4_apply_experts(st, x, ids, None, torch.zeros(4, 16, dtype=torch.bfloat16, device=dev))
    with pytest.raises(rs.LoraError):
        rs.lora_w4_apply_experts(st, torch.zeros(4, 68, dtype=torch.bfloat16, device=dev)[:, 2:66], ids)


# rows, d_in: one piece of 8 inputs, a last tile with one or nine, in one go and in chunks
@pytest.mark.parametrize("T,d_in", [(1, 8), (1, 136), (3, 200), (17, 136), (40, 136), (9, 4104), (16, 5128), (40, 4104)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_values_in_the_last_inputs(T, d_in, group, dtype):
    """The last tile's inputs alone count, at sums of |x| up to what lora.h
    states for bf16 (2^122 in a group), and where the formula ends for float32
    (15 |x| below 2^128)."""
    dev = device()
    note(f"w4 large {T} {d_in} {group} {dtype}")
    d_out = 40
    packed, s, z = make(140, 1, d_out, d_in, group, True, "bf16")
    s = np.exp2(np.round(np.log2(s)) - 20).astype(np.float32)
    x = acts(141, T, d_in, "bf16").astype(np.float64)
    x[:, d_in - 8:] = np.random.default_rng(142).choice([-1.0, 1.0, 0.5], (T, 8)) * 2.0 ** 118
    if dtype == "f32":
        x[:, d_in - 8:] = 0.0
        x[np.arange(T), d_in - 1 - np.arange(T) % 8] = 2.0 ** 123  # one input of a row: 15 |x| < 2^127
    x = x.astype(np.float32)
    st = pack(packed, s, z, group, "bf16", dev)
    y = rs.lora_w4_apply(st, torch.from_numpy(x).to(dev).to(DT[dtype]))
    a = (packed[0], s[0], z[0], group, x)
    assert_close(y, w4_apply_ref(*a), w4_magnitude_ref(*a), d_in, group, dtype)
    ids = torch.arange(T, dtype=torch.int32, device=dev).remainder(2).sub(1).abs().sub(1).unsqueeze(1).contiguous()  # 0, -1, 0, ...
    w = torch.full((T, 1), 0.5, device=dev)
    y = rs.lora_w4_apply_experts(st, torch.from_numpy(x).to(dev).to(DT[dtype]), ids, w)
    ref, mag = 0.5 * w4_apply_ref(*a), 0.5 * w4_magnitude_ref(*a)
    hole = ids.cpu().numpy()[:, 0] < 0
    ref[hole], mag[hole] = 0, 0
    assert_close(y, ref, mag, d_in, group, dtype, k=1)


@pytest.mark.parametrize("T,k", [(1, 4), (3, 2), (40, 4), (300, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("by_scale,by_weight,by_x", [(-80, -75, 100), (90, 70, -100), (-30, -120, 60), (30, 100, -60)])
def test_scale_times_weight_out_of_range(T, k, dtype, by_scale, by_weight, by_x):
    """Scales and weights whose products no float32 holds, rows that do."""
    dev = device()
    note(f"w4 weight {T} {k} {dtype} {by_scale}")
    E, d_in, d_out, group = 5, 264, 40, 64
    packed, s, z, x, ids, w = experts_case((T, k, E, d_in, d_out, group, True, "f32", dtype, False, True), 150, dev)
    s, w, x = (np.ldexp(v, e).astype(np.float32) for v, e in ((s, by_scale), (w, by_weight), (x, by_x)))
    st = pack(packed, s, z, group, "f32", dev)
    y = rs.lora_w4_apply_experts(st, torch.from_numpy(x).to(dev).to(DT[dtype]), torch.from_numpy(ids).to(dev),
                                 torch.from_numpy(w).to(dev))
    ref = experts_ref(packed, s, z, group, x, ids, w)
    mag = experts_ref(packed, s, z, group, x, ids, w, product=w4_magnitude_ref)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24  # tolerance() has 1e-30 in it: as large as these values
    tol = half * np.abs(ref) * (1 + 2.0 ** -8) + (64 + 5 + 32 + k + 2) * 2.0 ** -23 * mag
    assert np.isfinite(host(y)).all() and (np.abs(host(y) - ref) <= tol).all()
    assert np.abs(ref).max() > 0


@pytest.mark.parametrize("T", [1, 12, 300])
def test_weights_that_are_not_finite(T):
    """No finite value in such a token's row; the other tokens keep theirs."""
    dev = device()
    packed, s, z, x, ids, w = experts_case((T, 2, 4, 264, 40, 64, True, "bf16", "bf16", False, True), 160, dev, hole=False)
    st = pack(packed, s, z, 64, "bf16", dev)
    xd, idd, wd = torch.from_numpy(x).to(dev).bfloat16(), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev)
    good = rs.lora_w4_apply_experts(st, xd, idd, wd)
    for bad in (float("inf"), float("nan")):
        wb = wd.clone()
        wb[T // 2, 1] = bad
        y = rs.lora_w4_apply_experts(st, xd, idd, wb)
        keep = [t for t in range(T) if t != T // 2]
        assert np.array_equal(hbits(y[keep]), hbits(good[keep]))
        assert not bool(torch.isfinite(y[T // 2]).any())


def test_workspace_refused_on_the_gpu():
    """The calls check it before anything is launched."""
    dev = device()
    packed, s, z = make(170, 2, 16, 64, 32, False, "bf16")
    st = pack(packed, s, z, 32, "bf16", dev)
    x, ids = torch.zeros(400, 64, dtype=torch.bfloat16, device=dev), torch.zeros(400, 2, dtype=torch.int32, device=dev)
    need = rs.lora_w4_workspace_bytes(st, torch.bfloat16, 400, 2)
    assert need > 0
    for bad in (torch.zeros(1, dtype=torch.uint8, device=dev).expand(need), torch.zeros(2 * need, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            rs.lora_w4_apply_experts(st, x, ids, ws=bad)
    with pytest.raises(rs.LoraError):
        rs.lora_w4_apply_experts(st, x, ids, ws=torch.zeros(need - 1, dtype=torch.uint8, device=dev))
    rs.lora_w4_apply_experts(st, x, ids, ws=torch.zeros(need, dtype=torch.uint8, device=dev))


def one_input(T, d_in, d_out, group, seed=180):
    """Float32 rows with one input each, of 24 significant bits, codes a power
    of two from their zero points, scales powers of two: y is exact, and holds
    every bit of that input."""
    rng = np.random.default_rng(seed)
    packed, s, z = make(seed, 1, d_out, d_in, group, True, "f32")
    s = np.exp2(rng.integers(-3, 4, s.shape)).astype(np.float32)
    z = rng.integers(0, 8, z.shape).astype(np.uint8)
    step = rng.choice([1, 2, 4, 8], (1, d_out, d_in))
    q = z.repeat(group, -1)[..., :d_in] + np.where(step <= z.repeat(group, -1)[..., :d_in], rng.choice([-1, 1], step.shape), 1) * step
    assert q.min() >= 0 and q.max() <= 15
    packed = (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)
    x = np.zeros((T, d_in), np.float32)
    odd = rng.integers(2 ** 23, 2 ** 24, T) | 1  # all 24 bits from the first to the last
    x[np.arange(T), rng.integers(0, d_in, T)] = (odd * np.exp2(rng.integers(-40, 20, T).astype(float)) * rng.choice([-1, 1], T))
    return packed, s, z, x


@pytest.mark.parametrize("T,d_in,d_out,group", [(1, 520, 72, 32), (5, 4104, 40, 128), (17, 1032, 136, 64), (40, 264, 40, 32),
                                                (33, 5128, 24, 96), (300, 136, 24, 64)])
def test_float32_rows_are_whole(T, d_in, d_out, group):
    """Each of the three bf16 parts of x counts (test_w4_abi.py: without the
    last, no row would be right), for rows and for weighted sums."""
    dev = device()
    note(f"w4 whole float32 {T} {d_in} {group}")
    packed, s, z, x = one_input(T, d_in, d_out, group)
    st = pack(packed, s, z, group, "f32", dev)
    xd = torch.from_numpy(x).to(dev)
    ref = w4_apply_ref(packed[0], s[0], z[0], group, x)
    assert np.array_equal(ref, ref.astype(np.float32))
    assert np.array_equal(host(rs.lora_w4_apply(st, xd)), ref)
    ids = torch.zeros(T, 2, dtype=torch.int32, device=dev)
    ids[:, 1] = 1  # there is no such matrix
    y = rs.lora_w4_apply_experts(st, xd, ids, torch.full((T, 2), -0.5, device=dev))
    assert np.array_equal(host(y), -0.5 * ref)
    assert np.array_equal(host(rs.lora_w4_apply_experts(st, xd, ids)[::2]), ref)


def test_passes_in_turn_repeat():
    """Calls that nothing waits between, of several sizes and inputs in turn:
    each gives the bits of its first."""
    dev = device()
    jobs = []
    for i, (T, d_in, d_out, group) in enumerate([(1, 3584, 512, 128), (1, 1000, 2056, 64), (23, 3592, 520, 64), (7, 520, 136, 32)]):
        packed, s, z = make(190 + i, 1, d_out, d_in, group, i > 0, "bf16")
        st = pack(packed, s, z, group, "bf16", dev)
        jobs += [(st, torch.from_numpy(acts(195 + 2 * i + j, T, d_in, "bf16")).to(dev).bfloat16()) for j in range(2)]
    first = [rs.lora_w4_apply(st, x) for st, x in jobs]
    torch.cuda.synchronize()
    turns = [[rs.lora_w4_apply(st, x) for st, x in jobs] for _ in range(60)]
    for ys in turns:
        for y, want in zip(ys, first):
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))


FEW = [(1, 136, 40), (17, 520, 72), (40, 136, 40)]


@pytest.mark.parametrize("T,d_in,d_out,dtype,unit", [
    *[(*f, dtype, unit) for f in FEW for dtype, unit in (("bf16", -133), ("bf16", -126), ("f32", -133), ("f32", -126), ("f32", -112))],
    (301, 1032, 8200, "bf16", -133), (301, 1032, 8200, "bf16", -126)])
def test_smallest_values(T, d_in, d_out, dtype, unit):
    """x of a few of the smallest steps that lora.h says are kept, and near the
    smallest normal numbers, on large scales: exact."""
    dev = device()
    note(f"w4 smallest {T} {dtype} {unit}")
    packed, s, z = make(260, 1, d_out, d_in, 64, True, "bf16")
    s = np.exp2(np.random.default_rng(261).integers(98, 102, s.shape)).astype(np.float32)
    x = np.ldexp(np.random.default_rng(262).integers(-4, 5, (T, d_in)).astype(np.float64), unit)
    assert np.array_equal(x, x.astype(np.float32))
    x = x.astype(np.float32)
    y = rs.lora_w4_apply(pack(packed, s, z, 64, "bf16", dev), torch.from_numpy(x).to(dev).to(DT[dtype]))
    want = torch.from_numpy(w4_apply_ref(packed[0], s[0], z[0], 64, x)).to(DT[dtype])
    assert np.array_equal(host(y), host(want))
