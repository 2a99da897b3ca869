"""The many-rows kernel of the 4-bit products, at sizes whose plan names it
(test_w4_plan.py holds that: another choice of kernel fails there, and these
tests get new sizes).

Most tests are exact.  x holds small integers, scales and weights powers of
two: every product and every sum is a number of at most 24 bits, so y is the
oracle's value rounded once, bit for bit.  The bound of the others: the kernel
multiplies with q - z itself and x as f16 (exact: a value of at least 2^-31 of
its row's largest keeps its bits), so a sum passes through at most `gran`
additions in its group of `gran` <= 128 inputs, one scaling, and the additions
of groups, splits and choices, each 2^-23 (a matrix core may truncate) of
sum |s (q - z) x|, and y rounds once.
"""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, hbits, note
from oracle.w4_ref import w4_apply_ref, w4_matrix_ref
from test_gpu_w4 import acts, host, make, pack

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16

# T, d_in, d_out, rows per tile, splits of the inputs
DENSE = [(301, 1032, 8200, 64, 1), (601, 1032, 4104, 64, 1), (401, 2056, 4104, 64, 2), (997, 520, 4104, 96, 1), (470, 2056, 4104, 96, 3)]
# T, k, E, d_in, d_out, x per choice, weighted, rows per tile, splits
EXPERTS = [
    (600, 2, 3, 264, 200, False, False, 96, 1),
    (600, 2, 3, 264, 200, True, True, 96, 1),
    (419, 5, 5, 520, 328, False, True, 96, 1),
    (601, 2, 3, 4104, 72, True, False, 96, 7),
    (601, 2, 3, 4104, 72, False, True, 96, 7),
    (300, 1, 2, 1032, 264, False, False, 64, 2),
    (151, 4, 4, 1544, 264, True, True, 64, 3),
    (6700, 4, 1024, 136, 72, False, False, 64, 1),
    (6700, 4, 1024, 136, 72, False, True, 64, 1),
]
# group, zero points, scales
KINDS = [(32, True, "bf16"), (32, False, "f32"), (64, True, "f32"), (96, True, "bf16"), (128, False, "bf16"), (128, True, "bf16"),
         (256, True, "f32")]


def whole(seed, n, d_out, d_in, group, zeros):
    """Matrices with scales of powers of two."""
    packed, s, z = make(seed, n, d_out, d_in, group, zeros, "bf16")
    return packed, np.exp2(np.random.default_rng(seed).integers(-2, 2, s.shape)).astype(np.float32), z


def integers(seed, rows, d_in):
    return np.random.default_rng(seed).integers(-4, 5, (rows, d_in)).astype(np.float32)


def rounded(ref):
    """Exact float32 numbers as bf16 bits."""
    assert np.array_equal(ref, ref.astype(np.float32))
    return hbits(torch.from_numpy(ref.astype(np.float32)).to(BF16))


def by_expert(packed, s, z, group, x, ids, w=None):
    """Rows [T k, d_out], or with weights [T, d_out], an expert at a time."""
    T, k = ids.shape
    rows = np.zeros((T * k, packed.shape[1]))
    src = np.arange(T * k) if x.shape[0] == T * k else np.arange(T * k) // k
    for e in range(packed.shape[0]):
        at = np.flatnonzero(ids.reshape(-1) == e)
        if at.size:
            rows[at] = w4_apply_ref(packed[e], s[e], None if z is None else z[e], group, x[src[at]])
    if w is None:
        return rows
    return (rows.reshape(T, k, -1) * np.where((ids >= 0) & (ids < packed.shape[0]), w, 0.0)[:, :, None]).sum(1)


@pytest.mark.parametrize("group,zeros,scales", KINDS)
@pytest.mark.parametrize("T,d_in,d_out,bm,splits", DENSE)
def test_dense_exact(T, d_in, d_out, bm, splits, group, zeros, scales):
    dev = device()
    note(f"w4 many {T} {d_in} {d_out} {group} {zeros} {scales}")
    packed, s, z = whole(200, 1, d_out, d_in, group, zeros)
    x = integers(201, T, d_in)
    x[T // 2] = 0.0
    y = rs.lora_w4_apply(pack(packed, s, z, group, scales, dev), torch.from_numpy(x).to(dev).to(BF16))
    assert np.array_equal(hbits(y), rounded(w4_apply_ref(packed[0], s[0], None if z is None else z[0], group, x)))


@pytest.mark.parametrize("T,d_in,d_out,bm,splits", DENSE)
def test_values_beside_a_large_one(T, d_in, d_out, bm, splits):
    """Input 0 is 2^14, with codes equal to their zero point; the others are up
    to eight bits from 2^-24 on: f16's smallest numbers, and all of y."""
    dev = device()
    group = 64
    packed, s, z = whole(210, 1, d_out, d_in, group, True)
    packed[0, :, 0] = (packed[0, :, 0] & 0xF0) | z[0, :, 0]
    small = np.random.default_rng(211).integers(-255, 256, (T, d_in)) * 2.0 ** -24
    small[:, 0] = 0.0
    x = small.copy()
    x[:, 0] = 2.0 ** 14
    x = x.astype(np.float32)
    assert torch.equal(torch.from_numpy(x).to(BF16).float(), torch.from_numpy(x))
    y = rs.lora_w4_apply(pack(packed, s, z, group, "bf16", dev), torch.from_numpy(x).to(dev).to(BF16))
    ref = w4_apply_ref(packed[0], s[0], z[0], group, x)
    assert np.array_equal(ref, w4_apply_ref(packed[0], s[0], z[0], group, small))
    # sums are whole numbers of 2^-26 (scales from 2^-2), below 2^24 of them in absolute value
    assert (np.abs(small) @ np.abs(w4_matrix_ref(packed[0], s[0], z[0], group)).T).max() < 2.0 ** -26 * 2 ** 24
    assert np.array_equal(hbits(y), rounded(ref))


@pytest.mark.parametrize("T,d_in,d_out,bm,splits", DENSE)
def test_special_scales_and_zeros(T, d_in, d_out, bm, splits):
    """Scales of zero, negative and very small; whole groups of codes equal to
    their zero point; rows of very different size.  As near as the formula."""
    dev = device()
    group = 64
    packed, s, z = make(220, 1, d_out, d_in, group, True, "f32")
    s[0, 0] = 0.0
    s[0, 1] *= -1
    s[0, 2] = 1e-30
    s[0, 3, 1] = 0.0
    packed[0, 4], z[0, 4] = 0xBB, 11
    packed[0, 5], z[0, 5] = 0x00, 15
    packed[0, 6], z[0, 6] = 0xFF, 0
    x = acts(221, T, d_in, "bf16") * np.exp2(np.linspace(-60, 60, T).round())[:, None].astype(np.float32)
    y = rs.lora_w4_apply(pack(packed, s, z, group, "f32", dev), torch.from_numpy(x).to(dev).to(BF16))
    W = w4_matrix_ref(packed[0], s[0], z[0], group)
    ref, mag = x.astype(np.float64) @ W.T, np.abs(x.astype(np.float64)) @ np.abs(W).T
    steps = group + 1 + -(-d_in // group) + splits
    # Scale 1e-30 on rows of 2^-60 leaves values below 2^-126, where bf16's steps stay at 2^-133 (float32's at
    # 2^-149): a rounding there is off by up to half of one, whatever the value.
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + steps * 2.0 ** -23 * mag + 2.0 ** -134 + 2.0 ** -149
    assert bool(torch.isfinite(y).all()) and (np.abs(host(y) - ref) <= tol).all()
    assert bool((y[:, [0, 4]] == 0).all())


def routing(kind, T, k, E, seed=230):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "holes":
        ids[rng.random((T, k)) < 0.1] = -1
        ids[1] = E
        ids[T - 3:] = -(2 ** 31)
        ids[2] = ids[2, 0]
    elif kind == "skewed":
        ids[rng.random((T, k)) < 0.9] = E - 1
    elif kind == "one":
        ids[:] = E // 2
    return ids


@pytest.mark.parametrize("kind", ["uniform", "holes", "skewed", "one"])
@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_experts_exact(case, kind):
    T, k, E, d_in, d_out, per, weighted, bm, splits = case
    dev = device()
    for group, zeros, scales in (KINDS[:1] if E > 8 else KINDS[::2]):
        note(f"w4 many experts {case} {kind} {group}")
        packed, s, z = whole(231, E, d_out, d_in, group, zeros)
        ids = routing(kind, T, k, E)
        x = integers(232, T * k if per else T, d_in)
        w = np.random.default_rng(233).choice([0.5, 1.0, 2.0, -1.0, 0.0], (T, k)).astype(np.float32) if weighted else None
        xd = torch.from_numpy(x).to(dev).to(BF16)
        none = (ids < 0) | (ids >= E)
        wd = None
        if weighted:
            wd = torch.from_numpy(w).to(dev)
            wd[torch.from_numpy(none).to(dev)] = float("nan")
        if per:
            xd[torch.from_numpy(none.reshape(-1)).to(dev)] = float("nan")
        y = rs.lora_w4_apply_experts(pack(packed, s, z, group, scales, dev), xd, torch.from_numpy(ids).to(dev), wd)
        ref = by_expert(packed, s, z, group, x, ids, w)
        assert np.array_equal(ref, ref.astype(np.float32))
        assert np.array_equal(host(y), torch.from_numpy(ref).to(BF16).double().numpy())  # 0 and -0 alike


@pytest.mark.parametrize("case", EXPERTS[:5] + EXPERTS[8:], ids=lambda c: "-".join(map(str, c)))
def test_experts_captured(case):
    """Replays of one captured call on new inputs and choices, with eager calls
    between, and a second graph with a workspace of its own."""
    T, k, E, d_in, d_out, per, weighted, bm, splits = case
    dev = device()
    packed, s, z = whole(240, E, d_out, d_in, 64, True)
    st = pack(packed, s, z, 64, "bf16", dev)
    x = torch.from_numpy(integers(241, T * k if per else T, d_in)).to(dev).to(BF16)
    ids = torch.from_numpy(routing("holes", T, k, E)).to(dev)
    w = torch.rand(T, k, device=dev) if weighted else None
    first = rs.lora_w4_apply_experts(st, x, ids, w)
    nb = rs.lora_w4_workspace_bytes(st, BF16, T, k, weighted)
    graphs, outs, scratch = [], [], []
    for _ in range(2):
        outs.append(torch.empty_like(first))
        scratch.append(torch.empty(nb, dtype=torch.uint8, device=dev))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            rs.lora_w4_apply_experts(st, x, ids, w, outs[-1], ws=scratch[-1])
    for i in range(4):
        if i:
            x.copy_(torch.from_numpy(integers(242 + i, x.shape[0], d_in)).to(dev))
            ids.copy_(torch.from_numpy(routing(("skewed", "one", "uniform")[i - 1], T, k, E, 250 + i)).to(dev))
        for g, o, b in zip(graphs, outs, scratch):
            b.fill_(255)
            o.fill_(3.0)
            g.replay()
        want = rs.lora_w4_apply_experts(st, x, ids, w)
        torch.cuda.synchronize()
        for o in outs:
            assert np.array_equal(hbits(o), hbits(want)), i


@pytest.mark.parametrize("by", [-120, 80, 97])
@pytest.mark.parametrize("T,d_in,d_out,bm,splits", [DENSE[0], DENSE[3]])
def test_scales_at_their_bounds(T, d_in, d_out, bm, splits, by):
    """Rows of W that sum to up to the 2^113 that lora.h states; small ones."""
    dev = device()
    note(f"w4 scales {T} {d_in} 2^{by}")
    packed, s, z = whole(270, 1, d_out, d_in, 64, True)
    s = np.ldexp(s, by).astype(np.float32)
    assert np.abs(w4_matrix_ref(packed[0], s[0], z[0], 64)).sum(1).max() < 2.0 ** 113
    x = integers(271, T, d_in)
    y = rs.lora_w4_apply(pack(packed, s, z, 64, "bf16", dev), torch.from_numpy(x).to(dev).to(BF16))
    assert np.array_equal(hbits(y), rounded(w4_apply_ref(packed[0], s[0], z[0], 64, x)))
