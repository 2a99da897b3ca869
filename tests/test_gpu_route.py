"""The router on the GPU against the float64 oracle.

The chosen ids are exact: without a bias the order is that of the logits
themselves, and the bias cases' scores differ by more than float64 rounds.
Weights: a float32 exponential of l - l_max carries the difference's rounding
(2^-24 of |l - l_max|) and its own two or so units, the quotient and the last
rounding one each: (|l - l_max| + 8) 2^-24 relative.
"""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, note
from oracle.w4_ref import route_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(logits, dtype, k, bias=None, **kw):
    dev = device()
    l = torch.from_numpy(np.asarray(logits, np.float32)).to(dev).to(DT[dtype])
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(dev)
    ids, w = rs.lora_route(l, k, bias=b, **kw)
    lh = l.float().cpu().numpy().astype(np.float64)
    want, ww = route_ref(lh, k, bias=None if bias is None else np.asarray(bias, np.float32).astype(np.float64), **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    ih, wh = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(ih, want), np.argwhere(ih != want)[:5]
    spread = np.where(np.isfinite(lh), np.abs(lh), 0).clip(max=1e3)
    rel = (2 * spread.max(initial=0.0) + 8) * 2.0 ** -24
    assert (np.abs(wh - ww) <= rel * np.abs(ww) + 1e-44).all()
    assert (wh[want < 0] == 0).all()
    return ih, wh


CASES = [
    (1, 1, 1, "f32", dict()),
    (1, 64, 8, "bf16", dict()),
    (5, 3, 3, "f32", dict(renormalize=False)),
    (33, 65, 6, "bf16", dict(score="sigmoid")),
    (100, 128, 8, "f32", dict(renormalize=False, scale=2.5)),
    (7, 256, 32, "f32", dict(score="sigmoid", renormalize=False)),
    (9, 300, 4, "bf16", dict(groups=4, top_groups=2)),
    (40, 512, 8, "f32", dict(groups=64, top_groups=3)),
    (3, 1024, 31, "f32", dict(groups=2, top_groups=1)),
    (50, 256, 8, "f32", dict(score="sigmoid", groups=8, top_groups=4)),
    (21, 96, 5, "bf16", dict(score="sigmoid", groups=3, top_groups=1, scale=0.5)),
    (8, 16, 2, "f32", dict(score="sigmoid", groups=16, top_groups=2)),
]


@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-" + "-".join(map(str, c[4].values())))
def test_route(case, with_bias):
    T, E, k, dtype, kw = case
    note(f"route {case} bias={with_bias}")
    rng = np.random.default_rng(5)
    check(2 * rng.normal(size=(T, E)), dtype, k, 0.1 * rng.normal(size=E) if with_bias else None, **kw)


def test_ties_go_to_the_lowest_index():
    l = np.zeros((4, 200))
    l[1, ::3] = 1.0
    l[2, 150:] = -2.0
    l[3] = np.random.default_rng(1).integers(-2, 3, 200)
    l[3, 5], l[3, 6] = -0.0, 0.0
    ids, _ = check(l, "f32", 12)
    assert ids[0].tolist() == list(range(12)) and ids[1].tolist() == list(range(0, 36, 3))
    check(l, "bf16", 12, bias=np.zeros(200))
    check(l, "f32", 7, score="sigmoid", groups=10, top_groups=3)
    check(l, "f32", 7, groups=10, top_groups=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_logits(score, groups):
    """-inf and NaN logits are never chosen, whole rows of them included; +inf
    counts as the largest number; the lowest finite number can be chosen."""
    rng = np.random.default_rng(2)
    l = rng.normal(size=(9, 40)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 3:] = -np.inf
    l[3, ::2] = np.nan
    l[4, 7] = np.inf
    l[5, [3, 9]] = np.inf
    l[6] = np.finfo(np.float32).min
    l[7, :39] = -np.inf
    l[8, 5:] = -np.inf
    l[8, 5] = np.finfo(np.float32).min
    for bias in (None, 0.1 * rng.normal(size=40)):
        kw = dict(score=score, groups=groups, top_groups=2 if groups > 1 else 1)
        check(l, "f32", 6, bias, **kw)
    b = np.zeros(40)
    b[:38] = -np.inf
    b[38] = np.nan
    ids, w = check(rng.normal(size=(3, 40)), "f32", 4, b, score=score)
    assert ids.tolist() == [[39, -1, -1, -1]] * 3 and (w[:, 0] == 1).all()


def test_small_scores_keep_their_ratio():
    l = np.full((2, 8), -300.0)
    l[0, :3] = [-290, -291, -289]
    l[1] = [-80, -81, 60, -300, -79, -300, -300, -300]
    check(l, "f32", 3, score="sigmoid")
    # the bias leaves out the expert that the softmax is made of
    b = np.zeros(8)
    b[2] = -2.0
    check(l[1:], "f32", 3, b)
    check(l[1:], "f32", 3, groups=4, top_groups=2)


def test_strided_rows_and_outputs():
    dev = device()
    wide = torch.randn(11, 77, device=dev)
    ids, w = rs.lora_route(wide[:, 3:69], 5)
    want = rs.lora_route(wide[:, 3:69].contiguous(), 5)
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
    i2, w2 = torch.full_like(ids, 9), torch.full_like(w, 9.0)
    r = rs.lora_route(wide[:, 3:69], 5, ids=i2, weights=w2)
    assert r[0] is i2 and torch.equal(i2, ids) and torch.equal(w2, w)
    assert rs.lora_route(wide[:0, :8], 2)[0].shape == (0, 2)
    with pytest.raises(ValueError):
        rs.lora_route(wide.t(), 2)
    with pytest.raises(rs.LoraError):
        rs.lora_route(wide, 40)
    with pytest.raises(rs.LoraError):
        rs.lora_route(wide, 3, groups=2)


def test_captured():
    dev = device()
    l = torch.randn(64, 256, device=dev)
    b = 0.1 * torch.randn(256, device=dev)
    kw = dict(score="sigmoid", bias=b, groups=8, top_groups=3, scale=2.5)
    ids, w = torch.empty(64, 8, dtype=torch.int32, device=dev), torch.empty(64, 8, device=dev)
    rs.lora_route(l, 8, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.lora_route(l, 8, ids=ids, weights=w, **kw)
    for _ in range(4):
        l.normal_()
        graph.replay()
        want = rs.lora_route(l, 8, **kw)
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_an_expert(score, renormalize, dtype):
    """Rows with fewer experts than k, none among them, in every form: id -1
    and weight 0 where there is none, whatever the scale."""
    rng = np.random.default_rng(3)
    l = rng.normal(size=(8, 40)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, ::2], l[2, 1::2] = np.nan, -np.inf
    l[3, 2:] = -np.inf
    l[4, :39] = np.nan
    l[5, 4:] = -np.inf
    none = np.full(40, -np.inf)
    some = 0.1 * rng.normal(size=40)
    some[1:] = np.where(rng.random(39) < 0.9, -np.inf, some[1:])
    for bias in (None, np.zeros(40), some, none):
        for kw in (dict(), dict(groups=4, top_groups=2), dict(scale=2.5), dict(scale=-3.0, groups=5, top_groups=1)):
            ids, w = check(l, dtype, 6, bias, score=score, renormalize=renormalize, **kw)
            assert (ids[:3] == -1).all() and (w[:3] == 0).all()
            assert bias is not none or (ids == -1).all()
    dev = device()
    for scale in (float("inf"), float("nan")):
        ids, w = rs.lora_route(torch.from_numpy(l).to(dev), 6, score=score, renormalize=renormalize, scale=scale)
        assert bool((w[ids < 0] == 0).all()) and int((ids < 0).sum()) >= 18


SATURATED = [(8, 2, 1, 2), (8, 2, 2, 3), (64, 4, 2, 8), (96, 3, 1, 5), (96, 6, 3, 9), (60, 5, 2, 6), (256, 8, 4, 8), (130, 2, 1, 7),
             (1024, 64, 5, 12)]


@pytest.mark.parametrize("E,groups,top_groups,k", SATURATED)
def test_scores_that_saturate(E, groups, top_groups, k):
    """Sigmoid scores within 2^-53 of one, or of each other, in groups: without
    a bias the order is that of the logits, and a group's that of the exact
    sums, which such scores decide by what they lack of one."""
    rng = np.random.default_rng(6)
    kw = dict(score="sigmoid", groups=groups, top_groups=top_groups)
    if E == 8:
        ids, _ = check([[26, 26.5, 40, 45, 0, 0, 0, 0], [0, 0, 0, 0, 45, 40, 60, 50]], "f32", k, **kw)
        assert ids[:, 0].tolist() == [3, 6]
    for lo, hi in ((20, 60), (-60, -20), (36, 37), (-300, 300), (24.9, 25), (-700, 700)):
        l = rng.uniform(lo, hi, size=(20, E))
        check(l, "f32", k, **kw)
        check(l, "bf16", k, renormalize=False, **kw)


def test_group_sums_near_one():
    """Groups of one large and one small logit, whose sums differ from one by
    less than float64 holds beside it, of either sign; in between, sums of two
    of a kind."""
    rng = np.random.default_rng(9)
    for n in (2, 3, 5):
        l = np.full((60, 12 * n), -200.0)
        for t in range(60):
            for g in range(12):
                a, b = rng.uniform(30, 90), rng.uniform(-90, -30)
                l[t, g * n], l[t, g * n + n - 1] = (a, b) if t % 3 or g % 4 else rng.uniform(-1, 1, 2)
        for top_groups in (1, 5, 11):
            check(l, "f32", 2, score="sigmoid", groups=12, top_groups=top_groups)
    # by hand: 1 - 2e-18 + 1e-17, 1 - 1e-17 + 2e-18, 1 exactly, 1 + 1e-20
    l = np.log([[2e-18, 1e-17, 1e-17, 2e-18, 1e-19, 1e-19, 1e-20, 2e-20]])
    l[0, ::2] *= -1
    ids, _ = check(l, "f32", 2, score="sigmoid", groups=4, top_groups=1)
    assert ids.tolist() == [[0, 1]]
    ids, _ = check(l, "f32", 4, score="sigmoid", groups=4, top_groups=3)
    assert 2 not in ids
