"""The mixture-of-experts layer on the GPU where float32 holds the exact output
(tests/moe_exact.py): bits that are lost on the way are seen, in every form of
both kernels, whose sizes are those of tests/test_gpu_moe.py."""
import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from gpu_helpers import device, hbits, note
from moe_exact import ActLayer, ExactLayer
from oracle.moe_ref import act_ref
from test_gpu_moe import CASES, DT, pack

pytestmark = pytest.mark.gpu

# Rows that LDS does not hold at once, of x and of h: T, k, E, d, ffn, group, zeros, scales, dtype, act
LONG = [
    (40, 2, 2, 8200, 24, 128, False, "bf16", "f32", "silu"),
    (16, 2, 2, 8200, 24, 128, True, "bf16", "bf16", "silu"),
    (40, 2, 2, 24, 16384, 128, False, "bf16", "f32", "silu"),
    (40, 2, 2, 72, 16376, 32, True, "f32", "bf16", "silu"),
    (2, 2, 2, 24, 8200, 64, False, "f32", "f32", "gelu_tanh"),
    (1, 2, 3, 264, 18944, 128, True, "bf16", "bf16", "silu"),
    (33, 1, 2, 72, 32776, 64, True, "bf16", "bf16", "gelu_tanh"),
    (1, 1, 1, 40, 65544, 32, True, "f32", "f32", "silu"),
    (19, 2, 3, 24, 32776, 128, False, "f32", "f32", "silu"),
]


def exact_bounds(layer, x, ids, w):
    """y and what it may be off by: bf16 rows nothing (the exact sum rounded to
    bf16 once), float32 rows the k - 1 additions of k choices, half a step each
    of at most the terms' sum."""
    y, mag = layer.ref(x, ids, w)
    if layer.dtype == "bf16":
        return torch.from_numpy(y).to(torch.bfloat16).double().numpy(), np.zeros_like(y)
    return y, (ids.shape[1] - 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -10)


def act_bounds(layer, x, ids, w, act, dtype):
    """y and what it may be off by.

    g: bf16 rows exact; float32 rows the three parts of x are added, 2 steps of
    2^-24.  act: exp is off by 2 steps and by its argument's v 4 steps v (of gelu
    g's cube and the two products; of silu none), the sum, the quotient and the
    product with u = 1 by 1 each, g's own steps 2 (1 + 3 v).  So (8 + 2 + 10 v) 2^-24
    of |h|.  bf16 rows hold h to 16 bits, and a group of 32 features sums (32 + q) h
    and (32 + z) h, at most 94 |h| together, in 34 steps of 2^-23 at most, both parts
    of h within it.  The weighted sum adds k + 1 steps, and y rounds, half a step.
    The oracle's own gelu is g / 2 (1 + tanh): beside 1 tanh is off by up to 4 steps
    of 2^-53, which is all that is left of it at -5, so 2^-52 |g| more."""
    bf16 = dtype == "bf16"
    y, off = np.zeros((x.shape[0], layer.d_out)), np.zeros((x.shape[0], layer.d_out))
    k = ids.shape[1]
    for e in range(layer.n):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        g = layer.gates(x[t], e)
        h = act_ref(act, g)
        v = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
        dh = (10 + 10 * v) * 2.0 ** -24 * np.abs(h) + 1e-36 + 2.0 ** -52 * np.abs(g)
        if bf16:
            dh = dh + 2.0 ** -16 * np.abs(h)
            group = np.add.reduceat(np.abs(h) + dh, np.arange(0, layer.ffn, 32), 1)
            dy = dh[:, layer.f[e]] + 34 * 2.0 ** -23 * 94 * group[:, layer.f[e] // 32]
        else:
            dy = dh[:, layer.f[e]]
        scale = w[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, scale * h[:, layer.f[e]])
        np.add.at(off, t, scale * (dy + (k + 1) * 2.0 ** -24 * np.abs(h[:, layer.f[e]])))
    return y, off + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(y) + off)


def run(layer, group, group_down, scales, dtype, x, ids, w, act):
    dev = device()
    stores = [pack(m.packed(), g, scales, dev) for m, g in ((layer.gate, group), (layer.up, group), (layer.down, group_down))]
    return rs.lora_w4_moe(*stores, torch.from_numpy(x).to(dev).to(DT[dtype]), torch.from_numpy(ids).to(dev),
                          torch.from_numpy(w).to(dev), act=act)


@pytest.mark.parametrize("case", CASES + LONG, ids=lambda c: "-".join(map(str, c)))
def test_no_bit_is_lost(case):
    T, k, E, d, ffn, group, zeros, scales, dtype, act = case
    note(f"moe exact {case}")
    layer = ExactLayer(5, E, d, ffn, d, group, zeros, dtype)
    a = layer.inputs(6, T, k)
    got = run(layer, group, group, scales, dtype, *a, act)
    y, bound = exact_bounds(layer, *a)
    off = np.abs(got.double().cpu().numpy() - y)
    assert (off <= bound).all(), f"{int((off > bound).sum())} of {off.size} outputs"
    again = run(layer, group, group, scales, dtype, *a, act)
    assert np.array_equal(hbits(got), hbits(again))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_activations(case):
    T, k, E, d, ffn, group, zeros, scales, dtype, act = case
    note(f"moe act {case}")
    layer = ActLayer(7, E, d, ffn, d, group, zeros)
    x, ids, w = ExactLayer(5, E, d, ffn, d, group, zeros, dtype).inputs(8, T, k)
    y, bound = act_bounds(layer, x, ids, w, act, dtype)
    off = np.abs(run(layer, group, 32, scales, dtype, x, ids, w, act).double().cpu().numpy() - y)
    assert (off <= bound).all(), f"{float((off / bound).max()):.3g} of the bound"


def test_stores_past_31_bits():
    """The last experts of stores of more than 2^31 bytes of codes are those of
    the same stores in reverse order."""
    dev = device()
    g = torch.Generator(device=dev).manual_seed(11)
    n, d, ffn, group = 36, 4096, 32768, 128

    def random(d_out, d_in):
        q = torch.randint(0, 256, (n, d_out, d_in // 2), device=dev, generator=g, dtype=torch.uint8)
        assert q.numel() > 2 ** 31
        return q, (torch.rand(n, d_out, d_in // group, device=dev, generator=g) / (4 * d_in ** 0.5)).bfloat16()

    mats = [random(ffn, d), random(ffn, d), random(d, ffn)]
    stores = [rs.lora_w4_pack(q, s, group=group) for q, s in mats]
    turned = [rs.lora_w4_pack(q.flip(0), s.flip(0), group=group) for q, s in mats]
    del mats
    for T, k, dt in ((1, 3, torch.bfloat16), (50, 1, torch.bfloat16), (2, 2, torch.float32)):
        note(f"moe past 31 bits {T} {k} {dt}")
        x = torch.randn(T, d, device=dev, generator=g).to(dt)
        ids = (n - 1 - torch.arange(T * k, device=dev, dtype=torch.int32) % 7).view(T, k)
        w = torch.rand(T, k, device=dev, generator=g)
        y = rs.lora_w4_moe(*stores, x, ids, w)
        assert torch.isfinite(y).all() and y.float().std() > 0.01
        assert np.array_equal(hbits(y), hbits(rs.lora_w4_moe(*turned, x, n - 1 - ids, w)))


def test_calls_of_several_threads():
    """Host threads with a stream each, at once, on sizes whose kernels take
    different amounts of LDS, 8-bit layers among them: the results of calls made
    alone."""
    import threading

    dev = device()
    g = torch.Generator(device=dev).manual_seed(3)
    jobs = []
    layer = ExactLayer(8, 4, 4104, 136, 136, 64, True, "bf16")
    stores = [pack(m.packed(), 64, "bf16", dev) for m in (layer.gate, layer.up, layer.down)]
    for T in (1, 7, 40):
        x, ids, w = layer.inputs(T, T, 2)
        a = [torch.from_numpy(v).to(dev) for v in (x, ids, w)]
        a[0] = a[0].bfloat16()
        jobs.append(lambda a=a: rs.lora_w4_moe(*stores, *a))
    base = rs.lora_w8_pack(torch.randint(-127, 128, (520, 4104), dtype=torch.int8, device=dev, generator=g),
                           torch.rand(520, device=dev, generator=g))
    for T in (2, 40, 700):
        x = torch.randn(T, 4104, device=dev, generator=g).bfloat16()
        jobs.append(lambda x=x: rs.lora_w8_apply(base, x))
    got, failed = [None] * len(jobs), []
    start = threading.Barrier(len(jobs))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()

    def work(i):
        try:
            start.wait(60)
            with torch.cuda.stream(streams[i]):
                got[i] = [jobs[i]() for _ in range(20)]
            streams[i].synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for job, ys in zip(jobs, got):
        want = hbits(job())
        assert len(ys) == 20 and all(np.array_equal(hbits(y), want) for y in ys)


@pytest.mark.parametrize("T,dtype", [(2, "f32"), (24, "f32"), (64, "f32"), (24, "bf16"), (64, "bf16")])
def test_values_that_are_no_numbers(T, dtype):
    """An infinity or a NaN (of any payload) in a row reaches its own row alone, in
    the forms that tests/test_gpu_moe.py does not take."""
    dev = device()
    layer = ExactLayer(9, 16, 264, 4104, 136, 128, True, dtype)
    x, ids, w = layer.inputs(10, T, 4)
    stores = [pack(m.packed(), 128, "bf16", dev) for m in (layer.gate, layer.up, layer.down)]
    a = [torch.from_numpy(v).to(dev) for v in (x, ids, w)]
    a[0] = a[0].to(DT[dtype])
    base = hbits(rs.lora_w4_moe(*stores, *a))
    low = np.array([0x7F800001, 0xFF80FFFF], np.uint32).view(np.float32)  # NaNs whose upper half is an infinity's
    for bad in [np.inf, -np.inf, np.nan] + (list(low) if dtype == "f32" else []):
        z = x.copy()
        z[1, 263] = bad
        y = rs.lora_w4_moe(*stores, torch.from_numpy(z).to(dev).to(DT[dtype]), *a[1:])
        assert not torch.isfinite(y[1]).any(), bad
        keep = np.arange(T) != 1
        assert np.array_equal(hbits(y)[keep], base[keep]), bad
