"""The layers of tests/moe_exact.py on the CPU: they are what they say, and a
layer that loses a part of x or of h, the last features or the last inputs, or
takes the other activation, does not pass the GPU tests that use them."""
import numpy as np
import pytest
import torch

from moe_exact import ActLayer, ExactLayer, cut
from oracle.moe_ref import act_ref, moe_ref
from test_gpu_moe import CASES
from test_gpu_moe_exact import LONG, act_bounds, exact_bounds
from workloads import round_to_bf16


def held(v, dtype):
    """v as rows of `dtype`, float64."""
    return torch.from_numpy(v).to(torch.bfloat16 if dtype == "bf16" else torch.float32).double().numpy()


@pytest.mark.parametrize("T,k,n,d,ffn,group,zeros,dtype", [
    (1, 1, 1, 8, 8, 32, True, "bf16"), (5, 3, 4, 136, 72, 32, False, "bf16"), (3, 2, 3, 264, 40, 128, True, "bf16"),
    (1, 1, 2, 8, 16, 32, True, "f32"), (6, 3, 5, 136, 24, 64, False, "f32")])
def test_the_layers_are_the_oracles(T, k, n, d, ffn, group, zeros, dtype):
    layer = ExactLayer(1, n, d, ffn, d, group, zeros, dtype)
    x, ids, w = layer.inputs(2, T, k)
    if dtype == "bf16":
        assert np.array_equal(round_to_bf16(x), x)
    mats = [m.packed() for m in (layer.gate, layer.up, layer.down)]
    for act in ("silu", "gelu_tanh"):  # the identity at 64
        y, _ = moe_ref(*mats, group, group, x, ids, w, act)
        assert np.array_equal(y, layer.ref(x, ids, w)[0])
    f = np.float32(64)
    assert np.float32(1) + np.exp(-f) == 1 and f / (np.float32(1) + np.exp(-f)) == f


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_activations_layer_is_the_oracles(zeros, act):
    layer = ActLayer(3, 3, 72, 40, 136, 32, zeros)
    x, ids, w = ExactLayer(1, 3, 72, 40, 136, 32, zeros, "f32").inputs(4, 4, 2)
    y, _ = moe_ref(*[m.packed() for m in (layer.gate, layer.up, layer.down)], 32, 32, x, ids, w, act)
    assert np.allclose(y, act_bounds(layer, x, ids, w, act, "f32")[0], rtol=1e-13)


# Every case: with a fault, at least one output is out of its bounds.
@pytest.mark.parametrize("case", CASES + LONG, ids=lambda c: "-".join(map(str, c)))
def test_faults_are_seen(case):
    T, k, n, d, ffn, group, zeros, _, dtype, act = case
    layer = ExactLayer(5, n, d, ffn, d, group, zeros, dtype)
    a = layer.inputs(6, T, k)
    y, bound = exact_bounds(layer, *a)
    fine = lambda v: (np.abs(held(v, dtype) - y) <= bound).all()  # noqa: E731
    assert fine(layer.ref(*a)[0])
    faults = [dict(features=ffn - 8), dict(inputs=d - 8)] if d > 8 and ffn > 8 else []
    faults += [dict(features=ffn // 128 * 128)] if ffn % 128 and ffn > 128 else []
    faults += [dict(keep_h=8), dict(keep_h=12)] if layer.two else []
    faults += [dict(keep_x=16), dict(keep_h=16)] if dtype == "f32" else []
    for fault in faults:
        assert not fine(layer.ref(*a, **fault)[0]), fault
    # bf16 rows: 16 bits are what h needs
    if dtype == "bf16":
        assert fine(layer.ref(*a, keep_h=16)[0])
        assert all(np.array_equal(cut(layer.h(a[0], e), 16), layer.h(a[0], e)) for e in range(n))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_the_other_activation_is_seen(case):
    T, k, n, d, ffn, group, zeros, _, dtype, act = case
    layer = ActLayer(7, n, d, ffn, d, group, zeros)
    x, ids, w = ExactLayer(5, n, d, ffn, d, group, zeros, dtype).inputs(8, T, k)
    y, bound = act_bounds(layer, x, ids, w, act, dtype)
    other = act_bounds(layer, x, ids, w, "silu" if act == "gelu_tanh" else "gelu_tanh", dtype)[0]
    # Of tokens without an expert, or of gates that are all large, both are the same.
    assert (np.abs(other - y) > 3 * bound).any()
    assert act_ref("silu", 0.0) == 0
