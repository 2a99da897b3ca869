"""The mixture-of-experts layer on the CPU: sizes, refusals before any HIP
call, and the oracle against a layer written out."""
import ctypes as C

import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from oracle.moe_ref import act_ref, moe_ref
from oracle.w4_ref import experts_ref, w4_matrix_ref
from rank_specialized_amd import _lib as L

FAKE = 0x10000  # never dereferenced: every call below is refused, or has nothing to do
F32, BF16 = L.LORA_DTYPE_F32, L.LORA_DTYPE_BF16
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def store(n=4, d_in=64, d_out=40, group=32, scale_dtype=BF16, has_zeros=0):
    s = L.lora_w4_store()
    s.n, s.d_in, s.d_out, s.group, s.scale_dtype, s.has_zeros = n, d_in, d_out, group, scale_dtype, has_zeros
    s.codes = s.params = FAKE
    return s


def down(**kw):
    return store(**{**dict(d_in=40, d_out=64), **kw})


def test_workspace(lib):
    def need(T, k, g=store(), u=store(), d=down(), dt=BF16):
        return lib.lora_w4_moe_workspace_bytes(C.byref(g), C.byref(u), C.byref(d), dt, T, k)

    assert need(0, 2) == 0
    for T, k in ((1, 1), (1, 8), (7, 4), (64, 32)):
        assert need(T, k) >= T * k * 2 * 128 * 2 and need(T, k, dt=F32) > need(T, k)
    for bad in ((-1, 2), (1, 0), (L.LORA_W4_MOE_MAX_TOKENS + 1, 2), (1, L.LORA_W4_MOE_MAX_K + 1)):
        assert need(*bad) == 0
    assert need(1, 1, dt=9) == 0 and need(1, 1, d=down(d_in=48)) == 0
    assert lib.lora_w4_moe_workspace_bytes(None, C.byref(store()), C.byref(down()), BF16, 1, 1) == 0


def test_refusals(lib):
    def call(g=store(), u=store(), d=down(), dt=BF16, act=0, x=FAKE, ldx=64, y=FAKE, ldy=64, T=4, k=2, ids=FAKE, w=FAKE,
             ws=FAKE, wsb=BIG):
        ref = [C.byref(s) if s is not None else None for s in (g, u, d)]
        return lib.lora_w4_moe(*ref, dt, act, x, ldx, y, ldy, T, k, ids, w, ws, wsb, None)

    assert call(T=0) == 0 and call(T=0, x=None, y=None, ids=None, w=None, ws=None, wsb=0) == 0
    assert call(g=None) == 1 and call(u=None) == 1 and call(d=None) == 1
    assert call(T=-1) == 1 and call(k=0) == 1 and call(act=2) == 1 and call(act=-1) == 1
    assert call(x=None) == 1 and call(y=None) == 1 and call(ids=None) == 1 and call(w=None) == 1
    assert call(ldx=56) == 1 and call(ldy=56) == 1
    for other in (dict(n=5), dict(d_in=72), dict(d_out=48), dict(group=64), dict(scale_dtype=F32), dict(has_zeros=1)):
        assert call(u=store(**other)) == 1, other
    assert call(d=down(n=3)) == 1 and call(d=down(d_in=32)) == 1
    assert call(d=down(group=64, scale_dtype=F32, has_zeros=1), T=0) == 0  # may differ
    assert call(dt=3) == 2 and call(T=L.LORA_W4_MOE_MAX_TOKENS + 1) == 2 and call(k=L.LORA_W4_MOE_MAX_K + 1) == 2
    assert call(x=FAKE + 8) == 2 and call(y=FAKE + 4) == 2 and call(ids=FAKE + 2) == 2 and call(w=FAKE + 1) == 2
    assert call(ldx=68) == 2 and call(ldy=68) == 2
    big = L.LORA_W4_MOE_MAX_FFN + 8
    assert call(g=store(d_out=big), u=store(d_out=big), d=down(d_in=big)) == 2
    assert call(g=store(d_in=60), u=store(d_in=60)) == 2
    bad = store()
    bad.codes = None
    assert call(u=bad) == 1
    bad.codes = FAKE + 8
    assert call(u=bad) == 2
    need = lib.lora_w4_moe_workspace_bytes(C.byref(store()), C.byref(store()), C.byref(down()), BF16, 4, 2)
    assert call(ws=None) == 1 and call(wsb=need - 1) == 1 and call(ws=FAKE + 8) == 2
    assert lib.lora_last_hip_error() == 0


def test_experts_as_wide_as_any_matrix(lib):
    """h goes through LDS in pieces, as x does: ffn is bounded as every side of
    a 4-bit matrix is."""
    for ffn in (16392, 18944, 32776, 1 << 20):
        g, d = store(d_out=ffn), down(d_in=ffn)
        for dt, parts in ((BF16, 2), (F32, 3)):
            need = lib.lora_w4_moe_workspace_bytes(C.byref(g), C.byref(g), C.byref(d), dt, 64, 32)
            assert need >= 64 * 32 * parts * 2 * ffn, ffn
        assert lib.lora_w4_moe(C.byref(g), C.byref(g), C.byref(d), BF16, 0, None, 64, None, 64, 0, 2, None, None, None, 0, None) == 0
    assert lib.lora_last_hip_error() == 0


class Held:
    """What the binding's checks read of a store."""
    device_index, d_in, d_out, n = 0, 64, 40, 4


def test_binding_refusals():
    x, ids, w = torch.zeros(2, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    s = Held()
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        rs.lora_w4_moe(s, s, s, x.half(), ids, w)
    with pytest.raises(ValueError, match="ids"):
        rs.lora_w4_moe(s, s, s, x, ids.long(), w)
    with pytest.raises(ValueError, match="ids"):
        rs.lora_w4_moe(s, s, s, x, torch.zeros(2, 6, dtype=torch.int32)[:, ::2], w)
    with pytest.raises(ValueError, match="weights"):
        rs.lora_w4_moe(s, s, s, x, ids, w[:, :2])
    with pytest.raises(ValueError, match="weights"):
        rs.lora_w4_moe(s, s, s, x, ids, w.double())
    with pytest.raises(ValueError, match="x must"):
        rs.lora_w4_moe(s, s, s, x[:, :32], ids, w)
    with pytest.raises(ValueError, match="x must"):
        rs.lora_w4_moe(s, s, s, x[:1], ids, w)
    with pytest.raises(ValueError, match="act"):
        rs.lora_w4_moe(s, s, s, x, ids, w, act="relu")
    with pytest.raises(ValueError, match="not on cuda"):
        rs.lora_w4_moe(s, s, s, x, ids, w)
    other = Held()
    other.device_index = 1
    with pytest.raises(ValueError, match="one GPU"):
        rs.lora_w4_moe(s, s, other, x, ids, w)


# ------------------------------------------------------------ the oracle
def experts(rng, n, d_out, d_in, group, zeros):
    shape = (n, d_out, -(-d_in // group))
    return (rng.integers(0, 256, (n, d_out, d_in // 2), dtype=np.uint8), rng.normal(size=shape) / 40,
            rng.integers(0, 16, shape).astype(np.uint8) if zeros else None)


def test_oracle_act():
    g = np.linspace(-9, 9, 37)
    assert np.allclose(act_ref("silu", g), [v * (1 / (1 + np.exp(-v))) for v in g])
    v = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert np.allclose(act_ref("gelu_tanh", g), g / (1 + np.exp(-2 * v)), atol=1e-14)
    for kind in ("silu", "gelu_tanh"):  # the bound's slope
        f = np.linspace(-30, 30, 600001)
        assert np.abs(np.diff(act_ref(kind, f)) / np.diff(f)).max() < 1.13


def test_oracle_layer():
    rng = np.random.default_rng(0)
    G, U, D = experts(rng, 3, 24, 40, 32, True), experts(rng, 3, 24, 40, 32, True), experts(rng, 3, 16, 24, 64, False)
    x, ids, w = rng.normal(size=(4, 40)), np.array([[0, 2], [1, 1], [-1, 2], [3, -9]]), rng.random((4, 2))
    y, bound = moe_ref(G, U, D, 32, 64, x, ids, w)
    mat = lambda m, e, g: w4_matrix_ref(m[0][e], m[1][e], None if m[2] is None else m[2][e], g)  # noqa: E731
    layer = lambda t, e: mat(D, e, 64) @ (act_ref("silu", mat(G, e, 32) @ x[t]) * (mat(U, e, 32) @ x[t]))  # noqa: E731
    assert np.allclose(y[0], w[0, 0] * layer(0, 0) + w[0, 1] * layer(0, 2))
    assert np.allclose(y[1], w[1].sum() * layer(1, 1))
    assert np.allclose(y[2], w[2, 1] * layer(2, 2)) and not y[3].any()
    # the same layer out of the experts' products
    rows = [experts_ref(*m, 32, x, ids) for m in (G, U)]
    again = experts_ref(*D, 64, act_ref("silu", rows[0]) * rows[1], ids, w)
    assert np.allclose(y, again)
    assert (bound[:3] > 0).all() and not bound[3].any()
    # float32 arithmetic in one order of many stays within the bound
    f = lambda v: np.asarray(v, np.float32)  # noqa: E731
    for t in range(3):
        z = np.zeros(16, np.float32)
        for j in range(2):
            e = ids[t, j]
            if e >= 0:
                g, u = f(mat(G, e, 32)) @ f(x[t]), f(mat(U, e, 32)) @ f(x[t])
                h = g / (1 + np.exp(-g)) * u
                z = z + f(w[t, j]) * (f(mat(D, e, 64)) @ h)
        exact = moe_ref(G, U, D, 32, 64, f(x), ids, f(w))[0][t]
        assert (np.abs(z - exact) <= bound[t] + 2.0 ** -23 * np.abs(exact)).all()
