"""The 8-bit base products on the CPU: sizes, refusals before any HIP call, and
the oracle against exact fractions."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from oracle.w8_ref import w8_apply_ref, w8_product_ref, w8_quantize_ref
from rank_specialized_amd import _lib as L

FAKE = 0x10000  # never dereferenced: every call below is refused, or has nothing to do
F32, BF16 = L.LORA_DTYPE_F32, L.LORA_DTYPE_BF16
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def store(d_in=64, d_out=32):
    s = L.lora_w8_store()
    s.d_in, s.d_out = d_in, d_out
    s.codes = s.scales = FAKE
    return s


def test_bytes(lib):
    def sizes(d_in, d_out):
        c, p = C.c_size_t(), C.c_size_t()
        return lib.lora_w8_bytes(d_in, d_out, C.byref(c), C.byref(p)), c.value, p.value

    # blocks of 64 outputs x 64 inputs, a byte each; 64 float32 scales per block of outputs
    assert sizes(64, 64) == (0, 4096, 256)
    assert sizes(8, 8) == (0, 4096, 256)
    assert sizes(72, 200) == (0, 2 * 4 * 4096, 4 * 256)
    assert sizes(L.LORA_W8_MAX_IN, L.LORA_W8_MAX_OUT) == (0, 2048 * 64 * L.LORA_W8_MAX_OUT, 4 * L.LORA_W8_MAX_OUT)
    for bad in ((0, 64), (64, 0), (-8, 64)):
        assert sizes(*bad)[0] == 1, bad
    for bad in ((60, 64), (64, 4), (L.LORA_W8_MAX_IN + 8, 64), (64, L.LORA_W8_MAX_OUT + 8), (2**31 - 8, 64), (64, 2**31 - 8)):
        assert sizes(*bad)[0] == 2, bad
        s = store(*bad)
        assert lib.lora_w8_workspace_bytes(C.byref(s), 8, 0) == 0
    assert lib.lora_w8_bytes(64, 64, None, None) == 1
    assert 128 * 128 * L.LORA_W8_MAX_IN < 2**31 <= 128 * 128 * (L.LORA_W8_MAX_IN + 8)


def test_workspace(lib):
    s = store(3584, 512)
    for T in (1, 2, 5, 16, 64, 256, 257, 4096, L.LORA_W8_MAX_ROWS):
        n = lib.lora_w8_workspace_bytes(C.byref(s), T, 0)
        assert n == 0 or n >= T * (3584 + 4)  # rows of codes and their scales, or nothing
    for T in (-1, L.LORA_W8_MAX_ROWS + 1):
        assert lib.lora_w8_workspace_bytes(C.byref(s), T, 0) == 0
    assert lib.lora_w8_workspace_bytes(None, 8, 0) == 0


def test_pack_refusals(lib):
    out = L.lora_w8_store()

    def call(o=out, d_in=64, d_out=32, q=FAKE, s=FAKE, sd=F32, c=FAKE, p=FAKE):
        return lib.lora_w8_pack(C.byref(o) if o is not None else None, d_in, d_out, q, s, sd, c, p, None)

    assert call(o=None) == 1 and call(d_in=0) == 1 and call(d_out=-8) == 1
    assert call(q=None) == 1 and call(s=None) == 1 and call(c=None) == 1 and call(p=None) == 1
    assert call(q=FAKE + 4) == 2 and call(s=FAKE + 2) == 2 and call(s=FAKE + 1, sd=BF16) == 2
    assert call(c=FAKE + 8) == 2 and call(p=FAKE + 4) == 2 and call(sd=7) == 2 and call(d_in=68) == 2
    assert lib.lora_last_hip_error() == 0 and out.codes is None


def test_quantize_refusals(lib):
    def call(dt=BF16, x=FAKE, ldx=64, T=4, d_in=64, q=FAKE, ldq=64, s=FAKE):
        return lib.lora_w8_quantize(dt, x, ldx, T, d_in, q, ldq, s, None)

    assert call(T=0) == 0 and call(T=0, x=None, q=None, s=None) == 0
    assert call(T=-1) == 1 and call(d_in=0) == 1 and call(ldx=56) == 1 and call(ldq=48) == 1
    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1
    assert call(dt=5) == 2 and call(x=FAKE + 8) == 2 and call(ldx=68) == 2 and call(ldx=66, dt=F32) == 2
    assert call(q=FAKE + 8) == 2 and call(ldq=72) == 2 and call(s=FAKE + 2) == 2 and call(d_in=60) == 2
    assert call(ldq=L.LORA_W8_MAX_LDQ + 16) == 2 and call(T=L.LORA_W8_MAX_ROWS + 1) == 2
    assert call(d_in=L.LORA_W8_MAX_IN + 8, ldx=1 << 18, ldq=1 << 18) == 2
    assert lib.lora_last_hip_error() == 0


def test_apply_refusals(lib):
    def call(s=store(), dt=BF16, x=FAKE, ldx=64, y=FAKE, ldy=32, T=4, ws=FAKE, wsb=BIG):
        return lib.lora_w8_apply(C.byref(s) if s is not None else None, dt, x, ldx, y, ldy, T, ws, wsb, None)

    assert call(T=0) == 0 and call(T=0, x=None, y=None, ws=None, wsb=0) == 0
    assert call(s=None) == 1 and call(T=-1) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(ldx=56) == 1 and call(ldy=24) == 1
    assert call(dt=5) == 2 and call(x=FAKE + 8) == 2 and call(y=FAKE + 2) == 2 and call(ldx=68) == 2
    assert call(ldy=36) == 2 and call(ldx=66, dt=F32) == 2 and call(T=L.LORA_W8_MAX_ROWS + 1) == 2
    assert call(s=store(60)) == 2 and call(s=store(64, 36)) == 2
    bad = store()
    bad.codes = None
    assert call(s=bad) == 1
    bad.codes = FAKE + 8
    assert call(s=bad) == 2
    bad = store()
    bad.scales = FAKE + 4
    assert call(s=bad) == 2
    need = lib.lora_w8_workspace_bytes(C.byref(store()), 4096, 0)
    assert need > 0
    assert call(T=4096, ws=None) == 1 and call(T=4096, wsb=need - 1) == 1 and call(T=4096, ws=FAKE + 8) == 2
    assert lib.lora_last_hip_error() == 0


def test_apply_quantized_refusals(lib):
    def call(s=store(), q=FAKE, ldq=64, sc=FAKE, dt=BF16, y=FAKE, ldy=32, T=4, ws=FAKE, wsb=BIG):
        return lib.lora_w8_apply_quantized(C.byref(s) if s is not None else None, q, ldq, sc, dt, y, ldy, T, ws, wsb, None)

    assert call(T=0) == 0 and call(T=0, q=None, sc=None, y=None) == 0
    assert call(s=None) == 1 and call(T=-1) == 1 and call(q=None) == 1 and call(sc=None) == 1 and call(y=None) == 1
    assert call(ldq=48) == 1 and call(ldy=24) == 1
    assert call(q=FAKE + 8) == 2 and call(ldq=72) == 2 and call(sc=FAKE + 2) == 2 and call(dt=4) == 2
    assert call(y=FAKE + 8) == 2 and call(ldy=36) == 2 and call(T=L.LORA_W8_MAX_ROWS + 1) == 2
    assert call(ldq=L.LORA_W8_MAX_LDQ + 16) == 2
    need = lib.lora_w8_workspace_bytes(C.byref(store()), 4096, 1)
    if need:
        assert call(T=4096, ws=None) == 1 and call(T=4096, wsb=need - 1) == 1 and call(T=4096, ws=FAKE + 8) == 2
    assert lib.lora_last_hip_error() == 0


def test_binding_refusals():
    """The binding's own checks come before the library's."""
    q, s = torch.zeros(16, 64, dtype=torch.int8), torch.ones(16)
    with pytest.raises(ValueError, match="int8"):
        rs.lora_w8_pack(q.int(), s)
    with pytest.raises(ValueError, match="scales"):
        rs.lora_w8_pack(q, s[:8])
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        rs.lora_w8_pack(q, s.half())
    with pytest.raises(ValueError, match="GPU"):
        rs.lora_w8_pack(q, s)
    with pytest.raises(ValueError, match="GPU"):
        rs.lora_w8_quantize(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        rs.lora_w8_quantize(torch.zeros(2, 64).half())
    b = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        rs.W8Store(store(), b, torch.zeros(64))
    with pytest.raises(ValueError, match="GPU"):
        rs.W8Store(store(), b.to("meta"), torch.zeros(64).to("meta"))
    with pytest.raises(ValueError, match="out of range"):
        rs.lora_w8_bytes(2**32 + 64, 64)
    long = torch.empty(1, 1, dtype=torch.bfloat16, device="meta").expand(2**31, 8)
    with pytest.raises(ValueError, match="more rows"):
        rs.lora_w8_quantize(long)


def test_rows_of_codes_reach_to_a_multiple_of_16():
    """The kernels read rows of codes in pieces of 16 bytes: a last row that
    ends inside one at the end of its memory is refused."""
    ok = torch.zeros(3, 32, dtype=torch.int8)[:, :24]
    assert rs._codes(ok, 3, 24, "q") == 32 and rs._codes(ok[:1], 1, 24, "q") == 32
    assert rs._codes(torch.zeros(3, 64, dtype=torch.int8), 3, 64, "q") == 64
    for bad in (torch.zeros(88, dtype=torch.int8).as_strided((3, 24), (32, 1)), torch.zeros(1, 24, dtype=torch.int8)):
        with pytest.raises(ValueError, match="multiple of 16"):
            rs._codes(bad, bad.shape[0], 24, "q")
    for bad in (torch.zeros(3, 24), torch.zeros(3, 16, dtype=torch.int8), torch.zeros(4, 24, dtype=torch.int8)):
        with pytest.raises(ValueError, match="int8"):
            rs._codes(bad, 3, 24, "q")
    with pytest.raises(ValueError, match="unit column stride"):
        rs._codes(torch.zeros(3, 64, dtype=torch.int8)[:, ::2], 3, 32, "q")
    with pytest.raises(ValueError, match="unit column stride"):
        rs._codes(torch.zeros(1, 64, dtype=torch.int8)[:, ::2], 1, 32, "q")


# ------------------------------------------------------------ the oracle
def nearest(v: Fraction) -> int:
    return round(v)  # of a Fraction: exact, half to even


def test_oracle_quantize():
    rng = np.random.default_rng(0)
    rows = [rng.normal(size=40), np.zeros(40), np.full(40, -3.0), np.arange(-20, 20) / 2.0 * 1.984375, 1e-44 * np.arange(40),
            3e38 * rng.uniform(-1, 1, 40)]
    rows.append(np.concatenate([[254.0], np.arange(39) + 0.0]))  # steps of two: every odd value is a border
    x = np.array(rows).astype(np.float32)
    q, s = w8_quantize_ref(x)
    for t in range(x.shape[0]):
        a = max(Fraction(float(v)) for v in np.abs(x[t]))
        for k in range(40):
            assert q[t, k] == (nearest(127 * Fraction(float(x[t, k])) / a) if a else 0)
        assert s[t] == float(a) / 127
    assert q[6, 1:8].tolist() == [0, 0, 1, 2, 2, 2, 3]
    for bad in (np.nan, np.inf, -np.inf):
        x[0, 3] = bad
        q, s = w8_quantize_ref(x)
        assert np.isnan(s[0]) and not q[0].any() and s[2] == 3 / 127


def test_oracle_product():
    rng = np.random.default_rng(1)
    w, sw, x = rng.integers(-128, 128, (6, 24)), rng.random(6), rng.normal(size=(3, 24)).astype(np.float32)
    q, s = w8_quantize_ref(x)
    y = w8_product_ref(q, s, w, sw)
    for t in range(3):
        for o in range(6):
            assert np.isclose(y[t, o], s[t] * sw[o] * sum(int(a) * int(b) for a, b in zip(q[t], w[o])))
    # within half a step of each activation of the unrounded product
    full = x.astype(np.float64) @ (w * sw[:, None]).T
    assert (np.abs(w8_apply_ref(x, w, sw) - full) <= 0.5 * s[:, None] * (np.abs(w) * sw[:, None]).sum(1) + 1e-12).all()
    assert np.array_equal(w8_apply_ref(2 * x, w, sw), 2 * w8_apply_ref(x, w, sw))
