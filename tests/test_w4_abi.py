"""The 4-bit base products and the router on the CPU: sizes, refusals before
any HIP call, and the oracle against identities of its own."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import rank_specialized_amd as rs
from oracle.w4_ref import experts_ref, route_ref, unpack_ref, w4_apply_ref, w4_matrix_ref
from rank_specialized_amd import _lib as L

FAKE = 0x10000  # never dereferenced: every call below is refused, or has nothing to do
F32, BF16 = L.LORA_DTYPE_F32, L.LORA_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def store(n=1, d_in=64, d_out=32, group=32, scale_dtype=BF16, has_zeros=0):
    s = L.lora_w4_store()
    s.n, s.d_in, s.d_out, s.group, s.scale_dtype, s.has_zeros = n, d_in, d_out, group, scale_dtype, has_zeros
    s.codes = s.params = FAKE
    return s


def test_bytes(lib):
    def sizes(*a):
        c, p = C.c_size_t(), C.c_size_t()
        return lib.lora_w4_bytes(*a, C.byref(c), C.byref(p)), c.value, p.value

    # tiles of 16 x 128 codes, half a byte each; per tile 16 x (128 / gran) scales of 2, 4 or 8 bytes
    assert sizes(1, 128, 16, 128, BF16, 0) == (0, 1024, 32)
    assert sizes(1, 136, 24, 128, BF16, 0) == (0, 4 * 1024, 4 * 32)
    assert sizes(3, 128, 16, 64, BF16, 1) == (0, 3 * 1024, 3 * 16 * 2 * 4)
    assert sizes(1, 128, 16, 96, F32, 0) == (0, 1024, 16 * 4 * 8)
    assert sizes(1, 256, 16, 256, BF16, 0) == (0, 2048, 2 * 32)
    for bad in ((0, 128, 16, 128, BF16, 0), (1, 0, 16, 128, BF16, 0), (1, 128, -8, 128, BF16, 0),
                (1, 128, 16, 0, BF16, 0), (1, 128, 16, 128, BF16, 2)):
        assert sizes(*bad)[0] == 1, bad
    for bad in ((L.LORA_W4_MAX_N + 1, 128, 16, 128, BF16, 0), (1, 124, 16, 128, BF16, 0), (1, 128, 12, 128, BF16, 0),
                (1, 128, 16, 48, BF16, 0), (1, 128, 16, 128, 7, 0)):
        assert sizes(*bad)[0] == 2, bad
    assert lib.lora_w4_bytes(1, 128, 16, 128, BF16, 0, None, None) == 1


def test_sizes_at_their_limits(lib):
    """The largest sizes that are taken give the bytes that they should; one
    step more is refused, sizes near the largest int too."""
    d, n, big = L.LORA_W4_MAX_DIM, L.LORA_W4_MAX_N, 2**31 - 8
    c, p = C.c_size_t(), C.c_size_t()

    def status(n, d_in, d_out, group=128, kind=(BF16, 0)):
        return lib.lora_w4_bytes(n, d_in, d_out, group, *kind, C.byref(c), C.byref(p))

    assert status(n, d, d, 32, (F32, 1)) == 0
    assert (c.value, p.value) == (n * d * d // 2, n * d * (d // 32) * 8)
    # 2^31 - 32 is 96 more than a multiple of 128: four scales per tile row (gcd 32) of 2 bytes
    assert status(1, 64, 32, 2**31 - 32) == 0 and (c.value, p.value) == (2 * 1024, 2 * 16 * 4 * 2)
    for bad in ((1, d + 8, 16), (1, 128, d + 8), (1, big, 16), (1, 128, big), (n + 1, 128, 16)):
        assert status(*bad) == 2, bad
        s = store(n=bad[0], d_in=bad[1], d_out=bad[2], group=128)
        assert lib.lora_w4_workspace_bytes(C.byref(s), BF16, 4, 0, 0) == 0
    for T in (1, 16, 128, 4096, L.LORA_W4_MAX_ROWS):
        for k in (0, 1):
            for dt in (BF16, F32):  # the plan of every call that is taken can be made
                s = store(n=1 if k == 0 else n, d_in=d, d_out=d)
                assert 0 <= lib.lora_w4_workspace_bytes(C.byref(s), dt, T, k, k) < 1 << 56
    fake = 0x10000
    for T, want in ((0, 0), (L.LORA_ROUTE_MAX_TOKENS + 1, 2), (2**31 - 1, 2)):
        assert lib.lora_route(fake, 8, BF16, T, 8, 2, 0, None, 1, 1, 1, 1.0, fake, fake, None) == want
    assert lib.lora_last_hip_error() == 0


def test_pack_refusals(lib):
    out = L.lora_w4_store()

    def call(o=out, n=1, d_in=64, d_out=32, group=32, q=FAKE, s=FAKE, sd=BF16, z=None, c=FAKE, p=FAKE):
        return lib.lora_w4_pack(C.byref(o) if o is not None else None, n, d_in, d_out, group, q, s, sd, z, c, p, None)

    assert call(o=None) == 1
    assert call(n=0) == 1
    assert call(q=None) == 1 and call(s=None) == 1 and call(c=None) == 1 and call(p=None) == 1
    assert call(q=FAKE + 2) == 2 and call(s=FAKE + 1) == 2 and call(s=FAKE + 2, sd=F32) == 2
    assert call(c=FAKE + 8) == 2 and call(p=FAKE + 4) == 2
    assert call(group=40) == 2 and call(d_in=60) == 2 and call(sd=9) == 2
    assert lib.lora_last_hip_error() == 0


def test_apply_refusals(lib):
    big = 1 << 40

    def call(s=store(), dt=BF16, x=FAKE, ldx=64, y=FAKE, ldy=32, T=4, ws=FAKE, wsb=big):
        return lib.lora_w4_apply(C.byref(s) if s is not None else None, dt, x, ldx, y, ldy, T, ws, wsb, None)

    assert call(T=0) == 0 and call(T=0, x=None, y=None, ws=None, wsb=0) == 0
    assert call(s=None) == 1 and call(s=store(n=2)) == 1 and call(T=-1) == 1
    assert call(x=None) == 1 and call(y=None) == 1 and call(ldx=56) == 1 and call(ldy=24) == 1
    assert call(dt=5) == 2 and call(x=FAKE + 8) == 2 and call(y=FAKE + 2) == 2
    assert call(ldx=68) == 2 and call(ldy=36) == 2 and call(ldx=66, dt=F32) == 2
    assert call(s=store(d_in=60)) == 2 and call(s=store(group=16)) == 2
    assert call(T=L.LORA_W4_MAX_ROWS + 1) == 2
    bad = store()
    bad.codes = None
    assert call(s=bad) == 1
    bad.codes = FAKE + 8
    assert call(s=bad) == 2
    need = lib.lora_w4_workspace_bytes(C.byref(store()), BF16, 4096, 0, 0)
    if need:
        assert call(T=4096, ws=None) == 1 and call(T=4096, wsb=need - 1) == 1 and call(T=4096, ws=FAKE + 8) == 2
    assert lib.lora_last_hip_error() == 0


def test_experts_refusals(lib):
    big = 1 << 40
    st = store(n=4)

    def call(s=st, dt=BF16, x=FAKE, ldx=64, per=0, y=FAKE, ldy=32, T=4, k=2, ids=FAKE, w=None, ws=FAKE, wsb=big):
        return lib.lora_w4_apply_experts(C.byref(s) if s is not None else None, dt, x, ldx, per, y, ldy, T, k, ids, w,
                                         ws, wsb, None)

    assert call(T=0) == 0 and call(T=0, ids=None) == 0
    assert call(s=None) == 1 and call(k=0) == 1 and call(T=-1) == 1 and call(per=2) == 1 and call(ids=None) == 1
    assert call(x=None) == 1 and call(y=None) == 1 and call(ldx=8) == 1 and call(ldy=8) == 1
    assert call(dt=3) == 2 and call(x=FAKE + 4) == 2 and call(ids=FAKE + 2) == 2 and call(w=FAKE + 1) == 2
    assert call(T=L.LORA_W4_MAX_ROWS, k=2) == 2
    need = lib.lora_w4_workspace_bytes(C.byref(st), BF16, 512, 2, 1)
    assert need > 0
    assert call(T=512, w=FAKE, ws=None) == 1 and call(T=512, w=FAKE, wsb=need - 1) == 1
    assert call(T=512, w=FAKE, ws=FAKE + 4) == 2
    assert lib.lora_w4_workspace_bytes(None, BF16, 8, 1, 0) == 0
    assert lib.lora_w4_workspace_bytes(C.byref(st), BF16, -1, 1, 0) == 0
    assert lib.lora_last_hip_error() == 0


def test_route_refusals(lib):
    def call(l=FAKE, ldl=64, dt=F32, T=4, E=64, k=8, score=0, bias=None, g=1, tg=1, ids=FAKE, w=FAKE):
        return lib.lora_route(l, ldl, dt, T, E, k, score, bias, g, tg, 1, 1.0, ids, w, None)

    assert call(T=0) == 0 and call(T=0, l=None, ids=None, w=None) == 0
    assert call(T=-1) == 1 and call(E=0) == 1 and call(k=0) == 1 and call(ldl=63) == 1 and call(score=2) == 1
    assert call(g=0) == 1 and call(g=3) == 1 and call(g=8, tg=0) == 1 and call(g=8, tg=9) == 1
    assert call(g=16, tg=1, k=5) == 1  # more than the experts of one group
    assert call(k=65) == 1
    assert call(l=None) == 1 and call(ids=None) == 1 and call(w=None) == 1
    assert call(dt=4) == 2 and call(l=FAKE + 2) == 2 and call(ids=FAKE + 2) == 2 and call(bias=FAKE + 1) == 2
    assert call(k=L.LORA_ROUTE_MAX_K + 1) == 2
    assert call(E=L.LORA_ROUTE_MAX_EXPERTS + 64, ldl=2048) == 2
    assert call(E=512, ldl=512, g=128, tg=4) == 2
    assert lib.lora_last_hip_error() == 0


def test_binding_refusals():
    """The binding's own checks come before the library's."""
    q = torch.zeros(4, 16, 32, dtype=torch.uint8)
    s = torch.ones(4, 16, 2)
    with pytest.raises(ValueError, match="scales"):
        rs.lora_w4_pack(q, s[:, :, :1], group=32)
    with pytest.raises(ValueError, match="zeros"):
        rs.lora_w4_pack(q, s, torch.zeros(4, 16, 2), group=32)
    with pytest.raises(ValueError, match="uint8"):
        rs.lora_w4_pack(q.int(), s, group=32)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        rs.lora_w4_pack(q, s.half(), group=32)
    with pytest.raises(ValueError, match="GPU"):
        rs.lora_w4_pack(q, s, group=32)
    with pytest.raises(ValueError, match="group"):
        rs.lora_w4_pack(q, s, group=0)
    with pytest.raises(ValueError, match="GPU"):
        rs.lora_route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="score"):
        rs.lora_route(torch.zeros(2, 8), 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        rs.lora_route(torch.zeros(2, 8), 2, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="positive"):
        rs.lora_route(torch.zeros(2, 8), 0)


# ------------------------------------------------------------ the oracle
def test_oracle_unpack_and_matrix():
    packed = np.array([[0x21, 0x43, 0xF0, 0x8F]], np.uint8)
    assert unpack_ref(packed).tolist() == [[1, 2, 3, 4, 0, 15, 15, 8]]
    w = w4_matrix_ref(packed, np.array([[0.5]]), None, 32)
    assert w.tolist() == [[-3.5, -3.0, -2.5, -2.0, -4.0, 3.5, 3.5, 0.0]]
    w = w4_matrix_ref(packed, np.array([[1.0, 2.0]]), np.array([[1, 15]], np.uint8), 4)
    assert w.tolist() == [[0, 1, 2, 3, -30, 0, 0, -14]]


def test_oracle_products():
    rng = np.random.default_rng(0)
    packed = rng.integers(0, 256, (3, 8, 24), dtype=np.uint8)
    scales, zeros = rng.random((3, 8, 2)), rng.integers(0, 16, (3, 8, 2)).astype(np.uint8)
    x = rng.normal(size=(4, 48))
    ids = np.array([[0, 2], [1, 1], [-1, 2], [3, -7]])
    rows = experts_ref(packed, scales, zeros, 32, x, ids)
    assert np.allclose(rows[0], w4_apply_ref(packed[0], scales[0], zeros[0], 32, x[:1])[0])
    assert np.array_equal(rows[2], rows[3])
    assert not rows[4].any() and not rows[6].any() and not rows[7].any()
    w = rng.random((4, 2))
    y = experts_ref(packed, scales, zeros, 32, x, ids, w)
    assert np.allclose(y[0], w[0, 0] * rows[0] + w[0, 1] * rows[1]) and not y[3].any()
    # doubling the scales doubles the result; a code equal to its zero point adds nothing
    assert np.allclose(w4_apply_ref(packed[0], 2 * scales[0], zeros[0], 32, x), 2 * w4_apply_ref(packed[0], scales[0], zeros[0], 32, x))
    same = np.full((8, 24), 0x55, np.uint8)
    assert not w4_apply_ref(same, scales[0], np.full((8, 2), 5, np.uint8), 32, x).any()


def test_oracle_route():
    l = np.array([[1.0, 3.0, 3.0, -math.inf, 2.0, math.nan]])
    ids, w = route_ref(l, 4)
    assert ids.tolist() == [[1, 2, 4, 0]]  # the tie goes to the lower index
    assert np.allclose(w[0], np.exp([0, 0, -1, -2]) / np.exp([0, 0, -1, -2]).sum())
    ids, w = route_ref(l, 6, score="sigmoid", renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2, 4, 0, -1, -1]] and w[0, 4] == 0 and math.isclose(w[0, 0], 2 / (1 + math.exp(-3)))
    # two groups of three: sums of two, or the largest
    ids, _ = route_ref(np.array([[5.0, -9, -9, 2, 2, 0]]), 2, groups=2, top_groups=1)
    assert ids.tolist() == [[0, 1]]
    ids, _ = route_ref(np.array([[5.0, -9, -9, 2, 2, 0]]), 2, score="sigmoid", groups=2, top_groups=1)
    assert ids.tolist() == [[3, 4]]
    # the bias chooses, the score weighs
    ids, w = route_ref(np.array([[0.0, 1.0]]), 1, bias=[10.0, 0.0], renormalize=False)
    assert ids.tolist() == [[0]] and math.isclose(w[0, 0], 1 / (1 + math.e))
    ids, w = route_ref(np.full((1, 3), -math.inf), 2)
    assert ids.tolist() == [[-1, -1]] and not w.any()


def test_sizes_beyond_an_int():
    """ctypes cuts an int to 32 bits: the binding refuses what it would cut
    (a group of 2^32 + 32 would read scales that are not there)."""
    wrap = 2**32
    q, s = torch.zeros(16, 64, dtype=torch.uint8), torch.ones(16, 1)
    for bad in (wrap + 32, wrap + 128, -wrap + 32):
        with pytest.raises(ValueError, match="group"):
            rs.lora_w4_pack(q, s, group=bad)
    for bad in ((wrap + 1, 128, 16, 128), (1, wrap + 128, 16, 128), (1, 128, wrap + 16, 128), (1, 128, 16, wrap + 128)):
        with pytest.raises(ValueError, match="out of range"):
            rs.lora_w4_bytes(*bad, torch.bfloat16, False)
    long = torch.empty(1, 1, dtype=torch.bfloat16, device="meta").expand(2**31, 8)
    wide = torch.empty(1, 1, dtype=torch.bfloat16, device="meta").expand(1, 2**31)
    with pytest.raises(ValueError, match="more rows"):
        rs.lora_w4_apply(None, long)
    for bad in (long, wide):
        with pytest.raises(ValueError, match="more rows"):
            rs.lora_route(bad, 2)
    ids = torch.empty(1, 2**31, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="ids"):
        rs.lora_w4_apply_experts(None, wide, ids)
    with pytest.raises(ValueError, match="k is"):
        rs.lora_route(torch.zeros(1, 8), wrap + 2)


def test_oracle_pair_order():
    """Sums of two sigmoids in order, against 400-digit arithmetic, where
    they differ by more than float64 rounds (2^-50 of the sum, or of its
    distance from one or two)."""
    import decimal

    from oracle.w4_ref import pair_order

    rng, seen = np.random.default_rng(8), 0
    with decimal.localcontext() as ctx:
        ctx.prec = 400

        def exact(a, b):
            return sum(1 / (1 + (-decimal.Decimal(v)).exp()) for v in (a, b))

        for lo, hi in ((20, 60), (-60, -20), (-5, 5), (-300, 300), (40, 41)):
            for _ in range(60):
                p, q = rng.uniform(lo, hi, (2, 2)).astype(np.float32).astype(np.float64).tolist()
                if exact(*p) < exact(*q):
                    p, q = q, p
                sp, sq = exact(*p), exact(*q)
                if sp - sq > min(max(sp, sq), max(2 - sp, 2 - sq), max(abs(1 - sp), abs(1 - sq))) / 2**50:
                    seen += 1
                    assert pair_order(*p) > pair_order(*q), (p, q)
    assert seen > 295
    assert pair_order(-math.inf, 900.0) == pair_order(-math.inf, -math.inf) < pair_order(-800.0, -3e38)
    assert pair_order(0.0, 0.0) == pair_order(1.0, -1.0) == (1, 0.0)


def test_workspace_is_one_run_of_memory():
    """An expanded tensor or a strided view has more bytes by its shape than
    there are behind its address."""
    one = torch.zeros(1, dtype=torch.uint8)
    for bad in (one.expand(1 << 20), torch.zeros(64, 64)[:, ::2], torch.zeros(8, 16).t()):
        with pytest.raises(ValueError, match="contiguous"):
            rs._scratch(bad)
    assert rs._scratch(torch.zeros(64, 8)) == 2048 and rs._scratch(torch.zeros(64, 8)[8:24]) == 512


def test_float32_inputs_need_all_parts():
    """The inputs of the GPU's test of whole float32 rows tell three bf16 parts
    of x from two, in the oracle's product."""
    from test_gpu_w4 import one_input

    def part(v):
        return (v.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)

    for T, d_in, d_out, group in ((5, 4104, 40, 128), (300, 136, 24, 64)):
        packed, s, z, x = one_input(T, d_in, d_out, group)
        hi = part(x)
        mid = part(x - hi)
        assert np.array_equal(hi + mid + (x - hi - mid), x) and ((x - hi - mid).any(1)).all()
        whole = w4_apply_ref(packed[0], s[0], z[0], group, x)
        assert (whole != 0).all()
        assert (w4_apply_ref(packed[0], s[0], z[0], group, hi + mid) != whole).all()


def test_store_is_on_a_gpu():
    """Buffers moved to the host would pass for those of x on the host, and
    the kernels would be given host addresses."""
    b = torch.zeros(2048, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        rs.W4Store(store(), b, b)
    with pytest.raises(ValueError, match="GPU"):
        rs.W4Store(store(), b.to("meta"), b.to("meta"))
