"""The choice between the mixture-of-experts layer's kernels on the CPU: the rule
of csrc/moe.h and moe_layer.h restated, so that the GPU tests' sizes are known to
reach every kernel."""
import ctypes as C

import pytest

from rank_specialized_amd import _lib as L
from test_gpu_moe import CASES


def two_tiles(T, k, n, parts):
    return T > 16 // parts and 2 * T * k * parts > 16 * n


def kernels(case):
    """(rows' parts, tiles of 16 rows, blocks, waves to a block) of the first
    kernel, (tiles of 16 rows, blocks, waves to a wave's blocks) of the second."""
    T, k, n, d, ffn, group, _, _, dtype, _ = case
    x_parts, h_parts = (1, 2) if dtype == "bf16" else (3, 3)
    entries, h_tiles = min(T * k, n), -(-ffn // 128)
    if two_tiles(T, k, n, h_parts):
        down = (2, 8, 2)
    else:
        deep = entries * -(-d // 64) <= 256 and h_tiles >= 16
        down = (1, 4, 8 if deep else 2)
    if two_tiles(T, k, n, x_parts):
        return (x_parts, 2, 2, 4), down
    if dtype == "f32" and 2 * entries * h_tiles < 256:
        return (x_parts, 1, 1, 4), down
    if dtype == "bf16" and group % 128 == 0 and entries * h_tiles >= 512 and T * k >= 4 * n:
        return (x_parts, 1, 8, 1), down
    return (x_parts, 1, 4, 2), down


def test_sizes_reach_every_kernel():
    up, down = zip(*(kernels(c) for c in CASES))
    assert set(up) == {(1, 1, 4, 2), (1, 1, 8, 1), (1, 2, 2, 4), (3, 1, 1, 4), (3, 1, 4, 2), (3, 2, 2, 4)}
    assert set(zip((u[0] for u in up), down)) == {(p, d) for p in (1, 3) for d in ((1, 4, 2), (1, 4, 8), (2, 8, 2))}


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_workspace_follows(case):
    T, k, n, d, ffn, group, zeros, scales, dtype, _ = case
    s = [L.lora_w4_store() for _ in range(3)]
    for st, d_in, d_out in zip(s, (d, d, ffn), (ffn, ffn, d)):
        st.n, st.d_in, st.d_out, st.group, st.has_zeros = n, d_in, d_out, group, zeros
        st.scale_dtype, st.codes, st.params = (L.LORA_DTYPE_F32 if scales == "f32" else L.LORA_DTYPE_BF16), 0x10000, 0x10000
    need = L.lib().lora_w4_moe_workspace_bytes(*(C.byref(v) for v in s), L.LORA_DTYPE_F32 if dtype == "f32" else L.LORA_DTYPE_BF16, T, k)
    R, blocks = T * k, kernels(case)[1][1]
    groups = -(-(-(-d // 16)) // blocks)
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    h = R * (2 if dtype == "bf16" else 3) * -(-ffn // 128) * 256
    assert need == up(h) + up(min(R, n) * (8 + 6 * 64)) + up(groups * R * 16 * blocks * 4) + up(R) + up(4 * groups)
