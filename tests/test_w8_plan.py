"""The choice between the 8-bit products' kernels on the CPU: the rule of
csrc/w8.h restated, so that the GPU tests' sizes are known to reach every
kernel."""
import ctypes as C

import pytest

from rank_specialized_amd import _lib as L
from test_gpu_w8 import SIZES


def us(tile, T, d_out, kt):
    empty, load, start = {256: (0.52, 0.27, 4.0), 128: (0.17, 0.09, 4.5), 64: (0.055, 0.055, 4.5)}[tile]
    full, rest = divmod(-(-T // tile) * -(-d_out // tile), 256)
    return full * (kt * (empty + load) + start) + (kt * (empty + load * rest / 256) + start if rest else 0)


def kernel(T, d_in, d_out):
    """The tile of the many-rows kernel, or (tiles of rows, tiles of outputs,
    rounded in the kernel) of the few-rows kernel."""
    kt = -(-d_in // 64)
    blocks = -(-d_out // 64)
    if T > 32:
        for rt, nt in ((2, 1), (2, 2), (4, 2)):
            if blocks * (4 // rt) * -(-T // (16 * nt)) <= 256:
                return nt, rt, False
        small, mid, big = (us(t, T, d_out, kt) for t in (64, 128, 256))
        return (4, 4, False) if small <= mid and small <= big else (128 if mid < big else 256)
    rt = 4 if blocks >= 512 else (2 if blocks >= 128 else 1)
    return 1 if T <= 16 else 2, rt, T <= 16 and T * (-(-d_in // 512) * 512) <= 20480


def test_sizes_reach_every_kernel():
    assert {kernel(*s) for s in SIZES} == {128, 256, (4, 4, False)} | {(1, r, f) for r in (1, 2, 4) for f in (True, False)} | {
        (2, r, False) for r in (1, 2, 4)}


@pytest.mark.parametrize("T,d_in,d_out", SIZES)
def test_workspace_follows(T, d_in, d_out):
    s = L.lora_w8_store()
    s.d_in, s.d_out, s.codes, s.scales = d_in, d_out, 0x10000, 0x10000
    need = L.lib().lora_w8_workspace_bytes(C.byref(s), T, 0)
    plan = kernel(T, d_in, d_out)
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert need == (0 if isinstance(plan, tuple) and plan[2] else up(T * (-(-d_in // 16) * 16)) + up(4 * T))
