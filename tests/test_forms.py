"""The kernels' forms that calls of the experts' layer and of the 8-bit products
take, by csrc/moe.h and csrc/w8.h themselves, compiled for the CPU: at the sizes
of the GPU tests they are those that tests/test_moe_plan.py and
tests/test_w8_plan.py restate, every one of them among them."""
import os
import shutil
import subprocess

import pytest

from test_gpu_moe import CASES
from test_gpu_moe_exact import LONG
from test_gpu_w8 import SIZES
from test_moe_plan import kernels
from test_w8_plan import kernel

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MOE = """
#include <cstdio>
#include "moe.h"
using namespace lora;
int main() {
  int T, k, n, d, ffn, group, dtype;
  while (std::scanf("%d %d %d %d %d %d %d", &T, &k, &n, &d, &ffn, &group, &dtype) == 7) {
    const MoePlan p = moe_plan_call(n, ffn, d, dtype, T, k);
    const MoeForm u = kMoeUpForms[moe_up_form(p, dtype, w4_sub(group))], v = kMoeDownForms[moe_down_form(p)];
    std::printf("%d %d %d %d %d %d %d\\n", moe_x_parts(dtype), u.tiles, u.blocks, u.waves, v.tiles, moe_down_blocks(v.tiles == 2), v.waves);
  }
}
"""
W8 = """
#include <cstdio>
#include "w8.h"
int main() {
  int T, d_in, d_out;
  while (std::scanf("%d %d %d", &T, &d_in, &d_out) == 3) {
    const lora::W8Plan p = lora::w8_plan_call(d_in, d_out, T, false);
    std::printf("%d %d %d %d\\n", p.tile, p.nt, p.rt, (int)p.fused);
  }
}
"""


def forms(tmp_path, program, calls):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "t.cpp").write_text(program)
    subprocess.run([cxx, "-std=c++17", "-O1", f"-I{ROOT}/rank_specialized_amd/csrc", str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")],
                   check=True, timeout=120)
    lines = "\n".join(" ".join(map(str, c)) for c in calls)
    out = subprocess.run([str(tmp_path / "t")], input=lines, check=True, capture_output=True, text=True, timeout=30).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_experts_layer(tmp_path):
    got = forms(tmp_path, MOE, [(*c[:6], 1 if c[8] == "bf16" else 0) for c in CASES + LONG])
    assert got == [(*up, *down) for up, down in map(kernels, CASES + LONG)]
    assert {g[:4] for g in got} == {(1, 1, 4, 2), (1, 1, 8, 1), (1, 2, 2, 4), (3, 1, 1, 4), (3, 1, 4, 2), (3, 2, 2, 4)}
    assert {(g[0], *g[4:]) for g in got} == {(p, *d) for p in (1, 3) for d in ((1, 4, 2), (1, 4, 8), (2, 8, 2))}


def test_8_bit_products(tmp_path):
    got = forms(tmp_path, W8, SIZES)
    want = [kernel(*s) for s in SIZES]
    assert [(g[0] if g[0] else (*g[1:3], bool(g[3]))) for g in got] == want
    assert {g[0] for g in got} == {0, 128, 256} and {g[1:] for g in got if g[0] == 0} == {(4, 4, 0)} | {
        (1, r, f) for r in (1, 2, 4) for f in (0, 1)} | {(2, r, 0) for r in (1, 2, 4)}
