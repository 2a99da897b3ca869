"""Which kernel a call of the 4-bit products runs (csrc/w4.h, compiled for the
CPU), at the sizes of the GPU tests that mean to reach it."""
import os
import shutil
import subprocess

import pytest

from test_gpu_w4_many import DENSE, EXPERTS, KINDS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
#include <cstdio>
#include "w4.h"
int main() {
  lora_w4_store s{};
  int T, k, weighted;
  while (std::scanf("%d %d %d %d %d %d %d", &s.n, &s.d_in, &s.d_out, &s.group, &T, &k, &weighted) == 7) {
    const lora::W4Plan p = lora::w4_plan_call(s, LORA_DTYPE_BF16, T, k, weighted != 0);
    std::printf("%d %d\\n", p.bm, p.splits);
  }
}
"""


def plans(tmp_path, calls):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "t.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", f"-I{ROOT}/rank_specialized_amd/csrc", str(tmp_path / "t.cpp"), "-o", str(tmp_path / "t")],
                   check=True, timeout=120)
    lines = "\n".join(" ".join(map(str, c)) for c in calls)
    out = subprocess.run([str(tmp_path / "t")], input=lines, check=True, capture_output=True, text=True, timeout=30).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_sizes_of_the_many_rows_tests(tmp_path):
    calls, want = [], []
    for group, _, _ in KINDS:
        for T, d_in, d_out, bm, splits in DENSE:
            calls.append((1, d_in, d_out, group, T, 0, 0))
            want.append((bm, splits))
        for T, k, E, d_in, d_out, _, weighted, bm, splits in EXPERTS:
            calls.append((E, d_in, d_out, group, T, k, int(weighted)))
            want.append((bm, splits))
    assert plans(tmp_path, calls) == want
    # both tiles, whole and split, dense and by matrix, the latter weighted and not
    assert {(b, s > 1) for *_, b, s in DENSE} == {(b, s > 1) for *_, b, s in EXPERTS} == {(64, False), (64, True), (96, False), (96, True)}
    assert {(c[6], c[7]) for c in EXPERTS} == {(w, b) for w in (False, True) for b in (64, 96)}
