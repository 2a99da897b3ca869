"""The launchers' host helpers (csrc/host_util.h), compiled for the CPU over a
stand-in for the HIP runtime's few calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = """
#pragma once
#include <cstddef>
enum hipError_t { hipSuccess = 0, hipErrorInvalidDevice = 101 };
enum hipDeviceAttribute_t { hipDeviceAttributeMultiprocessorCount };
enum hipFuncAttribute { hipFuncAttributeMaxDynamicSharedMemorySize };
hipError_t hipGetDevice(int* dev);
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t a, int dev);
hipError_t hipFuncSetAttribute(const void* fn, hipFuncAttribute a, int value);
"""

# A thread that asks for the smaller size is inside the runtime's call when
# another asks for the larger one; the attribute is set where that call ends.
PROGRAM = """
#include <hip/hip_runtime.h>
#include "host_util.h"
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
static std::atomic<int> limit{0}, calls{0}, inside{0};
static void wait(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }
hipError_t hipGetDevice(int* dev) { *dev = 3; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 1; return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int value) {
  ++calls;
  ++inside;
  if (value < 100000) wait(300);
  limit = value;
  return hipSuccess;
}
int main() {
  static lora::DynLdsLimit lim;
  std::thread a([] { lora::ensure_dynamic_lds(lim, nullptr, 64 * 1024); });
  while (!inside) wait(1);
  std::thread b([] { lora::ensure_dynamic_lds(lim, nullptr, 128 * 1024); });
  a.join();
  b.join();
  const int after = limit, n = calls;
  lora::ensure_dynamic_lds(lim, nullptr, 100 * 1024);
  lora::ensure_dynamic_lds(lim, nullptr, 40 * 1024);
  std::printf("%d %d %d\\n", after, n, (int)calls);
}
"""


def test_the_lds_limit_never_falls(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(RUNTIME)
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe = tmp_path / "t"
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", f"-I{tmp_path}", f"-I{ROOT}/rank_specialized_amd/csrc",
                    str(tmp_path / "t.cpp"), "-o", str(exe)], check=True, timeout=120)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=30).stdout.split()
    assert out == [str(128 * 1024), "2", "2"]  # what covers a size is not set again
