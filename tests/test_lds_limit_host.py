"""A kernel's limit of dynamic LDS is set on every device that launches it, once each.  The
helper is compiled for the host against a runtime that counts."""
import glob
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_fine_tuning_nf4_amd", "csrc")

RUNTIME = r"""
#pragma once
enum hipError_t { hipSuccess = 0, hipErrorInvalidValue = 1 };
enum hipFuncAttribute { hipFuncAttributeMaxDynamicSharedMemorySize = 8 };
extern int device, asked, last_bytes;
extern hipError_t answer;
inline hipError_t hipGetDevice(int* d) { *d = device; return hipSuccess; }
inline hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int bytes) {
  ++asked; last_bytes = bytes; return answer;
}
"""

MAIN = r"""
#include <cstdio>
#include "lds_limit.h"
int device = 0, asked = 0, last_bytes = 0;
hipError_t answer = hipSuccess;
int main() {
  static qn::LdsLimit a, b;
  auto call = [&](qn::LdsLimit& l, int d) {
    device = d;
    const int before = asked;
    const int e = l(nullptr, 70000);
    std::printf("%d%d ", asked - before, e);
  };
  call(a, 0); call(a, 0); call(a, 3); call(a, 3); call(a, 0);  // once a device
  call(b, 0);                                                  // once a kernel
  answer = hipErrorInvalidValue; call(b, 5);                   // an error is not kept
  answer = hipSuccess; call(b, 5); call(b, 5);
  call(a, 63); call(a, 63); call(a, 64); call(a, 64); call(a, 100);
  std::printf("%d", last_bytes);
}
"""


def test_once_a_device(tmp_path):
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(RUNTIME)
    src, exe = tmp_path / "m.cpp", tmp_path / "m"
    src.write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-I", str(tmp_path), "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["10", "00", "10", "00", "00", "10", "11", "10", "00", "10", "00", "10", "10",
                   "10", "70000"]


def test_no_limit_is_set_once_a_process():
    """No kernel attribute is set while a static is initialised, which happens on the first
    device alone."""
    for path in glob.glob(os.path.join(CSRC, "*.hip")):
        text = open(path).read()
        for m in re.finditer(r"\bstatic\b[^;{]*\bhipError_t\b[^;=]*=", text):
            raise AssertionError((os.path.basename(path), m.group(0)))
