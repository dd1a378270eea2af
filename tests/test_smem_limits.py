"""The record of raised shared-memory limits: every kernel of every device has
its place, so that only the first call of each asks the runtime."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_attention_backward_gb300", "csrc")

PROGRAM = r"""
#include <stdint.h>
#include "smem_limits.h"
const void *kernel(int i) { return reinterpret_cast<const void *>(static_cast<uintptr_t>(64 + 16 * i)); }
int main() {
  abw::SmemLimits limits;
  for (int dev = 0; dev < 8; ++dev)
    for (int i = 0; i < 300; ++i) {
      if (limits.reaches(dev, kernel(i), 7 + dev, 1000)) return 1;     // another device's or kernel's
      limits.raised(dev, kernel(i), 7 + dev, 1000 + i);
    }
  for (int dev = 0; dev < 8; ++dev)
    for (int i = 0; i < 300; ++i) {
      if (!limits.reaches(dev, kernel(i), 7 + dev, 1000 + i)) return 2;
      if (limits.reaches(dev, kernel(i), 7 + dev, 1001 + i)) return 3;  // more than it was raised to
      if (limits.reaches(dev, kernel(i), 70 + dev, 1000)) return 4;     // a context made since
      if (limits.reaches(dev, kernel(i), 0, 1000)) return 5;            // an unknown one
    }
  limits.raised(3, kernel(5), 99, 2000);
  return limits.reaches(3, kernel(5), 99, 2000) && !limits.reaches(3, kernel(5), 10, 1000) ? 0 : 6;
}
"""


def test_every_kernel_has_its_place(tmp_path):
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_library_keeps_no_record_of_a_fixed_size():
    body = open(os.path.join(CSRC, "api.cu")).read()
    body = body[body.index("cudaError_t ensure_dynamic_smem"):]
    body = body[:body.index("\n}\n")]
    assert "SmemLimits" in body and not re.search(r"\w+\[\d+\];", body)
