"""How the token kernels cut rows (csrc/token_shape.h), for sizes that no memory holds too: what a
kernel that keeps a whole row copies to shared memory must fit there."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")
pytestmark = pytest.mark.skipif(CXX is None, reason="no C++ compiler")

PROGRAM = r"""
#include "token_shape.h"
#include <cstdio>
#include <initializer_list>
using namespace dps;
int main() {
  long seen[4] = {}, parted = 0;
  const int64_t rows[] = {1, 2, 33, 151, 152, 153, 304, 2047, 2048, 16384, 131072, (1 << 28) - 1, 1 << 28, 1 << 29,
                          (1 << 29) + 1, (1 << 30) - 1, 1 << 30, (1 << 30) + 7, 0x7fffffff};
  for (int P : {1, 3, 8, 64})
    for (int64_t T : rows) {
      if (P * T > 0x7fffffff) continue;
      for (int64_t v = 1; v <= 0x7fffffff; v += v / 37 + 1)
        for (int es : {2, 4}) {
          const int64_t row = v * es;
          const PolicyShape s = policy_shape(P, T, row, 152);
          const int nt = cta_threads(s.group);
          if (T * s.ctas > 0x7fffffff || int64_t{s.kcap} * 16 * nt > kMostKept) return printf("grid %ld\n", (long)v), 1;
          // a CTA's vectors (the row's first may start at any value), and its first thread's
          const int64_t nv = row / 16, part = (nv + s.ctas - 1) / s.ctas, n = (part + s.group - 1) / s.group;
          if (s.all && n > s.kcap) return printf("P %d T %ld V %ld: %ld vectors, %d fit\n", P, (long)T, (long)v, (long)n, s.kcap), 1;
          if (!s.all && s.group != 512) return printf("no such kernel: %d threads, a row in parts\n", s.group), 1;
          if (!s.all && s.ctas == 1) ++parted;
          ++seen[s.group == 32 ? 0 : s.group == 128 ? 1 : s.group == 256 ? 2 : 3];
        }
    }
  return seen[0] && seen[1] && seen[2] && seen[3] && parted ? 0 : 2;
}
"""


def test_policy_rows_fit_shared_memory(tmp_path):
    src, exe = tmp_path / "shape.cpp", tmp_path / "shape"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "gradient_sync_zero_gb300", "csrc")
    r = subprocess.run([CXX, "-std=c++17", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout)
