"""Which matrices may stand beside each other in one call: the overlap rule (csrc/rows_overlap.h)
against enumeration, and the calls' refusals of layouts that share a single element."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

import gradient_sync_zero_gb300 as dps
from gradient_sync_zero_gb300 import build as dbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

PROGRAM = r"""
#include "rows_overlap.h"
#include <cstdio>
#include <random>
#include <set>
using namespace dps;
int main() {
  std::mt19937_64 g(7);
  const auto in = [&](int lo, int hi) { return lo + static_cast<int>(g() % (hi - lo + 1)); };
  long yes = 0, no = 0, strided = 0;
  for (int k = 0; k < 400000; ++k) {
    RowSet m[2];
    const int P = in(1, 4), most = in(0, 3) ? 40 : 6;
    for (RowSet& s : m) s = {{in(0, 150), in(0, most), in(0, 7), in(1, 9)}, in(0, 60), P};
    if (in(0, 1)) m[1].rank_step = m[0].rank_step;
    if (in(0, 1)) m[1].first.step = m[0].first.step;
    if (in(0, 2) == 0) m[1].first.at += 1000 * (in(0, 1) ? 1 : 0);
    std::set<long> bytes;
    bool want = false;
    for (int w = 0; w < 2; ++w)
      for (int r = 0; r < P; ++r)
        for (int i = 0; i < m[w].first.n; ++i)
          for (int j = 0; j < m[w].first.len; ++j) {
            const long at = static_cast<long>(m[w].first.at + r * m[w].rank_step + i * m[w].first.step + j);
            if (w == 0) bytes.insert(at); else want = want || bytes.count(at);
          }
    if (sets_meet(m[0], m[1]) != want || sets_meet(m[1], m[0]) != want) return printf("case %d\n", k), 1;
    ++(want ? yes : no);
    // disjoint although their spans meet
    if (!want && m[0].first.n > 1 && m[1].first.n > 1 && m[1].first.at < 1000 && m[0].first.step != m[1].first.step)
      ++strided;
  }
  if (yes < 20000 || no < 20000 || strided < 2000) return printf("%ld %ld %ld\n", yes, no, strided), 2;
  // two rows of one matrix
  long apart = 0;
  for (int k = 0; k < 200000; ++k) {
    const RowSet s{{0, in(0, 30), in(1, 6), in(1, 9)}, in(0, 60), in(1, 4)};
    std::set<long> bytes;
    bool want = false;
    for (int r = 0; r < s.P; ++r)
      for (int i = 0; i < s.first.n; ++i)
        for (int j = 0; j < s.first.len; ++j)
          want = !bytes.insert(static_cast<long>(r * s.rank_step + i * s.first.step + j)).second || want;
    if (rows_meet(s) != want) return printf("rows %d\n", k), 5;
    if (!want && s.P > 1 && s.first.n > 1) ++apart;
  }
  if (apart < 2000) return 6;
  // strides and counts near their limits: rows of one byte at odd and at even places, and one apart
  const Wide big = Wide{1} << 61, n = Wide{1} << 30;
  const RowRun a{0, 2, n, 1}, b{1, 2, n, 1}, c{1, 3, n, 1}, e{big, big, 2, 4}, f{2 * big + 3, 5, n, 1};
  if (runs_meet(a, b) || !runs_meet(a, c) || !runs_meet(e, f) || runs_meet(e, RowRun{2 * big + 4, 5, n, 1})) return 3;
  // multiples of 2^20 - 1 and of 2^20 first agree at their product
  const Wide p = (1 << 20) - 1, q = 1 << 20;
  const RowRun u{p, p, q, 1}, v{q, q, p, 1}, x{p, p, q - 1, 1};
  return runs_meet(u, v) && !runs_meet(x, v) ? 0 : 4;
}
"""


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
def test_rule_against_enumeration(tmp_path):
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "gradient_sync_zero_gb300", "csrc")
    r = subprocess.run([CXX, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", inc, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout)


# ---- refusals of layouts one element into each other (fake addresses: nothing is launched) ----
BASE, TOK, WS = 1 << 30, C.c_void_p(1 << 34), C.c_void_p(1 << 36)


def R(at, rs, ws, dtype=dps.DP_BF16):
    """A matrix `at` bf16 elements from BASE."""
    return C.byref(dps.Rows(BASE + 2 * at, rs, ws, dtype, 0))


@pytest.fixture(scope="module", autouse=True)
def built():
    dbuild.build()


P, T, D, V = 3, 5, 64, 20


@pytest.mark.parametrize("x,out", [
    (R(0, 2 * T * D, D), R(T * D - 1, 2 * T * D, D)),              # buf[:, :T], buf[:, T:]
    (R(0, 2 * T * D, D), R(T * D + 1, 2 * T * D, D)),              # ... into the next rank's x
    (R(0, 2 * D, P * 2 * D), R(D - 1, 2 * D, P * 2 * D)),          # halves of [T][P][2 D]
    (R(0, 2 * D, P * 2 * D), R(D + 1, 2 * D, P * 2 * D)),
    (R(0, 4 * T * D, 2 * D), R(D + 1, 4 * T * D, 2 * D)),          # every second row
])
def test_dropout_refuses_one_shared_element(x, out):
    assert dps.lib().dp_dropout(x, None, out, P, T, D, None, None) == dps.DP_EINVAL
    assert "without being it" in dps.lib().dp_last_error().decode()


@pytest.mark.parametrize("out", [
    R(0, 3 * D - 1, 2 * D), R(0, 3 * D + 1, 2 * D),                # rank 1 in rank 0's gaps, but for an element
    R(0, 2 * D, 2 * D), R(0, 0, D), R(0, T * D - 1, D), R(0, D - 1, 2 * D), R(0, D, 2 * D - 1),
])
def test_output_rows_that_share_one_element_are_refused(out):
    x = C.byref(dps.Rows(1 << 40, T * D, D, dps.DP_BF16, 0))
    assert dps.lib().dp_dropout(x, None, out, 2, T, D, None, None) == dps.DP_EINVAL
    assert "out has rows that overlap" in dps.lib().dp_last_error().decode()


@pytest.mark.parametrize("slot,act", [(0, V * D - 1), (T * D - 1, 0), (0, 2 * (V + T) * D - T * D + 1)])
def test_embedding_refuses_one_element_shared_in_an_arena(slot, act):
    """An embedding's slot and its activations in one arena per rank."""
    lib, rank = dps.lib(), 2 * (V + T) * D
    args = (V, D, TOK, dps.DP_I64, P, T, 1.0, None)
    assert lib.dp_embedding_forward(R(slot, rank, D), *args, R(act, rank, D), None) == dps.DP_EINVAL
    assert "out overlaps table" in lib.dp_last_error().decode()
    assert lib.dp_embedding_backward(R(act, rank, D), TOK, dps.DP_I64, P, T, 1.0, None, R(slot, rank, D), V, D, 0, WS,
                                     1 << 40, None) == dps.DP_EINVAL
    assert "grad overlaps dout" in lib.dp_last_error().decode()
