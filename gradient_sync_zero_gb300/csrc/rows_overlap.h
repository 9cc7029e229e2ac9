// Whether matrices of strided rows share a byte, or two rows of one do: exact host arithmetic,
// apart from CUDA.
#pragma once

#include <cstdint>

namespace dps {

using Wide = __int128;   // addresses and products of strides and counts

// n rows of `len` bytes, `step` bytes apart, the first at `at`.
struct RowRun {
  Wide at, step, n, len;
};

// One run for each of P ranks, `rank_step` bytes apart.
struct RowSet {
  RowRun first;
  Wide rank_step;
  int P;
};

inline Wide floor_div(Wide a, Wide b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }   // b > 0

// The smallest i >= 0 with l <= a i mod m <= r, or -1 (0 <= a < m, 0 <= l <= r < m).  Where
// no multiple of a lies in [l, r], a i - m j does for the smallest j with m j mod a between -r
// and -l mod a: Euclid's steps, taken on the smaller of a and m - a.
inline Wide first_within(Wide a, Wide m, Wide l, Wide r) {
  if (l == 0) return 0;
  if (a == 0) return -1;
  if (2 * a > m) return first_within(m - a, m, m - r, m - l);
  const Wide i = (l + a - 1) / a;
  if (i * a <= r) return i;
  const Wide j = first_within(m % a, a, (a - r % a) % a, (a - l % a) % a);
  return j < 0 ? -1 : (l + m * j + a - 1) / a;
}

// Rows i of a and j of b share a byte iff lo <= a.at - b.at + i s - j t <= hi.
inline bool runs_meet(const RowRun& a, const RowRun& b) {
  if (a.n == 0 || b.n == 0) return false;
  const Wide s = a.n > 1 ? a.step : 0, t = b.n > 1 ? b.step : 0;
  const Wide lo = 1 - a.len, hi = b.len - 1, d = a.at - b.at, top = hi + (b.n - 1) * t;
  if (d > top || d + (a.n - 1) * s < lo) return false;
  // the rows of a that begin inside b's span (or end there)
  Wide i0 = 0, i1 = 0;
  if (s > 0) {
    i0 = d >= lo ? 0 : -floor_div(d - lo, s);
    i1 = floor_div(top - d, s);
    if (i1 > a.n - 1) i1 = a.n - 1;
    if (i0 > i1) return false;
  }
  const Wide w = hi - lo + 1;
  if (t == 0 || w >= t) return true;   // one row, or rows that leave no gap for a's
  const Wide x = (d + i0 * s - lo) % t;
  if (x < w) return true;
  const Wide k = first_within(s % t, t, t - x, t - x + w - 1);
  return k >= 0 && i0 + k <= i1;
}

// The ordinary case first, buffers apart: the pairs of 64 ranks would take 10 us.
inline bool sets_meet(const RowSet& a, const RowSet& b) {
  if (a.first.n == 0 || b.first.n == 0) return false;
  const auto end = [](const RowSet& m) {
    return m.first.at + (m.P - 1) * m.rank_step + (m.first.n - 1) * m.first.step + m.first.len;
  };
  if (a.first.at >= end(b) || b.first.at >= end(a)) return false;
  const auto at = [](const RowSet& m, Wide rank) {
    RowRun run = m.first;
    run.at += rank * m.rank_step;
    return run;
  };
  if (a.rank_step == b.rank_step) {   // only the ranks' distance counts
    for (int k = 1 - a.P; k < b.P; ++k)
      if (runs_meet(a.first, at(b, k))) return true;
    return false;
  }
  for (int r = 0; r < a.P; ++r)
    for (int q = 0; q < b.P; ++q)
      if (runs_meet(at(a, r), at(b, q))) return true;
  return false;
}

// Whether two rows of one matrix share a byte.
inline bool rows_meet(const RowSet& m) {
  if (m.first.n > 1 && m.first.step < m.first.len) return true;
  if (m.rank_step >= (m.first.n - 1) * m.first.step + m.first.len) return false;   // slice after slice
  for (int k = 1; k < m.P; ++k) {
    RowRun run = m.first;
    run.at += k * m.rank_step;
    if (runs_meet(m.first, run)) return true;
  }
  return false;
}

}  // namespace dps
