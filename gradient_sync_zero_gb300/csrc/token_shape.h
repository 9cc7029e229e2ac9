// How the token kernels cut their rows between threads and CTAs: host arithmetic on sizes
// alone, apart from CUDA so that it can be checked for sizes that no memory holds.
#pragma once

#include <cstdint>

namespace dps {

constexpr int kMaxCluster = 8;
constexpr int64_t kLongestKept = 112 * 1024;    // policy: bytes of a row per CTA, two CTAs per SM
constexpr int64_t kPart128 = 32 * 1024, kPart256 = 64 * 1024;   // policy: bytes of a row for 128 and 256 threads
constexpr int64_t kMostKept = 208 * 1024;       // shared memory of one CTA at most

template <int G>
constexpr int cta_of = G == 32 ? 128 : G;   // threads of a CTA
inline int cta_threads(int group) { return group == 32 ? cta_of<32> : group; }

// A row's threads are a group: a warp (four to a CTA) or the CTA.  A warp's row has
// no barrier and no second stage of its sums: 131072 rows of 4000 bf16 take 147 us
// against 196 with 128 threads each (policy loss 337 against 766), rows of 8000 147 against 158
// for half as many; from 12000 on a CTA is faster.  With few rows, a row's latency counts and
// more threads shorten it (264 rows of 4000: 3.1 us against 3.7) down to 1000 values.
inline bool warp_rows(int P, int64_t T, int64_t row_bytes) {
  return row_bytes <= 2048 || (row_bytes <= 16384 && P * T >= 2048);
}

// CTAs per row: more while a part is longer than `longest` bytes, or while the
// rows leave SMs without a CTA and a part still is 8 KB.  A grid has 2^31 - 1 of them.
inline int ctas_per_row(int P, int64_t T, int64_t row_bytes, int64_t longest, int64_t sms) {
  int C = 1;
  while (C < kMaxCluster && T * (2 * C) <= 0x7fffffff &&
         (row_bytes / C > longest || (P * T * C < 2 * sms && row_bytes / C >= 16384)))
    C *= 2;
  return C;
}

// The policy loss: threads of a group, CTAs per row, the vectors of a thread that its CTA's
// shared memory holds, and whether these are all.
struct PolicyShape {
  int group, ctas, kcap;
  bool all;
};

inline PolicyShape policy_shape(int P, int64_t T, int64_t row_bytes, int64_t sms) {
  PolicyShape s;
  const bool warps = warp_rows(P, T, row_bytes);
  s.ctas = warps ? 1 : ctas_per_row(P, T, row_bytes, kLongestKept, sms);
  // Threads of a group: enough vectors each that the row's reductions are a small part
  // of its work, and enough rows on an SM that one's loads cover another's sums.
  const int64_t part = row_bytes / s.ctas;
  s.group = warps ? 32 : part <= kPart128 ? 128 : part <= kPart256 ? 256 : 512;
  const int64_t vecs = (row_bytes / 16 + s.ctas - 1) / s.ctas, most = kMostKept / (16 * cta_threads(s.group));
  const int64_t per = (vecs + s.group - 1) / s.group;
  s.all = per <= most;
  s.kcap = static_cast<int>(s.all ? per : most);
  return s;
}

}  // namespace dps
