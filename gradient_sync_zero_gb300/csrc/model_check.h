// Argument checks that the C ABI entries of the operators share (host).
#pragma once

#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <initializer_list>
#include <string>

#include "model.h"
#include "rows_overlap.h"

namespace dps {

constexpr int64_t kMaxExtent = 0x7fffffff;
constexpr int64_t kMaxDim = 1 << 23;   // of an embedding row: 2^12 or 2^13 CTAs beside each other in the gradient

inline int bad(const char* fn, const std::string& what) { return fail(DP_EINVAL, std::string(fn) + ": " + what); }

inline int cuda_status(int err, const char* fn) {
  return err ? fail(DP_ECUDA, std::string(fn) + ": " + cudaGetErrorString(static_cast<cudaError_t>(err)))
             : DP_OK;
}

inline int check_sizes(const char* fn, int32_t P, int64_t T, int64_t cols, const char* cols_name) {
  if (P < 1 || P > kMaxP) return bad(fn, "P outside [1, 64]");
  if (T < 0 || T > kMaxExtent / P) return bad(fn, "T is negative or P * T is 2^31 or more");
  if (cols < 1 || cols > kMaxExtent) return bad(fn, std::string(cols_name) + " outside [1, 2^31)");
  return DP_OK;
}

inline int check_embedding(const char* fn, int32_t P, int64_t T, int64_t vocab, int64_t dim) {
  const int rc = check_sizes(fn, P, T, vocab, "vocab");
  if (rc) return rc;
  return dim < 1 || dim > kMaxDim ? bad(fn, "dim outside [1, 2^23]") : DP_OK;
}

inline RowSet row_set(const Mat& m, int32_t P, int64_t rows, int64_t cols) {
  const Wide es = esize(m.dtype);
  return {{static_cast<Wide>(reinterpret_cast<uintptr_t>(m.p)), es * m.ws, rows, es * cols}, es * m.rs, P};
}

// A dp_rows of [P][rows][cols].  An output's rows must be disjoint.
inline int check_rows(const char* fn, const char* name, const dp_rows* m, int32_t P, int64_t rows, int64_t cols,
               bool output, Mat* out) {
  if (!m) return bad(fn, std::string("NULL ") + name);
  if (m->dtype != DP_BF16 && m->dtype != DP_F32)
    return bad(fn, std::string(name) + " has an unknown type " + std::to_string(m->dtype));
  out->p = static_cast<uint8_t*>(m->data);
  out->rs = P > 1 ? m->rank_stride : 0;
  out->ws = rows > 1 ? m->row_stride : 0;
  out->dtype = m->dtype;
  if (rows == 0) return DP_OK;   // nothing is accessed
  if (!m->data) return bad(fn, std::string("NULL data in ") + name);
  if (reinterpret_cast<uintptr_t>(m->data) % esize(m->dtype))
    return fail(DP_EALIGN, std::string(fn) + ": " + name + " not aligned to its element type");
  if (out->rs < 0 || out->ws < 0) return bad(fn, std::string(name) + " has a negative stride");
  // the furthest element must be addressable
  const double last = static_cast<double>(P - 1) * static_cast<double>(out->rs) +
                      static_cast<double>(rows - 1) * static_cast<double>(out->ws) +
                      static_cast<double>(cols);
  if (last > 2.3e18) return bad(fn, std::string(name) + " has strides past the address space");
  if (output && rows_meet(row_set(*out, P, rows, cols))) return bad(fn, std::string(name) + " has rows that overlap");
  return DP_OK;
}

// An output may be an input itself, or share no element with it.
inline bool same_place(const Mat& a, const Mat& b) {
  return a.p == b.p && a.rs == b.rs && a.ws == b.ws && a.dtype == b.dtype;
}

inline bool overlap(const Mat& a, int64_t arows, int64_t acols, const Mat& b, int64_t brows, int64_t bcols, int32_t P) {
  if (!a.p || !b.p) return false;
  return sets_meet(row_set(a, P, arows, acols), row_set(b, P, brows, bcols));
}

inline int check_tokens(const char* fn, const void* tokens, int32_t type, int64_t n, TokenArgs* out) {
  if (type != DP_I32 && type != DP_I64) return bad(fn, "unknown token type " + std::to_string(type));
  out->p = tokens;
  out->wide = type == DP_I64;
  if (n == 0) return DP_OK;
  if (!tokens) return bad(fn, "NULL tokens");
  if (reinterpret_cast<uintptr_t>(tokens) % (out->wide ? 8 : 4))
    return fail(DP_EALIGN, std::string(fn) + ": tokens not aligned to their type");
  return DP_OK;
}

inline int check_dropout(const char* fn, const dp_dropout_cfg* c, DropArgs* out) {
  *out = DropArgs{};
  if (!c) return DP_OK;
  if (!(c->p >= 0.0 && c->p <= 1.0)) return bad(fn, "dropout p outside [0, 1]");
  if (reinterpret_cast<uintptr_t>(c->seed_dev) & 7u)
    return fail(DP_EALIGN, std::string(fn) + ": seed_dev not 8-byte aligned");
  const double thr = std::nearbyint(c->p * 4294967296.0);
  if (thr == 0.0) return DP_OK;   // nothing is dropped
  out->on = 1;
  out->last = static_cast<uint32_t>(thr - 1.0);
  out->inv = thr >= 4294967296.0 ? 0.0f : static_cast<float>(1.0 / (1.0 - c->p));
  out->seed = c->seed;
  out->offset = c->offset;
  out->rank0 = static_cast<uint32_t>(c->rank0);
  out->dev = c->seed_dev;
  return DP_OK;
}

// fp32 [P][T]; required unless `optional`.
inline int check_vec(const char* fn, const char* name, const float* p, int64_t n, bool optional) {
  if (!p) return optional || n == 0 ? DP_OK : bad(fn, std::string("NULL ") + name);
  if (reinterpret_cast<uintptr_t>(p) & 3u)
    return fail(DP_EALIGN, std::string(fn) + ": " + name + " not 4-byte aligned");
  return DP_OK;
}

// The scale and its product with log2(e), in fp32.
inline int check_scale(const char* fn, double s) {
  const float f = static_cast<float>(s);
  return f > 0.0f && std::isfinite(1.5f * f) ? DP_OK
                                             : bad(fn, "logit_scale must be positive and finite in fp32");
}

// The embedding's scale, and its product with the kept values' factor, in fp32: with an infinite
// one a dropped value would be NaN.
inline int check_factor(const char* fn, double scale, const DropArgs& d) {
  const double most = static_cast<double>(FLT_MAX);
  return std::fabs(scale) <= most && std::fabs(scale) * static_cast<double>(d.inv) <= most
             ? DP_OK
             : bad(fn, "scale, or scale / (1 - p), is not finite in fp32");
}

// An output vector apart from the other vectors, [P][T] fp32 each (`m` and `n` values).
inline int check_apart(const char* fn, const char* name, const float* out, int64_t m,
                std::initializer_list<const float*> others, int64_t n) {
  for (const float* p : others)
    if (out && p && out < p + n && p < out + m)
      return bad(fn, std::string(name) + " overlaps another vector of the call");
  return DP_OK;
}

// No exception leaves a C entry: the messages, and the maps of the launch helpers, allocate.
template <class F>
inline int guarded(F&& body) {
  try {
    return body();
  } catch (...) {
    try {
      return fail(DP_ENOMEM, "out of host memory");
    } catch (...) {
      return DP_ENOMEM;
    }
  }
}

}  // namespace dps

#define DP_TRY(call)           \
  do {                         \
    const int rc_ = (call);    \
    if (rc_) return rc_;       \
  } while (0)
