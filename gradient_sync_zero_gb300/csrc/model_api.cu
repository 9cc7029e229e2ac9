// C ABI entry points of the operators at the ends of a training step: argument
// checks and dispatch to the kernel launchers.  Everything a kernel indexes is
// checked here or bounded there, so a refused call enqueues nothing.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <initializer_list>
#include <string>

#include "model.h"
#include "rows_overlap.h"

using namespace dps;

namespace {

constexpr int64_t kMaxExtent = 0x7fffffff;
constexpr int64_t kMaxDim = 1 << 23;   // of an embedding row: 2^12 or 2^13 CTAs beside each other in the gradient

int bad(const char* fn, const std::string& what) { return fail(DP_EINVAL, std::string(fn) + ": " + what); }

int cuda_status(int err, const char* fn) {
  return err ? fail(DP_ECUDA, std::string(fn) + ": " + cudaGetErrorString(static_cast<cudaError_t>(err)))
             : DP_OK;
}

int check_sizes(const char* fn, int32_t P, int64_t T, int64_t cols, const char* cols_name) {
  if (P < 1 || P > kMaxP) return bad(fn, "P outside [1, 64]");
  if (T < 0 || T > kMaxExtent / P) return bad(fn, "T is negative or P * T is 2^31 or more");
  if (cols < 1 || cols > kMaxExtent) return bad(fn, std::string(cols_name) + " outside [1, 2^31)");
  return DP_OK;
}

int check_embedding(const char* fn, int32_t P, int64_t T, int64_t vocab, int64_t dim) {
  const int rc = check_sizes(fn, P, T, vocab, "vocab");
  if (rc) return rc;
  return dim < 1 || dim > kMaxDim ? bad(fn, "dim outside [1, 2^23]") : DP_OK;
}

RowSet row_set(const Mat& m, int32_t P, int64_t rows, int64_t cols) {
  const Wide es = esize(m.dtype);
  return {{static_cast<Wide>(reinterpret_cast<uintptr_t>(m.p)), es * m.ws, rows, es * cols}, es * m.rs, P};
}

// A dp_rows of [P][rows][cols].  An output's rows must be disjoint.
int check_rows(const char* fn, const char* name, const dp_rows* m, int32_t P, int64_t rows, int64_t cols,
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
bool same_place(const Mat& a, const Mat& b) {
  return a.p == b.p && a.rs == b.rs && a.ws == b.ws && a.dtype == b.dtype;
}

bool overlap(const Mat& a, int64_t arows, int64_t acols, const Mat& b, int64_t brows, int64_t bcols, int32_t P) {
  if (!a.p || !b.p) return false;
  return sets_meet(row_set(a, P, arows, acols), row_set(b, P, brows, bcols));
}

int check_tokens(const char* fn, const void* tokens, int32_t type, int64_t n, TokenArgs* out) {
  if (type != DP_I32 && type != DP_I64) return bad(fn, "unknown token type " + std::to_string(type));
  out->p = tokens;
  out->wide = type == DP_I64;
  if (n == 0) return DP_OK;
  if (!tokens) return bad(fn, "NULL tokens");
  if (reinterpret_cast<uintptr_t>(tokens) % (out->wide ? 8 : 4))
    return fail(DP_EALIGN, std::string(fn) + ": tokens not aligned to their type");
  return DP_OK;
}

int check_dropout(const char* fn, const dp_dropout_cfg* c, DropArgs* out) {
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
int check_vec(const char* fn, const char* name, const float* p, int64_t n, bool optional) {
  if (!p) return optional || n == 0 ? DP_OK : bad(fn, std::string("NULL ") + name);
  if (reinterpret_cast<uintptr_t>(p) & 3u)
    return fail(DP_EALIGN, std::string(fn) + ": " + name + " not 4-byte aligned");
  return DP_OK;
}

// The scale and its product with log2(e), in fp32.
int check_scale(const char* fn, double s) {
  const float f = static_cast<float>(s);
  return f > 0.0f && std::isfinite(1.5f * f) ? DP_OK
                                             : bad(fn, "logit_scale must be positive and finite in fp32");
}

// The embedding's scale, and its product with the kept values' factor, in fp32: with an infinite
// one a dropped value would be NaN.
int check_factor(const char* fn, double scale, const DropArgs& d) {
  const double most = static_cast<double>(FLT_MAX);
  return std::fabs(scale) <= most && std::fabs(scale) * static_cast<double>(d.inv) <= most
             ? DP_OK
             : bad(fn, "scale, or scale / (1 - p), is not finite in fp32");
}

// An output vector apart from the other vectors, [P][T] fp32 each (`m` and `n` values).
int check_apart(const char* fn, const char* name, const float* out, int64_t m,
                std::initializer_list<const float*> others, int64_t n) {
  for (const float* p : others)
    if (out && p && out < p + n && p < out + m)
      return bad(fn, std::string(name) + " overlaps another vector of the call");
  return DP_OK;
}

// No exception leaves a C entry: the messages, and the maps of the launch helpers, allocate.
template <class F>
int guarded(F&& body) {
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

}  // namespace

#define DP_TRY(call)           \
  do {                         \
    const int rc_ = (call);    \
    if (rc_) return rc_;       \
  } while (0)

extern "C" {

int dp_dropout(const dp_rows* x, const dp_rows* residual, const dp_rows* out, int32_t P, int64_t T,
               int64_t dim, const dp_dropout_cfg* cfg, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_dropout";
    clear_error();
    DP_TRY(check_sizes(fn, P, T, dim, "dim"));
    Mat mx, mr, mo;
    DP_TRY(check_rows(fn, "x", x, P, T, dim, false, &mx));
    if (residual) DP_TRY(check_rows(fn, "residual", residual, P, T, dim, false, &mr));
    DP_TRY(check_rows(fn, "out", out, P, T, dim, true, &mo));
    if ((!same_place(mo, mx) && overlap(mo, T, dim, mx, T, dim, P)) ||
        (!same_place(mo, mr) && overlap(mo, T, dim, mr, T, dim, P)))
      return bad(fn, "out overlaps x or residual without being it");
    DropArgs d;
    DP_TRY(check_dropout(fn, cfg, &d));
    if (dropout_ctas(T, dim) > kMaxExtent) return bad(fn, "T * dim needs 2^31 or more CTAs per rank");
    return cuda_status(launch_dropout(mx, mr, mo, P, T, dim, d, stream), fn);
  });
}

int dp_embedding_forward(const dp_rows* table, int64_t vocab, int64_t dim, const void* tokens,
                         int32_t token_type, int32_t P, int64_t T, double scale,
                         const dp_dropout_cfg* dropout, const dp_rows* out, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_embedding_forward";
    clear_error();
    DP_TRY(check_embedding(fn, P, T, vocab, dim));
    Mat mw, mo;
    TokenArgs tok;
    DropArgs d;
    DP_TRY(check_rows(fn, "table", table, P, vocab, dim, false, &mw));
    DP_TRY(check_rows(fn, "out", out, P, T, dim, true, &mo));
    DP_TRY(check_tokens(fn, tokens, token_type, P * T, &tok));
    DP_TRY(check_dropout(fn, dropout, &d));
    DP_TRY(check_factor(fn, scale, d));
    if (overlap(mo, T, dim, mw, vocab, dim, P)) return bad(fn, "out overlaps table");
    return cuda_status(launch_embedding_forward(mw, vocab, dim, tok, P, T, static_cast<float>(scale), d,
                                                mo, stream), fn);
  });
}

int dp_embedding_workspace_bytes(int32_t P, int64_t T, int64_t vocab, int64_t dim, int64_t* bytes) {
  return guarded([&]() -> int {
    const char* fn = "dp_embedding_workspace_bytes";
    clear_error();
    if (!bytes) return bad(fn, "NULL bytes");
    DP_TRY(check_embedding(fn, P, T, vocab, dim));
    *bytes = embedding_workspace_bytes(P, T, vocab, dim);
    return DP_OK;
  });
}

int dp_embedding_backward(const dp_rows* dout, const void* tokens, int32_t token_type, int32_t P,
                          int64_t T, double scale, const dp_dropout_cfg* dropout,
                          const dp_rows* grad, int64_t vocab, int64_t dim, int32_t accumulate,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_embedding_backward";
    clear_error();
    DP_TRY(check_embedding(fn, P, T, vocab, dim));
    Mat mx, mg;
    TokenArgs tok;
    DropArgs d;
    DP_TRY(check_rows(fn, "dout", dout, P, T, dim, false, &mx));
    DP_TRY(check_rows(fn, "grad", grad, P, vocab, dim, true, &mg));
    DP_TRY(check_tokens(fn, tokens, token_type, P * T, &tok));
    DP_TRY(check_dropout(fn, dropout, &d));
    DP_TRY(check_factor(fn, scale, d));
    if (overlap(mg, vocab, dim, mx, T, dim, P)) return bad(fn, "grad overlaps dout");
    if (embedding_backward_ctas(P, T, vocab, dim) > kMaxExtent)
      return bad(fn, "T * dim and vocab need 2^31 or more CTAs per rank");
    if (!workspace) return bad(fn, "NULL workspace");
    if (reinterpret_cast<uintptr_t>(workspace) & 31u)
      return fail(DP_EALIGN, std::string(fn) + ": workspace not 32-byte aligned");
    const int64_t need = embedding_workspace_bytes(P, T, vocab, dim);
    if (workspace_bytes < need)
      return bad(fn, "workspace holds " + std::to_string(workspace_bytes) + " bytes, needs " +
                         std::to_string(need));
    return cuda_status(launch_embedding_backward(mx, tok, P, T, static_cast<float>(scale), d, mg, vocab,
                                                 dim, accumulate != 0, static_cast<uint8_t*>(workspace),
                                                 stream), fn);
  });
}

int dp_token_logprob(const dp_rows* logits, int32_t P, int64_t T, int64_t vocab,
                     const void* tokens, int32_t token_type, double logit_scale, float* logp,
                     float* lse, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_token_logprob";
    clear_error();
    DP_TRY(check_sizes(fn, P, T, vocab, "vocab"));
    Mat mz;
    TokenArgs tok;
    DP_TRY(check_rows(fn, "logits", logits, P, T, vocab, false, &mz));
    DP_TRY(check_tokens(fn, tokens, token_type, P * T, &tok));
    DP_TRY(check_scale(fn, logit_scale));
    DP_TRY(check_vec(fn, "logp", logp, P * T, false));
    DP_TRY(check_vec(fn, "lse", lse, P * T, true));
    DP_TRY(check_apart(fn, "logp", logp, P * T, {lse}, P * T));
    return cuda_status(launch_token_logprob(mz, P, T, vocab, tok, static_cast<float>(logit_scale), logp,
                                            lse, stream), fn);
  });
}

int dp_token_logprob_backward(const dp_rows* logits, int32_t P, int64_t T, int64_t vocab,
                              const void* tokens, int32_t token_type, double logit_scale,
                              const float* lse, const float* dlogp, const dp_rows* dlogits,
                              void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_token_logprob_backward";
    clear_error();
    DP_TRY(check_sizes(fn, P, T, vocab, "vocab"));
    Mat mz, mg;
    TokenArgs tok;
    DP_TRY(check_rows(fn, "logits", logits, P, T, vocab, false, &mz));
    DP_TRY(check_rows(fn, "dlogits", dlogits, P, T, vocab, true, &mg));
    DP_TRY(check_tokens(fn, tokens, token_type, P * T, &tok));
    DP_TRY(check_scale(fn, logit_scale));
    DP_TRY(check_vec(fn, "lse", lse, P * T, false));
    DP_TRY(check_vec(fn, "dlogp", dlogp, P * T, false));
    if (mg.dtype != mz.dtype) return bad(fn, "dlogits must have the logits' type");
    if (!same_place(mg, mz) && overlap(mg, T, vocab, mz, T, vocab, P))
      return bad(fn, "dlogits overlaps logits without being it");
    return cuda_status(launch_token_logprob_backward(mz, P, T, vocab, tok, static_cast<float>(logit_scale),
                                                     lse, dlogp, mg, stream), fn);
  });
}

int dp_policy_loss(const dp_rows* logits, int32_t P, int64_t T, int64_t vocab, const void* tokens,
                   int32_t token_type, const float* old_logp, const float* ref_logp,
                   const float* advantage, const float* weight, const dp_policy_cfg* cfg,
                   float* logp, float* stats, const dp_rows* dlogits, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_policy_loss";
    clear_error();
    DP_TRY(check_sizes(fn, P, T, vocab, "vocab"));
    Mat mz, mg;
    TokenArgs tok;
    DP_TRY(check_rows(fn, "logits", logits, P, T, vocab, false, &mz));
    if (dlogits) {
      DP_TRY(check_rows(fn, "dlogits", dlogits, P, T, vocab, true, &mg));
      if (mg.dtype != mz.dtype) return bad(fn, "dlogits must have the logits' type");
      if (!same_place(mg, mz) && overlap(mg, T, vocab, mz, T, vocab, P))
        return bad(fn, "dlogits overlaps logits without being it");
    }
    DP_TRY(check_tokens(fn, tokens, token_type, P * T, &tok));
    DP_TRY(check_vec(fn, "old_logp", old_logp, P * T, false));
    DP_TRY(check_vec(fn, "ref_logp", ref_logp, P * T, true));
    DP_TRY(check_vec(fn, "advantage", advantage, P * T, false));
    DP_TRY(check_vec(fn, "weight", weight, P * T, true));
    DP_TRY(check_vec(fn, "logp", logp, P * T, false));
    DP_TRY(check_vec(fn, "stats", stats, 1, false));
    if (!cfg) return bad(fn, "NULL cfg");
    DP_TRY(check_scale(fn, cfg->logit_scale));
    if (!(cfg->clip_low >= 0.0 && cfg->clip_low <= 1.0 && cfg->clip_high >= 0.0 &&
          std::isfinite(cfg->clip_high)))
      return bad(fn, "clip_low outside [0, 1] or clip_high not finite and >= 0");
    if (!(cfg->kl_beta >= 0.0 && std::isfinite(cfg->kl_beta))) return bad(fn, "kl_beta must be finite and >= 0");
    if (cfg->kl_beta > 0.0 && !ref_logp) return bad(fn, "kl_beta > 0 needs ref_logp");
    DP_TRY(check_apart(fn, "logp", logp, P * T, {old_logp, ref_logp, advantage, weight}, P * T));
    DP_TRY(check_apart(fn, "stats", stats, 4 * P, {old_logp, ref_logp, advantage, weight, logp}, P * T));
    PolicyArgs a;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.adv = advantage;
    a.weight = weight;
    a.lo = static_cast<float>(1.0 - cfg->clip_low);
    a.hi = static_cast<float>(1.0 + cfg->clip_high);
    a.beta = static_cast<float>(cfg->kl_beta);
    return cuda_status(launch_policy_loss(mz, P, T, vocab, tok, static_cast<float>(cfg->logit_scale), a,
                                          logp, stats, mg, stream), fn);
  });
}

}  // extern "C"
