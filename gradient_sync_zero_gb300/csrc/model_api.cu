// C ABI entry points of the operators at the ends of a training step: argument
// checks and dispatch to the kernel launchers.  Everything a kernel indexes is
// checked here or bounded there, so a refused call enqueues nothing.
#include "model_check.h"

using namespace dps;

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
