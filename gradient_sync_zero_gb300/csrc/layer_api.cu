// C ABI entry points of the dense layer, the orthogonalisation and the Muon step: argument
// checks and dispatch.  A refused call enqueues nothing.
#include <algorithm>
#include <memory>
#include <new>
#include <set>

#include "layer.h"
#include "model_check.h"

using namespace dps;

namespace {

// A bias: one row for each rank.
int check_bias(const char* fn, const char* name, const dp_rows* m, int32_t P, int64_t N, bool output, Mat* out) {
  return check_rows(fn, name, m, P, 1, N, output, out);
}

int need_bf16(const char* fn, const char* name, const Mat& m) {
  return m.dtype == DP_BF16 ? DP_OK : bad(fn, std::string(name) + " must be DP_BF16");
}

int check_linear(const char* fn, int32_t P, int64_t T, int64_t in_dim, int64_t out_dim) {
  const int rc = check_sizes(fn, P, T, in_dim, "in_dim");
  if (rc) return rc;
  if (out_dim < 1 || out_dim > kMaxExtent) return bad(fn, "out_dim outside [1, 2^31)");
  if (std::max(T, std::max(in_dim, out_dim)) > kMaxExtent - 1023)   // a last tile's rows are counted in 31 bits too
    return bad(fn, "T, in_dim or out_dim above 2^31 - 1024");
  // their tiles and CTAs are counted in 31 bits
  const double t = static_cast<double>(T), k = static_cast<double>(in_dim), n = static_cast<double>(out_dim);
  const double most = 1e12 / P;
  return t * k > most || t * n > most || k * n > most ? bad(fn, "a matrix of more than 1e12 elements") : DP_OK;
}

int check_act(const char* fn, int32_t act) {
  return act < DP_ACT_NONE || act > DP_ACT_SILU ? bad(fn, "unknown activation " + std::to_string(act)) : DP_OK;
}

int check_workspace(const char* fn, const void* ws, int64_t have, int64_t need) {
  if (need == 0) return DP_OK;
  if (!ws) return bad(fn, "NULL workspace");
  if (reinterpret_cast<uintptr_t>(ws) & 31u) return fail(DP_EALIGN, std::string(fn) + ": workspace not 32-byte aligned");
  return have < need ? bad(fn, "workspace holds " + std::to_string(have) + " bytes, needs " + std::to_string(need))
                     : DP_OK;
}

// Bytes [p, p + n) outside every row of m.
bool apart(const void* p, int64_t n, const Mat& m, int64_t rows, int64_t cols, int32_t P) {
  if (!p || n <= 0 || !m.p || rows == 0) return true;
  const RowSet one{{static_cast<Wide>(reinterpret_cast<uintptr_t>(p)), 0, 1, n}, 0, 1};
  return !sets_meet(one, row_set(m, P, rows, cols));
}

struct Part {
  const char* name;
  const Mat* m;
  int64_t rows, cols;
};

int check_ns(const char* fn, const dp_newton_schulz_cfg* c, NewtonSchulz* out) {
  if (!c) return bad(fn, "NULL cfg");
  const double most = static_cast<double>(FLT_MAX);
  if (!(std::fabs(c->a) <= most && std::fabs(c->b) <= most && std::fabs(c->c) <= most))
    return bad(fn, "a, b or c not finite in fp32");
  if (!(c->eps >= 1e-30 && c->eps <= 1e30)) return bad(fn, "eps outside [1e-30, 1e30]");
  if (c->steps < 1 || c->steps > 64) return bad(fn, "steps outside [1, 64]");
  *out = {static_cast<float>(c->a), static_cast<float>(c->b), static_cast<float>(c->c), static_cast<float>(c->eps), c->steps};
  return DP_OK;
}

constexpr int64_t kMaxSide = 1 << 20;

int check_sides(const char* fn, int64_t rows, int64_t cols) {
  return rows < 1 || rows > kMaxSide || cols < 1 || cols > kMaxSide ? bad(fn, "rows or cols outside [1, 2^20]") : DP_OK;
}

const Muon* as_muon(const dp_muon* m) { return reinterpret_cast<const Muon*>(m); }

}  // namespace

extern "C" {

int dp_linear_workspace_bytes(const dp_rows* x, const dp_rows* w, int32_t P, int64_t T, int64_t in_dim,
                              int64_t out_dim, int32_t backward, int64_t* bytes) {
  return guarded([&]() -> int {
    const char* fn = "dp_linear_workspace_bytes";
    clear_error();
    if (!bytes) return bad(fn, "NULL bytes");
    DP_TRY(check_linear(fn, P, T, in_dim, out_dim));
    Mat mx, mw;
    DP_TRY(check_rows(fn, "x", x, P, T, in_dim, false, &mx));
    DP_TRY(check_rows(fn, "w", w, P, out_dim, in_dim, false, &mw));
    *bytes = linear_workspace_bytes(mx, mw, P, T, in_dim, out_dim, backward != 0);
    return DP_OK;
  });
}

int dp_linear_forward(const dp_rows* x, const dp_rows* w, const dp_rows* bias, const dp_rows* residual,
                      const dp_rows* z, const dp_rows* y, int32_t P, int64_t T, int64_t in_dim, int64_t out_dim,
                      int32_t act, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_linear_forward";
    clear_error();
    DP_TRY(check_linear(fn, P, T, in_dim, out_dim));
    DP_TRY(check_act(fn, act));
    LinearArgs a;
    a.P = P;
    a.T = T;
    a.K = in_dim;
    a.N = out_dim;
    a.act = act;
    DP_TRY(check_rows(fn, "x", x, P, T, in_dim, false, &a.x));
    DP_TRY(check_rows(fn, "w", w, P, out_dim, in_dim, false, &a.w));
    DP_TRY(check_rows(fn, "y", y, P, T, out_dim, true, &a.y));
    if (bias) DP_TRY(check_bias(fn, "bias", bias, P, out_dim, false, &a.bias));
    if (residual) DP_TRY(check_rows(fn, "residual", residual, P, T, out_dim, false, &a.residual));
    if (z) DP_TRY(check_rows(fn, "z", z, P, T, out_dim, true, &a.z));
    DP_TRY(need_bf16(fn, "x", a.x));
    DP_TRY(need_bf16(fn, "w", a.w));
    const Part ins[] = {{"x", &a.x, T, in_dim}, {"w", &a.w, out_dim, in_dim}, {"bias", &a.bias, 1, out_dim}};
    for (const Part& o : {Part{"y", &a.y, T, out_dim}, Part{"z", &a.z, T, out_dim}})
      for (const Part& i : ins)
        if (overlap(*o.m, o.rows, o.cols, *i.m, i.rows, i.cols, P))
          return bad(fn, std::string(o.name) + " overlaps " + i.name);
    if (overlap(a.z, T, out_dim, a.y, T, out_dim, P)) return bad(fn, "z overlaps y");
    if (overlap(a.z, T, out_dim, a.residual, T, out_dim, P)) return bad(fn, "z overlaps residual");
    if (!same_place(a.y, a.residual) && overlap(a.y, T, out_dim, a.residual, T, out_dim, P))
      return bad(fn, "y overlaps residual without being it");
    if (T == 0) return DP_OK;
    const int64_t need = linear_workspace_bytes(a.x, a.w, P, T, in_dim, out_dim, false);
    DP_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    for (const Part& i : {ins[0], ins[1], ins[2], Part{"y", &a.y, T, out_dim}, Part{"z", &a.z, T, out_dim},
                          Part{"residual", &a.residual, T, out_dim}})
      if (!apart(workspace, need, *i.m, i.rows, i.cols, P)) return bad(fn, std::string("workspace overlaps ") + i.name);
    return cuda_status(launch_linear_forward(a, static_cast<uint8_t*>(workspace), stream), fn);
  });
}

int dp_linear_backward(const dp_rows* dy, const dp_rows* z, const dp_rows* x, const dp_rows* w, const dp_rows* dx,
                       const dp_rows* dw, const dp_rows* dbias, int32_t P, int64_t T, int64_t in_dim,
                       int64_t out_dim, int32_t act, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                       void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_linear_backward";
    clear_error();
    DP_TRY(check_linear(fn, P, T, in_dim, out_dim));
    DP_TRY(check_act(fn, act));
    LinearArgs a;
    a.P = P;
    a.T = T;
    a.K = in_dim;
    a.N = out_dim;
    a.act = act;
    a.accumulate = accumulate != 0;
    DP_TRY(check_rows(fn, "dy", dy, P, T, out_dim, false, &a.dy));
    DP_TRY(check_rows(fn, "x", x, P, T, in_dim, false, &a.x));
    DP_TRY(check_rows(fn, "w", w, P, out_dim, in_dim, false, &a.w));
    if (act != DP_ACT_NONE) DP_TRY(check_rows(fn, "z", z, P, T, out_dim, false, &a.z));
    if (!dx && !dw && !dbias) return bad(fn, "dx, dw and dbias are all NULL");
    if (dx) DP_TRY(check_rows(fn, "dx", dx, P, T, in_dim, true, &a.dx));
    if (dw) DP_TRY(check_rows(fn, "dw", dw, P, out_dim, in_dim, true, &a.dw));
    if (dbias) DP_TRY(check_bias(fn, "dbias", dbias, P, out_dim, true, &a.dbias));
    DP_TRY(need_bf16(fn, "x", a.x));
    DP_TRY(need_bf16(fn, "w", a.w));
    const Part ins[] = {{"dy", &a.dy, T, out_dim}, {"x", &a.x, T, in_dim}, {"w", &a.w, out_dim, in_dim},
                        {"z", &a.z, T, out_dim}};
    const Part outs[] = {{"dx", &a.dx, T, in_dim}, {"dw", &a.dw, out_dim, in_dim}, {"dbias", &a.dbias, 1, out_dim}};
    for (const Part& o : outs)
      for (const Part& i : ins)
        if (overlap(*o.m, o.rows, o.cols, *i.m, i.rows, i.cols, P))
          return bad(fn, std::string(o.name) + " overlaps " + i.name);
    for (int i = 0; i < 3; ++i)
      for (int j = 0; j < i; ++j)
        if (overlap(*outs[i].m, outs[i].rows, outs[i].cols, *outs[j].m, outs[j].rows, outs[j].cols, P))
          return bad(fn, std::string(outs[i].name) + " overlaps " + outs[j].name);
    const int64_t need = linear_workspace_bytes(a.x, a.w, P, T, in_dim, out_dim, true);
    DP_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    for (const Part& i : {ins[0], ins[1], ins[2], ins[3], outs[0], outs[1], outs[2]})
      if (!apart(workspace, need, *i.m, i.rows, i.cols, P)) return bad(fn, std::string("workspace overlaps ") + i.name);
    return cuda_status(launch_linear_backward(a, static_cast<uint8_t*>(workspace), stream), fn);
  });
}

int dp_orthogonalize_workspace_bytes(int32_t P, int64_t rows, int64_t cols, int64_t* bytes) {
  return guarded([&]() -> int {
    const char* fn = "dp_orthogonalize_workspace_bytes";
    clear_error();
    if (!bytes) return bad(fn, "NULL bytes");
    if (P < 1 || P > kMaxP) return bad(fn, "P outside [1, 64]");
    DP_TRY(check_sides(fn, rows, cols));
    *bytes = orthogonalize_workspace_bytes(P, rows, cols);
    return DP_OK;
  });
}

int dp_orthogonalize(const dp_rows* x, const dp_rows* out, int32_t P, int64_t rows, int64_t cols,
                     const dp_newton_schulz_cfg* cfg, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_orthogonalize";
    clear_error();
    if (P < 1 || P > kMaxP) return bad(fn, "P outside [1, 64]");
    DP_TRY(check_sides(fn, rows, cols));
    Mat mx, mo;
    NewtonSchulz ns;
    DP_TRY(check_rows(fn, "x", x, P, rows, cols, false, &mx));
    DP_TRY(check_rows(fn, "out", out, P, rows, cols, true, &mo));
    DP_TRY(need_bf16(fn, "out", mo));
    DP_TRY(check_ns(fn, cfg, &ns));
    if (!same_place(mo, mx) && overlap(mo, rows, cols, mx, rows, cols, P))
      return bad(fn, "out overlaps x without being it");
    const int64_t need = orthogonalize_workspace_bytes(P, rows, cols);
    DP_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    if (!apart(workspace, need, mx, rows, cols, P) || !apart(workspace, need, mo, rows, cols, P))
      return bad(fn, "workspace overlaps x or out");
    return cuda_status(launch_orthogonalize(mx, mo, P, rows, cols, ns, static_cast<uint8_t*>(workspace), stream), fn);
  });
}

int dp_muon_create(const dp_plan* plan, const int32_t* tensors, const int64_t* rows, const int64_t* cols, int32_t n,
                   dp_muon** out) {
  return guarded([&]() -> int {
    const char* fn = "dp_muon_create";
    clear_error();
    if (!out) return bad(fn, "NULL out");
    *out = nullptr;
    const Plan* pl = as_plan(plan);
    if (!pl) return bad(fn, "NULL plan");
    if (n < 0 || (n > 0 && (!tensors || !rows || !cols))) return bad(fn, "n is negative, or NULL tensors, rows or cols");
    auto m = std::make_unique<Muon>();
    m->plan_id = pl->id;
    m->P = pl->P;
    m->L = pl->L;
    m->stride = pl->stride;
    m->plan_ws = pl->workspace_bytes;
    std::set<int32_t> seen;
    for (int32_t i = 0; i < n; ++i) {
      const int32_t t = tensors[i];
      if (t < 0 || static_cast<size_t>(t) >= pl->sizes.size()) return bad(fn, "tensor " + std::to_string(t) + " is not in the plan");
      if (!seen.insert(t).second) return bad(fn, "tensor " + std::to_string(t) + " is listed twice");
      DP_TRY(check_sides(fn, rows[i], cols[i]));
      const size_t at = static_cast<size_t>(t);
      if (rows[i] * cols[i] != pl->sizes[at])
        return bad(fn, "tensor " + std::to_string(t) + " holds " + std::to_string(pl->sizes[at]) + " elements, not " +
                           std::to_string(rows[i]) + " x " + std::to_string(cols[i]));
      MuonGroup* g = nullptr;
      for (MuonGroup& c : m->groups)
        if (c.rows == rows[i] && c.cols == cols[i]) g = &c;
      if (!g) {
        m->groups.push_back({rows[i], cols[i], {}});
        g = &m->groups.back();
      }
      g->off.push_back(pl->t_off[at]);
    }
    *out = reinterpret_cast<dp_muon*>(m.release());
    return DP_OK;
  });
}

int dp_muon_free(dp_muon* muon) {
  clear_error();
  delete reinterpret_cast<Muon*>(muon);
  return DP_OK;
}

int dp_muon_workspace_bytes(const dp_muon* muon, int64_t* bytes) {
  return guarded([&]() -> int {
    const char* fn = "dp_muon_workspace_bytes";
    clear_error();
    if (!muon || !bytes) return bad(fn, "NULL muon or bytes");
    *bytes = muon_workspace_bytes(*as_muon(muon));
    return DP_OK;
  });
}

int dp_muon_step(const dp_muon* muon, void* plan_workspace, const float* mean, float* master, float* momentum,
                 void* params, int32_t use_clip_coef, const float* coef_dev, const dp_muon_cfg* cfg, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const char* fn = "dp_muon_step";
    clear_error();
    const Muon* m = as_muon(muon);
    if (!m) return bad(fn, "NULL muon");
    if (!plan_workspace) return bad(fn, "NULL plan_workspace");
    if (!cfg) return bad(fn, "NULL cfg");
    for (const void* p : {static_cast<const void*>(plan_workspace), static_cast<const void*>(mean),
                          static_cast<const void*>(master), static_cast<const void*>(momentum),
                          static_cast<const void*>(params)}) {
      if (!p && !m->groups.empty()) return bad(fn, "NULL device pointer");
      if (reinterpret_cast<uintptr_t>(p) & 31u) return fail(DP_EALIGN, std::string(fn) + ": device pointer not 32-byte aligned");
    }
    MuonArgs a{};
    if (coef_dev && !use_clip_coef) return bad(fn, "coef_dev given with use_clip_coef = 0");
    if (reinterpret_cast<uintptr_t>(coef_dev) & 3u) return fail(DP_EALIGN, std::string(fn) + ": coef_dev not 4-byte aligned");
    if (use_clip_coef)
      a.coef = coef_dev ? coef_dev
                        : reinterpret_cast<const float*>(static_cast<uint8_t*>(plan_workspace) + DP_WS_COEF_OFFSET);
    if (reinterpret_cast<uintptr_t>(cfg->lr_dev) & 3u) return fail(DP_EALIGN, std::string(fn) + ": lr_dev not 4-byte aligned");
    if (!(cfg->lr >= 0.0 && cfg->lr <= 1e30)) return bad(fn, "lr must be finite and >= 0");
    if (!(cfg->momentum >= 0.0 && cfg->momentum < 1.0)) return bad(fn, "momentum outside [0, 1)");
    if (!(cfg->weight_decay >= 0.0 && cfg->weight_decay <= 1e30)) return bad(fn, "weight_decay must be finite and >= 0");
    if (cfg->scale != DP_MUON_SPECTRAL && cfg->scale != DP_MUON_MATCH_RMS)
      return bad(fn, "unknown scale " + std::to_string(cfg->scale));
    DP_TRY(check_ns(fn, &cfg->newton_schulz, &a.ns));
    // the fp32 arrays, the replicas and the workspaces, each apart from the others (the mean is only read: it
    // may be the plan workspace's stage)
    const int64_t state = 4 * m->L, reps = 2 * m->P * m->stride, need = muon_workspace_bytes(*m);
    const struct {
      const char* name;
      const void* p;
      int64_t n;
    } parts[] = {{"mean", mean, state}, {"master", master, state}, {"momentum", momentum, state}, {"params", params, reps},
                 {"workspace", workspace, need}, {"plan_workspace", plan_workspace, m->plan_ws}};
    DP_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    for (int i = 0; i < 6; ++i)
      for (int j = i == 5 ? 1 : 0; j < i; ++j) {
        const auto *p = static_cast<const uint8_t*>(parts[i].p), *q = static_cast<const uint8_t*>(parts[j].p);
        if (parts[i].n > 0 && parts[j].n > 0 && p < q + parts[j].n && q < p + parts[i].n)
          return bad(fn, std::string(parts[i].name) + " overlaps " + parts[j].name);
      }
    a.mean = mean;
    a.master = master;
    a.momentum = momentum;
    a.params = static_cast<uint8_t*>(params);
    a.lr_dev = cfg->lr_dev;
    a.lr = static_cast<float>(cfg->lr);
    a.weight_decay = static_cast<float>(cfg->weight_decay);
    a.mu = static_cast<float>(cfg->momentum);
    a.rest = static_cast<float>(1.0 - cfg->momentum);
    a.nesterov = cfg->nesterov != 0;
    a.match_rms = cfg->scale == DP_MUON_MATCH_RMS;
    a.hdr = plan_workspace;
    return cuda_status(launch_muon(*m, a, static_cast<uint8_t*>(workspace), stream), fn);
  });
}

int64_t dp_product_timeouts(int32_t reset) {
  clear_error();
  const int64_t a = product_timeouts_linear(reset != 0), b = product_timeouts_orthogonal(reset != 0);
  return a < 0 || b < 0 ? -2 : a + b;
}

}  // extern "C"
