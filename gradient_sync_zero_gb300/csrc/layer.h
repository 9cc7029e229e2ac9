// The dense layer and the update of its weights: what the C ABI entries (layer_api.cu) hand to
// the kernel launchers (kernels_linear.cu, kernels_orthogonal.cu).  Arguments are checked before.
#pragma once

#include <cstdint>
#include <vector>

#include "model.h"

namespace dps {

struct LinearArgs {
  Mat x, w, bias, residual, z, y;   // forward; bias one row
  Mat dy, dx, dw, dbias;            // backward (p = nullptr: not wanted)
  int P = 1;
  int64_t T = 0, K = 0, N = 0;
  int act = 0;
  bool accumulate = false;
};

// Rows that the tensor core's copies can read in place: 16-byte boundaries, strides they can hold,
// and no row shown twice.
bool copyable(const Mat& m, int64_t rows, int64_t cols);
int64_t linear_workspace_bytes(const Mat& x, const Mat& w, int P, int64_t T, int64_t K, int64_t N, bool backward);
int launch_linear_forward(const LinearArgs& a, uint8_t* ws, void* stream);
int launch_linear_backward(const LinearArgs& a, uint8_t* ws, void* stream);

struct NewtonSchulz {
  float a, b, c, eps;
  int steps;
};
int64_t orthogonalize_workspace_bytes(int P, int64_t rows, int64_t cols);
int launch_orthogonalize(const Mat& x, const Mat& out, int P, int64_t rows, int64_t cols, const NewtonSchulz& ns,
                         uint8_t* ws, void* stream);

// The matrices of one shape, in the order they were given.
struct MuonGroup {
  int64_t rows, cols;
  std::vector<int64_t> off;   // flat offsets
};
struct Muon {
  uint64_t plan_id;
  int32_t P;
  int64_t L, stride;          // of the plan's flat space, of its replicas
  int64_t plan_ws;            // bytes of the plan's workspace
  std::vector<MuonGroup> groups;
};
struct MuonArgs {
  const float* mean;
  float *master, *momentum;
  uint8_t* params;
  const float* coef;          // device, or nullptr
  const float* lr_dev;
  float lr, weight_decay, mu, rest;   // rest = 1 - mu
  bool nesterov, match_rms;
  NewtonSchulz ns;
  void* hdr;                  // DevHeader of the plan's workspace
};
int64_t muon_workspace_bytes(const Muon& m);
int launch_muon(const Muon& m, const MuonArgs& a, uint8_t* ws, void* stream);

// Bounded waits of the products that gave up (-2: the counters cannot be read).
int64_t product_timeouts_linear(bool reset);
int64_t product_timeouts_orthogonal(bool reset);

}  // namespace dps
