// Newton-Schulz orthogonalisation of a batch of matrices, and the Muon step built on it.
//
//   X = x / max(|x|, eps);  steps times: G = X X^T (X^T X where X is tall),
//   Q = b G + c G^2,  X <- a X + Q X (a X + X Q)
//
// An odd polynomial of X: it acts on the singular values alone and drives them towards 1.  Three
// products a step on k_product (product.cuh).  G and Q are symmetric, so only the tiles of their
// lower halves are formed, the others written as their mirror: 3 m^2 n + m^3 operations a step
// where plain products take 4 m^2 n + 2 m^3 (m the smaller side).
//
// The products' operands are fp16 (their sums fp32): an iterate's singular values stay near or
// below 1, so the range is known and bf16's three bits less would buy nothing (errors of the
// result measured 1e-2 to 3e-2 with bf16, 1e-3 with fp16).  X is held times a power of two, S, that
// brings a flat spectrum's entries near 1: an entry of S X is at most about 1.3 S < 2^16.  What
// rounding X loses would be scaled up with the small singular values by a X, step after
// step, so X is kept as fp16 and what that leaves out, lo, as 8 bits: the products read X, the
// epilogue adds a (X + lo).  (Simulated in 64 bits: without lo a matrix of rank 1 comes out 0.15 off
// and a spectrum that falls like 1/i 3.7e-3, with it 5e-4 and 4e-4; lo in e5m2 leaves 7e-3.  a
// on the diagonal of Q would spare the epilogue X, but takes Q's last bits: 1.5e-3.)
//
// On GB300, five steps, in bursts: four 2048 x 5632 matrices 1.22 to 1.27 ms (1280 TFLOP/s of the operations
// above), one 7680 x 2560 0.69 to 0.74 ms (55 of its tiles on 76 pairs in two of three products).  A
// step of the four: G 62 us, Q 33, X 126: X's epilogue moves eight bytes a value through the SM
// beside the products and takes as long as they do.
#include <algorithm>
#include <cmath>
#include <memory>
#include <utility>
#include <vector>

#include "layer.h"
#include "product.cuh"

namespace dps {
namespace {

constexpr int kMaxBatch = 64;

// ---- fp16 rows of a workspace matrix: pitches are multiples of 32 elements ----
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
__device__ __forceinline__ void store_half(__half* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_half(f[0], f[1]), pack_half(f[2], f[3]), pack_half(f[4], f[5]), pack_half(f[6], f[7]));
}

// What fp16 leaves out of a value, up to half of hi's last place, as 8 bits in 1/254 of that place
// (-127 .. 127, biased by 128), so the pair holds 19 bits.  A place is 2^(e - 10) for hi in
// [2^e, 2^(e + 1)), 2^-24 below 2^-14; powers of two are multiplied by adding exponents.
__device__ __forceinline__ uint32_t exponent_of(float hi) {
  return max(__float_as_uint(hi) & 0x7f800000u, 0x38800000u);   // (e + 127) << 23
}
__device__ __forceinline__ uint32_t lo_of(float f, float hi) {   // in the low byte; the others are not 0
  const float per = __uint_as_float((271u << 23) + 0x7e0000u - exponent_of(hi));   // 254 / 256 * 2^(18 - e)
  return __float_as_uint(fmaf(f - hi, per, 12582912.0f + 128.0f));                 // rounds to an integer
}
__device__ __forceinline__ float with_lo(float hi, uint32_t word, int byte) {
  const float q = __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u | byte)) - (8388608.0f + 128.0f);
  return fmaf(q, __uint_as_float(exponent_of(hi) - (18u << 23) + 0x10204u), hi);   // 256 / 254 * 2^(e - 18)
}
// f rounded to hi, and what that left out.
__device__ __forceinline__ void store_pair(__half* hi, uint8_t* lo, const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = lo_of(f[4 * j + i], __half2float(__float2half_rn(f[4 * j + i])));
    w[j] = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
  }
  store_half(hi, f);
  *reinterpret_cast<uint2*>(lo) = make_uint2(w[0], w[1]);
}

struct HalfMat {
  __half* p;
  int64_t step;    // from matrix to matrix
  int32_t pitch;
  __device__ __forceinline__ int64_t at(int b, int m, int n) const { return b * step + int64_t{m} * pitch + n; }
};

// The plan's workspace of a Muon step (hdr NULL: none): what the step may still write depends on it.
struct PlanState {
  DevHeader* hdr;
  uint64_t plan_id;
  // This plan's, and no bounded wait gave up: sums that were not waited for must not reach the weights.
  __device__ __forceinline__ bool sound() const {
    return hdr->plan_id == plan_id && !(*reinterpret_cast<const volatile int32_t*>(&hdr->status) & DP_STATUS_TIMEOUT);
  }
  __device__ __forceinline__ void report(int32_t bit) const {
    if (hdr) atomicOr(&hdr->status, bit);
  }
};

// Both halves of a symmetric matrix: blocks of 256 above the diagonal mirror those below.
struct Symmetric {
  static constexpr bool kSwap = false, kMirror = true, kBefore = false, kAsks = false;
  HalfMat out;
  PlanState plan;
  __device__ __forceinline__ void gave_up() const { plan.report(DP_STATUS_TIMEOUT); }
  struct Cols {};
  __device__ __forceinline__ void fetch_cols(int, int, Cols&) const {}
  __device__ __forceinline__ bool whole(int) const { return true; }   // pitches hold whole vectors
  __device__ __forceinline__ void apply_rows(int, int, int, int, const float*, int) const {}
  __device__ __forceinline__ void mirror(int b, int n, int m, const float (&v)[8]) const {
    store_half(out.p + out.at(b, n, m), v);
  }
  // Eight values that were joined, and their mirror one by one.
  __device__ __forceinline__ void store_both(int b, int m, int n, const float (&v)[8], int valid) const {
    store_half(out.p + out.at(b, m, n), v);
    if (m / kTileM > n / kTileM) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) out.p[out.at(b, n + j, m)] = __float2half_rn(v[j]);
    }
  }
  static __device__ __forceinline__ bool above(int m, int n) { return n / kTileM > m / kTileM; }
};

// G = X X^T / S^2.
struct GramEpi : Symmetric {
  static constexpr bool kJoins = true;
  using Straight = GramEpi;
  float alpha;
  struct Pre {};
  __device__ __forceinline__ bool ahead(int) const { return false; }
  __device__ __forceinline__ void fetch(int, int, int, Pre&) const {}
  __device__ __forceinline__ void before(float (&)[8], const Pre&) const {}
  __device__ __forceinline__ void scale(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= alpha;
  }
  __device__ __forceinline__ void apply(int b, int m, int n, float (&v)[8], const Pre&, const Cols&) const {
    scale(v);
    store_half(out.p + out.at(b, m, n), v);
  }
  __device__ __forceinline__ void join(int b, int m, int n, float (&v)[8], int valid) const {
    if (above(m, n)) return;
    scale(v);
    store_both(b, m, n, v, valid);
  }
};

// Q = b G + c G G.
struct PolyEpi : Symmetric {
  static constexpr bool kJoins = false;
  HalfMat g;
  float b1, c1;
  struct Pre {
    uint4 q;
  };
  __device__ __forceinline__ bool ahead(int) const { return true; }
  __device__ __forceinline__ void fetch(int b, int m, int n, Pre& pre) const { pre.q = ld_again(g.p + g.at(b, m, n)); }
  __device__ __forceinline__ void before(float (&)[8], const Pre&) const {}
  __device__ __forceinline__ void combine(float (&v)[8], const Pre& pre) const {
    const uint32_t w[4] = {pre.q.x, pre.q.y, pre.q.z, pre.q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_half(w[i]);
      v[2 * i] = fmaf(c1, v[2 * i], b1 * t.x);
      v[2 * i + 1] = fmaf(c1, v[2 * i + 1], b1 * t.y);
    }
  }
  __device__ __forceinline__ void apply(int b, int m, int n, float (&v)[8], const Pre& pre, const Cols&) const {
    combine(v, pre);
    store_half(out.p + out.at(b, m, n), v);
  }
};

// ---- where the last iterate goes ----
// The matrices of a launch.
struct MuonTable {
  int64_t off[kMaxBatch];
  int32_t rows[kMaxBatch], cols[kMaxBatch];
  float scale[kMaxBatch];     // s of the update
};
struct MuonOut {
  float* master;
  __nv_bfloat16* params;
  int64_t stride;
  PlanState plan;
  const float* lr_dev;
  float lr, decay;            // theta <- (1 - lr decay) theta - lr s O
  int32_t P;
  MuonTable of;
  __device__ __forceinline__ bool vec(int b) const { return of.cols[b] % 8 == 0; }   // offsets are multiples of eight
};

enum { kIterate = 0, kMatrix = 1, kMuon = 2 };

// What becomes of the last iterate: a matrix of the caller's, or the Muon update (whose kernels ask
// the plan's state before).
struct Finish {
  int32_t mode, vec;
  Mat out;
  MuonOut mu;

  // Eight columns of which `valid` exist; v ends as what was stored.
  __device__ __forceinline__ void finish(int b, int m, int n0, float (&v)[8], int valid) const {
    constexpr int C = 8;
    if (mode == kMatrix) {
      __nv_bfloat16* p = row_ptr<__nv_bfloat16>(out, b, m) + n0;
      store_bf16(p, v, valid, vec);
      return;
    }
    const float lr = mu.lr_dev ? *mu.lr_dev : mu.lr;
    const float keep = 1.0f - lr * mu.decay, step = lr * mu.of.scale[b];
    const int64_t cols = mu.of.cols[b];
    const bool wide = mu.vec(b);
    const int64_t at = mu.of.off[b] + m * cols + n0;
    float* w = mu.master + at;
    if (wide && valid == C) {
#pragma unroll
      for (int j = 0; j < C; j += 4) {
        const uint4 q = ld_again(w + j);
        v[j] = fmaf(-step, v[j], keep * __uint_as_float(q.x));
        v[j + 1] = fmaf(-step, v[j + 1], keep * __uint_as_float(q.y));
        v[j + 2] = fmaf(-step, v[j + 2], keep * __uint_as_float(q.z));
        v[j + 3] = fmaf(-step, v[j + 3], keep * __uint_as_float(q.w));
      }
#pragma unroll
      for (int j = 0; j < C; j += 8) put_f8(w + j, v + j);   // offsets are multiples of eight
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j < valid) w[j] = v[j] = fmaf(-step, v[j], keep * w[j]);
    }
    for (int r = 0; r < mu.P; ++r) store_bf16(mu.params + r * mu.stride + at, v, valid, wide);
  }

  // Column n of rows m0 .. : scale times column `lane` of the block.
  __device__ __forceinline__ void finish_rows(int b, int m0, int rows, int n, const float* block, int lane, float scale) const {
    if (mode == kMatrix) {
#pragma unroll 8
      for (int i = 0; i < rows; ++i) st_elem(row_ptr<__nv_bfloat16>(out, b, m0 + i) + n, scale * block_at(block, i, lane));
      return;
    }
    const float lr = mu.lr_dev ? *mu.lr_dev : mu.lr;
    const float keep = 1.0f - lr * mu.decay, step = lr * mu.of.scale[b];
    const int64_t cols = mu.of.cols[b];
#pragma unroll 1
    for (int r = 0; r < rows; r += 8) {
      const int64_t at = mu.of.off[b] + (m0 + r) * cols + n;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r + i < rows ? mu.master[at + i * cols] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = fmaf(-step, scale * block_at(block, r + i, lane), keep * v[i]);
        if (r + i < rows) mu.master[at + i * cols] = v[i];
      }
      for (int p = 0; p < mu.P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r + i < rows) st_elem(mu.params + p * mu.stride + at + i * cols, v[i]);
    }
  }

  static __device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&v)[8], int valid, bool vec) {
    if (vec && valid == 8) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack2_rne(v[0], v[1]), pack2_rne(v[2], v[3]), pack2_rne(v[4], v[5]), pack2_rne(v[6], v[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) st_elem(p + j, v[j]);
    }
  }
};

// X <- a (X + lo) + Q X: the next iterate, or the last.
struct ApplyEpi : Finish {
  static constexpr bool kSwap = false, kMirror = false, kBefore = true, kJoins = false, kAsks = true;
  const __half* hi;           // X, lo and the next X are laid out alike
  HalfMat hi_out;
  uint8_t* lo;
  float a, inv;               // inv = 1 / S

  struct Pre {
    uint4 h;
    uint2 q;
  };
  struct Cols {};
  __device__ __forceinline__ bool live() const { return mode != kMuon || mu.plan.sound(); }
  __device__ __forceinline__ void gave_up() const { mu.plan.report(DP_STATUS_TIMEOUT); }
  __device__ __forceinline__ void fetch_cols(int, int, Cols&) const {}
  __device__ __forceinline__ bool ahead(int) const { return true; }
  __device__ __forceinline__ void fetch(int b, int m, int n, Pre& pre) const {
    const int64_t at = hi_out.at(b, m, n);
    pre.h = ld_again(hi + at);
    asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(pre.q.x), "=r"(pre.q.y) : "l"(lo + at) : "memory");
  }
  __device__ __forceinline__ void before(float (&v)[8], const Pre& pre) const {
    const uint32_t x[4] = {pre.h.x, pre.h.y, pre.h.z, pre.h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = unpack_half(x[i]);
      const uint32_t w = i < 2 ? pre.q.x : pre.q.y;
      v[2 * i] = fmaf(a, with_lo(h.x, w, 2 * i & 3), v[2 * i]);
      v[2 * i + 1] = fmaf(a, with_lo(h.y, w, (2 * i & 3) + 1), v[2 * i + 1]);
    }
  }
  // The caller's rows in whole vectors (one shape a launch); the next iterate's always are.
  __device__ __forceinline__ bool whole(int valid) const {
    return mode == kIterate || (valid == 32 && (mode == kMuon ? mu.vec(0) : vec));
  }
  __device__ __forceinline__ void apply(int b, int m, int n, float (&v)[8], const Pre& pre, const Cols&) const {
    before(v, pre);
    if (mode == kIterate) {
      const int64_t at = hi_out.at(b, m, n);
      store_pair(hi_out.p + at, lo + at, v);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
    finish(b, m, n, v, 8);
  }
  __device__ __forceinline__ void apply_rows(int b, int m0, int rows, int n, const float* block, int lane) const {
    finish_rows(b, m0, rows, n, block, lane, inv);
  }
  __device__ __forceinline__ void mirror(int, int, int, const float (&)[8]) const {}
};

// ---- from the caller's matrices to the first iterate ----
// Sources give eight columns j .. j + 7 of row i of matrix b, of which `valid` exist (others 0):
// ahead() issues the loads of whole vectors, first() and again() use them, so that a thread's loads
// are all on their way before its first store.
template <class T>
__device__ __forceinline__ void take_eight(const Oct<T>& o, const T* p, int valid, bool vec, float (&f)[8]) {
  if (vec && valid == 8) {
    o.get(f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < valid ? ld_elem(p + k) : 0.0f;
  }
}

template <class T>
struct MatSource {
  Mat x;
  int32_t vec, rows, cols;
  struct Ahead {
    Oct<T> x;
  };
  __device__ __forceinline__ int rows_of(int) const { return rows; }
  __device__ __forceinline__ int cols_of(int) const { return cols; }
  static constexpr bool kGuarded = false;
  __device__ __forceinline__ bool ready() const { return true; }   // for all threads of a CTA
  __device__ __forceinline__ void ahead(int b, int64_t i, int64_t j, int valid, bool, Ahead& o) const {
    if (vec && valid == 8) o.x.load_again(row_ptr<const T>(x, b, i) + j);
  }
  __device__ __forceinline__ void first(int b, int64_t i, int64_t j, int valid, const Ahead& o, float (&f)[8]) const {
    take_eight(o.x, row_ptr<const T>(x, b, i) + j, valid, vec, f);
  }
  __device__ __forceinline__ void again(int b, int64_t i, int64_t j, int valid, const Ahead& o, float (&f)[8]) const {
    first(b, i, j, valid, o, f);
  }
  __device__ __forceinline__ void not_finite() const {}
};

// buf <- mu buf + (1 - mu) g and u = mu buf + (1 - mu) g (or buf), g = coef mean.  The second
// pass reads what the first wrote and forms the same u.
struct MuonSource {
  const float* mean;
  float* momentum;
  const float* coef;
  PlanState plan;
  float mu, rest;
  int32_t nesterov;
  MuonTable of;
  struct Ahead {
    Oct<float> g, m;
  };
  __device__ __forceinline__ int rows_of(int b) const { return of.rows[b]; }
  __device__ __forceinline__ int cols_of(int b) const { return of.cols[b]; }
  // The same in the whole CTA: one thread reads what another stream's kernel may be changing.
  static constexpr bool kGuarded = true;
  __device__ __forceinline__ bool ready() const {
    __shared__ bool ok;
    if (threadIdx.x == 0) {
      ok = plan.sound();
      if (plan.hdr->plan_id != plan.plan_id) plan.report(DP_STATUS_PLAN_MISMATCH);
    }
    __syncthreads();
    return ok;
  }
  __device__ __forceinline__ int64_t at(int b, int64_t i, int64_t j) const { return of.off[b] + i * of.cols[b] + j; }
  __device__ __forceinline__ bool vec(int b) const { return of.cols[b] % 8 == 0; }
  __device__ __forceinline__ void ahead(int b, int64_t i, int64_t j, int valid, bool is_first, Ahead& o) const {
    if (!vec(b) || valid != 8) return;
    o.m.load_again(momentum + at(b, i, j));
    if (is_first || nesterov) o.g.load_again(mean + at(b, i, j));
  }
  __device__ __forceinline__ void gradient(int b, int64_t p, int valid, const Ahead& o, float (&g)[8]) const {
    take_eight(o.g, mean + p, valid, vec(b), g);
    if (coef) {
      const float c = *coef;
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] *= c;
    }
  }
  __device__ __forceinline__ void look_ahead(const float (&g)[8], float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = nesterov ? fmaf(mu, f[k], rest * g[k]) : f[k];
  }
  __device__ __forceinline__ void first(int b, int64_t i, int64_t j, int valid, const Ahead& o, float (&f)[8]) const {
    float* p = momentum + at(b, i, j);
    float g[8];
    gradient(b, at(b, i, j), valid, o, g);
    take_eight(o.m, static_cast<const float*>(p), valid, vec(b), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = fmaf(mu, f[k], rest * g[k]);
    if (vec(b) && valid == 8) {
      put_f8(p, f);   // offsets are multiples of eight
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < valid) p[k] = f[k];
    }
    look_ahead(g, f);
  }
  __device__ __forceinline__ void again(int b, int64_t i, int64_t j, int valid, const Ahead& o, float (&f)[8]) const {
    take_eight(o.m, static_cast<const float*>(momentum) + at(b, i, j), valid, vec(b), f);
    if (!nesterov) return;
    float g[8];
    gradient(b, at(b, i, j), valid, o, g);
    look_ahead(g, f);
  }
  __device__ __forceinline__ void not_finite() const { plan.report(DP_STATUS_NONFINITE); }
};

constexpr int kStageThreads = 256, kStageOcts = 4;   // groups of eight values a thread

// Squares are summed in fp32 in units of the CTA's largest value's power of two, so that none over- or
// underflows, and one thread goes on in double.  (FP64 is so slow on this GPU that a few
// double operations of every thread took most of these kernels' time.)
struct Unit {
  uint32_t e;   // biased exponent
  __device__ __forceinline__ float inverse() const { return __uint_as_float((254 - e) << 23); }
  __device__ __forceinline__ double squared(float sum) const {
    const double u = __hiloint2double(static_cast<int>(e + 896) << 20, 0);
    return static_cast<double>(sum) * u * u;
  }
};
// most: this thread's largest magnitude, as its bits (NaN above all).
__device__ __forceinline__ Unit block_unit(uint32_t most) {
  __shared__ uint32_t of[32];
  most = __reduce_max_sync(0xffffffffu, most);
  if (threadIdx.x % 32 == 0) of[threadIdx.x / 32] = most;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) most = max(most, of[i]);
  const uint32_t e = most >> 23;
  return {e > 253 ? 253 : e};
}
// The sum over the CTA, in thread 0.
__device__ __forceinline__ float block_sum(float s) {
  __shared__ float of[32];
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (threadIdx.x % 32 == 0) of[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < static_cast<int>(blockDim.x) / 32; ++i) s += of[i];
  return s;
}
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

template <class Src>
__global__ void __launch_bounds__(kStageThreads)
k_ns_squares(const __grid_constant__ Src src, int64_t rows, int64_t cols, Div8 per, double* parts) {
  wait_for_predecessor();
  if (!src.ready()) return;
  const int b = blockIdx.y;
  const int64_t n = rows * per.n;
  float f[kStageOcts][8] = {};
  typename Src::Ahead o[kStageOcts];
  int64_t i[kStageOcts], j[kStageOcts];
  int valid[kStageOcts];
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k) {
    const int64_t x = (int64_t{blockIdx.x} * kStageOcts + k) * kStageThreads + threadIdx.x;
    valid[k] = 0;
    if (x < n) {
      per.split(x, i[k], j[k]);
      j[k] *= 8;
      valid[k] = static_cast<int>(cols - j[k] < 8 ? cols - j[k] : 8);
      src.ahead(b, i[k], j[k], valid[k], true, o[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k)
    if (valid[k]) src.first(b, i[k], j[k], valid[k], o[k], f[k]);
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) most = max(most, magnitude(f[k][q]));
  const Unit unit = block_unit(most);
  const float inv = unit.inverse();
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float v = f[k][q] * inv;
      s = fmaf(v, v, s);
    }
  s = block_sum(s);
  if (threadIdx.x == 0) parts[int64_t{b} * gridDim.x + blockIdx.x] = unit.squared(s);
}

// The norm of each matrix, from its parts in their order.
constexpr int kNormThreads = 128;
template <class Src>
__global__ void __launch_bounds__(kNormThreads)
k_ns_norm(const __grid_constant__ Src src, const double* parts, int n_parts, double* norms) {
  __shared__ double of[kNormThreads];
  wait_for_predecessor();
  if (!src.ready()) return;
  const double* p = parts + int64_t{blockIdx.x} * n_parts;
  double s = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += kNormThreads) s += p[i];
  of[threadIdx.x] = s;
  for (int d = kNormThreads / 2; d > 0; d /= 2) {
    __syncthreads();
    if (threadIdx.x < d) of[threadIdx.x] += of[threadIdx.x + d];
  }
  if (threadIdx.x != 0) return;
  const double norm = sqrt(of[0]);
  norms[blockIdx.x] = norm;
  if (!isfinite(norm)) src.not_finite();
}

// 1 / max(norm, eps) times `to`; NaN where the norm is not finite.
__device__ __forceinline__ float norm_scale(double norm, float eps, double to) {
  return isfinite(norm) ? static_cast<float>(to / (norm < eps ? static_cast<double>(eps) : norm)) : __int_as_float(0x7fffffff);
}

// 1 / max(norm, eps) as two factors: of a long matrix of fp32's largest values it is below the normal
// numbers (9 bits of it are left at 64 x 2^18).  (S / norm never is: S grows with the matrix as its norm may.)
struct TwoFactors {
  float first, then;
  __device__ __forceinline__ float of(float v) const { return v * first * then; }
};
__device__ __forceinline__ TwoFactors inverse_norm(double norm, float eps) {
  const float first = norm > 0x1p96 ? 0x1p-64f : 1.0f;
  return {first, norm_scale(norm, eps, norm > 0x1p96 ? 0x1p64 : 1.0)};
}

// S X as hi and lo.
template <class Src>
__global__ void __launch_bounds__(kStageThreads)
k_ns_stage(const __grid_constant__ Src src, int64_t rows, int64_t cols, Div8 per, const double* norms, float S, float eps,
           HalfMat hi, uint8_t* lo) {
  __shared__ float scale_of;
  wait_for_predecessor();
  if (!src.ready()) return;
  const int b = blockIdx.y;
  const int64_t n = rows * per.n;
  typename Src::Ahead o[kStageOcts];
  int64_t i[kStageOcts], j[kStageOcts];
  int valid[kStageOcts];
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k) {
    const int64_t x = (int64_t{blockIdx.x} * kStageOcts + k) * kStageThreads + threadIdx.x;
    valid[k] = 0;
    if (x < n) {
      per.split(x, i[k], j[k]);
      j[k] *= 8;
      valid[k] = static_cast<int>(cols - j[k] < 8 ? cols - j[k] : 8);
      src.ahead(b, i[k], j[k], valid[k], false, o[k]);
    }
  }
  if (threadIdx.x == 0) scale_of = norm_scale(norms[b], eps, S);
  __syncthreads();
  const float scale = scale_of;
#pragma unroll
  for (int k = 0; k < kStageOcts; ++k) {
    if (!valid[k]) break;
    float f[8];
    src.again(b, i[k], j[k], valid[k], o[k], f);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] *= scale;
    const int64_t at = b * hi.step + i[k] * hi.pitch + j[k];
    store_pair(hi.p + at, lo + at, f);
  }
}

// ---- small matrices: the whole iteration in the shared memory of a cluster ----
// In fp32 on the ordinary multipliers: a matrix too small to fill tiles costs the tensor cores three
// launches a step (115 us for 3 x 48 x 131), here a step is a few thousand cycles, and nothing is
// rounded to fewer bits.  X lies as [m][n] whichever side is longer; each CTA of the cluster has all m
// rows of a slice of n.  A step: its part of G, one cluster barrier, the sum of the parts in the
// CTAs' order through distributed shared memory, Q (in every CTA), its slice of a X + Q X.
// A thread forms 4 x 4 values from four rows (of k) of each operand at a time: eight 16-byte
// reads for 64 multiply-adds.  3 x 48 x 131 take 36 us, 6 of them a step: three quarters of that is the latency of
// reads, shuffles and barriers (one CTA for a matrix took 43 us).
constexpr int64_t kSmallFloats = 56 * 1024;   // of shared memory
constexpr int kSmallNsThreads = 512;
constexpr int kSmallLong = 256;               // from here on eight CTAs share a matrix, below four

// Rows of `ld` floats start 4 banks apart, so eight rows' 16-byte reads meet no bank twice.
__host__ __device__ inline int small_ld(int64_t n) { return static_cast<int>((n + 27) / 32 * 32 + 4); }
// Columns of a CTA: whole groups of eight.
__host__ __device__ inline int small_slice(int64_t n, int ctas) { return static_cast<int>((n + 8 * ctas - 1) / (8 * ctas) * 8); }
inline int small_ctas(int64_t n) { return n > kSmallLong ? 8 : 4; }
// X, Y, two parts of G (peers may still read the last one), G and Q.
inline int64_t small_floats(int64_t m, int64_t n, int ctas) {
  const int64_t m4 = (m + 3) / 4 * 4;
  return 2 * m4 * small_ld(small_slice(n, ctas)) + 4 * m4 * small_ld(m);
}
bool fits_small(int64_t rows, int64_t cols) {
  const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  return m <= 128 && n <= kSmallFloats && small_floats(m, n, small_ctas(n)) <= kSmallFloats;
}

// acc[i][j] += sum over k = k0, k0 + 4 step .. < kn (and the three after each) of a[i][k] b[j][k]
__device__ __forceinline__ void rows_by_rows(const float* a, int lda, const float* b, int ldb, int k0, int kn, int step,
                                             float (&acc)[4][4]) {
#pragma unroll 2
  for (int k = k0; k < kn; k += 4 * step) {
    float4 p[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = *reinterpret_cast<const float4*>(a + i * lda + k);
      q[i] = *reinterpret_cast<const float4*>(b + i * ldb + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(p[i].x, q[j].x, fmaf(p[i].y, q[j].y, fmaf(p[i].z, q[j].z, fmaf(p[i].w, q[j].w, acc[i][j]))));
  }
}

// acc[u][v] += sum over k likewise of q[u][k] x[k][v]
__device__ __forceinline__ void rows_by_cols(const float* q, int ldq, const float* x, int ldx, int k0, int kn, int step,
                                             float (&acc)[4][4]) {
#pragma unroll 2
  for (int k = k0; k < kn; k += 4 * step) {
    float4 p[4], r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      p[u] = *reinterpret_cast<const float4*>(q + u * ldq + k);
      r[u] = *reinterpret_cast<const float4*>(x + (k + u) * ldx);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w[4] = {p[u].x, p[u].y, p[u].z, p[u].w};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[u][0] = fmaf(w[v], r[v].x, acc[u][0]);
        acc[u][1] = fmaf(w[v], r[v].y, acc[u][1]);
        acc[u][2] = fmaf(w[v], r[v].z, acc[u][2]);
        acc[u][3] = fmaf(w[v], r[v].w, acc[u][3]);
      }
    }
  }
}

// A tile's k is shared by neighbouring lanes (1, 2 or 4 of them) where there are fewer tiles than
// threads; their sums are added in the same order in each, and each writes its part of the tile's rows.
template <int SHARE>
__device__ __forceinline__ void add_shares(float (&acc)[4][4]) {
#pragma unroll
  for (int d = 1; d < SHARE; d *= 2)
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[u][v] += __shfl_xor_sync(0xffffffffu, acc[u][v], d);
}
// Calls f with the share as a constant (divisions by it are shifts).
template <class F>
__device__ __forceinline__ void with_share(int tiles, F&& f) {
  if (4 * tiles <= kSmallNsThreads) return f(std::integral_constant<int, 4>{});
  if (2 * tiles <= kSmallNsThreads) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

// Y = a X + Q X, tiles of four rows and four columns, for the whole CTA.
__device__ __forceinline__ void apply_tiles(float a, const float* q, int ldq, const float* x, float* y, int ldx, int m4, int n4) {
  const int tiles = m4 * n4;
  with_share(tiles, [&](auto s) {
    constexpr int kShare = decltype(s)::value;
    const int sub = threadIdx.x % kShare;
    for (int t0 = 0; t0 < tiles; t0 += kSmallNsThreads / kShare) {
      const int t = t0 + static_cast<int>(threadIdx.x) / kShare;
      const int i = t / n4, j = t - i * n4;
      float acc[4][4] = {};
      if (t < tiles) rows_by_cols(q + 4 * i * ldq, ldq, x + 4 * j, ldx, 4 * sub, 4 * m4, kShare, acc);
      add_shares<kShare>(acc);
      if (t < tiles) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u % kShare == sub) {
            const float4 p = *reinterpret_cast<const float4*>(x + (4 * i + u) * ldx + 4 * j);
            *reinterpret_cast<float4*>(y + (4 * i + u) * ldx + 4 * j) = make_float4(
                fmaf(a, p.x, acc[u][0]), fmaf(a, p.y, acc[u][1]), fmaf(a, p.z, acc[u][2]), fmaf(a, p.w, acc[u][3]));
          }
      }
    }
  });
}

// Row and column of the tiles of a lower half, found once.
constexpr int kLowerTiles = 32 * 33 / 2;   // of up to 128 rows
__device__ __forceinline__ void list_tiles(uint16_t* list, int m4) {
  for (int i = threadIdx.x; i < m4 * m4; i += kSmallNsThreads) {
    const int r = i / m4, c = i - r * m4;
    if (c <= r) list[r * (r + 1) / 2 + c] = static_cast<uint16_t>(r << 8 | c);
  }
}

// A symmetric product by its lower half: `to` = rows of `from` by rows of `from`, or with g (then from is
// G) Q = b G + c G G.
__device__ __forceinline__ void symmetric_tiles(const uint16_t* list, const float* from, int ld, int kn, float* to,
                                                const float* g, int ldg, int m4, float b1, float c1) {
  const int tiles = m4 * (m4 + 1) / 2;
  with_share(tiles, [&](auto s) {
    constexpr int kShare = decltype(s)::value;
    const int sub = threadIdx.x % kShare;
    for (int t0 = 0; t0 < tiles; t0 += kSmallNsThreads / kShare) {
      const int t = t0 + static_cast<int>(threadIdx.x) / kShare;
      const int at = list[t < tiles ? t : 0], i = at >> 8, j = at & 255;
      float acc[4][4] = {};
      if (t < tiles) rows_by_rows(from + 4 * i * ld, ld, from + 4 * j * ld, ld, 4 * sub, kn, kShare, acc);
      add_shares<kShare>(acc);
      if (t < tiles) {
        if (g) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 p = *reinterpret_cast<const float4*>(g + (4 * i + u) * ldg + 4 * j);
            acc[u][0] = fmaf(c1, acc[u][0], b1 * p.x);
            acc[u][1] = fmaf(c1, acc[u][1], b1 * p.y);
            acc[u][2] = fmaf(c1, acc[u][2], b1 * p.z);
            acc[u][3] = fmaf(c1, acc[u][3], b1 * p.w);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u % kShare == sub) {
            *reinterpret_cast<float4*>(to + (4 * i + u) * ldg + 4 * j) = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
            *reinterpret_cast<float4*>(to + (4 * j + u) * ldg + 4 * i) = make_float4(acc[0][u], acc[1][u], acc[2][u], acc[3][u]);
          }
      }
    }
  });
}

__device__ __forceinline__ float4 peer_float4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ double peer_double(uint32_t cluster_addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <class Src, int CTAS>
__global__ void __launch_bounds__(kSmallNsThreads)
k_ns_small(const __grid_constant__ Src src, float a1, float b1, float c1, float eps, int steps,
           const __grid_constant__ Finish last) {
  extern __shared__ __align__(16) float small_smem[];
  __shared__ double squares;
  __shared__ TwoFactors scale_of;
  __shared__ uint32_t ready, go;   // this CTA's reading, and whether all of the cluster's agree: CTAs that read
                                   // each other's memory leave together
  __shared__ uint16_t list[kLowerTiles];
  wait_for_predecessor();
  const int batch = blockIdx.x / CTAS, tid = threadIdx.x, rank = static_cast<int>(cluster_rank());
  const bool allowed = src.ready();
  if (tid == 0) ready = allowed;
  const int rows = src.rows_of(batch), cols = src.cols_of(batch);
  const bool tall = rows > cols;
  const int m = tall ? cols : rows, whole = tall ? rows : cols, slice = small_slice(whole, CTAS), first = rank * slice;
  const int n = whole - first < slice ? (whole > first ? whole - first : 0) : slice;   // of this CTA
  const int m4 = (m + 3) / 4, n4 = slice / 4, ldx = small_ld(slice), ldg = small_ld(m), gs = 4 * m4 * ldg;
  float *x = small_smem, *y = x + 4 * m4 * ldx, *part = y + 4 * m4 * ldx, *g = part + 2 * gs, *q = g + gs;
  for (int i = tid; i < m4 * ldx; i += kSmallNsThreads) reinterpret_cast<float4*>(x)[i] = make_float4(0, 0, 0, 0);
  list_tiles(list, m4);
  __syncthreads();
  const int r0 = tall ? first : 0, k0 = tall ? 0 : first;               // this CTA's rows and columns ...
  const int lines = tall ? n : m, wide = tall ? m : n, per = (wide + 7) / 8;   // ... and how many
  uint32_t most = 0;
  for (int t = tid; allowed && t < lines * per; t += kSmallNsThreads) {
    const int i = t / per, j = (t - i * per) * 8, valid = wide - j < 8 ? wide - j : 8;
    float f[8];
    typename Src::Ahead o;
    src.ahead(batch, r0 + i, k0 + j, valid, true, o);
    src.first(batch, r0 + i, k0 + j, valid, o, f);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < valid) {
        x[tall ? (j + k) * ldx + i : i * ldx + j + k] = f[k];
        most = max(most, magnitude(f[k]));
      }
  }
  const Unit unit = block_unit(most);
  const float inv = unit.inverse();
  float sq = 0.0f;
  for (int i = tid; i < 4 * m4 * ldx; i += kSmallNsThreads) {   // what pads the rows is 0
    const float v = x[i] * inv;
    sq = fmaf(v, v, sq);
  }
  sq = block_sum(sq);
  if (tid == 0) squares = unit.squared(sq);
  cluster_sync_all();
  if (tid == 0) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CTAS; ++c) s += peer_double(peer_addr(&squares, c));
    go = 1;
    if (Src::kGuarded) {
#pragma unroll
      for (int c = 0; c < CTAS; ++c) go &= peer_u32(peer_addr(&ready, c));
    }
    const double norm = sqrt(s);
    scale_of = inverse_norm(norm, eps);
    if (!isfinite(norm) && rank == 0) src.not_finite();
  }
  __syncthreads();
  if (!go) steps = 0;
  const TwoFactors scale = scale_of;
  for (int i = tid; i < 4 * m4 * ldx; i += kSmallNsThreads) x[i] = scale.of(x[i]);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    float* mine = part + (s & 1) * gs;
    symmetric_tiles(list, x, ldx, slice, mine, nullptr, ldg, m4, 0.0f, 0.0f);
    cluster_sync_all();
    for (int i = tid; i < m4 * ldg; i += kSmallNsThreads) {
      float4 p[CTAS];
#pragma unroll
      for (int c = 0; c < CTAS; ++c) p[c] = peer_float4(peer_addr(mine + 4 * i, c));
#pragma unroll
      for (int c = 1; c < CTAS; ++c) {
        p[0].x += p[c].x;
        p[0].y += p[c].y;
        p[0].z += p[c].z;
        p[0].w += p[c].w;
      }
      *reinterpret_cast<float4*>(g + 4 * i) = p[0];
    }
    __syncthreads();
    symmetric_tiles(list, g, ldg, 4 * m4, q, g, ldg, m4, b1, c1);
    __syncthreads();
    apply_tiles(a1, q, ldg, x, y, ldx, m4, n4);
    __syncthreads();
    float* t = x;
    x = y;
    y = t;
  }
  for (int t = tid; go && t < lines * per; t += kSmallNsThreads) {
    const int i = t / per, j = (t - i * per) * 8, valid = wide - j < 8 ? wide - j : 8;
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < valid ? x[tall ? (j + k) * ldx + i : i * ldx + j + k] : 0.0f;
    last.finish(batch, r0 + i, k0 + j, f, valid);
  }
  cluster_sync_all();   // a CTA's parts are read until its peers are here
}

// ---- thin matrices: up to 64 rows (or columns), too long for one CTA's shared memory ----
// In fp32 too: a step needs m^2 n multiply-adds for G and as many for Q X, few enough beside X's
// own bytes, and with few rows the roundings of G and Q to fp16 would not average out (3.3e-3
// of the result for 2 x 20000).  X lies as [m][np] fp32; a CTA takes runs of kThinCols columns,
// applies Q to them and sums what they add to the next G; k_ns_thin_join adds the CTAs' sums in order.
constexpr int kThinRows = 64, kThinCols = 128, kThinLd = kThinCols + 4, kThinLdg = kThinRows + 4;
constexpr int kThinCtas = 128;   // runs of columns, at most, of one matrix
constexpr int kThinSmem = 4 * (2 * kThinRows * kThinLd + 2 * kThinRows * kThinLdg);

struct ThinArgs {
  float* x;                 // [batch][m][np]
  const float* g;           // [batch][m4 * 4][kThinLdg]
  float* sums;              // [batch][ctas][m4 * 4][kThinLdg]
  const double* norms;
  int64_t np;
  int32_t rows, cols, run, last;   // run: columns of a CTA
  float a, b, c, eps;
};

// FIRST: from the source, X = x / max(|x|, eps).  Otherwise X <- a X + Q X, to `finish` after the last.
template <class Src, bool FIRST>
__global__ void __launch_bounds__(kSmallNsThreads)
k_ns_thin(const __grid_constant__ Src src, const ThinArgs t, const __grid_constant__ Finish finish) {
  extern __shared__ __align__(16) float small_smem[];
  wait_for_predecessor();
  if (!src.ready()) return;
  const int batch = blockIdx.y, tid = threadIdx.x;
  const bool tall = t.rows > t.cols;
  const int m = tall ? t.cols : t.rows, n = tall ? t.rows : t.cols, m4 = (m + 3) / 4;
  float *x = small_smem, *y = x + kThinRows * kThinLd, *g = y + kThinRows * kThinLd, *q = g + kThinRows * kThinLdg;
  TwoFactors scale{1.0f, 1.0f};
  __shared__ uint16_t list[kLowerTiles];
  if (FIRST) {
    __shared__ TwoFactors scale_of;
    if (tid == 0) scale_of = inverse_norm(t.norms[batch], t.eps);
    __syncthreads();
    scale = scale_of;
  } else {
    list_tiles(list, m4);
    for (int i = tid; i < 4 * m4 * kThinLdg; i += kSmallNsThreads) g[i] = t.g[batch * int64_t{kThinRows * kThinLdg} + i];
    __syncthreads();
    symmetric_tiles(list, g, kThinLdg, 4 * m4, q, g, kThinLdg, m4, t.b, t.c);
  }
  const int ti = tid / 32, tj = tid / 2 % 16, sub = tid % 2;   // this thread's half of a tile of G
  float acc[4][4] = {};
  const int64_t c0 = int64_t{blockIdx.x} * t.run, c1 = c0 + t.run < n ? c0 + t.run : n;
  float* xg = t.x + batch * int64_t{m} * t.np;
  for (int64_t c = c0; c < c1; c += kThinCols) {
    const int w = static_cast<int>(c1 - c < kThinCols ? c1 - c : kThinCols);
    __syncthreads();   // the previous run of columns is done with
    if (FIRST) {
      for (int i = tid; i < 4 * m4 * kThinLd; i += kSmallNsThreads) x[i] = 0.0f;
      __syncthreads();
      const int per = tall ? (m + 7) / 8 : (w + 7) / 8, lines = tall ? w : m;
      for (int k = tid; k < lines * per; k += kSmallNsThreads) {
        const int i = k / per, j = (k - i * per) * 8, left = (tall ? m : w) - j, valid = left < 8 ? left : 8;
        float f[8];
        typename Src::Ahead o;
        const int64_t row = tall ? c + i : i, col = tall ? j : c + j;
        src.ahead(batch, row, col, valid, false, o);
        src.again(batch, row, col, valid, o, f);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (u < valid) x[tall ? (j + u) * kThinLd + i : i * kThinLd + j + u] = scale.of(f[u]);
      }
      __syncthreads();
    } else {
      for (int k = tid; k < 4 * m4 * kThinCols; k += kSmallNsThreads) {
        const int i = k / kThinCols, j = k % kThinCols;
        y[i * kThinLd + j] = i < m && j < w ? xg[i * t.np + c + j] : 0.0f;
      }
      __syncthreads();
      apply_tiles(t.a, q, kThinLdg, y, x, kThinLd, m4, kThinCols / 4);
      __syncthreads();
    }
    if (!FIRST && t.last) {
      const int per = tall ? (m + 7) / 8 : (w + 7) / 8, lines = tall ? w : m;
      for (int k = tid; k < lines * per; k += kSmallNsThreads) {
        const int i = k / per, j = (k - i * per) * 8, left = (tall ? m : w) - j, valid = left < 8 ? left : 8;
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] = u < valid ? x[tall ? (j + u) * kThinLd + i : i * kThinLd + j + u] : 0.0f;
        if (tall)
          finish.finish(batch, static_cast<int>(c + i), j, f, valid);
        else
          finish.finish(batch, i, static_cast<int>(c + j), f, valid);
      }
      continue;
    }
    for (int k = tid; k < m * w; k += kSmallNsThreads) {
      const int i = k / w, j = k - i * w;
      xg[i * t.np + c + j] = x[i * kThinLd + j];
    }
    if (ti < m4 && tj < m4) rows_by_rows(x + 4 * ti * kThinLd, kThinLd, x + 4 * tj * kThinLd, kThinLd, 4 * sub, kThinCols, 2, acc);
  }
  if (!FIRST && t.last) return;
  add_shares<2>(acc);
  if (ti >= m4 || tj >= m4) return;
  float* out = t.sums + (int64_t{batch} * gridDim.x + blockIdx.x) * (kThinRows * kThinLdg);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u % 2 == sub) *reinterpret_cast<float4*>(out + (4 * ti + u) * kThinLdg + 4 * tj) = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
}

__global__ void __launch_bounds__(128) k_ns_thin_join(const float* sums, int ctas, float* g) {
  wait_for_predecessor();
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= kThinRows * kThinLdg) return;
  const float* p = sums + int64_t{blockIdx.y} * ctas * (kThinRows * kThinLdg) + i;
  float s = 0.0f;
  for (int k = 0; k < ctas; ++k) s += p[int64_t{k} * (kThinRows * kThinLdg)];
  g[int64_t{blockIdx.y} * (kThinRows * kThinLdg) + i] = s;
}

// ---- how a batch is laid out ----
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

struct Layout {
  int64_t rows, cols, m, n;
  int batch;
  int64_t xp, gp;                      // pitches
  int64_t hi[2], lo, g, q, parts, partial, bytes;
  int64_t n_parts, run;
  int ctas;                            // of a thin matrix, each with `run` columns
  ProductCut gram, poly, apply;
};

int64_t lower_tiles(int64_t mt, int bn) { return mt * (mt + 1) / 2 * (kTileM / bn); }

Layout layout(int64_t rows, int64_t cols, int batch) {
  Layout l{};
  l.rows = rows;
  l.cols = cols;
  l.batch = batch;
  if (fits_small(rows, cols)) return l;
  l.m = rows < cols ? rows : cols;
  l.n = rows < cols ? cols : rows;
  const auto take = [&](int64_t bytes) {
    const int64_t here = l.bytes;
    l.bytes += up(bytes, 256);
    return here;
  };
  l.n_parts = cut(rows * cut(cols, 8), kStageThreads * kStageOcts);
  l.parts = take(8 * batch * (l.n_parts + 1));   // and the norms
  if (l.m <= kThinRows) {
    // whole runs of kThinCols columns for each CTA, enough CTAs to fill the GPU
    const int64_t runs = cut(l.n, kThinCols);
    const int64_t most = cut(4 * kThinCtas, batch);
    l.run = cut(runs, most < kThinCtas ? most : kThinCtas) * kThinCols;
    l.ctas = static_cast<int>(cut(l.n, l.run));
    l.xp = up(l.n, 32);
    l.hi[0] = take(4 * batch * l.m * l.xp);
    l.g = take(4 * int64_t{batch} * kThinRows * kThinLdg);
    l.partial = take(4 * int64_t{batch} * l.ctas * kThinRows * kThinLdg);
    return l;
  }
  l.xp = up(cols, 32);
  l.gp = up(l.m, 32);
  const int64_t mt = cut(l.m, kTileM);
  const double mm = static_cast<double>(l.m) * static_cast<double>(l.m) * batch;
  const auto lower = [&](int bn) { return lower_tiles(mt, bn) * batch; };
  l.gram = cut_product_of(lower, l.n, mm, 256, 128, least_parts(l.n, false));
  // Q's and X's K is the smaller side m, in parts it pays at no size: fewer tiles than pairs mean m up to
  // 2816, whose m / 64 blocks at 512 cycles are worth less than joining m^2 values and a launch (by the
  // costs above: m = 512 4096 cycles against 5000, m = 2816 22528 against 77000)
  l.poly = cut_product_of(lower, l.m, mm, 256, 128, 1, true);
  l.apply = cut_product_of([&](int bn) { return cut(rows, kTileM) * cut(cols, bn) * batch; }, l.m,
                           static_cast<double>(rows) * static_cast<double>(cols) * batch, 256, 128, 1, true);
  for (int i = 0; i < 2; ++i) l.hi[i] = take(2 * batch * rows * l.xp);
  l.lo = take(batch * rows * l.xp);
  l.g = take(2 * batch * l.m * l.gp);
  l.q = take(2 * batch * l.m * l.gp);
  l.partial = take(l.gram.splits > 1 ? 4 * l.gram.splits * batch * l.m * l.m : 0);
  return l;
}

// The matrices that go through the steps together: enough to fill the GPU, in bounded memory.
constexpr int64_t kBatchBytes = int64_t{1} << 30;
int batch_of(int64_t rows, int64_t cols, int64_t count) {
  const int64_t most = kBatchBytes / (5 * rows * cols + 1);
  const int64_t n = most < 1 ? 1 : most;
  return static_cast<int>(count < n ? (count < kMaxBatch ? count : kMaxBatch) : (n < kMaxBatch ? n : kMaxBatch));
}

template <bool AMN, bool BMN, bool SYM, class Epi>
int run_product(const ProductCut& c, const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, int batch,
                float* partial, const Epi& epi, void* stream) {
  return c.bn == 256 ? launch_product<256, AMN, BMN, SYM>(a, b, M, N, K, batch, false, c.splits, partial, epi, stream)
                   : launch_product<128, AMN, BMN, SYM>(a, b, M, N, K, batch, false, c.splits, partial, epi, stream);
}

int64_t short_side(int64_t rows, int64_t cols) { return rows < cols ? rows : cols; }
int64_t long_side(int64_t rows, int64_t cols) { return rows < cols ? cols : rows; }

// floats: of shared memory, the most that any of the launch's matrices takes in `ctas` parts.
template <class Src>
int iterate_small(const Src& src, int batch, int ctas, int64_t floats, const NewtonSchulz& ns, const Finish& last,
                  void* stream) {
  const auto kernel = ctas == 8 ? k_ns_small<Src, 8> : k_ns_small<Src, 4>;
  const cudaError_t ce = ensure_dyn_smem(kernel, 4 * kSmallFloats);
  if (ce != cudaSuccess) return static_cast<int>(ce);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(batch * ctas));
  cfg.blockDim = dim3(kSmallNsThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(4 * floats);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, src, ns.a, ns.b, ns.c, ns.eps, ns.steps, last);
  const cudaError_t after = cudaGetLastError();
  return static_cast<int>(e != cudaSuccess ? e : after);
}

// The two passes before the first step: the norms, and S X.
template <class Src>
int squares(const Layout& l, const Src& src, dim3 grid, const Div8& per, double* parts, double* norms, void* stream) {
  const int e = launch_g(k_ns_squares<Src>, grid, kStageThreads, 0, stream, src, l.rows, l.cols, per, parts);
  if (e) return e;
  return launch_g(k_ns_norm<Src>, dim3(static_cast<unsigned>(l.batch)), kNormThreads, 0, stream, src,
                  static_cast<const double*>(parts), static_cast<int>(l.n_parts), norms);
}

// Matrices of one shape on their way through the steps.
struct Run {
  Layout l;
  HalfMat hi, next;           // X, and where the next one goes
  uint8_t* lo;
  Operand og, oq;             // G and Q
  GramEpi gram;
  PolyEpi poly;
  Finish last;
  float S, a;

  Run(const Layout& layout, const NewtonSchulz& ns, const Finish& finish, uint8_t* ws) : l(layout), last(finish), a(ns.a) {
    const auto half = [&](int64_t at) { return reinterpret_cast<__half*>(ws + at); };
    hi = next = {half(l.hi[0]), l.rows * l.xp, static_cast<int32_t>(l.xp)};
    next.p = half(l.hi[1]);
    lo = ws + l.lo;
    const HalfMat g{half(l.g), l.m * l.gp, static_cast<int32_t>(l.gp)};
    HalfMat q = g;
    q.p = half(l.q);
    og = {g.p, l.m, l.m, l.gp, g.step};
    oq = {q.p, l.m, l.m, l.gp, q.step};
    // S: the power of two next to sqrt(m n), at most 2^15
    S = 1.0f;
    while (S < 32768.0f && 2.0 * S * S < static_cast<double>(l.m) * static_cast<double>(l.n)) S *= 2.0f;
    gram.plan = poly.plan = finish.mu.plan;
    gram.out = g;
    gram.alpha = 1.0f / (S * S);
    poly.out = q;
    poly.g = g;
    poly.b1 = ns.b;
    poly.c1 = ns.c;
  }
  Operand x() const { return {hi.p, l.cols, l.rows, l.xp, hi.step}; }
  // The step's last product; X and the next one change places.
  ApplyEpi next_apply(bool final_step) {
    ApplyEpi e{};
    static_cast<Finish&>(e) = last;
    if (!final_step) e.mode = kIterate;
    e.hi = hi.p;
    e.lo = lo;
    e.hi_out = next;
    e.a = a;
    e.inv = 1.0f / S;
    std::swap(hi.p, next.p);
    return e;
  }
};
template <class Src>
int stage(const Run& r, const Src& src, dim3 grid, const Div8& per, const double* norms, const NewtonSchulz& ns, void* stream) {
  return launch_g(k_ns_stage<Src>, grid, kStageThreads, 0, stream, src, r.l.rows, r.l.cols, per, norms, r.S, ns.eps, r.hi, r.lo);
}

template <class Src>
int iterate(const Layout& l, const Src& src, const NewtonSchulz& ns, const Finish& last, uint8_t* ws, void* stream) {
  if (fits_small(l.rows, l.cols)) {
    const int64_t m = short_side(l.rows, l.cols), n = long_side(l.rows, l.cols);
    return iterate_small(src, l.batch, small_ctas(n), small_floats(m, n, small_ctas(n)), ns, last, stream);
  }
  double* parts = reinterpret_cast<double*>(ws + l.parts);
  float* partial = reinterpret_cast<float*>(ws + l.partial);
  double* norms = parts + l.batch * l.n_parts;
  const Div8 per(cut(l.cols, 8));
  const dim3 grid(static_cast<unsigned>(l.n_parts), static_cast<unsigned>(l.batch));
  int e = squares(l, src, grid, per, parts, norms, stream);
  if (l.m <= kThinRows) {
    ThinArgs t{reinterpret_cast<float*>(ws + l.hi[0]), reinterpret_cast<float*>(ws + l.g), partial, norms, l.xp,
               static_cast<int32_t>(l.rows), static_cast<int32_t>(l.cols), static_cast<int32_t>(l.run), 0,
               ns.a, ns.b, ns.c, ns.eps};
    const dim3 ctas(static_cast<unsigned>(l.ctas), static_cast<unsigned>(l.batch));
    for (const auto kernel : {k_ns_thin<Src, true>, k_ns_thin<Src, false>}) {
      const cudaError_t ce = ensure_dyn_smem(kernel, kThinSmem);
      if (ce != cudaSuccess) return static_cast<int>(ce);
    }
    if (!e) e = launch_g(k_ns_thin<Src, true>, ctas, kSmallNsThreads, kThinSmem, stream, src, t, last);
    for (int k = 0; k < ns.steps && !e; ++k) {
      t.last = k + 1 == ns.steps;
      e = launch_g(k_ns_thin_join, dim3(cut(kThinRows * kThinLdg, 128), static_cast<unsigned>(l.batch)), 128, 0, stream,
                   static_cast<const float*>(partial), l.ctas, reinterpret_cast<float*>(ws + l.g));
      if (!e) e = launch_g(k_ns_thin<Src, false>, ctas, kSmallNsThreads, kThinSmem, stream, src, t, last);
    }
    return e;
  }
  if (e) return e;
  Run r(l, ns, last, ws);
  e = stage(r, src, grid, per, norms, ns, stream);
  for (int k = 0; k < ns.steps && !e; ++k) {
    const Operand x = r.x();
    const bool tall = l.rows > l.cols;
    e = tall ? run_product<true, true, true>(l.gram, x, x, l.m, l.m, l.n, l.batch, partial, r.gram, stream)
             : run_product<false, false, true>(l.gram, x, x, l.m, l.m, l.n, l.batch, partial, r.gram, stream);
    if (!e) e = run_product<false, false, true>(l.poly, r.og, r.og, l.m, l.m, l.m, l.batch, partial, r.poly, stream);
    const ApplyEpi apply = r.next_apply(k + 1 == ns.steps);
    if (!e)
      e = tall ? run_product<false, false, false>(l.apply, x, r.oq, l.rows, l.cols, l.m, l.batch, partial, apply, stream)
               : run_product<false, true, false>(l.apply, r.oq, x, l.rows, l.cols, l.m, l.batch, partial, apply, stream);
  }
  return e;
}

// Matrices of several shapes together: each step's products of all of them in one launch each, so that
// the last round of one shape's tiles and its epilogue run beside another's.
constexpr int kTogether = 8;
struct Piece {
  Layout l;
  MuonSource src;
  Finish last;
  int64_t at;                 // in the workspace
};
int iterate_together(Piece* pieces, int n, const NewtonSchulz& ns, uint8_t* ws, void* stream) {
  // the longest sums first: the short ones fill the end
  std::stable_sort(pieces, pieces + n, [](const Piece& a, const Piece& b) { return a.l.n > b.l.n; });
  std::vector<Run> runs;
  int e = 0;
  for (int i = 0; i < n && !e; ++i) {
    const Piece& p = pieces[i];
    const Layout& l = p.l;
    runs.emplace_back(l, ns, p.last, ws + p.at);
    double* parts = reinterpret_cast<double*>(ws + p.at + l.parts);
    double* norms = parts + l.batch * l.n_parts;
    const Div8 per(cut(l.cols, 8));
    const dim3 grid(static_cast<unsigned>(l.n_parts), static_cast<unsigned>(l.batch));
    e = squares(l, p.src, grid, per, parts, norms, stream);
    if (!e) e = stage(runs.back(), p.src, grid, per, norms, ns, stream);
  }
  auto grams = std::make_unique<Problems<GramEpi, kTogether>>();
  auto polys = std::make_unique<Problems<PolyEpi, kTogether>>();
  auto applies = std::make_unique<Problems<ApplyEpi, kTogether>>();
  grams->n = polys->n = applies->n = n;
  for (int k = 0; k < ns.steps && !e; ++k) {
    for (int i = 0; i < n && !e; ++i) {
      Run& r = runs[static_cast<size_t>(i)];
      const Layout& l = r.l;
      const Operand x = r.x();
      const bool tall = l.rows > l.cols;
      e = fill_problem<256, true>(grams->p + i, x, tall, x, tall, l.m, l.m, l.n, l.batch, false, 1, nullptr, r.gram, false);
      if (!e)
        e = fill_problem<256, true>(polys->p + i, r.og, false, r.og, false, l.m, l.m, l.m, l.batch, false, 1, nullptr, r.poly,
                                    false);
      const ApplyEpi apply = r.next_apply(k + 1 == ns.steps);
      if (!e)
        e = fill_problem<256, false>(applies->p + i, tall ? x : r.oq, false, tall ? r.oq : x, !tall, l.rows, l.cols, l.m,
                                     l.batch, false, 1, nullptr, apply, false);
    }
    if (!e) e = launch_problems<256, kAsked, kAsked, true>(*grams, stream);
    if (!e) e = launch_problems<256, 0, 0, true>(*polys, stream);
    if (!e) e = launch_problems<256, 0, kAsked, false>(*applies, stream);
  }
  return e;
}

Mat ranks_from(const Mat& m, int r) {
  Mat s = m;
  s.p += r * m.rs * esize(m.dtype);
  return s;
}

}  // namespace

int64_t orthogonalize_workspace_bytes(int P, int64_t rows, int64_t cols) {
  const int n = batch_of(rows, cols, P);
  int64_t most = layout(rows, cols, n).bytes;
  if (P % n) {   // a smaller last batch may be cut into more parts
    const int64_t rest = layout(rows, cols, P % n).bytes;
    most = rest > most ? rest : most;
  }
  return most;
}

int launch_orthogonalize(const Mat& x, const Mat& out, int P, int64_t rows, int64_t cols, const NewtonSchulz& ns,
                         uint8_t* ws, void* stream) {
  const int n = batch_of(rows, cols, P);
  for (int r = 0; r < P; r += n) {
    const int batch = P - r < n ? P - r : n;
    const Layout l = layout(rows, cols, batch);
    Finish last{};
    last.mode = kMatrix;
    last.out = ranks_from(out, r);
    last.vec = oct_rows(out);
    const Mat from = ranks_from(x, r);
    const int vec = oct_rows(x), r32 = static_cast<int>(rows), c32 = static_cast<int>(cols);
    const int e = x.dtype == DP_BF16 ? iterate(l, MatSource<__nv_bfloat16>{from, vec, r32, c32}, ns, last, ws, stream)
                                     : iterate(l, MatSource<float>{from, vec, r32, c32}, ns, last, ws, stream);
    if (e) return e;
  }
  return cudaSuccess;
}

// The rounds of a Muon step beside its small matrices: pieces of one shape each that go through the steps
// together, in bounded memory; thin matrices have kernels and a round of their own, and so have those
// so long that G's sums are formed in parts.
namespace {
constexpr int64_t kRoundBytes = int64_t{4} << 30;
struct Part {
  const MuonGroup* group;
  int from;
  Layout l;
  int64_t at;
};
std::vector<std::vector<Part>> muon_rounds(const Muon& m) {
  std::vector<std::vector<Part>> rounds;
  int64_t bytes = 0;
  bool open = false;
  for (const MuonGroup& g : m.groups) {
    if (fits_small(g.rows, g.cols)) continue;
    const int count = static_cast<int>(g.off.size()), n = batch_of(g.rows, g.cols, count);
    const bool alone = short_side(g.rows, g.cols) <= kThinRows || least_parts(long_side(g.rows, g.cols), false) > 1;
    for (int k = 0; k < count; k += n) {
      const Layout l = layout(g.rows, g.cols, count - k < n ? count - k : n);
      if (!open || alone || rounds.back().size() == kTogether || bytes + l.bytes > kRoundBytes) {
        rounds.emplace_back();
        bytes = 0;
      }
      rounds.back().push_back({&g, k, l, bytes});
      bytes += l.bytes;
      open = !alone;
    }
  }
  return rounds;
}
}  // namespace

int64_t muon_workspace_bytes(const Muon& m) {
  int64_t most = 0;
  for (const auto& round : muon_rounds(m)) most = std::max(most, round.back().at + round.back().l.bytes);
  return most;
}

int launch_muon(const Muon& m, const MuonArgs& a, uint8_t* ws, void* stream) {
  MuonSource src{};
  src.mean = a.mean;
  src.momentum = a.momentum;
  src.coef = a.coef;
  src.plan = {static_cast<DevHeader*>(a.hdr), m.plan_id};
  src.mu = a.mu;
  src.rest = a.rest;
  src.nesterov = a.nesterov;
  Finish last{};
  last.mode = kMuon;
  last.mu.master = a.master;
  last.mu.params = reinterpret_cast<__nv_bfloat16*>(a.params);
  last.mu.stride = m.stride;
  last.mu.plan = src.plan;
  last.mu.lr_dev = a.lr_dev;
  last.mu.lr = a.lr;
  last.mu.decay = a.weight_decay;
  last.mu.P = m.P;
  int filled = 0;
  const auto add = [&](const MuonGroup& g, int64_t off) {
    const double big = static_cast<double>(g.rows > g.cols ? g.rows : g.cols);
    const double aspect = static_cast<double>(g.rows) / static_cast<double>(g.cols);
    src.of.off[filled] = off;
    src.of.rows[filled] = static_cast<int32_t>(g.rows);
    src.of.cols[filled] = static_cast<int32_t>(g.cols);
    src.of.scale[filled++] = static_cast<float>(a.match_rms ? 0.2 * std::sqrt(big) : std::sqrt(aspect > 1.0 ? aspect : 1.0));
  };
  // small matrices of all shapes together, in as many parts as the longest takes
  int ctas = 0;
  for (const MuonGroup& g : m.groups)
    if (fits_small(g.rows, g.cols)) ctas = std::max(ctas, small_ctas(long_side(g.rows, g.cols)));
  int64_t floats = 0;
  const auto small = [&]() {
    if (filled == 0) return 0;
    last.mu.of = src.of;
    const int e = iterate_small(src, filled, ctas, floats, a.ns, last, stream);
    filled = 0;
    floats = 0;
    return e;
  };
  for (const MuonGroup& g : m.groups) {
    if (!fits_small(g.rows, g.cols)) continue;
    for (const int64_t off : g.off) {
      add(g, off);
      floats = std::max(floats, small_floats(short_side(g.rows, g.cols), long_side(g.rows, g.cols), ctas));
      if (filled == kMaxBatch) {
        const int e = small();
        if (e) return e;
      }
    }
  }
  if (const int e = small()) return e;
  for (const auto& round : muon_rounds(m)) {
    std::vector<Piece> pieces;
    for (const Part& part : round) {
      filled = 0;
      for (int i = 0; i < part.l.batch; ++i) add(*part.group, part.group->off[static_cast<size_t>(part.from + i)]);
      last.mu.of = src.of;
      pieces.push_back({part.l, src, last, part.at});
    }
    const int e = pieces.size() == 1
                      ? iterate(pieces[0].l, src, a.ns, last, ws, stream)
                      : iterate_together(pieces.data(), static_cast<int>(pieces.size()), a.ns, ws, stream);
    if (e) return e;
  }
  return cudaSuccess;
}

int64_t product_timeouts_orthogonal(bool reset) {
  unsigned long long n = 0, z = 0;
  if (cudaMemcpyFromSymbol(&n, g_product_timeouts, sizeof n) != cudaSuccess) return -2;
  if (reset && cudaMemcpyToSymbol(g_product_timeouts, &z, sizeof z) != cudaSuccess) return -2;
  return static_cast<int64_t>(n);
}

}  // namespace dps
