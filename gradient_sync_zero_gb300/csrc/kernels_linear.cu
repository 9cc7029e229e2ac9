// The linear layer over P ranks: y = residual + act(x w^T + bias), and its gradients
//   dz = dy * act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum over rows of dz.
//
// All three products run on k_product (product.cuh); which operand is K-major follows from how
// the matrices lie: x and w are both K-major forward, w is MN-major in dx, dz and x both are in dw.
//
// On GB300, in bursts: 8 x 1024 tokens 2560 -> 10240 with bias, GELU and z 252 to 271 us (1590 to 1700
// TFLOP/s; cuBLAS's plain product 223); gradients of 8 x 2048 tokens 2048 -> 5632 with SiLU 535 us, of which
// dz 90 (554 MB) and each product 222 (1700 TFLOP/s).
#include "layer.h"
#include "product.cuh"

namespace dps {
namespace {

// ---- activations ----
// By erfc and the logistic function, whose small values keep their relative accuracy.  The logistic
// function is two approximate instructions (2^-22 each) beside a multiply and an add: with expf and an
// IEEE division the epilogue of 8 x 1024 x 2560 -> 10240 took longer than its products.
__device__ __forceinline__ float logistic(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
__device__ __forceinline__ float tanh_arg(float z) { return 1.5957691f * fmaf(0.044715f * z * z, z, z); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  switch (ACT) {
    case DP_ACT_RELU: return z > 0.0f ? z : z == z ? 0.0f : z;
    case DP_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678f);
    case DP_ACT_GELU_TANH: return z * logistic(tanh_arg(z));   // (1 + tanh u) / 2 is logistic(2 u)
    case DP_ACT_SILU: return z * logistic(z);
    default: return z;
  }
}

// Slopes are 0 or 1 in fp32 far from 0: z is held there, so that no product of its powers overflows.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  z = z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z;   // NaN stays
  switch (ACT) {
    case DP_ACT_RELU: return z > 0.0f ? 1.0f : z == z ? 0.0f : z;
    case DP_ACT_GELU: return 0.5f * erfcf(z * -0.70710678f) + z * 0.39894228f * __expf(-0.5f * z * z);
    case DP_ACT_GELU_TANH: {
      const float q = logistic(tanh_arg(z));
      return fmaf(z * q * (1.0f - q), 1.5957691f * fmaf(0.134145f * z, z, 1.0f), q);
    }
    case DP_ACT_SILU: {
      const float q = logistic(z);
      return q * fmaf(z, 1.0f - q, 1.0f);
    }
    default: return 1.0f;
  }
}

// Calls f with the activation as a constant.
template <class F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case DP_ACT_RELU: return f(std::integral_constant<int, DP_ACT_RELU>{});
    case DP_ACT_GELU: return f(std::integral_constant<int, DP_ACT_GELU>{});
    case DP_ACT_GELU_TANH: return f(std::integral_constant<int, DP_ACT_GELU_TANH>{});
    case DP_ACT_SILU: return f(std::integral_constant<int, DP_ACT_SILU>{});
    default: return f(std::integral_constant<int, DP_ACT_NONE>{});
  }
}

// ---- rows of a Mat ----
// Eight consecutive values of which `valid` exist, one by one.
template <class T>
__device__ __forceinline__ void load_ones(const T* p, int valid, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j < valid ? ld_elem(p + j) : 0.0f;
}

// Eight values from column j of row i, on a 16-byte boundary.
__device__ __forceinline__ void store_row(const Mat& m, int r, int64_t i, int64_t j, const float (&f)[8]) {
  if (m.dtype == DP_BF16) {
    *reinterpret_cast<uint4*>(row_ptr<__nv_bfloat16>(m, r, i) + j) =
        make_uint4(pack2_rne(f[0], f[1]), pack2_rne(f[2], f[3]), pack2_rne(f[4], f[5]), pack2_rne(f[6], f[7]));
  } else {
    float* p = row_ptr<float>(m, r, i) + j;
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

__device__ __forceinline__ float load_one(const Mat& m, int r, int64_t i, int64_t j) {
  return m.dtype == DP_BF16 ? ld_elem(row_ptr<const __nv_bfloat16>(m, r, i) + j) : row_ptr<const float>(m, r, i)[j];
}
__device__ __forceinline__ void store_one(const Mat& m, int r, int64_t i, int64_t j, float v) {
  if (m.dtype == DP_BF16)
    st_elem(row_ptr<__nv_bfloat16>(m, r, i) + j, v);
  else
    row_ptr<float>(m, r, i)[j] = v;
}

__device__ __forceinline__ void add_oct(float* v, const uint4& q) {
  Oct<__nv_bfloat16> o;
  o.q = q;
  float f[8];
  o.get(f);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] += f[k];
}

__device__ __forceinline__ void add_eight(float* v, const float* p) {
  Oct<float> o;
  o.load_again(p);
  float f[8];
  o.get(f);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] += f[k];
}

// out = residual + act(v + bias), z = v + bias.
struct LinearOut {
  Mat bias, z, residual, out;
  int32_t act, vec;
};

// SWAP: the product's rows are the output's columns.
template <bool SWAP>
struct LinearEpi : LinearOut {
  static constexpr bool kSwap = SWAP, kMirror = false, kBefore = false, kJoins = true, kAsks = false;
  using Straight = LinearEpi<false>;
  LinearEpi() = default;
  LinearEpi(const LinearOut& o) : LinearOut(o) {}
  // A bf16 residual and bias (fp32 ones, twice the registers, are loaded where they are used).
  struct Pre {
    uint4 residual;
  };
  struct Cols {
    uint4 bias;
  };
  __device__ __forceinline__ void fetch_cols(int b, int n, Cols& cols) const {
    if (bias.p && bias.dtype == DP_BF16) cols.bias = ld_again(row_ptr<const __nv_bfloat16>(bias, b, 0) + n);
  }
  __device__ __forceinline__ bool whole(int valid) const { return vec && valid == 32; }
  __device__ __forceinline__ bool ahead(int valid) const { return !SWAP && whole(valid); }
  __device__ __forceinline__ void fetch(int b, int m, int n, Pre& pre) const {
    if (residual.p && residual.dtype == DP_BF16) pre.residual = ld_again(row_ptr<const __nv_bfloat16>(residual, b, m) + n);
  }
  __device__ __forceinline__ void before(float (&)[8], const Pre&) const {}
  __device__ __forceinline__ void mirror(int, int, int, const float (&)[8]) const {}
  __device__ __forceinline__ void gave_up() const {}

  __device__ __forceinline__ void apply(int b, int m, int n, float (&v)[8], const Pre& pre, const Cols& cols) const {
    if (bias.p) {
      if (bias.dtype == DP_BF16)
        add_oct(v, cols.bias);
      else
        add_eight(v, row_ptr<const float>(bias, b, 0) + n);
    }
    if (z.p) store_row(z, b, m, n, v);
    with_act(act, [&](auto a) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_value<decltype(a)::value>(v[j]);
    });
    if (residual.p) {
      if (residual.dtype == DP_BF16)
        add_oct(v, pre.residual);
      else
        add_eight(v, row_ptr<const float>(residual, b, m) + n);
    }
    store_row(out, b, m, n, v);
  }

  // Eight rows' loads, then their stores.
  __device__ __forceinline__ void apply_rows(int b, int m0, int rows, int n, const float* block, int lane) const {
    const float add = bias.p ? load_one(bias, b, 0, n) : 0.0f;
#pragma unroll 1
    for (int r = 0; r < rows; r += 8) {
      float v[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        q[i] = residual.p && r + i < rows ? load_one(residual, b, m0 + r + i, n) : 0.0f;
        v[i] = block_at(block, r + i, lane) + add;
      }
      if (z.p) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r + i < rows) store_one(z, b, m0 + r + i, n, v[i]);
      }
      with_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value<decltype(a)::value>(v[i]);
      });
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i < rows) store_one(out, b, m0 + r + i, n, v[i] + q[i]);
    }
  }

  // SWAP: rows n0 .. of the output's column m; lanes hold consecutive columns.
  __device__ __forceinline__ void apply_cols(int b, int m, int n0, int valid, const float* block, int lane) const {
    const float add = bias.p ? load_one(bias, b, 0, m) : 0.0f;
#pragma unroll 4
    for (int j = 0; j < valid; ++j) one(b, n0 + j, m, block_at(block, lane, j) + add);
  }
  // z and out at one place.
  __device__ __forceinline__ void one(int b, int64_t row, int64_t col, float s) const {
    if (z.p) store_one(z, b, row, col, s);
    const float q = residual.p ? load_one(residual, b, row, col) : 0.0f;
    with_act(act, [&](auto a) { s = act_value<decltype(a)::value>(s); });
    store_one(out, b, row, col, s + q);
  }

  __device__ __forceinline__ void join(int b, int m, int n, float (&v)[8], int valid) const {
    if (vec && valid == 8) {
      Pre pre;
      Cols cols;
      fetch(b, m, n, pre);
      fetch_cols(b, n, cols);
      apply(b, m, n, v, pre, cols);
      return;
    }
#pragma unroll 1
    for (int j = 0; j < valid; ++j) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s = k == j ? v[k] : s;
      one(b, m, n + j, bias.p ? s + load_one(bias, b, 0, n + j) : s);
    }
  }
};

// vec: rows can be loaded and stored in whole vectors.
LinearOut linear_out(const Mat& bias, const Mat& z, const Mat& residual, const Mat& out, int act) {
  return {bias, z, residual, out, act, oct_rows(bias) && oct_rows(z) && oct_rows(residual) && oct_rows(out)};
}

// ---- operands that the copies cannot read in place ----
// [P][rows][cols] bf16 into rows of `pitch` (a multiple of eight) elements; lanes take consecutive
// pairs of columns, so that reads of unaligned rows coalesce too.  Up to two matrices a launch.
struct PackOne {
  Mat src;
  __nv_bfloat16* dst;
  int64_t rows, cols, pitch, pairs;   // pairs: rows * pitch / 2
  Div8 half;                          // by pitch / 2
};
constexpr int kPackThreads = 256, kPackPairs = 4;
__global__ void __launch_bounds__(kPackThreads) k_pack(PackOne a, PackOne b) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const int64_t x0 = int64_t{blockIdx.x} * (kPackThreads * kPackPairs) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kPackPairs; ++k) {
    int64_t x = x0 + k * kPackThreads;
    const bool second = x >= a.pairs;
    const PackOne& m = second ? b : a;
    if (second) x -= a.pairs;
    if (x >= m.pairs) break;
    int64_t i, j;
    m.half.split(x, i, j);
    j *= 2;
    const __nv_bfloat16* p = row_ptr<const __nv_bfloat16>(m.src, r, i) + j;
    const float lo = j < m.cols ? ld_elem(p) : 0.0f, hi = j + 1 < m.cols ? ld_elem(p + 1) : 0.0f;
    *reinterpret_cast<uint32_t*>(m.dst + (r * m.rows + i) * m.pitch + j) = pack2_rne(lo, hi);
  }
}

// ---- dz and the bias's gradient ----
// A CTA takes kDzRows rows of kDzCols columns: dz (bf16, where `dz` is given: the products' operand, so
// it is rounded here; its column sums are not) and the sums of its columns in fp32, joined over the
// CTAs in the order of their rows by k_dbias.  A thread issues the loads of kDzBatch rows before it
// uses any.
constexpr int kDzThreads = 256, kDzCols = 128, kDzRows = 128, kDzBatch = 8;   // 205 -> 86 us for 8 x 2048 x 5632, SiLU, sums alone

// VEC: eight whole values on 16-byte boundaries, and every row of the chunk exists.
template <class TY, class TZ, int ACT, bool VEC>
__device__ __forceinline__ void dz_rows(const Mat& dy, const Mat& z, __nv_bfloat16* dz, int64_t pitch, int r, int64_t t0,
                                        int64_t T, int64_t j, int valid, float (&sum)[8]) {
  constexpr bool kZ = ACT != DP_ACT_NONE;
  const TY* py = row_ptr<const TY>(dy, r, t0) + j;
  const TZ* pz = kZ ? row_ptr<const TZ>(z, r, t0) + j : nullptr;
  __nv_bfloat16* to = dz ? dz + t0 * pitch + j : nullptr;
#pragma unroll 1
  for (int k = 0; k < kDzRows / 16; k += kDzBatch) {
    Oct<TY> a[kDzBatch];
    Oct<TZ> b[kDzBatch];
    if (VEC) {
#pragma unroll
      for (int u = 0; u < kDzBatch; ++u) {
        a[u].load(py + (k + u) * 16 * dy.ws);
        if (kZ) b[u].load(pz + (k + u) * 16 * z.ws);
      }
    }
#pragma unroll
    for (int u = 0; u < kDzBatch; ++u) {
      float f[8], q[8];
      if (VEC) {
        a[u].get(f);
        if (kZ) b[u].get(q);
      } else {
        if (t0 + (k + u) * 16 >= T) return;
        load_ones(py + (k + u) * 16 * dy.ws, valid, f);
        if (kZ) load_ones(pz + (k + u) * 16 * z.ws, valid, q);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (kZ) f[i] *= act_slope<ACT>(q[i]);
        sum[i] += VEC || i < valid ? f[i] : 0.0f;
      }
      if (to)
        *reinterpret_cast<uint4*>(to + (k + u) * 16 * pitch) =
            make_uint4(pack2_rne(f[0], f[1]), pack2_rne(f[2], f[3]), pack2_rne(f[4], f[5]), pack2_rne(f[6], f[7]));
    }
  }
}

// Rows off 16-byte boundaries: lanes take consecutive columns, kDzOddRows rows a CTA.
constexpr int kDzOddRows = 32;
template <class TY, class TZ>
__global__ void __launch_bounds__(kDzThreads)
k_dz_odd(Mat dy, Mat z, int act, __nv_bfloat16* dz, int64_t pitch, int64_t rank_step, float* sums, int64_t T, int64_t N,
         int64_t col_blocks) {
  __shared__ float part[kDzThreads / kDzCols][kDzCols];
  wait_for_predecessor();
  constexpr int kLanes = kDzThreads / kDzCols, kRows = kDzOddRows / kLanes;
  const int r = blockIdx.y;
  const int64_t chunk = blockIdx.x / col_blocks, cb = blockIdx.x - chunk * col_blocks;
  const int col = threadIdx.x % kDzCols, lane = threadIdx.x / kDzCols;
  const int64_t j = cb * kDzCols + col, t0 = chunk * kDzOddRows + lane;
  float sum = 0.0f;
  if (j < N) {
    float f[kRows], q[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t t = t0 + k * kLanes;
      f[k] = t < T ? ld_elem(row_ptr<const TY>(dy, r, t) + j) : 0.0f;
      if (act != DP_ACT_NONE) q[k] = t < T ? ld_elem(row_ptr<const TZ>(z, r, t) + j) : 0.0f;
    }
    if (act != DP_ACT_NONE)
      with_act(act, [&](auto a) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) f[k] *= act_slope<decltype(a)::value>(q[k]);
      });
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t t = t0 + k * kLanes;
      sum += f[k];
      if (dz && t < T) st_elem(dz + r * rank_step + t * pitch + j, f[k]);
    }
  }
  if (!sums) return;
  part[lane][col] = sum;
  __syncthreads();
  if (threadIdx.x < kDzCols && j < N) {
    float s = 0.0f;
    for (int i = 0; i < kLanes; ++i) s += part[i][col];
    sums[(chunk * gridDim.y + r) * N + j] = s;
  }
}

template <class TY, class TZ>
__global__ void __launch_bounds__(kDzThreads)
k_dz(Mat dy, Mat z, int act, __nv_bfloat16* dz, int64_t pitch, int64_t rank_step, float* sums, int64_t T, int64_t N,
     int64_t col_blocks) {
  __shared__ float part[kDzThreads / 16][kDzCols + 4];
  wait_for_predecessor();
  const int r = blockIdx.y;
  const int64_t chunk = blockIdx.x / col_blocks, cb = blockIdx.x - chunk * col_blocks;
  const int oct = threadIdx.x % 16, lane = threadIdx.x / 16;
  const int64_t j = cb * kDzCols + oct * 8;
  const int valid = static_cast<int>(N - j < 8 ? (N - j > 0 ? N - j : 0) : 8);
  float sum[8] = {};
  if (valid > 0) {
    __nv_bfloat16* to = dz ? dz + r * rank_step : nullptr;
    const int64_t t0 = chunk * kDzRows + lane;
    with_act(act, [&](auto a) {
      if (valid == 8 && (chunk + 1) * kDzRows <= T)
        dz_rows<TY, TZ, decltype(a)::value, true>(dy, z, to, pitch, r, t0, T, j, valid, sum);
      else
        dz_rows<TY, TZ, decltype(a)::value, false>(dy, z, to, pitch, r, t0, T, j, valid, sum);
    });
  }
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) part[lane][oct * 8 + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < kDzCols && cb * kDzCols + c < N) {
    float s = 0.0f;
    for (int i = 0; i < kDzThreads / 16; ++i) s += part[i][c];
    sums[(chunk * gridDim.y + r) * N + cb * kDzCols + c] = s;
  }
}

__global__ void __launch_bounds__(256) k_dbias(const float* sums, int64_t chunks, Mat dbias, int64_t N, bool accumulate) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const int64_t j = int64_t{blockIdx.x} * 256 + threadIdx.x;
  if (j >= N) return;
  float s = 0.0f;
  for (int64_t c = 0; c < chunks; ++c) s += sums[(c * gridDim.y + r) * N + j];
  store_one(dbias, r, 0, j, accumulate ? s + load_one(dbias, r, 0, j) : s);
}

// ---- a few tokens ----
// Up to kFewRows tokens: bound by the weights' bytes, so a warp takes kFewCols rows of w, its lanes eight
// values of each at a time with kFewAhead such loads of each row in flight, on the ordinary
// multipliers.  Sums in fp32 over the lanes in a fixed order.  2048 -> 5632 with cold weights: one
// token 6.2 us (3.7 TB/s; as a column of the tensor core's tile 9.9), two 7.2; four 9.2 and over 8
// ranks 55, where the tile takes 10.5 and 35: the instructions, not the bytes.
constexpr int64_t kFewRows = 2;
constexpr int kFewThreads = 128, kFewCols = 2, kFewAhead = 4;
template <int T>
__global__ void __launch_bounds__(kFewThreads) k_few(Mat x, Mat w, int64_t K, int64_t N, LinearEpi<false> epi) {
  wait_for_predecessor();
  const int r = blockIdx.y, lane = threadIdx.x % 32;
  const int64_t n0 = (int64_t{blockIdx.x} * (kFewThreads / 32) + threadIdx.x / 32) * kFewCols;
  if (n0 >= N) return;
  const __nv_bfloat16 *px[T], *pw[kFewCols];
#pragma unroll
  for (int t = 0; t < T; ++t) px[t] = row_ptr<const __nv_bfloat16>(x, r, t);
#pragma unroll
  for (int c = 0; c < kFewCols; ++c) pw[c] = row_ptr<const __nv_bfloat16>(w, r, n0 + c < N ? n0 + c : n0);
  float acc[kFewCols][T] = {};
  for (int64_t k0 = lane * 8; k0 < K; k0 += 256 * kFewAhead) {
    Oct<__nv_bfloat16> a[kFewCols][kFewAhead], b[T];
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u)
#pragma unroll
      for (int c = 0; c < kFewCols; ++c) {
        a[c][u].q = make_uint4(0, 0, 0, 0);
        if (k0 + 256 * u < K) a[c][u].load(pw[c] + k0 + 256 * u);
      }
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) {
      if (k0 + 256 * u >= K) break;
#pragma unroll
      for (int t = 0; t < T; ++t) b[t].load_again(px[t] + k0 + 256 * u);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float f[8], q[8];
        b[t].get(f);
#pragma unroll
        for (int c = 0; c < kFewCols; ++c) {
          a[c][u].get(q);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c][t] = fmaf(f[i], q[i], acc[c][t]);
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kFewCols; ++c)
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int d = 16; d > 0; d /= 2) acc[c][t] += __shfl_xor_sync(0xffffffffu, acc[c][t], d);
      if (lane == c * T + t && n0 + c < N)
        epi.one(r, t, n0 + c, epi.bias.p ? acc[c][t] + load_one(epi.bias, r, 0, n0 + c) : acc[c][t]);
    }
}
// Whole vectors of x and w.
bool few(const Mat& x, const Mat& w, int64_t T, int64_t K) {
  return T <= kFewRows && K % 8 == 0 && oct_rows(x) && oct_rows(w);
}

// ---- how a call is cut ----
constexpr int64_t kSwapRows = 128;   // up to here a token is a column of the tensor core's tile

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }
int64_t pitch8(int64_t n) { return (n + 7) / 8 * 8; }

struct Cut {
  int bn;
  bool swap;
  int splits;
  bool long_sums;
};
// fp32 results of a long K need several accumulators, for which a tile 256 wide has no room.
Cut cut_product(int64_t M, int64_t N, int64_t K, int P, bool f32) {
  const ProductCut c = cut_product_of([&](int bn) { return cut(M, kTileM) * cut(N, bn) * P; }, K,
                                      static_cast<double>(M) * static_cast<double>(N) * P,
                                      f32 && sum_segments(K) > 1 ? 128 : 256, 128, least_parts(K, f32));
  return {c.bn, false, c.splits, f32};
}
Cut cut_forward(int64_t T, int64_t K, int64_t N, int P, bool f32) {
  if (T > kSwapRows) return cut_product(T, N, K, P, f32);
  const int bn = T <= 64 ? 64 : 128;
  const ProductCut c = cut_product_of([&](int) { return cut(N, kTileM) * P; }, K,
                                      static_cast<double>(T) * static_cast<double>(N) * P, bn, bn, least_parts(K, f32));
  return {bn, true, c.splits, f32};
}

// Where things lie in the workspace; `bytes` in all.
struct LinearLayout {
  int64_t x = -1, w = -1, dz = -1, sums = -1, partial = 0, bytes = 0;
  Cut fwd{}, dx{}, dw{};
};
// f32_first, f32_dw: whether y (or z), or dx, and dw are kept in fp32.
LinearLayout layout(const Mat& x, const Mat& w, int P, int64_t T, int64_t K, int64_t N, bool backward,
                    bool f32_first = false, bool f32_dw = false) {
  LinearLayout l;
  const auto take = [&](int64_t n) {
    const int64_t at = l.bytes;
    l.bytes += align256(n);
    return at;
  };
  const bool direct = !backward && few(x, w, T, K);   // by ordinary loads, which read any rows in place
  if (!direct && !copyable(x, T, K)) l.x = take(2 * P * T * pitch8(K));
  if (!direct && !copyable(w, N, K)) l.w = take(2 * P * N * pitch8(K));
  int64_t part = 0;
  // room for the parts whichever type the results have
  const auto parts = [&](auto&& how, bool f32, int64_t values) {
    for (const Cut& c : {how(false), how(true)})
      if (c.splits > 1 && 4 * c.splits * values > part) part = 4 * c.splits * values;
    return how(f32);
  };
  if (backward) {
    l.dz = take(2 * P * T * pitch8(N));
    l.sums = take(4 * P * cut(T, kDzOddRows) * N);
    if (T > 0) {
      l.dx = parts([&](bool f) { return cut_product(T, K, N, P, f); }, f32_first, P * T * K);
      l.dw = parts([&](bool f) { return cut_product(N, K, T, P, f); }, f32_dw, P * N * K);
    }
  } else if (T > 0 && !direct) {
    l.fwd = parts([&](bool f) { return cut_forward(T, K, N, P, f); }, f32_first, P * T * N);
  }
  l.partial = take(part);
  return l;
}

Operand operand(const Mat& m, int64_t rows, int64_t cols) { return {m.p, cols, rows, m.ws, m.rs}; }

// The operands x and w [P][rows][K]: in place, or copies made by one launch.
struct Operands {
  Operand x, w;
};
int pack_operands(const LinearArgs& a, const LinearLayout& l, bool need_x, bool need_w, uint8_t* ws, void* stream,
                  Operands* out) {
  PackOne jobs[2] = {{Mat{}, nullptr, 0, 0, 0, 0, Div8(1)}, {Mat{}, nullptr, 0, 0, 0, 0, Div8(1)}};
  int n = 0;
  const auto one = [&](const Mat& m, int64_t at, int64_t rows, bool need) {
    if (at < 0 || !need) return operand(m, rows, a.K);
    const int64_t pitch = pitch8(a.K);
    jobs[n++] = {m, reinterpret_cast<__nv_bfloat16*>(ws + at), rows, a.K, pitch, rows * (pitch / 2), Div8(pitch / 2)};
    return Operand{ws + at, a.K, rows, pitch, rows * pitch};
  };
  *out = {one(a.x, l.x, a.T, need_x), one(a.w, l.w, a.N, need_w)};
  if (n == 0) return cudaSuccess;
  const int64_t ctas = cut(jobs[0].pairs + jobs[1].pairs, kPackThreads * kPackPairs);
  return launch_g(k_pack, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(a.P)), kPackThreads, 0, stream, jobs[0],
                  jobs[1]);
}

template <bool AMN, bool BMN>
int product(const Cut& c, const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, int P, float* partial,
            const LinearOut& o, void* stream) {
  const LinearEpi<false> epi(o);
  return c.bn == 256 ? launch_product<256, AMN, BMN, false>(a, b, M, N, K, P, true, c.splits, partial, epi, stream, c.long_sums)
                     : launch_product<128, AMN, BMN, false>(a, b, M, N, K, P, true, c.splits, partial, epi, stream, c.long_sums);
}

}  // namespace

bool copyable(const Mat& m, int64_t rows, int64_t cols) {
  if (rows > 1 && m.ws < cols) return false;
  constexpr int64_t kMost = int64_t{1} << 39;   // elements: tensor maps hold strides below 2^40 bytes
  return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.rs % 8 == 0 && m.ws % 8 == 0 && m.rs < kMost && m.ws < kMost;
}

int64_t linear_workspace_bytes(const Mat& x, const Mat& w, int P, int64_t T, int64_t K, int64_t N, bool backward) {
  return layout(x, w, P, T, K, N, backward).bytes;
}

int launch_linear_forward(const LinearArgs& a, uint8_t* ws, void* stream) {
  if (a.T == 0) return cudaSuccess;
  const LinearLayout l = layout(a.x, a.w, a.P, a.T, a.K, a.N, false,
                                a.y.dtype == DP_F32 || (a.z.p && a.z.dtype == DP_F32));
  const LinearOut o = linear_out(a.bias, a.z, a.residual, a.y, a.act);
  if (few(a.x, a.w, a.T, a.K)) {
    const dim3 grid(static_cast<unsigned>(cut(a.N, kFewThreads / 32 * kFewCols)), static_cast<unsigned>(a.P));
    const LinearEpi<false> epi(o);
    const auto go = [&](auto kernel) { return launch_g(kernel, grid, kFewThreads, 0, stream, a.x, a.w, a.K, a.N, epi); };
    return a.T == 1 ? go(k_few<1>) : go(k_few<2>);
  }
  Operands in;
  const int e = pack_operands(a, l, true, true, ws, stream, &in);
  if (e) return e;
  const Operand &x = in.x, &w = in.w;
  float* partial = reinterpret_cast<float*>(ws + l.partial);
  if (!l.fwd.swap) return product<false, false>(l.fwd, x, w, a.T, a.N, a.K, a.P, partial, o, stream);
  const LinearEpi<true> epi(o);
  return l.fwd.bn == 64
             ? launch_product<64, false, false, false>(w, x, a.N, a.T, a.K, a.P, true, l.fwd.splits, partial, epi, stream,
                                                       l.fwd.long_sums)
             : launch_product<128, false, false, false>(w, x, a.N, a.T, a.K, a.P, true, l.fwd.splits, partial, epi, stream,
                                                        l.fwd.long_sums);
}

int launch_linear_backward(const LinearArgs& a, uint8_t* ws, void* stream) {
  const LinearLayout l = layout(a.x, a.w, a.P, a.T, a.K, a.N, true, a.dx.p && a.dx.dtype == DP_F32,
                                a.dw.p && a.dw.dtype == DP_F32);
  const Mat none{};
  const LinearOut odw = linear_out(none, none, a.accumulate ? a.dw : none, a.dw, DP_ACT_NONE);
  float* sums = reinterpret_cast<float*>(ws + l.sums);
  const dim3 bias_grid(static_cast<unsigned>(cut(a.N, 256)), static_cast<unsigned>(a.P));
  if (a.T == 0) {   // empty sums
    if (a.accumulate) return cudaSuccess;
    int e = 0;
    if (a.dbias.p) e = launch_g(k_dbias, bias_grid, 256, 0, stream, static_cast<const float*>(sums), int64_t{0}, a.dbias, a.N, false);
    if (!e && a.dw.p) {
      const int64_t want = cut(a.P * a.N * cut(a.K, 8), kJoinThreads);
      e = launch_g(k_join<LinearEpi<false>>, dim3(static_cast<unsigned>(want < 4096 ? want : 4096)), kJoinThreads, 0, stream,
                   static_cast<const float*>(sums), static_cast<int>(a.N), static_cast<int>(a.K), a.P, 0, LinearEpi<false>(odw));
    }
    return e;
  }
  Operand dz = operand(a.dy, a.T, a.N);
  const bool own = (a.dx.p || a.dw.p) && (a.act != DP_ACT_NONE || a.dy.dtype != DP_BF16 || !copyable(a.dy, a.T, a.N));
  if (own) dz = {ws + l.dz, a.N, a.T, pitch8(a.N), a.T * pitch8(a.N)};
  int e = 0;
  if (own || a.dbias.p) {
    const bool vec = oct_rows(a.dy) && (a.act == DP_ACT_NONE || oct_rows(a.z));
    const int64_t cols = cut(a.N, kDzCols), chunks = cut(a.T, vec ? kDzRows : kDzOddRows);
    const dim3 grid(static_cast<unsigned>(cols * chunks), static_cast<unsigned>(a.P));
    __nv_bfloat16* to = own ? reinterpret_cast<__nv_bfloat16*>(ws + l.dz) : nullptr;
    e = with_type(a.dy.dtype, [&](auto* ty) {
      return with_type(a.act == DP_ACT_NONE ? a.dy.dtype : a.z.dtype, [&](auto* tz) {
        using TY = std::remove_pointer_t<decltype(ty)>;
        using TZ = std::remove_pointer_t<decltype(tz)>;
        float* into = a.dbias.p ? sums : nullptr;
        return vec ? launch_g(k_dz<TY, TZ>, grid, kDzThreads, 0, stream, a.dy, a.z, a.act, to, pitch8(a.N), a.T * pitch8(a.N),
                              into, a.T, a.N, cols)
                   : launch_g(k_dz_odd<TY, TZ>, grid, kDzThreads, 0, stream, a.dy, a.z, a.act, to, pitch8(a.N),
                              a.T * pitch8(a.N), into, a.T, a.N, cols);
      });
    });
    if (!e && a.dbias.p)
      e = launch_g(k_dbias, bias_grid, 256, 0, stream, static_cast<const float*>(sums), chunks, a.dbias, a.N, a.accumulate);
    if (e) return e;
  }
  float* partial = reinterpret_cast<float*>(ws + l.partial);
  Operands in;
  e = pack_operands(a, l, a.dw.p != nullptr, a.dx.p != nullptr, ws, stream, &in);
  if (!e && a.dx.p)
    e = product<false, true>(l.dx, dz, in.w, a.T, a.K, a.N, a.P, partial, linear_out(none, none, none, a.dx, DP_ACT_NONE), stream);
  if (!e && a.dw.p) e = product<true, true>(l.dw, dz, in.x, a.N, a.K, a.T, a.P, partial, odw, stream);
  return e;
}

int64_t product_timeouts_linear(bool reset) {
  unsigned long long n = 0, z = 0;
  if (cudaMemcpyFromSymbol(&n, g_product_timeouts, sizeof n) != cudaSuccess) return -2;
  if (reset && cudaMemcpyToSymbol(g_product_timeouts, &z, sizeof z) != cudaSuccess) return -2;
  return static_cast<int64_t>(n);
}

}  // namespace dps
