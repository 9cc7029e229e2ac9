// Token log-probabilities, their gradient, and the clipped policy loss, over rows
// of logits.
#include <cmath>

#include "model.cuh"

namespace dps {
namespace {

constexpr int kRowThreads = 512;
constexpr int kStatThreads = 256;

// A softmax's running statistics: the largest value seen and the sum of
// exp(value - largest).
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.s + b.s};   // no term yet (or NaN in one of the sums)
  return {m, a.s * __expf(a.m - m) + b.s * __expf(b.m - m)};
}

template <int NT>
__device__ MaxSum block_merge(MaxSum v, MaxSum* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = merge(v, {__shfl_xor_sync(~0u, v.m, o), __shfl_xor_sync(~0u, v.s, o)});
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int w = 1; w < NT / 32; ++w) v = merge(v, sh[w]);
  __syncthreads();
  return v;
}

// One row's softmax statistics by one CTA: the maximum, then the sum.
template <class T>
__device__ MaxSum row_stats(const T* x, int64_t V, float scale, MaxSum* sh) {
  float m = -INFINITY;
  bool nan = false;
  for (int64_t j = threadIdx.x; j < V; j += kRowThreads) {
    const float z = ld_elem(x + j) * scale;
    nan |= z != z;
    m = fmaxf(m, z);
  }
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < V; j += kRowThreads)
    s += m == -INFINITY ? 0.0f : expf(ld_elem(x + j) * scale - m);
  return block_merge<kRowThreads>({m, nan ? NAN : s}, sh);
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
k_logprob(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, float* logp, float* lse) {
  wait_for_predecessor();
  __shared__ MaxSum sh[kRowThreads / 32];
  const int r = blockIdx.y;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const int64_t i = r * N + t, v = token_at(tok, i, V);
    float lp = 0.0f, le = 0.0f;
    if (v >= 0) {
      const T* x = row_ptr<T>(logits, r, t);
      const MaxSum a = row_stats(x, V, scale, sh);
      const float ls = logf(a.s);
      le = a.m + ls;
      lp = (ld_elem(x + v) * scale - a.m) - ls;
    }
    if (threadIdx.x == 0) {
      logp[i] = lp;
      if (lse) lse[i] = le;
    }
  }
}

// dlogits = g * (1[v = token] - exp(z - lse)), g = dlogp * scale.
template <class T>
__device__ void write_grad(const T* x, T* dx, int64_t V, float scale, float lse, float g, int64_t v) {
  for (int64_t j = threadIdx.x; j < V; j += kRowThreads) {
    const float p = expf(ld_elem(x + j) * scale - lse);
    st_elem(dx + j, g * ((j == v ? 1.0f : 0.0f) - p));
  }
}

template <class T>
__device__ void write_zeros(T* dx, int64_t V) {
  for (int64_t j = threadIdx.x; j < V; j += kRowThreads) st_elem(dx + j, 0.0f);
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
k_logprob_grad(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, const float* lse,
               const float* dlogp, Mat dlogits) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const int64_t i = r * N + t, v = token_at(tok, i, V);
    const float g = dlogp[i] * scale;
    T* dx = row_ptr<T>(dlogits, r, t);
    if (v < 0 || g == 0.0f)
      write_zeros(dx, V);
    else
      write_grad(row_ptr<T>(logits, r, t), dx, V, scale, lse[i], g, v);
  }
}

// One row of the policy loss: its terms and the slope dloss/dlogp, without w.
struct PolicyRow {
  float pg, kl, slope;
  bool clipped;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, int64_t i, float logp) {
  PolicyRow o;
  const float q = expf(logp - a.old_logp[i]), A = a.adv[i];
  const float plain = q * A, held = fminf(fmaxf(q, a.lo), a.hi) * A;
  o.clipped = held < plain;
  o.pg = -(o.clipped ? held : plain);
  o.slope = o.clipped ? 0.0f : -plain;
  o.kl = 0.0f;
  if (a.ref_logp) {
    const float d = a.ref_logp[i] - logp, e = expm1f(d);
    o.kl = e - d;
    if (a.beta != 0.0f) o.slope -= a.beta * e;
  }
  return o;
}

__device__ __forceinline__ float weight_of(const PolicyArgs& a, int64_t i) {
  return a.weight ? a.weight[i] : 1.0f;
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
k_policy(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, PolicyArgs a, float* logp,
         Mat dlogits) {
  wait_for_predecessor();
  __shared__ MaxSum sh[kRowThreads / 32];
  const int r = blockIdx.y;
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    const int64_t i = r * N + t, v = token_at(tok, i, V);
    const float w = weight_of(a, i);
    T* dx = dlogits.p ? row_ptr<T>(dlogits, r, t) : nullptr;
    if (v < 0 || w == 0.0f) {
      if (threadIdx.x == 0) logp[i] = 0.0f;
      if (dx) write_zeros(dx, V);
      continue;
    }
    const T* x = row_ptr<T>(logits, r, t);
    const MaxSum st = row_stats(x, V, scale, sh);
    const float ls = logf(st.s);
    const float lp = (ld_elem(x + v) * scale - st.m) - ls;
    if (threadIdx.x == 0) logp[i] = lp;
    if (dx) {
      __syncthreads();   // dlogits may be logits: every thread has its token's logit
      const float g = w * policy_row(a, i, lp).slope * scale;
      if (g == 0.0f)
        write_zeros(dx, V);
      else
        write_grad(x, dx, V, scale, st.m + ls, g, v);
    }
  }
}

// The loss and its parts, one CTA per rank: rows in a fixed order, sums in double.
__global__ void __launch_bounds__(kStatThreads)
k_policy_stats(int64_t N, int64_t V, TokenArgs tok, PolicyArgs a, const float* logp, float* stats) {
  wait_for_predecessor();
  __shared__ double sh[4][kStatThreads / 32];
  const int r = blockIdx.x;
  double s[4] = {0, 0, 0, 0};
  for (int64_t t = threadIdx.x; t < N; t += kStatThreads) {
    const int64_t i = r * N + t;
    const float w = weight_of(a, i);
    if (w == 0.0f || token_at(tok, i, V) < 0) continue;
    const PolicyRow o = policy_row(a, i, logp[i]);
    s[0] += static_cast<double>(w) * (a.beta != 0.0f ? o.pg + a.beta * o.kl : o.pg);
    s[1] += static_cast<double>(w) * o.pg;
    s[2] += static_cast<double>(w) * o.kl;
    s[3] += o.clipped ? static_cast<double>(w) : 0.0;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s[k] += __shfl_xor_sync(~0u, s[k], o);
    if ((threadIdx.x & 31) == 0) sh[k][threadIdx.x >> 5] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    double v = 0;
    for (int w = 0; w < kStatThreads / 32; ++w) v += sh[threadIdx.x][w];
    stats[4 * r + threadIdx.x] = static_cast<float>(v);
  }
}

dim3 row_grid(int P, int64_t N) {
  return dim3(static_cast<unsigned>(N < (1 << 20) ? N : (1 << 20)), static_cast<unsigned>(P));
}

}  // namespace

int launch_token_logprob(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                         float scale, float* logp, float* lse, void* stream) {
  if (T == 0) return cudaSuccess;
  return with_type(logits.dtype, [&](auto* z) {
    return launch_g(k_logprob<std::remove_pointer_t<decltype(z)>>, row_grid(P, T), kRowThreads, 0, stream,
                    logits, T, V, tok, scale, logp, lse);
  });
}

int launch_token_logprob_backward(const Mat& logits, int P, int64_t T, int64_t V,
                                  const TokenArgs& tok, float scale, const float* lse,
                                  const float* dlogp, const Mat& dlogits, void* stream) {
  if (T == 0) return cudaSuccess;
  return with_type(logits.dtype, [&](auto* z) {
    return launch_g(k_logprob_grad<std::remove_pointer_t<decltype(z)>>, row_grid(P, T), kRowThreads, 0,
                    stream, logits, T, V, tok, scale, lse, dlogp, dlogits);
  });
}

int launch_policy_loss(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                       float scale, const PolicyArgs& a, float* logp, float* stats,
                       const Mat& dlogits, void* stream) {
  if (T > 0) {
    const int e = with_type(logits.dtype, [&](auto* z) {
      return launch_g(k_policy<std::remove_pointer_t<decltype(z)>>, row_grid(P, T), kRowThreads, 0, stream,
                      logits, T, V, tok, scale, a, logp, dlogits);
    });
    if (e) return e;
  }
  return launch_g(k_policy_stats, dim3(static_cast<unsigned>(P)), kStatThreads, 0, stream, T, V, tok, a,
                  static_cast<const float*>(logp), stats);
}

}  // namespace dps
