// Token log-probabilities, their gradient, and the clipped policy loss, over rows
// of logits.
//
// All three are bound by HBM: a logit is read once (2 or 4 bytes) and, where a
// gradient is wanted, one is written, for an exponential or two and a handful of
// other operations.  In base 2, with c = scale * log2(e) and any reference m near the
// largest c x,
//   s = sum_v 2^(c x_v - m),   lse = (m + log2 s) / log2(e),   logp = (c x_t - m - log2 s) / log2(e),
// and the softmax is 2^(c x_v - m) / s.  c x - m is one fused operation and m the same
// float everywhere, so m's own rounding, up to 32 where |m| is just below 2^30, cancels.
// Two values go through each multiply-add (fma.f32x2; with one each the log-probabilities below ran 11% slower).
// All of it is fp32, and a gradient is rounded once, to its type, when it is stored.
//
// Measured on GB300 (HBM copy 6.79 TB/s): log-probabilities of 16384 rows of 32000 bf16
// 148 us (7.1 TB/s), the gradient of 8192 rows of 50257 bf16 234 us (6.7 TB/s), the policy
// loss of 16384 rows of 50304 bf16, a quarter left out, 435 us (6.6 TB/s).
//
// Rows whose largest c x is 2^30 or more in magnitude (a row of one large mask value, of
// -inf alone, one with an infinity at its top) would take 2^(c x - m) past fp32, for m's
// rounding, or overflow in c x: they are computed again from differences x - max x (far_row).
//
// A row is cut at the first 16-byte boundary: up to 7 leading and trailing values
// go alone, the rest as 16-byte vectors, whatever the row's alignment.
#include <cmath>

#include "model.cuh"
#include "token_shape.h"

namespace dps {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ---- pairs of fp32 ----
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(ex2(a), ex2(b));
}

// ---- 16-byte vectors: N values, as N/2 pairs ----
template <class T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void pairs(const uint4& q, uint64_t (&f)[4]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 store(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpack2(f[i], a, b);
      w[i] = pack2_rne(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // A vector of -inf.
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  // The largest value (a NaN is passed over: it reaches the sum by itself).
  static __device__ __forceinline__ float top(const uint4& q) {
    __nv_bfloat162 h[4];
    memcpy(h, &q, 16);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void pairs(const uint4& q, uint64_t (&f)[2]) {
    f[0] = pack2(__uint_as_float(q.x), __uint_as_float(q.y));
    f[1] = pack2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  static __device__ __forceinline__ uint4 store(const uint64_t (&f)[2]) {
    float a, b, c, d;
    unpack2(f[0], a, b);
    unpack2(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ __forceinline__ float top(const uint4& q) {
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                 fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
};

__device__ __forceinline__ void copy_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- a softmax's running statistics: the largest c x, and sum 2^(c x - m) ----
struct alignas(8) Run {   // moves as one 8-byte access (cluster_run)
  float m, s;
};

// Below 2^30 half a unit in the last place of m is 32 at most: 2^(c x - m) stays within
// 2^32 and the sum of a row within 2^63.  (From 2^34 on it may be 2^512.)  And two different
// x of one sign whose c x are about 2^30 differ there by 64 or more, so a value below -2^30 has
// no weight beside one above: 2^-64, where a row has fewer than 2^31 values.
constexpr float kFar = 1073741824.0f;   // 2^30

// The reference a sum is taken against: 0 where only values below -kFar, which have no
// weight in a row whose largest is above, were seen (then the sum is 0).
__device__ __forceinline__ float ref_of(float m) { return m < -kFar ? 0.0f : m; }

__device__ __forceinline__ Run merge(Run a, Run b) {
  const float m = fmaxf(a.m, b.m), r = ref_of(m);
  // a side that saw nothing has s = 0 (or NaN, which must stay)
  const float ea = a.m < -kFar ? 1.0f : ex2(a.m - r), eb = b.m < -kFar ? 1.0f : ex2(b.m - r);
  return {m, a.s * ea + b.s * eb};
}

__device__ __forceinline__ void raise(Run& a, float m) {
  if (m > a.m) {
    if (a.m >= -kFar) a.s *= ex2(a.m - m);
    a.m = m;
  }
}

// K vectors more.
template <class T, int K>
__device__ __forceinline__ void take(Run& a, const uint4 (&q)[K], float c) {
  constexpr int H = Vec16<T>::N / 2;
  float m = Vec16<T>::top(q[0]);
#pragma unroll
  for (int k = 1; k < K; ++k) m = fmaxf(m, Vec16<T>::top(q[k]));
  raise(a, m * c);
  const float r = -ref_of(a.m);
  const uint64_t r2 = pack2(r, r), c2 = pack2(c, c), one = pack2(1.0f, 1.0f);
  uint64_t s2 = pack2(a.s, 0.0f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    uint64_t f[H];
    Vec16<T>::pairs(q[k], f);
#pragma unroll
    for (int h = 0; h < H; ++h) s2 = fma2(ex2_2(fma2(f[h], c2, r2)), one, s2);
  }
  float lo, hi;
  unpack2(s2, lo, hi);
  a.s = lo + hi;
}

__device__ __forceinline__ void take_one(Run& a, float x, float c) {
  raise(a, x * c);
  a.s += ex2(fmaf(x, c, -ref_of(a.m)));
}

// A warp's: the largest first, then every lane's sum against it.
__device__ __forceinline__ Run warp_run(Run a) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(a.m));
  // a lane that saw nothing has s = 0 (or NaN, which must stay)
  float s = a.m < -kFar ? a.s : a.s * ex2(a.m - ref_of(m));
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return {m, s};
}

// The group's; the same value in every thread.  What the group read of its row comes before
// what it writes from here on, which may be the same row: a warp's shuffles order no memory.
template <int G>
__device__ __forceinline__ Run group_run(Run a) {
  a = warp_run(a);
  if constexpr (G == 32) __syncwarp();
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    __shared__ Run sh[W];
    const int lane = threadIdx.x & 31;
    if (lane == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    a = warp_run(lane < W ? sh[lane] : Run{-INFINITY, 0.0f});
  }
  return a;
}

// ---- clusters: C CTAs share a row when there are few rows, or long ones ----
// The row's statistics from its CTAs' (cluster_arrive() was called at the start: a
// CTA's shared memory is written from outside only once it runs).
__device__ Run cluster_run(Run a, int C) {
  __shared__ Run part[kMaxCluster];
  static_assert(sizeof(Run) == 8 && alignof(Run) == 8, "written as st.v2.f32");
  cluster_wait();
  if (threadIdx.x < static_cast<unsigned>(C)) {
    uint32_t dst;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(dst)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&part[cluster_rank()]))), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(a.m), "f"(a.s) : "memory");
  }
  cluster_arrive();
  cluster_wait();
  a = part[0];
  for (int k = 1; k < C; ++k) a = merge(a, part[k]);
  return a;
}

// A group's part of a row (c of C), and its thread's single values: vectors [v0, v0 + n) of the row's aligned body, and
// the values around the body (the leading ones with the first part, the trailing
// ones with the last; at most one of each per thread).
template <class T>
struct Slice {
  const uint4* xv;    // the part's first vector
  int64_t j0;         // its first value's column
  int n;              // vectors
  int64_t edge;       // this thread's single column, or -1
  int64_t edge2;

  __device__ __forceinline__ Slice(const T* x, int64_t V, int c, int C, int tid) {
    constexpr int N = Vec16<T>::N;
    const int off = (16 - static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15)) & 15;
    const int up = off / static_cast<int>(sizeof(T));
    const int64_t lead = up < V ? up : V;
    const int nv = static_cast<int>((V - lead) / N), per = C == 1 ? nv : (nv + C - 1) / C;
    const int v0 = int64_t{c} * per < nv ? c * per : nv;
    n = v0 + per < nv ? per : nv - v0;
    j0 = lead + int64_t{N} * v0;
    xv = reinterpret_cast<const uint4*>(x + j0);
    edge = c == 0 && tid < lead ? tid : -1;
    const int64_t at = lead + int64_t{N} * nv + tid;
    edge2 = c == C - 1 && at < V ? at : -1;
  }
};

// The statistics of a row that c x overflows in, by one group, value by value: the
// largest x, and sum 2^(c (x - max)).  A row of -inf alone gives {-inf, 0}; +inf or NaN
// gives NaN.
template <class T, int G>
__device__ __noinline__ Run far_row(const T* x, int64_t V, float c) {
  __shared__ float part[2][G / 32];
  const int tid = threadIdx.x & (G - 1);
  float m = -INFINITY, s = 0.0f;
  for (int64_t j = tid; j < V; j += G) m = fmaxf(m, ld_elem(x + j));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  if constexpr (G > 32) {
    if ((tid & 31) == 0) part[0][tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < G / 32; ++w) m = fmaxf(m, part[0][w]);
  }
  const float r = m == -INFINITY ? 0.0f : m;
  for (int64_t j = tid; j < V; j += G) s += ex2((ld_elem(x + j) - r) * c);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  if constexpr (G > 32) {
    if ((tid & 31) == 0) part[1][tid >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < G / 32; ++w) s += part[1][w];
  } else {
    __syncwarp();   // as in group_run
  }
  return {m, s};
}

// logp and lse of a far row.
__device__ __forceinline__ void far_result(Run a, float xt, float scale, float& logp, float& lse) {
  const float m = a.m == -INFINITY ? 0.0f : a.m, ls = logf(a.s);
  logp = (xt - m) * scale - ls;
  lse = m * scale + ls;
}

constexpr float kLn2 = 0.6931471805599453f;

// ---- one row of the policy loss: its terms and the slope dloss/dlogp, without w ----
struct PolicyRow {
  float pg, kl, slope;
  bool clipped;
};

struct PolicyIn {
  float old_logp, adv, ref_logp;
  __device__ __forceinline__ PolicyIn(const PolicyArgs& a, int64_t i)
      : old_logp(a.old_logp[i]), adv(a.adv[i]), ref_logp(a.ref_logp ? a.ref_logp[i] : 0.0f) {}
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, const PolicyIn& in, float logp) {
  PolicyRow o;
  const float q = expf(logp - in.old_logp), A = in.adv;
  const float plain = q * A, held = fminf(fmaxf(q, a.lo), a.hi) * A;
  o.clipped = held < plain;
  o.pg = -(o.clipped ? held : plain);
  o.slope = o.clipped ? 0.0f : -plain;
  o.kl = 0.0f;
  if (a.ref_logp) {
    const float d = in.ref_logp - logp, e = expm1f(d);
    o.kl = e - d;
    if (a.beta != 0.0f) o.slope -= a.beta * e;
  }
  return o;
}

__device__ __forceinline__ float weight_of(const PolicyArgs& a, int64_t i) {
  return a.weight ? a.weight[i] : 1.0f;
}

// ---- forward: one row per group, or per cluster ----
// A thread has four vectors in flight; what is past the row's end reads as -inf, so that
// a last short round costs no second loop.  Bound by HBM reads.
constexpr int kRowThreads = 128;   // 256 ran 2% and 512 11% slower: the reduction's share per thread

template <class T, int G, bool CL>
__global__ void __launch_bounds__(cta_of<G>)
k_logprob(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, float* logp, float* lse, int C) {
  constexpr int NT = cta_of<G>, K = 4;
  wait_for_predecessor();
  const int r = blockIdx.y, part = CL ? static_cast<int>(cluster_rank()) : 0, tid = threadIdx.x & (G - 1);
  const int64_t t = CL ? blockIdx.x / C : blockIdx.x * int64_t{NT / G} + threadIdx.x / G;
  if (G < NT && t >= N) return;
  const int64_t i = r * N + t, v = token_at(tok, i, V);
  if (v < 0) {
    if (tid == 0 && part == 0) {
      logp[i] = 0.0f;
      if (lse) lse[i] = 0.0f;
    }
    return;
  }
  if (CL) cluster_arrive();
  const float c = scale * kLog2e;
  const T* x = row_ptr<T>(logits, r, t);
  const float xt = ld_elem(x + v);
  const Slice<T> sl(x, V, part, CL ? C : 1, tid);
  Run a{-INFINITY, 0.0f};
  const uint4* p = sl.xv + tid;
  for (int left = sl.n - tid; left > 0; left -= K * G, p += K * G) {
    uint4 q[K];
#pragma unroll
    for (int u = 0; u < K; ++u) q[u] = u * G < left ? ld_stream(p + u * G) : Vec16<T>::nothing();
    take<T>(a, q, c);
  }
  if (sl.edge >= 0) take_one(a, ld_elem(x + sl.edge), c);
  if (sl.edge2 >= 0) take_one(a, ld_elem(x + sl.edge2), c);
  a = group_run<G>(a);
  if (CL) a = cluster_run(a, C);
  float lp, le;
  if (fabsf(a.m) < kFar) {
    const float ls = log2f(a.s);
    lp = (fmaf(xt, c, -a.m) - ls) * kLn2;
    le = (a.m + ls) * kLn2;
  } else {
    far_result(far_row<T, G>(x, V, c), xt, scale, lp, le);
  }
  if (tid == 0 && part == 0) {
    logp[i] = lp;
    if (lse) lse[i] = le;
  }
}

// ---- gradients: g (1[v = token] - p) ----
template <class T>
__device__ __forceinline__ void st_vec(T* dx, const uint64_t (&f)[Vec16<T>::N / 2], bool aligned) {
  if (aligned) {
    st_stream(reinterpret_cast<uint4*>(dx), Vec16<T>::store(f));
  } else {   // dlogits sits at another phase of 16 bytes than logits
#pragma unroll
    for (int h = 0; h < Vec16<T>::N / 2; ++h) {
      float a, b;
      unpack2(f[h], a, b);
      st_elem(dx + 2 * h, a);
      st_elem(dx + 2 * h + 1, b);
    }
  }
}

// Adds g to the value at place `at` of a vector (at outside [0, N): none).
template <int H>
__device__ __forceinline__ void add_at(uint64_t (&f)[H], int64_t at, float g) {
  if (at < 0 || at >= 2 * H) return;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    float a, b;
    unpack2(f[h], a, b);
    f[h] = pack2(a + (at == 2 * h ? g : 0.0f), b + (at == 2 * h + 1 ? g : 0.0f));
  }
}

template <class T>
__device__ __forceinline__ bool vec_aligned(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Zeros over a row's part (cut by dlogits' own alignment).
template <class T, int G>
__device__ void zero_slice(T* dx, int64_t V, int part, int C) {
  const int tid = threadIdx.x & (G - 1);
  const Slice<T> sl(dx, V, part, C, tid);
  uint4* p = const_cast<uint4*>(sl.xv);
  for (int k = tid; k < sl.n; k += G) st_stream(p + k, make_uint4(0, 0, 0, 0));
  if (sl.edge >= 0) st_elem(dx + sl.edge, 0.0f);
  if (sl.edge2 >= 0) st_elem(dx + sl.edge2, 0.0f);
}

// From a given lse: no sums, so a row is cut into parts of kGradVecs vectors a
// thread, all of a thread's loads in flight at once, and a CTA lives for one round of
// loads and stores.  Bound by HBM, reads and writes alike.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

template <class T, int G>
__global__ void __launch_bounds__(cta_of<G>, 8)   // 32 registers at 256 threads: 4% faster than with 48
k_logprob_grad(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, const float* lse,
               const float* dlogp, Mat dlogits, int parts) {
  constexpr int NT = cta_of<G>, VN = Vec16<T>::N, H = VN / 2;
  wait_for_predecessor();
  const int r = blockIdx.y, tid = threadIdx.x & (G - 1);
  const int part = G < NT ? 0 : static_cast<int>(blockIdx.x % static_cast<unsigned>(parts));
  const int64_t t = G < NT ? blockIdx.x * int64_t{NT / G} + threadIdx.x / G : blockIdx.x / static_cast<unsigned>(parts);
  if (G < NT && t >= N) return;
  const int64_t i = r * N + t, v = token_at(tok, i, V);
  const float g = dlogp[i] * scale, le = lse[i];
  T* dx = row_ptr<T>(dlogits, r, t);
  if (v < 0 || g == 0.0f) {
    zero_slice<T, G>(dx, V, part, parts);
    return;
  }
  const T* x = row_ptr<T>(logits, r, t);
  const Slice<T> sl(x, V, part, parts, tid);
  T* dv = dx + sl.j0;
  const bool al = vec_aligned(dv);
  const uint64_t s2 = pack2(scale, scale), l2 = pack2(-le, -le), e2 = pack2(kLog2e, kLog2e), g2 = pack2(-g, -g);
  for (int k0 = tid; k0 < sl.n; k0 += kGradVecs * G) {
    uint4 q[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
      if (k0 + u * G < sl.n) q[u] = ld_stream(sl.xv + k0 + u * G);
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int k = k0 + u * G;
      if (k >= sl.n) break;
      uint64_t f[H];
      Vec16<T>::pairs(q[u], f);
#pragma unroll
      for (int h = 0; h < H; ++h) f[h] = fma2(ex2_2(fma2(fma2(f[h], s2, l2), e2, 0)), g2, 0);
      add_at(f, v - (sl.j0 + int64_t{VN} * k), g);
      st_vec<T>(dv + int64_t{VN} * k, f, al);
    }
  }
  const auto one = [&](int64_t j) {
    const float p = ex2(fmaf(ld_elem(x + j), scale, -le) * kLog2e);
    st_elem(dx + j, (j == v ? g : 0.0f) - g * p);
  };
  if (sl.edge >= 0) one(sl.edge);
  if (sl.edge2 >= 0) one(sl.edge2);
}

// ---- the policy loss: statistics and gradient in one pass over HBM ----
// Two passes from global memory would read every logit twice (half as much traffic
// again); a row of 50304 bf16 fits shared memory twice per SM, so that one row's loads and
// stores overlap another's sums.  What is left to HBM's rate is the issue of the two
// passes' instructions (64% of the issue slots busy).
// One row per group, or per cluster.  A thread copies its vectors to shared memory
// (all of them in flight at once, waited for in four groups) and reads only its
// own back, once for the sum and once for the gradient, so the copies need no
// barrier.  Vectors past `kcap` per thread, which shared memory has no room for,
// are read from global memory both times.  Every read of the row comes before the
// row's barrier or is the writer's own, so dlogits may be logits.
template <class T, int G, bool CL, bool ALL>
__global__ void __launch_bounds__(cta_of<G>, G == 512 ? 2 : 1024 / cta_of<G>)
k_policy(Mat logits, int64_t N, int64_t V, TokenArgs tok, float scale, PolicyArgs pa, float* logp,
         Mat dlogits, int C, int kcap) {
  constexpr int NT = cta_of<G>, VN = Vec16<T>::N, H = VN / 2, K = 4;
  extern __shared__ uint4 keep[];   // [kcap][NT]
  wait_for_predecessor();
  const int r = blockIdx.y, part = CL ? static_cast<int>(cluster_rank()) : 0, nc = CL ? C : 1;
  const int tid = threadIdx.x & (G - 1);
  const int64_t t = CL ? blockIdx.x / C : blockIdx.x * int64_t{NT / G} + threadIdx.x / G;
  if (G < NT && t >= N) return;
  const int64_t i = r * N + t, v = token_at(tok, i, V);
  const float w = weight_of(pa, i);
  T* dx = dlogits.p ? row_ptr<T>(dlogits, r, t) : nullptr;
  if (v < 0 || w == 0.0f) {
    if (tid == 0 && part == 0) logp[i] = 0.0f;
    if (dx) zero_slice<T, G>(dx, V, part, nc);
    return;
  }
  if (CL) cluster_arrive();
  const float c = scale * kLog2e;
  const T* x = row_ptr<T>(logits, r, t);
  const Slice<T> sl(x, V, part, nc, tid);
  uint4* mine = keep + threadIdx.x;
  const int n = (sl.n + G - 1 - tid) / G;   // this thread's vectors
  const int quarter = ((n + 3) / 4 + K - 1) / K * K, kept = ALL || n < kcap ? n : kcap;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    for (int k = g * quarter; k < (g + 1) * quarter && k < kept; ++k)
      copy_async16(mine + k * NT, sl.xv + k * int64_t{G} + tid);
    copy_commit();
  }
  const float xt = ld_elem(x + v);
  const PolicyIn in(pa, i);
  float xe = -INFINITY, xe2 = -INFINITY;
  if (sl.edge >= 0) xe = ld_elem(x + sl.edge);
  if (sl.edge2 >= 0) xe2 = ld_elem(x + sl.edge2);
  const auto vec = [&](int k) {
    return ALL || k < kept ? mine[k * NT] : ld_stream(sl.xv + k * int64_t{G} + tid);
  };
  Run a{-INFINITY, 0.0f};
  const auto group = [&](int g) {
    const int end = (g + 1) * quarter < n ? (g + 1) * quarter : n;
    int k = g * quarter;
    for (; k + K - 1 <= end; k += K) {   // the last of a round may be missing
      uint4 q[K];
#pragma unroll
      for (int u = 0; u < K; ++u) q[u] = u < K - 1 || k + u < end ? vec(k + u) : Vec16<T>::nothing();
      take<T>(a, q, c);
    }
    for (; k < end; ++k) {
      const uint4 q[1] = {vec(k)};
      take<T>(a, q, c);
    }
  };
  copy_wait<3>();
  group(0);
  copy_wait<2>();
  group(1);
  copy_wait<1>();
  group(2);
  copy_wait<0>();
  group(3);
  if (sl.edge >= 0) take_one(a, xe, c);
  if (sl.edge2 >= 0) take_one(a, xe2, c);
  a = group_run<G>(a);
  if (CL) a = cluster_run(a, C);
  const bool far = !(fabsf(a.m) < kFar);
  float lp = (fmaf(xt, c, -a.m) - log2f(a.s)) * kLn2, le;
  if (far) {
    a = far_row<T, G>(x, V, c);
    far_result(a, xt, scale, lp, le);
    if (CL) {   // every CTA of the row has read it: dlogits may be logits
      cluster_arrive();
      cluster_wait();
    }
  }
  if (tid == 0 && part == 0) logp[i] = lp;
  if (!dx) return;
  const float g = w * policy_row(pa, in, lp).slope * scale, gs = g / a.s;
  if (g == 0.0f) {
    zero_slice<T, G>(dx, V, part, nc);
    return;
  }
  const auto one = [&](int64_t j, float xj) {
    const float p = ex2(far ? (xj - (a.m == -INFINITY ? 0.0f : a.m)) * c : fmaf(xj, c, -a.m));
    st_elem(dx + j, (j == v ? g : 0.0f) - gs * p);
  };
  if (sl.edge >= 0) one(sl.edge, xe);
  if (sl.edge2 >= 0) one(sl.edge2, xe2);
  if (far) {
    for (int k = 0; k < n; ++k)
      for (int u = 0; u < VN; ++u) {
        const int64_t j = sl.j0 + (k * int64_t{G} + tid) * VN + u;
        one(j, ld_elem(x + j));
      }
    return;
  }
  // the thread's vector that holds the token, and its place there
  const int64_t tv = v - sl.j0;
  int hit = -1;
  if (tv >= 0 && tv / VN < sl.n) {
    const int k = static_cast<int>(tv / VN);
    if (k % G == tid) hit = k / G;
  }
  T* dv = dx + sl.j0 + VN * tid;
  const bool al = vec_aligned(dv);
  const uint64_t r2 = pack2(-a.m, -a.m), c2 = pack2(c, c), g2 = pack2(-gs, -gs);
#pragma unroll 2
  for (int k = 0; k < n; ++k) {
    uint64_t f[H];
    Vec16<T>::pairs(vec(k), f);
#pragma unroll
    for (int h = 0; h < H; ++h) f[h] = fma2(ex2_2(fma2(f[h], c2, r2)), g2, 0);
    if (k == hit) add_at(f, tv % VN, g);
    st_vec<T>(dv, f, al);
    dv += G * VN;
  }
}

// The loss and its parts, a cluster of C CTAs per rank: every thread its rows in order,
// the threads' sums in a fixed order, all in double.
constexpr int kStatThreads = 256;

__global__ void __launch_bounds__(kStatThreads)
k_policy_stats(int64_t N, int64_t V, TokenArgs tok, PolicyArgs a, const float* logp, float* stats, int C) {
  wait_for_predecessor();
  __shared__ double sh[4][kStatThreads / 32];
  __shared__ double all[kMaxCluster][4];   // the first CTA's: every CTA's sums
  if (C > 1) cluster_arrive();
  const int part = C > 1 ? static_cast<int>(cluster_rank()) : 0, r = blockIdx.x / C;
  double s[4] = {0, 0, 0, 0};
  for (int64_t t = part * kStatThreads + threadIdx.x; t < N; t += C * kStatThreads) {
    const int64_t i = r * N + t;
    const float w = weight_of(a, i);
    if (w == 0.0f || token_at(tok, i, V) < 0) continue;
    const PolicyRow o = policy_row(a, PolicyIn(a, i), logp[i]);
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
  double v = 0;
  if (threadIdx.x < 4)
    for (int w = 0; w < kStatThreads / 32; ++w) v += sh[threadIdx.x][w];
  if (C > 1) {
    cluster_wait();
    if (threadIdx.x < 4) {
      uint32_t dst;
      asm("mapa.shared::cluster.u32 %0, %1, 0;"
          : "=r"(dst)
          : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&all[part][threadIdx.x]))));
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dst), "d"(v) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    if (part > 0 || threadIdx.x >= 4) return;
    v = 0;
    for (int k = 0; k < C; ++k) v += all[k][threadIdx.x];
  }
  if (threadIdx.x < 4) stats[4 * r + threadIdx.x] = static_cast<float>(v);
}

// ---- launches ----
// A launch without opt-in has 48 KB of shared memory, the kernel's static variables (a few
// hundred bytes: partial sums by warp or CTA) among them.
constexpr size_t kStaticMost = 1024;

// Launch with clusters of C CTAs along x.
template <class K, class... A>
int launch_cluster(K kernel, dim3 grid, int C, int threads, size_t smem, void* stream, A... args) {
  if (smem + kStaticMost > 48 * 1024) {
    const cudaError_t e = ensure_dyn_smem(kernel, smem);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl_enabled()) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (C > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = static_cast<unsigned>(C);
    attr[na].val.clusterDim.y = 1;
    attr[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(na);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  const cudaError_t last = cudaGetLastError();
  return static_cast<int>(e != cudaSuccess ? e : last);
}

constexpr int64_t kLongestRead = 256 * 1024;    // forward: bytes of a row per CTA

}  // namespace

// Rows of a launch whose groups are warps.
dim3 short_grid(int P, int64_t T) { return dim3(static_cast<unsigned>((T + 3) / 4), static_cast<unsigned>(P)); }

int launch_token_logprob(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                         float scale, float* logp, float* lse, void* stream) {
  if (T == 0) return cudaSuccess;
  return with_type(logits.dtype, [&](auto* z) {
    using E = std::remove_pointer_t<decltype(z)>;
    const int64_t row = V * static_cast<int64_t>(sizeof(E));
    const auto go = [&](auto kernel, dim3 grid, int C) {
      return launch_cluster(kernel, grid, C, kRowThreads, 0, stream, logits, T, V, tok, scale, logp, lse, C);
    };
    if (warp_rows(P, T, row)) return go(k_logprob<E, 32, false>, short_grid(P, T), 1);
    const int C = ctas_per_row(P, T, row, kLongestRead, sm_count());
    const dim3 grid(static_cast<unsigned>(T * C), static_cast<unsigned>(P));
    return go(C > 1 ? k_logprob<E, kRowThreads, true> : k_logprob<E, kRowThreads, false>, grid, C);
  });
}

int launch_token_logprob_backward(const Mat& logits, int P, int64_t T, int64_t V,
                                  const TokenArgs& tok, float scale, const float* lse,
                                  const float* dlogp, const Mat& dlogits, void* stream) {
  if (T == 0) return cudaSuccess;
  return with_type(logits.dtype, [&](auto* z) {
    using E = std::remove_pointer_t<decltype(z)>;
    if (warp_rows(P, T, V * static_cast<int64_t>(sizeof(E))))
      return launch_g(k_logprob_grad<E, 32>, short_grid(P, T), cta_of<32>, 0, stream, logits, T, V, tok, scale, lse,
                      dlogp, dlogits, 1);
    const int64_t share = int64_t{kGradThreads} * kGradVecs * Vec16<E>::N;
    int64_t parts = (V + share - 1) / share;
    if (T * parts > 0x7fffffff) parts = 1;   // a thread then loops over its vectors
    return launch_g(k_logprob_grad<E, kGradThreads>, dim3(static_cast<unsigned>(T * parts), static_cast<unsigned>(P)),
                    kGradThreads, 0, stream, logits, T, V, tok, scale, lse, dlogp, dlogits,
                    static_cast<int>(parts));
  });
}

int launch_policy_loss(const Mat& logits, int P, int64_t T, int64_t V, const TokenArgs& tok,
                       float scale, const PolicyArgs& a, float* logp, float* stats,
                       const Mat& dlogits, void* stream) {
  if (T > 0) {
    const int e = with_type(logits.dtype, [&](auto* z) {
      using E = std::remove_pointer_t<decltype(z)>;
      const int64_t row = V * static_cast<int64_t>(sizeof(E));
      const PolicyShape sh = policy_shape(P, T, row, sm_count());
      const int g = sh.group, C = sh.ctas, nt = cta_threads(g);
      const dim3 grid = g == 32 ? short_grid(P, T) : dim3(static_cast<unsigned>(T * C), static_cast<unsigned>(P));
      const auto go = [&](auto kernel) {
        return launch_cluster(kernel, grid, C, nt, static_cast<size_t>(sh.kcap) * 16 * nt, stream, logits, T,
                              V, tok, scale, a, logp, dlogits, C, sh.kcap);
      };
      if (g == 32) return go(k_policy<E, 32, false, true>);
      if (g == 128) return C > 1 ? go(k_policy<E, 128, true, true>) : go(k_policy<E, 128, false, true>);
      if (g == 256) return C > 1 ? go(k_policy<E, 256, true, true>) : go(k_policy<E, 256, false, true>);
      // longer than eight CTAs' shared memory, or than one's where T leaves no grid for more
      if (!sh.all) return go(k_policy<E, 512, true, false>);
      return C > 1 ? go(k_policy<E, 512, true, true>) : go(k_policy<E, 512, false, true>);
    });
    if (e) return e;
  }
  const int C = T > 2 * kStatThreads ? kMaxCluster : 1;
  return launch_cluster(k_policy_stats, dim3(static_cast<unsigned>(P * C)), C, kStatThreads, 0, stream, T, V, tok, a,
                        static_cast<const float*>(logp), stats, C);
}

}  // namespace dps
