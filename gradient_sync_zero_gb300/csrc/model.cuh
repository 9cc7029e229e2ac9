// Device-side building blocks of the operators at the ends of a training step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include <type_traits>

#include "launch.cuh"
#include "model.h"

namespace dps {

// The kernels are launched as programmatic dependents of the previous kernel in
// their stream: no global memory is touched before this returns.
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16-byte accesses of data that is used once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.cs.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
// ... that other CTAs may read too.
__device__ __forceinline__ uint4 ld_again(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void st_stream(void* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// The token of row i, or -1 where it is outside [0, V).
__device__ __forceinline__ int64_t token_at(const TokenArgs& t, int64_t i, int64_t V) {
  const int64_t k = t.wide ? static_cast<const int64_t*>(t.p)[i]
                           : static_cast<int64_t>(static_cast<const int32_t*>(t.p)[i]);
  return k >= 0 && k < V ? k : -1;
}

// Philox4x32-10 (Salmon, Moraes, Dror & Shaw, SC 2011): ten rounds of two 32 x 32
// -> 64 bit products, each round's key one Weyl step further.  M counters advance
// together, so that a round's key is formed once and their chains of dependent
// products overlap.
template <int M>
__device__ __forceinline__ void philox4(uint4 (&c)[M], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint64_t a = static_cast<uint64_t>(c[m].x) * 0xD2511F53u;
      const uint64_t b = static_cast<uint64_t>(c[m].z) * 0xCD9E8D57u;
      c[m] = make_uint4(static_cast<uint32_t>(b >> 32) ^ c[m].y ^ k0, static_cast<uint32_t>(b),
                        static_cast<uint32_t>(a >> 32) ^ c[m].w ^ k1, static_cast<uint32_t>(a));
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// What a kernel needs to draw: the key, and the two counter words that do not
// depend on the element.  Values are only selected here; the factor 1 / (1 - p)
// goes into the multiplication that the kernel has anyway.
struct Drop {
  uint32_t k0, k1, c2, c3, last;

  __device__ __forceinline__ Drop(const DropArgs& d, int rank)
      : c2(d.rank0 + static_cast<uint32_t>(rank)), last(d.last) {
    uint64_t seed = d.seed;
    c3 = d.offset;
    if (d.dev) {
      seed = d.dev[0];
      c3 = static_cast<uint32_t>(d.dev[1]);
    }
    k0 = static_cast<uint32_t>(seed);
    k1 = static_cast<uint32_t>(seed >> 32);
  }
  __device__ __forceinline__ uint4 counter(uint64_t b) const {
    return make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32), c2, c3);
  }
  // A dropped value is 0 whatever it was (an infinity or NaN too).
  __device__ __forceinline__ float keep(float x, uint32_t word) const { return word > last ? x : 0.0f; }
  // The four words of elements 4b .. 4b+3 of this rank.
  __device__ __forceinline__ uint4 words(uint64_t b) const {
    uint4 c[1] = {counter(b)};
    philox4(c, k0, k1);
    return c[0];
  }
  // Elements 8 g[u] .. 8 g[u] + 7, for U groups.
  template <int U>
  __device__ __forceinline__ void octs(float (&f)[U][8], const int64_t (&g)[U]) const {
    uint4 c[2 * U];
#pragma unroll
    for (int h = 0; h < 2 * U; ++h) c[h] = counter(2 * static_cast<uint64_t>(g[h / 2]) + (h & 1));
    philox4(c, k0, k1);
#pragma unroll
    for (int h = 0; h < 2 * U; ++h) {
      float* q = f[h / 2] + 4 * (h & 1);
      q[0] = keep(q[0], c[h].x);
      q[1] = keep(q[1], c[h].y);
      q[2] = keep(q[2], c[h].z);
      q[3] = keep(q[3], c[h].w);
    }
  }
};

// Eight consecutive values: 16 bytes of bf16, 32 of fp32.
template <class T>
struct Oct;
template <>
struct Oct<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = ld_stream(p); }
  __device__ __forceinline__ void load_again(const __nv_bfloat16* p) { q = ld_again(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Oct<float> {
  uint4 q[2];
  __device__ __forceinline__ void load(const float* p) {
    q[0] = ld_stream(p);
    q[1] = ld_stream(p + 4);
  }
  __device__ __forceinline__ void load_again(const float* p) {
    q[0] = ld_again(p);
    q[1] = ld_again(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(q[i].x);
      f[4 * i + 1] = __uint_as_float(q[i].y);
      f[4 * i + 2] = __uint_as_float(q[i].z);
      f[4 * i + 3] = __uint_as_float(q[i].w);
    }
  }
};
__device__ __forceinline__ void store_oct(__nv_bfloat16* p, const float (&f)[8]) {
  st_stream(p, make_uint4(pack2_rne(f[0], f[1]), pack2_rne(f[2], f[3]), pack2_rne(f[4], f[5]),
                          pack2_rne(f[6], f[7])));
}
__device__ __forceinline__ void store_oct(float* p, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    st_stream(p + 4 * i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                    __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
}

// Every row of m starts on a 16-byte boundary (host; an absent matrix does).
inline bool oct_rows(const Mat& m) {
  const int64_t es = esize(m.dtype);
  return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.rs * es % 16 == 0 && m.ws * es % 16 == 0);
}

// g / n and g mod n for group numbers.  Those below 2^32 (nearly always) divide in
// 32 bits, a third of the instructions of the 64-bit division.
struct Div8 {
  int64_t n;
  explicit Div8(int64_t n_) : n(n_) {}
  __device__ __forceinline__ void split(int64_t g, int64_t& q, int64_t& r) const {
    if ((static_cast<uint64_t>(g) | static_cast<uint64_t>(n)) >> 32) {
      q = g / n;
      r = g - q * n;
    } else {
      const uint32_t a = static_cast<uint32_t>(g), b = static_cast<uint32_t>(n), k = a / b;
      q = k;
      r = a - k * b;
    }
  }
};

template <class T>
__device__ __forceinline__ T* row_ptr(const Mat& m, int r, int64_t i) {
  return reinterpret_cast<T*>(m.p) + (r * m.rs + i * m.ws);
}

// launch_k for grids of more than one dimension.
template <class K, class... A>
int launch_g(K kernel, dim3 grid, int threads, size_t smem, void* stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  const cudaError_t last = cudaGetLastError();
  return static_cast<int>(e != cudaSuccess ? e : last);
}

// Calls f with a null pointer of the element type: with_type(t, [&](auto* z) { ... }).
template <class F>
inline int with_type(int32_t dtype, F&& f) {
  return dtype == DP_BF16 ? f(static_cast<__nv_bfloat16*>(nullptr)) : f(static_cast<float*>(nullptr));
}

}  // namespace dps
