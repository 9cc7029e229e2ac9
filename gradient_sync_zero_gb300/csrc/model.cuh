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

// The token of row i, or -1 where it is outside [0, V).
__device__ __forceinline__ int64_t token_at(const TokenArgs& t, int64_t i, int64_t V) {
  const int64_t k = t.wide ? static_cast<const int64_t*>(t.p)[i]
                           : static_cast<int64_t>(static_cast<const int32_t*>(t.p)[i]);
  return k >= 0 && k < V ? k : -1;
}

// Philox4x32-10 (Salmon, Moraes, Dror & Shaw, SC 2011): ten rounds of two 32 x 32
// -> 64 bit products, each round's key one Weyl step further.
__device__ __forceinline__ uint4 philox4(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// What a kernel needs to draw: the key, and the two counter words that do not
// depend on the element.
struct Drop {
  uint32_t k0, k1, c2, c3, thr;
  float inv;   // 1 / (1 - p)
  bool all;

  __device__ __forceinline__ Drop(const DropArgs& d, int rank)
      : c2(d.rank0 + static_cast<uint32_t>(rank)), thr(d.thr), inv(d.inv), all(d.all != 0) {
    uint64_t seed = d.seed;
    c3 = d.offset;
    if (d.dev) {
      seed = d.dev[0];
      c3 = static_cast<uint32_t>(d.dev[1]);
    }
    k0 = static_cast<uint32_t>(seed);
    k1 = static_cast<uint32_t>(seed >> 32);
  }
  // The four words of elements 4b .. 4b+3 of this rank.
  __device__ __forceinline__ uint4 words(uint64_t b) const {
    return philox4(make_uint4(static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32), c2, c3), k0,
                   k1);
  }
  // A dropped value is 0 whatever it was (an infinity or NaN too).
  __device__ __forceinline__ float apply(float x, uint32_t word) const {
    return word >= thr && !all ? x * inv : 0.0f;
  }
  __device__ __forceinline__ float one(float x, uint64_t i) const {
    const uint4 w = words(i >> 2);
    const uint32_t k = static_cast<uint32_t>(i) & 3u;
    return apply(x, k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w);
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
