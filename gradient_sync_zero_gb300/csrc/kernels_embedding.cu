// Embedding lookup and its gradient, over the replicas' embedding slots.
#include "model.cuh"

namespace dps {
namespace {

constexpr int kLookupThreads = 256;
constexpr int kGradThreads = 256;
constexpr int kGradCols = 1024;   // columns of one CTA, four per thread

// One CTA per row.
template <class TW, class TO>
__global__ void __launch_bounds__(kLookupThreads)
k_lookup(Mat table, int64_t V, int64_t D, TokenArgs tok, int64_t T, float scale, DropArgs d, Mat out) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const Drop drop(d, r);
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int64_t v = token_at(tok, r * T + t, V);
    for (int64_t j = threadIdx.x; j < D; j += kLookupThreads) {
      float x = 0.0f;
      if (v >= 0) {
        x = ld_elem(row_ptr<TW>(table, r, v) + j) * scale;
        if (d.on) x = drop.one(x, t * D + j);
      }
      st_elem(row_ptr<TO>(out, r, t) + j, x);
    }
  }
}

// One CTA per (rank, vocabulary row, kGradCols columns): the tokens that name the
// row are found in order, 256 positions at a time.
template <class TX, class TG>
__global__ void __launch_bounds__(kGradThreads)
k_embedding_grad(Mat dout, TokenArgs tok, int64_t T, float scale, DropArgs d, Mat grad, int64_t V,
                 int64_t D, int accumulate) {
  wait_for_predecessor();
  __shared__ int warp_n[kGradThreads / 32];
  __shared__ int64_t hit[kGradThreads];
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j0 = blockIdx.z * int64_t{kGradCols} + threadIdx.x;
  const Drop drop(d, r);
  for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
    float acc[kGradCols / kGradThreads] = {};
    bool any = false;
    for (int64_t t0 = 0; t0 < T; t0 += kGradThreads) {
      const int64_t t = t0 + threadIdx.x;
      const bool is = t < T && token_at(tok, r * T + t, V) == v;
      const unsigned m = __ballot_sync(~0u, is);
      if (lane == 0) warp_n[warp] = __popc(m);
      __syncthreads();
      int at = __popc(m & ((1u << lane) - 1u)), n = 0;
      for (int w = 0; w < kGradThreads / 32; ++w) {
        if (w < warp) at += warp_n[w];
        n += warp_n[w];
      }
      if (is) hit[at] = t;
      __syncthreads();
      for (int k = 0; k < n; ++k) {
        const int64_t th = hit[k];
#pragma unroll
        for (int c = 0; c < kGradCols / kGradThreads; ++c) {
          const int64_t j = j0 + c * kGradThreads;
          if (j >= D) break;
          const float x = ld_elem(row_ptr<TX>(dout, r, th) + j);
          acc[c] += d.on ? drop.one(x, th * D + j) : x;
        }
      }
      any |= n > 0;
      __syncthreads();
    }
    if (!any && accumulate) continue;
#pragma unroll
    for (int c = 0; c < kGradCols / kGradThreads; ++c) {
      const int64_t j = j0 + c * kGradThreads;
      if (j >= D) break;
      TG* g = row_ptr<TG>(grad, r, v) + j;
      st_elem(g, acc[c] * scale + (accumulate ? ld_elem(g) : 0.0f));
    }
  }
}

}  // namespace

int launch_embedding_forward(const Mat& table, int64_t V, int64_t D, const TokenArgs& tok, int P,
                             int64_t T, float scale, const DropArgs& d, const Mat& out,
                             void* stream) {
  if (T == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(T < (1 << 20) ? T : (1 << 20)), static_cast<unsigned>(P));
  return with_type(table.dtype, [&](auto* tw) {
    return with_type(out.dtype, [&](auto* to) {
      return launch_g(k_lookup<std::remove_pointer_t<decltype(tw)>, std::remove_pointer_t<decltype(to)>>,
                      grid, kLookupThreads, 0, stream, table, V, D, tok, T, scale, d, out);
    });
  });
}

int64_t embedding_workspace_bytes(int, int64_t, int64_t, int64_t) { return 256; }

int launch_embedding_backward(const Mat& dout, const TokenArgs& tok, int P, int64_t T, float scale,
                              const DropArgs& d, const Mat& grad, int64_t V, int64_t D,
                              bool accumulate, uint8_t*, void* stream) {
  const dim3 grid(static_cast<unsigned>(V < (1 << 20) ? V : (1 << 20)), static_cast<unsigned>(P),
                  static_cast<unsigned>((D + kGradCols - 1) / kGradCols));
  return with_type(dout.dtype, [&](auto* tx) {
    return with_type(grad.dtype, [&](auto* tg) {
      return launch_g(k_embedding_grad<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(tg)>>,
                      grid, kGradThreads, 0, stream, dout, tok, T, scale, d, grad, V, D,
                      accumulate ? 1 : 0);
    });
  });
}

}  // namespace dps
