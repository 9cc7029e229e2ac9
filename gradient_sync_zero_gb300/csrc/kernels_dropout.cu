// Dropout with an optional residual, over [P][T][D].
#include "model.cuh"

namespace dps {
namespace {

constexpr int kDropThreads = 256;

// One thread per four consecutive elements (one generator call).
template <class TX, class TR, class TO>
__global__ void __launch_bounds__(kDropThreads)
k_dropout(Mat x, Mat res, Mat out, int64_t n, int64_t D, DropArgs d) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const Drop drop(d, r);
  const int64_t nb = (n + 3) / 4;
  for (int64_t b = blockIdx.x * int64_t{kDropThreads} + threadIdx.x; b < nb;
       b += int64_t{gridDim.x} * kDropThreads) {
    const uint4 w = drop.words(b);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = 4 * b + k;
      if (i >= n) break;
      const int64_t t = i / D, j = i - t * D;
      float v = ld_elem(row_ptr<TX>(x, r, t) + j);
      v = d.on ? drop.apply(v, ws[k]) : v;
      if (res.p) v += ld_elem(row_ptr<TR>(res, r, t) + j);
      st_elem(row_ptr<TO>(out, r, t) + j, v);
    }
  }
}

}  // namespace

int launch_dropout(const Mat& x, const Mat& res, const Mat& out, int P, int64_t T, int64_t D,
                   const DropArgs& d, void* stream) {
  const int64_t n = T * D;
  if (n == 0) return cudaSuccess;
  const int64_t nb = (n + 3) / 4, want = (nb + kDropThreads - 1) / kDropThreads;
  const dim3 grid(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20)), static_cast<unsigned>(P));
  return with_type(x.dtype, [&](auto* tx) {
    return with_type(res.p ? res.dtype : x.dtype, [&](auto* tr) {
      return with_type(out.dtype, [&](auto* to) {
        return launch_g(k_dropout<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(tr)>,
                                  std::remove_pointer_t<decltype(to)>>,
                        grid, kDropThreads, 0, stream, x, res, out, n, D, d);
      });
    });
  });
}

}  // namespace dps
