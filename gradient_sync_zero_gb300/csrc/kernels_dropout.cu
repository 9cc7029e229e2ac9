// Dropout with an optional residual, over [P][T][D].
//
// Bound by HBM: a value is read (and its residual) and one is written.  The
// generator costs 20 wide multiplies and about as many logic operations for four
// values, which fit beside the loads: a thread issues the loads of its groups of
// eight values first and draws their words while they are on the way.
//
// Measured on GB300 (HBM copy 6.79 TB/s): 50.3M bf16 values with a residual 50 us (6.0
// TB/s, 0.89 of copy).  Two groups a thread took 53 us, one 59; with the counters advanced
// one after the other (each round's keys formed for each) 74 us.
#include "model.cuh"

namespace dps {
namespace {

constexpr int kDropThreads = 128;
constexpr int kDropCtas = 8;     // per SM at least: registers for kDropGroups groups, and half the warps
constexpr int kDropGroups = 4;   // groups of eight values per thread

// A thread takes kDropGroups groups of eight consecutive elements, kDropThreads
// groups apart.  D a multiple of eight and rows on 16-byte boundaries; ONE: a single
// row, so no division.
template <class TX, class TR, class TO, bool ONE>
__global__ void __launch_bounds__(kDropThreads, kDropCtas)
k_dropout_vec(Mat x, Mat res, Mat out, int64_t groups, Div8 rowdiv, DropArgs d) {
  const int r = blockIdx.y;
  wait_for_predecessor();
  const Drop drop(d, r);
  const int64_t g0 = blockIdx.x * int64_t{kDropThreads * kDropGroups} + threadIdx.x;
  Oct<TX> a[kDropGroups];
  Oct<TR> b[kDropGroups];
  int64_t g[kDropGroups], t[kDropGroups], j[kDropGroups];
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    g[u] = j[u] = g0 + u * kDropThreads;
    t[u] = 0;
    if (!ONE) rowdiv.split(g[u], t[u], j[u]);
    if (g[u] < groups) {
      a[u].load(row_ptr<TX>(x, r, t[u]) + 8 * j[u]);
      if (res.p) b[u].load(row_ptr<TR>(res, r, t[u]) + 8 * j[u]);
    }
  }
  float f[kDropGroups][8];
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) a[u].get(f[u]);
  if (d.on) drop.octs(f, g);
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    if (g[u] >= groups) break;
    if (res.p) {
      float q[8];
      b[u].get(q);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[u][k] = fmaf(f[u][k], d.inv, q[k]);
    } else if (d.on) {   // a pass-through keeps every bit
#pragma unroll
      for (int k = 0; k < 8; ++k) f[u][k] *= d.inv;
    }
    store_oct(row_ptr<TO>(out, r, t[u]) + 8 * j[u], f[u]);
  }
}

// Elements [i0, n) one by one, four (one generator call) per thread.
template <class TX, class TR, class TO>
__global__ void __launch_bounds__(kDropThreads)
k_dropout(Mat x, Mat res, Mat out, int64_t i0, int64_t n, int64_t D, DropArgs d) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const Drop drop(d, r);
  const int64_t nb = (n + 3) / 4;
  for (int64_t b = i0 / 4 + blockIdx.x * int64_t{kDropThreads} + threadIdx.x; b < nb;
       b += int64_t{gridDim.x} * kDropThreads) {
    const uint4 w = drop.words(b);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    int64_t t = 4 * b / D, j = 4 * b - t * D;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (4 * b + k >= n) break;
      float v = ld_elem(row_ptr<TX>(x, r, t) + j);
      v = d.on ? drop.keep(v, ws[k]) : v;
      v = res.p ? fmaf(v, d.inv, ld_elem(row_ptr<TR>(res, r, t) + j)) : d.on ? v * d.inv : v;
      st_elem(row_ptr<TO>(out, r, t) + j, v);
      if (++j == D) {
        j = 0;
        ++t;
      }
    }
  }
}

// Rows that follow each other without a gap are one row of T * D.
bool one_row(const Mat& m, int64_t T, int64_t D) { return !m.p || T == 1 || m.ws == D; }

}  // namespace

int64_t dropout_ctas(int64_t T, int64_t D) { return T * D / (8 * kDropThreads * kDropGroups) + 1; }

int launch_dropout(const Mat& x0, const Mat& res0, const Mat& out0, int P, int64_t T, int64_t D,
                   const DropArgs& d, void* stream) {
  if (T == 0) return cudaSuccess;
  Mat x = x0, res = res0, out = out0;
  if (one_row(x, T, D) && one_row(res, T, D) && one_row(out, T, D)) {
    D *= T;
    T = 1;
    x.ws = res.ws = out.ws = 0;
  }
  const int64_t n = T * D;
  // Vectors where every group of eight starts on a 16-byte boundary.  A single row's
  // last D mod 8 values go one by one.
  const bool vec = (T == 1 || D % 8 == 0) && oct_rows(x) && oct_rows(res) && oct_rows(out);
  const int64_t groups = vec ? n / 8 : 0, rest = n - 8 * groups;
  return with_type(x.dtype, [&](auto* tx) {
    return with_type(res.p ? res.dtype : x.dtype, [&](auto* tr) {
      return with_type(out.dtype, [&](auto* to) {
        using TX = std::remove_pointer_t<decltype(tx)>;
        using TR = std::remove_pointer_t<decltype(tr)>;
        using TO = std::remove_pointer_t<decltype(to)>;
        if (groups > 0) {
          const int64_t per = kDropThreads * kDropGroups;
          const dim3 grid(static_cast<unsigned>((groups + per - 1) / per), static_cast<unsigned>(P));
          const auto go = [&](auto kernel) {
            return launch_g(kernel, grid, kDropThreads, 0, stream, x, res, out, groups, Div8(D / 8), d);
          };
          const int e = T == 1 ? go(k_dropout_vec<TX, TR, TO, true>) : go(k_dropout_vec<TX, TR, TO, false>);
          if (e) return e;
        }
        if (rest == 0) return 0;
        const int64_t want = ((rest + 3) / 4 + kDropThreads - 1) / kDropThreads;
        return launch_g(k_dropout<TX, TR, TO>,
                        dim3(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20)), static_cast<unsigned>(P)),
                        kDropThreads, 0, stream, x, res, out, 8 * groups, n, D, d);
      });
    });
  });
}

}  // namespace dps
