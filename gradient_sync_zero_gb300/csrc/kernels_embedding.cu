// Embedding lookup and its gradient, over the replicas' embedding slots.
//
// Both are bound by HBM.  The lookup reads the rows that are named (the frequent
// ones from L2) and writes one row per token.  The gradient reads one row per
// token and writes the whole slot, most rows of which no token names.
#include "model.cuh"

namespace dps {
namespace {

// ---- lookup ----
#ifndef LG
#define LG 4
#endif
#ifndef LT
#define LT 128
#endif
#ifndef LB
#define LB 10
#endif
constexpr int kLookupThreads = LT;
constexpr int kLookupGroups = LG;   // groups of eight values per thread

// Every thread has the tokens of its groups in flight together, then the values:
// two rounds of latency for four groups.
template <class TW, class TO>
__global__ void __launch_bounds__(kLookupThreads, LB)
k_lookup_vec(Mat table, int64_t V, Div8 rowdiv, TokenArgs tok, int64_t T, float scale, DropArgs d, Mat out) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const Drop drop(d, r);
  const int64_t groups = T * rowdiv.n;
  const int64_t g0 = blockIdx.x * int64_t{kLookupThreads * kLookupGroups} + threadIdx.x;
  int64_t t[kLookupGroups], j[kLookupGroups], v[kLookupGroups];
#pragma unroll
  for (int u = 0; u < kLookupGroups; ++u) {
    const int64_t g = g0 + u * kLookupThreads;
    rowdiv.split(g, t[u], j[u]);
    v[u] = g < groups ? token_at(tok, r * T + t[u], V) : -1;
  }
  Oct<TW> a[kLookupGroups];
#pragma unroll
  for (int u = 0; u < kLookupGroups; ++u)
    if (v[u] >= 0) a[u].load_again(row_ptr<TW>(table, r, v[u]) + 8 * j[u]);
  const float factor = scale * d.inv;
#pragma unroll
  for (int u0 = 0; u0 < kLookupGroups; u0 += 2) {   // two groups' generators at a time
    float f[2][8];
    const int64_t g[2] = {g0 + u0 * kLookupThreads, g0 + (u0 + 1) * kLookupThreads};
#pragma unroll
    for (int h = 0; h < 2; ++h) a[u0 + h].get(f[h]);
    if (d.on) drop.octs(f, g);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (g[h] >= groups) break;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[h][k] = v[u0 + h] >= 0 ? f[h][k] * factor : 0.0f;
      store_oct(row_ptr<TO>(out, r, t[u0 + h]) + 8 * j[u0 + h], f[h]);
    }
  }
}

// Rows that are not on 16-byte boundaries: one CTA per row, value by value.
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
        x = ld_elem(row_ptr<TW>(table, r, v) + j);
        if (d.on) x = drop.one(x, t * D + j);
        x *= scale * d.inv;
      }
      st_elem(row_ptr<TO>(out, r, t) + j, x);
    }
  }
}

// ---- gradient ----
// 1. Each rank's (token, position) pairs are sorted by token, stably, so that the
//    tokens of a row follow each other in order of position.
// 2. The sorted pairs are cut into windows of kWindow, whatever the tokens: one CTA
//    sums the rows of dout that its window names, in fp32, run of equal tokens by run.
//    A run inside the window goes to its gradient row; one that reaches over the
//    window's end or start goes to the workspace as a partial sum.  So a token that
//    fills half the batch costs each CTA what any other does.
// 3. The window in which such a run starts adds its partial sums, in order.
// Rows that no token names are written beside step 1.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMost = 16 * kSortThreads;   // pairs that one CTA sorts
constexpr int kWindow = 32;
constexpr int kScanKeys = 1024;                // vocabulary rows per CTA of the scan
constexpr int kZeroBits = 8 * kSortWarps * 256 * 4;   // rows whose marks fit the sort's counters

// The workspace.  Pairs sorted by token: tok[P][T] (V for a token outside the
// vocabulary, so these come last), pos[P][T].  With more than one chunk of
// kSortMost positions per rank, also each chunk's own sorted pairs (ctok, cpos), the
// chunks' counts per row (cnt[P][K][V + 1]), and the rows' first places (base).
struct GradWs {
  int32_t *tok, *pos, *ctok, *cpos, *cnt, *base, *bsum;
  float* part;   // [P][windows][2][D]: a window's run from before it, and over its end
};

int64_t chunks_of(int64_t T) { return (T + kSortMost - 1) / kSortMost; }
int64_t windows_of(int64_t T) { return (T + kWindow - 1) / kWindow; }
int64_t scan_blocks(int64_t V) { return (V + 1 + kScanKeys - 1) / kScanKeys; }

int64_t lay_out(int P, int64_t T, int64_t V, int64_t D, uint8_t* ws, GradWs* w) {
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    uint8_t* p = ws + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t n = P * T, K = chunks_of(T);
  w->tok = reinterpret_cast<int32_t*>(take(4 * n));
  w->pos = reinterpret_cast<int32_t*>(take(4 * n));
  w->part = reinterpret_cast<float*>(take(8 * P * windows_of(T) * D));
  if (K > 1) {
    w->ctok = reinterpret_cast<int32_t*>(take(4 * n));
    w->cpos = reinterpret_cast<int32_t*>(take(4 * n));
    w->cnt = reinterpret_cast<int32_t*>(take(4 * P * K * (V + 1)));
    w->base = reinterpret_cast<int32_t*>(take(4 * P * (V + 1)));
    w->bsum = reinterpret_cast<int32_t*>(take(4 * P * scan_blocks(V)));
  }
  return at > 256 ? at : 256;
}

// Zeros over a row by one warp, whatever its alignment.
template <class T>
__device__ __forceinline__ void zero_row(T* p, int64_t D) {
  const int lane = threadIdx.x & 31;
  const int64_t off = ((16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15)) & 15) /
                      static_cast<int64_t>(sizeof(T));
  constexpr int64_t N = 16 / sizeof(T);
  const int64_t lead = off < D ? off : D, nv = (D - lead) / N, rest = lead + nv * N;
  if (lane < lead) st_elem(p + lane, 0.0f);
  for (int64_t k = lane; k < nv; k += 32) st_stream(p + lead + k * N, make_uint4(0, 0, 0, 0));
  if (rest + lane < D) st_elem(p + rest + lane, 0.0f);
}

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sum, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  uint32_t before = lane < warp ? warp_sum[lane] : 0, all = warp_sum[lane];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(~0u, before, o);
    all += __shfl_xor_sync(~0u, all, o);
  }
  *total = all;
  return before + s - v;
}

// Stable sort of one chunk's pairs in shared memory, eight bits a pass: each warp
// ranks its run of the positions 32 at a time (equal digits find each other with
// match), the warps' counters are summed digit by digit, and every pair moves to
// its place.  ITEMS pairs per thread stay in registers in between.
template <int ITEMS>
__device__ void sort_chunk(const TokenArgs& tok, int64_t first, int n, int64_t V, int passes, uint8_t* smem,
                           uint32_t* key, uint16_t* pos) {
  uint32_t(*hist)[256] = reinterpret_cast<uint32_t(*)[256]>(smem);
  __shared__ uint32_t warp_sum[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = warp * (ITEMS * 32) + lane;
  uint32_t k[ITEMS];
  uint32_t p[ITEMS];   // position, and the rank in the pass's upper half
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int e = e0 + 32 * i;
    const int64_t v = e < n ? token_at(tok, first + e, V) : 0;
    k[i] = e < n ? static_cast<uint32_t>(v < 0 ? V : v) : 0xffffffffu;   // what is past n sorts last
    p[i] = static_cast<uint32_t>(e);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = 8 * pass;
    for (int h = threadIdx.x; h < kSortWarps * 256; h += kSortThreads) hist[0][h] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t dg = (k[i] >> shift) & 255u;
      const uint32_t same = __match_any_sync(~0u, dg);
      const uint32_t seen = hist[warp][dg], below = __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (below == 0) hist[warp][dg] = seen + __popc(same);
      __syncwarp();
      p[i] = (p[i] & 0xffffu) | ((seen + below) << 16);
    }
    __syncthreads();
    {   // thread t: digit t / 4, eight warps' counters
      const int dg = threadIdx.x >> 2, w0 = (threadIdx.x & 3) * (kSortWarps / 4);
      uint32_t c[kSortWarps / 4], sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps / 4; ++w) sum += c[w] = hist[w0 + w][dg];
      uint32_t total;
      uint32_t at = block_exclusive(sum, warp_sum, &total);
#pragma unroll
      for (int w = 0; w < kSortWarps / 4; ++w) {
        hist[w0 + w][dg] = at;
        at += c[w];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t at = hist[warp][(k[i] >> shift) & 255u] + (p[i] >> 16);
      key[at] = k[i];
      pos[at] = static_cast<uint16_t>(p[i]);
    }
    __syncthreads();
    if (pass + 1 < passes) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        k[i] = key[e0 + 32 * i];
        p[i] = pos[e0 + 32 * i];
      }
      __syncthreads();
    }
  }
}

// CTAs [0, P * K): one chunk of one rank each.  The rest, `zeroers` per rank, write
// the rows that no token names: each marks the named ones among its rows (blocks
// of 2^log_rows, dealt round-robin) in shared memory and writes the others.
template <class TG, int ITEMS>
__global__ void __launch_bounds__(kSortThreads)
k_embedding_sort(TokenArgs tok, int P, int64_t T, int64_t V, int64_t K, int passes, GradWs w, Mat grad,
                 int64_t D, int zeroers, int log_rows) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  wait_for_predecessor();
  const int64_t sorters = P * K;
  if (blockIdx.x < sorters) {
    uint32_t* key = reinterpret_cast<uint32_t*>(sort_smem + kSortWarps * 256 * 4);
    uint16_t* pos = reinterpret_cast<uint16_t*>(key + ITEMS * kSortThreads);
    const int64_t r = blockIdx.x / K, c = blockIdx.x % K, t0 = c * kSortMost;
    const int n = static_cast<int>(T - t0 < kSortMost ? T - t0 : kSortMost);
    sort_chunk<ITEMS>(tok, r * T + t0, n, V, passes, sort_smem, key, pos);
    int32_t* to = (K > 1 ? w.ctok : w.tok) + r * T + t0;
    int32_t* po = (K > 1 ? w.cpos : w.pos) + r * T + t0;
    int32_t* cnt = K > 1 ? w.cnt + (r * K + c) * (V + 1) : nullptr;
    for (int e = threadIdx.x; e < n; e += kSortThreads) {
      const uint32_t k = key[e];
      to[e] = static_cast<int32_t>(k);
      po[e] = static_cast<int32_t>(t0 + pos[e]);
      if (K > 1) {   // the run's length, from its two ends
        if (e == 0 || key[e - 1] != k) atomicAdd(cnt + k, -e);
        if (e == n - 1 || key[e + 1] != k) atomicAdd(cnt + k, e + 1);
      }
    }
    return;
  }
  uint32_t* mark = reinterpret_cast<uint32_t*>(sort_smem);
  const unsigned z = static_cast<unsigned>(blockIdx.x - sorters), Z = static_cast<unsigned>(zeroers);
  const int r = static_cast<int>(z / Z);
  const unsigned c = z % Z;
  const int64_t nb = ((V - 1) >> log_rows) + 1;   // blocks of rows
  const int64_t rows = ((nb - c + Z - 1) / Z) << log_rows;
  for (int64_t l0 = 0; l0 < rows; l0 += kZeroBits) {
    const int64_t len = rows - l0 < kZeroBits ? rows - l0 : kZeroBits;
    for (int64_t i = threadIdx.x; i < (len + 31) / 32; i += kSortThreads) mark[i] = 0;
    __syncthreads();
    for (int64_t t = threadIdx.x; t < T; t += kSortThreads) {
      const int64_t v = token_at(tok, r * T + t, V);
      if (v < 0) continue;
      const unsigned b = static_cast<unsigned>(v >> log_rows);
      if (b % Z != c) continue;
      const int64_t l = (static_cast<int64_t>(b / Z) << log_rows) + (v & ((int64_t{1} << log_rows) - 1)) - l0;
      if (l >= 0 && l < len) atomicOr(mark + (l >> 5), 1u << (l & 31));
    }
    __syncthreads();
    for (int64_t l = threadIdx.x >> 5; l < len; l += kSortWarps) {
      const int64_t row = l0 + l;
      const int64_t v = (((row >> log_rows) * Z + c) << log_rows) + (row & ((int64_t{1} << log_rows) - 1));
      if (v < V && !((mark[l >> 5] >> (l & 31)) & 1u)) zero_row(row_ptr<TG>(grad, r, v), D);
    }
    __syncthreads();
  }
}

// ---- more than one chunk: the chunks' sorted pairs become one sorted list ----
__global__ void __launch_bounds__(kSortThreads) k_embedding_clear(int32_t* p, int64_t n) {
  wait_for_predecessor();
  for (int64_t i = blockIdx.x * int64_t{kSortThreads} + threadIdx.x; i < n; i += int64_t{gridDim.x} * kSortThreads)
    p[i] = 0;
}

// Per row: the count of the chunks before (in place of the chunk's own), the whole
// count, and the sums of kScanKeys rows.
__global__ void __launch_bounds__(kScanKeys) k_embedding_totals(GradWs w, int64_t V, int64_t K) {
  wait_for_predecessor();
  __shared__ uint32_t warp_sum[kScanKeys / 32];
  const int r = blockIdx.y;
  const int64_t v = blockIdx.x * int64_t{kScanKeys} + threadIdx.x;
  uint32_t sum = 0;
  if (v <= V) {
    int32_t* cnt = w.cnt + r * K * (V + 1) + v;
    for (int64_t k = 0; k < K; ++k) {
      const int32_t c = cnt[k * (V + 1)];
      cnt[k * (V + 1)] = static_cast<int32_t>(sum);
      sum += static_cast<uint32_t>(c);
    }
    w.base[r * (V + 1) + v] = static_cast<int32_t>(sum);
  }
  uint32_t total;
  block_exclusive(sum, warp_sum, &total);
  if (threadIdx.x == 0) w.bsum[r * gridDim.x + blockIdx.x] = static_cast<int32_t>(total);
}

// Per row: its first place in the sorted list.  Rows without a token are written.
template <class TG>
__global__ void __launch_bounds__(kScanKeys)
k_embedding_offsets(GradWs w, int64_t V, Mat grad, int64_t D, int accumulate) {
  wait_for_predecessor();
  __shared__ uint32_t warp_sum[kScanKeys / 32];
  __shared__ uint32_t warp_sum2[kScanKeys / 32];
  __shared__ uint8_t empty[kScanKeys];
  const int r = blockIdx.y;
  const int64_t v0 = blockIdx.x * int64_t{kScanKeys}, v = v0 + threadIdx.x;
  uint32_t before = 0, offset, total;
  for (int64_t b = threadIdx.x; b < blockIdx.x; b += kScanKeys) before += w.bsum[r * gridDim.x + b];
  block_exclusive(before, warp_sum, &offset);
  const uint32_t n = v <= V ? w.base[r * (V + 1) + v] : 0;
  const uint32_t at = block_exclusive(n, warp_sum2, &total) + offset;
  if (v <= V) w.base[r * (V + 1) + v] = static_cast<int32_t>(at);
  if (accumulate) return;
  empty[threadIdx.x] = v < V && n == 0;
  __syncthreads();
  for (int k = threadIdx.x >> 5; k < kScanKeys; k += kScanKeys / 32)
    if (empty[k]) zero_row(row_ptr<TG>(grad, r, v0 + k), D);
}

// Every pair of a chunk to its place: the row's first place, the chunks before, and
// the place in the chunk's own run (whose start a binary search finds).
__global__ void __launch_bounds__(kSortThreads) k_embedding_merge(GradWs w, int64_t T, int64_t V, int64_t K) {
  extern __shared__ __align__(16) uint8_t merge_smem[];
  wait_for_predecessor();
  int32_t* key = reinterpret_cast<int32_t*>(merge_smem);
  const int64_t r = blockIdx.x / K, c = blockIdx.x % K, t0 = c * kSortMost, o = r * T + t0;
  const int n = static_cast<int>(T - t0 < kSortMost ? T - t0 : kSortMost);
  for (int e = threadIdx.x; e < n; e += kSortThreads) key[e] = w.ctok[o + e];
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kSortThreads) {
    const int32_t k = key[e];
    int lo = 0, hi = e;   // the first place of k lies in [lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (key[mid] < k) lo = mid + 1; else hi = mid;
    }
    const int64_t at = int64_t{w.base[r * (V + 1) + k]} + w.cnt[(r * K + c) * (V + 1) + k] + (e - lo);
    w.tok[r * T + at] = k;
    w.pos[r * T + at] = w.cpos[o + e];
  }
}

// ---- windows ----
constexpr int kSumThreads = 256;   // at most; a thread has eight columns (one when unaligned)

// Columns j .. j+C-1 of a thread's sums.
template <class T, int C>
struct Cols {
  Oct<T> q;
  __device__ __forceinline__ void load(const T* p) { q.load(p); }
  __device__ __forceinline__ void add(float (&acc)[C], const DropArgs& d, const Drop& drop, int64_t i) const {
    float f[1][8];
    q.get(f[0]);
    const int64_t g[1] = {i >> 3};
    if (d.on) drop.octs(f, g);
#pragma unroll
    for (int k = 0; k < C; ++k) acc[k] += f[0][k];
  }
};
template <class T>
struct Cols<T, 1> {
  float x;
  __device__ __forceinline__ void load(const T* p) { x = ld_elem(p); }
  __device__ __forceinline__ void add(float (&acc)[1], const DropArgs& d, const Drop& drop, int64_t i) const {
    acc[0] += d.on ? drop.one(x, i) : x;
  }
};

template <class T, int C>
__device__ __forceinline__ void store_grad(T* p, float (&acc)[C], float scale, int accumulate) {
#pragma unroll
  for (int k = 0; k < C; ++k) acc[k] *= scale;
  if constexpr (C == 8) {
    if (accumulate) {
      Oct<T> old;
      old.load(p);
      float f[8];
      old.get(f);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += f[k];
    }
    store_oct(p, acc);
  } else {
    st_elem(p, accumulate ? acc[0] + ld_elem(p) : acc[0]);
  }
}

template <class TX, class TG, int C>
__global__ void __launch_bounds__(kSumThreads)
k_embedding_sum(GradWs w, Mat dout, int64_t T, float scale, DropArgs d, Mat grad, int64_t V, int64_t D,
                int accumulate) {
  constexpr int U = sizeof(Oct<TX>) == 16 ? 8 : 4;   // rows in flight
  __shared__ int32_t stok[kWindow + 2];   // the window's tokens, and one on either side
  __shared__ int32_t spos[kWindow];
  wait_for_predecessor();
  const int r = blockIdx.z, lane = threadIdx.x & 31;
  const int64_t a = blockIdx.x * int64_t{kWindow};
  const int len = static_cast<int>(T - a < kWindow ? T - a : kWindow);
  const int32_t* tok = w.tok + r * T;
  for (int i = threadIdx.x; i < len + 2; i += blockDim.x) {
    const int64_t k = a - 1 + i;
    stok[i] = k >= 0 && k < T ? tok[k] : -1;
  }
  for (int i = threadIdx.x; i < len; i += blockDim.x) spos[i] = w.pos[r * T + a + i];
  __syncthreads();
  const int n = __popc(__ballot_sync(~0u, lane < len && stok[1 + lane] < V));   // those named come first
  const int64_t j = (blockIdx.y * int64_t{blockDim.x} + threadIdx.x) * C;
  if (j >= D) return;
  const Drop drop(d, r);
  float* part = w.part + (r * int64_t{gridDim.x} + blockIdx.x) * 2 * D + j;
  float acc[C] = {};
  bool inner = stok[0] != stok[1];   // the run began in this window
  for (int i0 = 0; i0 < n; i0 += U) {
    Cols<TX, C> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < n) x[u].load(row_ptr<TX>(dout, r, spos[i0 + u]) + j);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      x[u].add(acc, d, drop, int64_t{spos[i]} * D + j);
      const int32_t v = stok[1 + i];
      const bool last = i + 1 == len;   // of the window
      if (!last && stok[2 + i] == v) continue;
      if (inner && !(last && stok[2 + i] == v)) {
        store_grad<TG, C>(row_ptr<TG>(grad, r, v) + j, acc, scale, accumulate);
      } else {
        float* p = part + (inner ? D : 0);
        if constexpr (C == 8) {
          store_oct(p, acc);
        } else {
          *p = acc[0];
        }
      }
#pragma unroll
      for (int k = 0; k < C; ++k) acc[k] = 0.0f;
      inner = true;
    }
  }
}

// A run over a window's end, summed by the window in which it starts.
template <class TG, int C>
__global__ void __launch_bounds__(kSumThreads)
k_embedding_join(GradWs w, int64_t T, float scale, Mat grad, int64_t V, int64_t D, int accumulate) {
  constexpr int U = 8;
  wait_for_predecessor();
  const int r = blockIdx.z, lane = threadIdx.x & 31;
  const int64_t win = blockIdx.x, a = win * kWindow, b = a + kWindow;   // never the last window
  const int32_t* tok = w.tok + r * T;
  const int32_t v = tok[b];
  if (v >= V || tok[b - 1] != v || (a > 0 && tok[a - 1] == v)) return;
  int64_t more = 1;   // windows after this one that the run reaches into
  for (;;) {
    const int64_t k = b + (more + lane) * kWindow;
    const unsigned in = __ballot_sync(~0u, k < T && tok[k] == v);
    more += in == ~0u ? 32 : __ffs(~in) - 1;
    if (in != ~0u) break;
  }
  const int64_t j = (blockIdx.y * int64_t{blockDim.x} + threadIdx.x) * C;
  if (j >= D) return;
  const float* part = w.part + (r * (gridDim.x + int64_t{1}) + win) * 2 * D + j;
  float acc[C];
  Cols<float, C> x[U];
  const DropArgs none;
  const Drop undropped(none, 0);
#pragma unroll
  for (int k = 0; k < C; ++k) acc[k] = 0.0f;
  x[0].load(part + D);
  x[0].add(acc, none, undropped, 0);
  for (int64_t m0 = 1; m0 <= more; m0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m0 + u <= more) x[u].load(part + (m0 + u) * 2 * D);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m0 + u <= more) x[u].add(acc, none, undropped, 0);
  }
  store_grad<TG, C>(row_ptr<TG>(grad, r, v) + j, acc, scale, accumulate);
}

int bits_of(int64_t v) {
  int b = 0;
  while (v >> b) ++b;
  return b;
}

}  // namespace

int launch_embedding_forward(const Mat& table, int64_t V, int64_t D, const TokenArgs& tok, int P,
                             int64_t T, float scale, const DropArgs& d, const Mat& out,
                             void* stream) {
  if (T == 0) return cudaSuccess;
  // T * D may pass 2^31 CTAs' worth of groups only past any GPU's memory; row by row then
  const int64_t per = kLookupThreads * kLookupGroups, ctas = (T * (D / 8) + per - 1) / per;
  const bool vec = D % 8 == 0 && oct_rows(table) && oct_rows(out) && ctas <= 0x7fffffff;
  return with_type(table.dtype, [&](auto* tw) {
    return with_type(out.dtype, [&](auto* to) {
      using TW = std::remove_pointer_t<decltype(tw)>;
      using TO = std::remove_pointer_t<decltype(to)>;
      if (vec)
        return launch_g(k_lookup_vec<TW, TO>, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(P)),
                        kLookupThreads, 0, stream, table, V, Div8(D / 8), tok, T, scale, d, out);
      return launch_g(k_lookup<TW, TO>,
                      dim3(static_cast<unsigned>(T < (1 << 20) ? T : (1 << 20)), static_cast<unsigned>(P)),
                      kLookupThreads, 0, stream, table, V, D, tok, T, scale, d, out);
    });
  });
}

int64_t embedding_workspace_bytes(int P, int64_t T, int64_t V, int64_t D) {
  GradWs w{};
  return lay_out(P, T, V, D, nullptr, &w);
}

int launch_embedding_backward(const Mat& dout, const TokenArgs& tok, int P, int64_t T, float scale,
                              const DropArgs& d, const Mat& grad, int64_t V, int64_t D,
                              bool accumulate, uint8_t* ws, void* stream) {
  if (T == 0 && accumulate) return cudaSuccess;
  GradWs w{};
  lay_out(P, T, V, D, ws, &w);
  scale *= d.inv;   // the sums are of kept values, unscaled
  const int64_t K = chunks_of(T), windows = windows_of(T);
  const int acc = accumulate ? 1 : 0, passes = (bits_of(V) + 7) / 8;
  const int sms = sm_count();
  return with_type(grad.dtype, [&](auto* tg) {
    using TG = std::remove_pointer_t<decltype(tg)>;
    // Rows without a token: beside the sort on the SMs that it leaves, in blocks of 4 KB at
    // least.  With several chunks the scan knows them and writes them.
    const int zeroers = accumulate || K > 1 ? 0 : (sms > 2 * P ? (sms - P) / P : 1);
    int log_rows = 0;
    while (log_rows < 12 && (D * static_cast<int64_t>(sizeof(TG)) << log_rows) < 4096) ++log_rows;
    int e = 0;
    if (K > 1) {
      const int64_t n = P * K * (V + 1);
      e = launch_g(k_embedding_clear, dim3(static_cast<unsigned>(n / kSortThreads + 1 < 4096 ? n / kSortThreads + 1 : 4096)),
                   kSortThreads, 0, stream, w.cnt, n);
      if (e) return e;
    }
    const auto sort = [&](auto kernel, int items) {
      const size_t smem = kSortWarps * 256 * 4 + static_cast<size_t>(items) * kSortThreads * 6;
      const cudaError_t ce = ensure_dyn_smem(kernel, smem);
      if (ce != cudaSuccess) return static_cast<int>(ce);
      return launch_g(kernel, dim3(static_cast<unsigned>(P * K + int64_t{P} * zeroers)), kSortThreads, smem, stream,
                      tok, P, T, V, K, passes, w, grad, D, zeroers, log_rows);
    };
    e = T <= kSortThreads       ? sort(k_embedding_sort<TG, 1>, 1)
        : T <= 4 * kSortThreads ? sort(k_embedding_sort<TG, 4>, 4)
                                : sort(k_embedding_sort<TG, 16>, 16);
    if (e || T == 0) return e;
    if (K > 1) {
      const dim3 scan(static_cast<unsigned>(scan_blocks(V)), static_cast<unsigned>(P));
      if ((e = launch_g(k_embedding_totals, scan, kScanKeys, 0, stream, w, V, K))) return e;
      if ((e = launch_g(k_embedding_offsets<TG>, scan, kScanKeys, 0, stream, w, V, grad, D, acc))) return e;
      const cudaError_t ce = ensure_dyn_smem(k_embedding_merge, 4 * kSortMost);
      if (ce != cudaSuccess) return static_cast<int>(ce);
      e = launch_g(k_embedding_merge, dim3(static_cast<unsigned>(P * K)), kSortThreads, 4 * kSortMost, stream, w, T,
                   V, K);
      if (e) return e;
    }
    return with_type(dout.dtype, [&](auto* tx) {
      using TX = std::remove_pointer_t<decltype(tx)>;
      const auto sums = [&](auto cols) {
        constexpr int C = decltype(cols)::value;
        const int64_t need = (D + C - 1) / C;
        const int nt = need < kSumThreads ? static_cast<int>((need + 31) / 32 * 32) : kSumThreads;
        const unsigned blocks = static_cast<unsigned>((need + nt - 1) / nt);
        int s = launch_g(k_embedding_sum<TX, TG, C>, dim3(static_cast<unsigned>(windows), blocks, static_cast<unsigned>(P)),
                         nt, 0, stream, w, dout, T, scale, d, grad, V, D, acc);
        if (s || windows == 1) return s;
        return launch_g(k_embedding_join<TG, C>,
                        dim3(static_cast<unsigned>(windows - 1), blocks, static_cast<unsigned>(P)), nt, 0, stream, w, T,
                        scale, grad, V, D, acc);
      };
      if (D % 8 == 0 && oct_rows(dout) && oct_rows(grad)) return sums(std::integral_constant<int, 8>{});
      return sums(std::integral_constant<int, 1>{});
    });
  });
}

}  // namespace dps
