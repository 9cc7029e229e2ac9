// Embedding lookup and its gradient, over the replicas' embedding slots.
//
// Both are bound by HBM.  The lookup reads the rows that are named (the frequent
// ones from L2) and writes one row per token.  The gradient reads one row per
// token and writes the whole slot, most rows of which no token names.
//
// Measured on GB300 (HBM copy 6.79 TB/s): lookup of 8 x 8192 tokens in 50257 x 768 bf16
// 22.6 us (6.5 TB/s), with dropout 45 us; the gradient of 8 x 16384 tokens in 32000 x 2048
// bf16 259 us (6.1 TB/s).
#include "model.cuh"

namespace dps {
namespace {

// ---- lookup ----
constexpr int kLookupThreads = 128;

// A row of out is written by 2^log_lanes neighbouring threads, groups of eight values
// apart: the token is read and the rows' addresses are formed once per row.  With
// dropout the generator's instructions take the time, though no pipe is full (ALU 58%,
// multiply-add 42%, issue slots 61% busy): a thread draws for two groups at once (one at a
// time took 50 us where this takes 45) and has the next two loads in flight; without, four
// loads.  Flat groups, each with its row's division, token and addresses, took 62 us.
template <class TW, class TO, bool DROP>
__global__ void __launch_bounds__(kLookupThreads)
k_lookup_vec(Mat table, int64_t V, int groups, TokenArgs tok, int64_t T, float factor, DropArgs d, Mat out,
             int log_lanes) {
  constexpr int U = DROP ? 2 : 4;
  wait_for_predecessor();
  const int r = blockIdx.y, lanes = 1 << log_lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t t = (blockIdx.x * int64_t{kLookupThreads} + threadIdx.x) >> log_lanes;
  if (t >= T) return;
  const int64_t v = token_at(tok, r * T + t, V);
  TO* to = row_ptr<TO>(out, r, t) + 8 * lane;
  if (v < 0) {
    const float zero[8] = {};
    for (int j = lane; j < groups; j += lanes, to += 8 * lanes) store_oct(to, zero);
    return;
  }
  const TW* from = row_ptr<TW>(table, r, v) + 8 * lane;
  if constexpr (DROP) {
    const Drop drop(d, r);
    int64_t g[U];
    Oct<TW> a[U], next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      g[u] = t * groups + lane + u * lanes;
      if (lane + u * lanes < groups) a[u].load_again(from + 8 * u * lanes);
    }
    for (int j = lane; j < groups; j += U * lanes) {
      from += 8 * U * lanes;
      float f[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + (U + u) * lanes < groups) next[u].load_again(from + 8 * u * lanes);
        a[u].get(f[u]);
      }
      drop.octs(f, g);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u * lanes < groups) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[u][k] *= factor;
          store_oct(to + 8 * u * lanes, f[u]);
        }
        a[u] = next[u];
        g[u] += U * lanes;
      }
      to += 8 * U * lanes;
    }
  } else {
    for (int j = lane; j < groups; j += U * lanes) {
      Oct<TW> a[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j + u * lanes < groups) a[u].load_again(from + 8 * u * lanes);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j + u * lanes >= groups) break;
        float f[8];
        a[u].get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= factor;
        store_oct(to + 8 * u * lanes, f);
      }
      from += 8 * U * lanes;
      to += 8 * U * lanes;
    }
  }
}

// Rows that are not on 16-byte boundaries, value by value: without dropout a warp per
// row; with it a thread takes four consecutive elements of the rank (one generator call).
template <class TW, class TO>
__global__ void __launch_bounds__(kLookupThreads)
k_lookup_plain(Mat table, int64_t V, int64_t D, TokenArgs tok, int64_t T, float factor, Mat out) {
  constexpr int U = 8;
  wait_for_predecessor();
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x * int64_t{kLookupThreads / 32} + (threadIdx.x >> 5);
  if (t >= T) return;
  const int64_t v = token_at(tok, r * T + t, V);
  TO* to = row_ptr<TO>(out, r, t) + lane;
  const TW* from = v >= 0 ? row_ptr<TW>(table, r, v) + lane : nullptr;
  for (int64_t left = D - lane; left > 0; left -= 32 * U, to += 32 * U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = from && 32 * u < left ? ld_elem(from + 32 * u) : 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (32 * u < left) st_elem(to + 32 * u, from ? x[u] * factor : 0.0f);
    if (from) from += 32 * U;
  }
}

template <class TW, class TO>
__global__ void __launch_bounds__(kLookupThreads)
k_lookup(Mat table, int64_t V, Div8 rowdiv, TokenArgs tok, int64_t T, float factor, DropArgs d, Mat out) {
  wait_for_predecessor();
  const int r = blockIdx.y;
  const Drop drop(d, r);
  const int64_t D = rowdiv.n, n = T * D;
  for (int64_t i0 = 4 * (blockIdx.x * int64_t{kLookupThreads} + threadIdx.x); i0 < n;
       i0 += 4 * int64_t{gridDim.x} * kLookupThreads) {
    int64_t t[4], j[4], v[4];
    rowdiv.split(i0, t[0], j[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      const bool next = j[k - 1] + 1 == D;
      t[k] = t[k - 1] + (next ? 1 : 0);
      j[k] = next ? 0 : j[k - 1] + 1;
    }
    float x[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i0 + k < n ? token_at(tok, r * T + t[k], V) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v[k] >= 0) x[k] = ld_elem(row_ptr<TW>(table, r, v[k]) + j[k]) * factor;
    const uint4 w = drop.words(i0 >> 2);
    x[0] = drop.keep(x[0], w.x);
    x[1] = drop.keep(x[1], w.y);
    x[2] = drop.keep(x[2], w.z);
    x[3] = drop.keep(x[3], w.w);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k < n) st_elem(row_ptr<TO>(out, r, t[k]) + j[k], x[k]);
  }
}

// ---- gradient ----
// 1. Each rank's (token, position) pairs are sorted by token, stably, so that the
//    tokens of a row follow each other in order of position.
// 2. The sorted pairs are cut into windows (window_of), whatever the tokens: one CTA
//    sums the rows of dout that its window names, in fp32, run of equal tokens by run.
//    A run inside the window goes to its gradient row; one that reaches over the
//    window's end or start goes to the workspace as a partial sum.  So a token that
//    fills half the batch costs each window's sums what any other does.
// 3. The last of a run's windows to finish adds its partial sums, in their order:
//    which CTA that is changes nothing in the result.  It adds them alone: 65536 tokens of
//    768 bf16 values in 50257 rows take 112 us where the tokens are spread, 249 where one token
//    is half of them and 371 where it is all.
// (A launch of its own for the joins took 28 us where the sums take 120: most of its CTAs
// found nothing to do, and cost a wave's latency each.)
// Rows that no token names are written beside both: the last ones by the SMs that the
// sort leaves idle, as many as its time allows; the others by CTAs dealt between the
// windows', where HBM moves the mix of reads and writes faster than writes alone.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMost = 16 * kSortThreads;   // pairs that one CTA sorts
constexpr int kWindow = 32;                    // at most (a warp looks at one at a time)
constexpr int kScanKeys = 1024;                // vocabulary rows per CTA of the scan
constexpr int kZeroBits = 8 * kSortWarps * 256 * 4;   // rows whose marks fit the sort's counters

// The workspace.  Pairs sorted by token: tok[P][T] (V for a token outside the
// vocabulary, so these come last), pos[P][T].  With more than one chunk of
// kSortMost positions per rank, also each chunk's own sorted pairs (ctok, cpos), the
// chunks' counts per row (cnt[P][K][V + 1]), and the rows' first places (base).
struct GradWs {
  int32_t *tok, *pos, *ctok, *cpos, *cnt, *base, *bsum;
  float* part;   // [P][windows][2][D]: a window's run from before it, and over its end
  uint32_t* named;  // [P][words_of(V)]: a bit for each row that a token names
  uint32_t* done;   // [P][windows][column blocks]: windows finished of the run that starts there
};

int64_t chunks_of(int64_t T) { return (T + kSortMost - 1) / kSortMost; }
// Pairs per window.  Long windows have fewer partial sums (at most two rows of fp32 for
// each 32 rows read); short ones give every SM a CTA when there are few tokens, and a CTA one
// or two rounds of loads (777 tokens a rank of 131 values: 12.5 us against 20).
int window_of(int P, int64_t T) { return P * T < 8192 ? 8 : kWindow; }
int64_t windows_of(int P, int64_t T) { return (T + window_of(P, T) - 1) / window_of(P, T); }
__host__ __device__ inline int64_t words_of(int64_t V) { return (V + 31) / 32; }
int64_t scan_blocks(int64_t V) { return (V + 1 + kScanKeys - 1) / kScanKeys; }

// Columns per thread: eight, or four (value by value) where rows are not on 16-byte
// boundaries.
constexpr int kSumThreads = 256;   // at most
int col_threads(int64_t D, int C) {
  const int64_t need = (D + C - 1) / C;
  return need < kSumThreads ? static_cast<int>((need + 31) / 32 * 32) : kSumThreads;
}
int64_t col_blocks(int64_t D, int C) {
  const int64_t per = int64_t{col_threads(D, C)} * C;
  return (D + per - 1) / per;
}

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
  w->part = reinterpret_cast<float*>(take(8 * P * windows_of(P, T) * D));
  w->named = reinterpret_cast<uint32_t*>(take(4 * P * words_of(V)));
  w->done = reinterpret_cast<uint32_t*>(take(4 * P * windows_of(P, T) * col_blocks(D, 4)));   // the most
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

// A row on 16-byte boundaries that is shorter than a warp's store.
template <class T>
__host__ __device__ inline bool short_row(int64_t D, bool vec) {
  return vec && D * static_cast<int64_t>(sizeof(T)) < 512;
}

// Zeros in those of 32 rows from v0 on whose bit is not set, by `n` threads.  Short rows
// go as one run of vectors, others a warp each.
template <class T>
__device__ __forceinline__ void zero_rows(const Mat& grad, int r, int64_t v0, int64_t V, uint32_t named, int64_t D,
                                          bool vec, int tid, int n) {
  if (short_row<T>(D, vec)) {
    const unsigned per = static_cast<unsigned>(D * static_cast<int64_t>(sizeof(T)) / 16);
    for (unsigned i = tid; i < 32 * per; i += n) {
      const unsigned k = i / per, j = i - k * per;
      if (v0 + k < V && !((named >> k) & 1u))
        st_stream(row_ptr<T>(grad, r, v0 + k) + j * (16 / sizeof(T)), make_uint4(0, 0, 0, 0));
    }
    return;
  }
  for (int k = tid >> 5; k < 32; k += n >> 5)
    if (v0 + k < V && !((named >> k) & 1u)) zero_row(row_ptr<T>(grad, r, v0 + k), D);
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
// ranks its run of the positions 32 at a time, the warps' counters are summed digit
// by digit, and every pair moves to its place.  ITEMS pairs per thread stay in registers in between.
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
      // The lanes with this digit: by turns from match and from ballots, bit by bit, which
      // different units execute (all match 39 us for 16384 pairs, all ballots 34).
      uint32_t same = ~0u;
      if (i & 1) {
        same = __match_any_sync(~0u, dg);
      } else {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const uint32_t set = __ballot_sync(~0u, (dg >> b) & 1u);
          same &= (dg >> b) & 1u ? set : ~set;
        }
      }
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
      if (!DP_IN_BOUNDS(at < ITEMS * kSortThreads)) continue;
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

// Zeros in the rows [v0, V) that no token names, by `Z` CTAs of which this is the c-th: it
// takes every Z-th block of 2^log_rows rows, marks the named ones in shared memory
// and writes the others.
template <class TG>
__device__ void zero_unnamed(const TokenArgs& tok, int r, int64_t T, int64_t V, int64_t v0, unsigned c, unsigned Z,
                             int log_rows, uint32_t* mark, const Mat& grad, int64_t D, bool vec) {
  const int64_t nb = (V - v0 + (int64_t{1} << log_rows) - 1) >> log_rows;
  const int64_t rows = ((nb - c + Z - 1) / Z) << log_rows, in_block = (int64_t{1} << log_rows) - 1;
  for (int64_t l0 = 0; l0 < rows; l0 += kZeroBits) {
    const int64_t len = rows - l0 < kZeroBits ? rows - l0 : kZeroBits;
    for (int64_t i = threadIdx.x; i < (len + 31) / 32; i += kSortThreads) mark[i] = 0;
    __syncthreads();
    for (int64_t t = threadIdx.x; t < T; t += kSortThreads) {
      const int64_t v = token_at(tok, r * T + t, V) - v0;
      if (v < 0) continue;
      const unsigned b = static_cast<unsigned>(v >> log_rows);
      if (b % Z != c) continue;
      const int64_t l = (static_cast<int64_t>(b / Z) << log_rows) + (v & in_block) - l0;
      if (l >= 0 && l < len) atomicOr(mark + (l >> 5), 1u << (l & 31));
    }
    __syncthreads();
    const auto row_of = [&](int64_t l) {
      const int64_t row = l0 + l;
      return v0 + (((row >> log_rows) * Z + c) << log_rows) + (row & in_block);
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (short_row<TG>(D, vec)) {   // blocks of 32 rows at least
      for (int64_t l = 32 * warp; l < len; l += 32 * kSortWarps)
        zero_rows<TG>(grad, r, row_of(l), V, mark[l >> 5], D, vec, lane, 32);
    } else {
      for (int64_t l = warp; l < len; l += kSortWarps)
        if (row_of(l) < V && !((mark[l >> 5] >> (l & 31)) & 1u)) zero_row(row_ptr<TG>(grad, r, row_of(l)), D);
    }
    __syncthreads();
  }
}

// One CTA per chunk of a rank; then, `zeroers` per rank, those of zero_unnamed.
template <class TG, int ITEMS>
__global__ void __launch_bounds__(kSortThreads)
k_embedding_sort(TokenArgs tok, int P, int64_t T, int64_t V, int64_t K, int passes, GradWs w, int W, int64_t windows,
                 int64_t ny, Mat grad, int64_t D, bool vec, int64_t v0, int zeroers, int log_rows) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  wait_for_predecessor();
  if (blockIdx.x >= P * K) {
    const unsigned z = static_cast<unsigned>(blockIdx.x - P * K), Z = static_cast<unsigned>(zeroers);
    zero_unnamed<TG>(tok, static_cast<int>(z / Z), T, V, v0, z % Z, Z, log_rows,
                     reinterpret_cast<uint32_t*>(sort_smem), grad, D, vec);
    return;
  }
  uint32_t* key = reinterpret_cast<uint32_t*>(sort_smem + kSortWarps * 256 * 4);
  uint16_t* pos = reinterpret_cast<uint16_t*>(key + ITEMS * kSortThreads);
  const int64_t r = blockIdx.x / K, c = blockIdx.x % K, t0 = c * kSortMost;
  const int n = static_cast<int>(T - t0 < kSortMost ? T - t0 : kSortMost);
  const int64_t win0 = t0 / W, wins = (n + W - 1) / W;
  uint32_t* named = w.named + r * words_of(V);
  if (K == 1)   // with more, k_embedding_clear has
    for (int64_t i = threadIdx.x; i < words_of(V); i += kSortThreads) named[i] = 0;
  for (int64_t i = threadIdx.x; i < wins * ny; i += kSortThreads) w.done[(r * windows + win0) * ny + i] = 0;
  sort_chunk<ITEMS>(tok, r * T + t0, n, V, passes, sort_smem, key, pos);
  int32_t* to = (K > 1 ? w.ctok : w.tok) + r * T + t0;
  int32_t* po = (K > 1 ? w.cpos : w.pos) + r * T + t0;
  int32_t* cnt = K > 1 ? w.cnt + (r * K + c) * (V + 1) : nullptr;
  for (int e = threadIdx.x; e < n; e += kSortThreads) {
    const uint32_t k = key[e];
    to[e] = static_cast<int32_t>(k);
    po[e] = static_cast<int32_t>(t0 + pos[e]);
    const bool head = e == 0 || key[e - 1] != k;
    if (head && k < V) atomicOr(named + (k >> 5), 1u << (k & 31));
    if (K > 1) {   // the run's length, from its two ends
      if (head) atomicAdd(cnt + k, -e);
      if (e == n - 1 || key[e + 1] != k) atomicAdd(cnt + k, e + 1);
    }
  }
}

// ---- more than one chunk: the chunks' sorted pairs become one sorted list ----
__global__ void __launch_bounds__(kSortThreads)
k_embedding_clear(int32_t* cnt, int64_t n, uint32_t* named, int64_t words) {
  wait_for_predecessor();
  const int64_t i0 = blockIdx.x * int64_t{kSortThreads} + threadIdx.x, step = int64_t{gridDim.x} * kSortThreads;
  for (int64_t i = i0; i < n; i += step) cnt[i] = 0;
  for (int64_t i = i0; i < words; i += step) named[i] = 0;
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

// Per row: its first place in the sorted list.
__global__ void __launch_bounds__(kScanKeys) k_embedding_offsets(GradWs w, int64_t V) {
  wait_for_predecessor();
  __shared__ uint32_t warp_sum[kScanKeys / 32];
  __shared__ uint32_t warp_sum2[kScanKeys / 32];
  const int r = blockIdx.y;
  const int64_t v = blockIdx.x * int64_t{kScanKeys} + threadIdx.x;
  uint32_t before = 0, offset, total;
  for (int64_t b = threadIdx.x; b < blockIdx.x; b += kScanKeys) before += w.bsum[r * gridDim.x + b];
  block_exclusive(before, warp_sum, &offset);
  const uint32_t n = v <= V ? w.base[r * (V + 1) + v] : 0;
  const uint32_t at = block_exclusive(n, warp_sum2, &total) + offset;
  if (v <= V) w.base[r * (V + 1) + v] = static_cast<int32_t>(at);
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
    if (!DP_IN_BOUNDS(at >= 0 && at < T)) continue;
    w.tok[r * T + at] = k;
    w.pos[r * T + at] = w.cpos[o + e];
  }
}

// ---- windows ----
// Columns j .. j+C-1 of a thread's sums: C = 8 as vectors; C = 4 value by value, of which
// the row has `n`.
template <class T, int C>
struct Cols {
  Oct<T> q;
  __device__ __forceinline__ void load(const T* p, int) { q.load(p); }
  template <bool DROP>
  __device__ __forceinline__ void add(float (&acc)[C], const Drop& drop, int64_t i) const {
    float f[1][8];
    q.get(f[0]);
    const int64_t g[1] = {i >> 3};
    if (DROP) drop.octs(f, g);
#pragma unroll
    for (int k = 0; k < C; ++k) acc[k] += f[0][k];
  }
};
template <class T>
struct Cols<T, 4> {
  float x[4];
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = k < n ? ld_elem(p + k) : 0.0f;
  }
  template <bool DROP>
  __device__ __forceinline__ void add(float (&acc)[4], const Drop& drop, int64_t i) const {
    if (DROP) {   // the four elements lie in two of the generator's blocks, at most
      uint4 c[2] = {drop.counter(static_cast<uint64_t>(i) >> 2), drop.counter((static_cast<uint64_t>(i) >> 2) + 1)};
      philox4(c, drop.k0, drop.k1);
      const int at = static_cast<int>(i & 3);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = at + k;
        const uint4 w = e < 4 ? c[0] : c[1];
        acc[k] += drop.keep(x[k], (e & 3) == 0 ? w.x : (e & 3) == 1 ? w.y : (e & 3) == 2 ? w.z : w.w);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += x[k];
    }
  }
};

// Partial sums; another SM may have written them, so they are read past the L1.
template <int C>
struct PartCols {
  float x[C];
  __device__ __forceinline__ void load(const float* p, int n) {
    if constexpr (C == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 q = __ldcg(reinterpret_cast<const float4*>(p) + h);
        x[4 * h] = q.x;
        x[4 * h + 1] = q.y;
        x[4 * h + 2] = q.z;
        x[4 * h + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) x[k] = k < n ? __ldcg(p + k) : 0.0f;
    }
  }
  __device__ __forceinline__ void add(float (&acc)[C]) const {
#pragma unroll
    for (int k = 0; k < C; ++k) acc[k] += x[k];
  }
};
template <int C>
__device__ __forceinline__ void store_part(float* p, const float (&acc)[C], int n) {
  if constexpr (C == 8) {
    store_oct(p, acc);
  } else {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < n) p[k] = acc[k];
  }
}

template <class T, int C>
__device__ __forceinline__ void store_grad(T* p, float (&acc)[C], int n, float scale, int accumulate) {
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
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k < n) st_elem(p + k, accumulate ? acc[k] + ld_elem(p + k) : acc[k]);
  }
}

// Of the run of v that window `win` is in: its first and last windows.  Looks at the
// windows' first tokens, 32 windows at a time.
__device__ __forceinline__ void run_windows(const int32_t* tok, int64_t T, int W, int64_t win, int32_t v,
                                            int64_t& first, int64_t& last) {
  const int lane = threadIdx.x & 31;
  last = win;
  for (;;) {
    const int64_t k = (last + 1 + lane) * W;
    const unsigned in = __ballot_sync(~0u, k < T && tok[k] == v);
    last += in == ~0u ? 32 : __ffs(~in) - 1;
    if (in != ~0u) break;
  }
  first = win;   // the first of the windows before that begin with v, and the one before it
  if (tok[win * W] != v) return;   // if v reaches back into it
  for (;;) {
    const int64_t k = (first - 1 - lane) * W;
    const unsigned in = __ballot_sync(~0u, k >= 0 && tok[k] == v);
    first -= in == ~0u ? 32 : __ffs(~in) - 1;
    if (in != ~0u) break;
  }
  if (first > 0 && tok[first * W - 1] == v) --first;
}

// This CTA's share of a run's partial sums is written: the last CTA to say so adds them.
template <class TG, int C>
__device__ __forceinline__ void finish_run(const GradWs& w, const int32_t* tok, int64_t T, int W, int64_t win,
                                           int32_t v, int64_t windows, int64_t ny, int col, int r, int64_t j, int64_t D, const Mat& grad, float scale,
                                           int accumulate, uint32_t* ticket) {
  constexpr int U = C == 8 ? 4 : 8;   // partial sums in flight
  int64_t first, last;
  run_windows(tok, T, W, win, v, first, last);
  __syncthreads();
  if (threadIdx.x == 0) {
    // release: the CTA's partial sums (ordered before by the barrier); acquire: the others'
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(before)
                 : "l"(w.done + (r * windows + first) * ny + col)
                 : "memory");
    *ticket = before;
  }
  __syncthreads();
  if (*ticket != static_cast<uint32_t>(last - first) || j >= D) return;
  if (!DP_IN_BOUNDS(first >= 0 && first < last && last < windows)) return;
  const float* part = w.part + (r * windows + first) * 2 * D + j;
  const int more = static_cast<int>(last - first);
  const int cols = D - j < C ? static_cast<int>(D - j) : C;
  float acc[C] = {};
  PartCols<C> x[U];
  x[0].load(part + D, cols);
  x[0].add(acc);
  for (int m0 = 1; m0 <= more; m0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m0 + u <= more) x[u].load(part + (m0 + u) * 2 * D, cols);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m0 + u <= more) x[u].add(acc);
  }
  store_grad<TG, C>(row_ptr<TG>(grad, r, v) + j, acc, cols, scale, accumulate);
}

template <class TX, class TG, int C, bool DROP>
__global__ void __launch_bounds__(kSumThreads, DROP ? 3 : 4)
k_embedding_sum(GradWs w, Mat dout, int64_t T, float scale, DropArgs d, Mat grad, int64_t V, int64_t D,
                int accumulate, int W, int64_t windows, int64_t ny, int64_t v0, int64_t zeroers,
                int zero_words) {
  constexpr int U = sizeof(Oct<TX>) == 16 ? 8 : 4;   // rows in flight
  __shared__ int32_t stok[kWindow + 2];   // the window's tokens, and one on either side
  __shared__ int32_t spos[kWindow];
  __shared__ uint32_t ticket;
  wait_for_predecessor();
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  // The rank's CTAs: windows * ny of sums and `zeroers` of rows that no token names,
  // dealt evenly.
  const int64_t sums = windows * ny, all = sums + zeroers;
  const int64_t mine = blockIdx.x * sums / all;
  if ((blockIdx.x + int64_t{1}) * sums / all == mine) {
    for (int64_t word = (blockIdx.x - mine) * zero_words; word < (blockIdx.x - mine + 1) * zero_words; ++word)
      if (word * 32 < v0)
        zero_rows<TG>(grad, r, word * 32, v0, w.named[r * words_of(V) + word], D, C == 8, threadIdx.x, blockDim.x);
    return;
  }
  const int64_t win = mine / ny, a = win * W;
  const int col = static_cast<int>(mine - win * ny);
  const int len = static_cast<int>(T - a < W ? T - a : W);
  const int32_t* tok = w.tok + r * T;
  for (int i = threadIdx.x; i < len + 2; i += blockDim.x) {
    const int64_t k = a - 1 + i;
    stok[i] = k >= 0 && k < T ? tok[k] : -1;
  }
  for (int i = threadIdx.x; i < len; i += blockDim.x) {
    const int32_t p = w.pos[r * T + a + i];
    spos[i] = DP_IN_BOUNDS(p >= 0 && p < T && tok[a + i] >= 0 && tok[a + i] <= V) ? p : 0;
  }
  __syncthreads();
  const int n = __popc(__ballot_sync(~0u, lane < len && stok[1 + lane] < V));   // those named come first
  if (n == 0) return;
  const int64_t j = (col * int64_t{blockDim.x} + threadIdx.x) * C;
  if (j < D) {
    const Drop drop(d, r);
    const int cols = D - j < C ? static_cast<int>(D - j) : C;
    float* part = w.part + (r * windows + win) * 2 * D + j;
    float acc[C] = {};
    bool inner = stok[0] != stok[1];   // the run began in this window
    for (int i0 = 0; i0 < n; i0 += U) {
      Cols<TX, C> x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < n) x[u].load(row_ptr<TX>(dout, r, spos[i0 + u]) + j, cols);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        if (i >= n) break;
        x[u].template add<DROP>(acc, drop, int64_t{spos[i]} * D + j);
        const int32_t v = stok[1 + i];
        const bool last = i + 1 == len;   // of the window
        if (!last && stok[2 + i] == v) continue;
        if (inner && !(last && stok[2 + i] == v)) {
          store_grad<TG, C>(row_ptr<TG>(grad, r, v) + j, acc, cols, scale, accumulate);
        } else {
          store_part<C>(part + (inner ? D : 0), acc, cols);
        }
#pragma unroll
        for (int k = 0; k < C; ++k) acc[k] = 0.0f;
        inner = true;
      }
    }
  }
  // the run from before the window, and another one over its end
  const int32_t lead = stok[1], tail = stok[len];
  const bool before = stok[0] == lead, after = n == len && stok[len + 1] == tail;
  if (before) finish_run<TG, C>(w, tok, T, W, win, lead, windows, ny, col, r, j, D, grad, scale, accumulate, &ticket);
  if (after && !(before && tail == lead)) {
    __syncthreads();   // the ticket is free again
    finish_run<TG, C>(w, tok, T, W, win, tail, windows, ny, col, r, j, D, grad, scale, accumulate, &ticket);
  }
}

int bits_of(int64_t v) {
  int b = 0;
  while (v >> b) ++b;
  return b;
}

}  // namespace

int64_t bounds_violations_embedding(bool reset) {
#ifdef DPSYNC_CHECKED
  unsigned long long n = 0;
  if (cudaMemcpyFromSymbol(&n, g_bounds_violations, sizeof n) != cudaSuccess) return -2;
  if (reset) {
    const unsigned long long z = 0;
    if (cudaMemcpyToSymbol(g_bounds_violations, &z, sizeof z) != cudaSuccess) return -2;
  }
  return static_cast<int64_t>(n);
#else
  (void)reset;
  return -1;
#endif
}

int launch_embedding_forward(const Mat& table, int64_t V, int64_t D, const TokenArgs& tok, int P,
                             int64_t T, float scale, const DropArgs& d, const Mat& out,
                             void* stream) {
  if (T == 0) return cudaSuccess;
  const bool vec = D % 8 == 0 && oct_rows(table) && oct_rows(out);
  const int groups = static_cast<int>(D / 8);
  int log_lanes = 0;   // a warp per row, or the part of one that a short row fills
  while (log_lanes < 5 && (2 << log_lanes) <= groups) ++log_lanes;
  if (log_lanes == 5 && d.on && (groups + 31) / 32 % 2) --log_lanes;   // an even number of groups each
  const int64_t rows = kLookupThreads >> log_lanes;
  const float factor = scale * d.inv;
  return with_type(table.dtype, [&](auto* tw) {
    return with_type(out.dtype, [&](auto* to) {
      using TW = std::remove_pointer_t<decltype(tw)>;
      using TO = std::remove_pointer_t<decltype(to)>;
      if (vec)
        return launch_g(d.on ? k_lookup_vec<TW, TO, true> : k_lookup_vec<TW, TO, false>,
                        dim3(static_cast<unsigned>((T + rows - 1) / rows), static_cast<unsigned>(P)), kLookupThreads, 0,
                        stream, table, V, groups, tok, T, factor, d, out, log_lanes);
      if (!d.on)
        return launch_g(k_lookup_plain<TW, TO>, dim3(static_cast<unsigned>((T + 3) / 4), static_cast<unsigned>(P)),
                        kLookupThreads, 0, stream, table, V, D, tok, T, factor, out);
      const int64_t want = (T * D + 4 * kLookupThreads - 1) / (4 * kLookupThreads);
      return launch_g(k_lookup<TW, TO>,
                      dim3(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20)), static_cast<unsigned>(P)),
                      kLookupThreads, 0, stream, table, V, Div8(D), tok, T, factor, d, out);
    });
  });
}

int64_t embedding_workspace_bytes(int P, int64_t T, int64_t V, int64_t D) {
  GradWs w{};
  return lay_out(P, T, V, D, nullptr, &w);
}

int64_t embedding_backward_ctas(int P, int64_t T, int64_t V, int64_t D) {
  return windows_of(P, T) * col_blocks(D, 4) + words_of(V);
}

int launch_embedding_backward(const Mat& dout, const TokenArgs& tok, int P, int64_t T, float scale,
                              const DropArgs& d, const Mat& grad, int64_t V, int64_t D,
                              bool accumulate, uint8_t* ws, void* stream) {
  if (T == 0 && accumulate) return cudaSuccess;
  GradWs w{};
  lay_out(P, T, V, D, ws, &w);
  scale *= d.inv;   // the sums are of kept values, unscaled
  const int W = window_of(P, T), passes = (bits_of(V) + 7) / 8;
  const int64_t K = chunks_of(T), windows = windows_of(P, T);
  const bool vec = D % 8 == 0 && oct_rows(dout) && oct_rows(grad);
  const int nt = col_threads(D, vec ? 8 : 4);
  const int64_t ny = col_blocks(D, vec ? 8 : 4);
  // Rows [v0, V) are written beside the sort: what the SMs without a CTA of it write, at
  // 5.5 MB a microsecond, while it takes 4 us and 1.8 more for each 1024 positions.
  const int64_t row = D * esize(grad.dtype), sms = sm_count();
  int zeroers = 0, log_rows = 0;
  int64_t v0 = V;
  if (!accumulate && K == 1 && sms >= 2 * P) {
    zeroers = static_cast<int>((sms - P) / P);
    const double time = 4.0 + 1.8 * static_cast<double>((T + kSortThreads - 1) / kSortThreads);
    const double rows = 5.5e6 * time / (static_cast<double>(P) * static_cast<double>(row));
    v0 = rows >= static_cast<double>(V) ? 0 : (V - static_cast<int64_t>(rows)) / 32 * 32;
    while (log_rows < 12 && (row << log_rows) < 4096) ++log_rows;   // blocks of 4 KB at least
    if (vec && row < 512 && log_rows < 5) log_rows = 5;
  }
  int e = 0;
  if (K != 1) {
    const int64_t n = P * K * (V + 1), words = P * words_of(V), want = (n > words ? n : words) / kSortThreads + 1;
    e = launch_k(k_embedding_clear, static_cast<int>(want < 4096 ? want : 4096), kSortThreads, 0, stream, w.cnt, n,
                 w.named, words);
    if (e) return e;
  }
  if (K > 0) {
    const auto sort = [&](auto kernel, int items) {
      const size_t smem = kSortWarps * 256 * 4 + static_cast<size_t>(items) * kSortThreads * 6;
      const cudaError_t ce = smem > 48 * 1024 ? ensure_dyn_smem(kernel, smem) : cudaSuccess;
      if (ce != cudaSuccess) return static_cast<int>(ce);
      return launch_k(kernel, static_cast<int>(P * (K + zeroers)), kSortThreads, smem, stream, tok, P, T, V, K, passes,
                      w, W, windows, ny, grad, D, vec, v0, zeroers, log_rows);
    };
    e = with_type(grad.dtype, [&](auto* tg) {
      using TG = std::remove_pointer_t<decltype(tg)>;
      return T <= kSortThreads       ? sort(k_embedding_sort<TG, 1>, 1)
             : T <= 4 * kSortThreads ? sort(k_embedding_sort<TG, 4>, 4)
                                     : sort(k_embedding_sort<TG, 16>, 16);
    });
    if (e) return e;
  }
  if (K > 1) {
    const dim3 scan(static_cast<unsigned>(scan_blocks(V)), static_cast<unsigned>(P));
    if ((e = launch_g(k_embedding_totals, scan, kScanKeys, 0, stream, w, V, K))) return e;
    if ((e = launch_g(k_embedding_offsets, scan, kScanKeys, 0, stream, w, V))) return e;
    const cudaError_t ce = ensure_dyn_smem(k_embedding_merge, 4 * kSortMost);
    if (ce != cudaSuccess) return static_cast<int>(ce);
    e = launch_k(k_embedding_merge, static_cast<int>(P * K), kSortThreads, 4 * kSortMost, stream, w, T, V, K);
    if (e) return e;
  }
  // CTAs of at least 16 KB of rows [0, v0)
  const int zero_words = row * 32 >= 16384 ? 1 : static_cast<int>(16384 / (row * 32));
  const int64_t writers = accumulate ? 0 : (words_of(v0) + zero_words - 1) / zero_words;
  const dim3 grid(static_cast<unsigned>(windows * ny + writers), static_cast<unsigned>(P));
  return with_type(dout.dtype, [&](auto* tx) {
    return with_type(grad.dtype, [&](auto* tg) {
      using TX = std::remove_pointer_t<decltype(tx)>;
      using TG = std::remove_pointer_t<decltype(tg)>;
      const auto kernel = d.on ? (vec ? k_embedding_sum<TX, TG, 8, true> : k_embedding_sum<TX, TG, 4, true>)
                               : (vec ? k_embedding_sum<TX, TG, 8, false> : k_embedding_sum<TX, TG, 4, false>);
      return launch_g(kernel, grid, nt, 0, stream, w, dout, T, scale, d, grad, V, D, accumulate ? 1 : 0, W, windows, ny,
                      v0, writers, zero_words);
    });
  });
}

}  // namespace dps
