// Batched products D = A B^T of 16-bit matrices with fp32 sums and a fused epilogue, on
// tcgen05 by pairs of CTAs.
//
// A tile of D is 256 x BN: each CTA of a pair holds 128 rows of A and BN / 2 rows of B
// in shared memory and 128 x BN sums in its tensor memory; the pair's products read both
// CTAs' halves of B, so B crosses each SM's shared memory half as often as it would for one
// CTA's tile.  K advances in blocks of 64 (one 128-byte swizzled row) through a ring of
// kStages stages that TMA fills.  One warp of each CTA copies, one of the first CTA issues
// products, eight of each CTA run the epilogue on one of two accumulators while the next
// tile's products fill the other.  The grid is persistent: as many pairs as are resident,
// each walking work units (a tile, or a part of its K) round-robin.
//
// Bound by the tensor cores: 512 cycles of them for each block of K of a 256-wide tile, in which the
// pair copies 64 KB.  On GB300 8192^3 in bf16 runs at 1840 to 1910 TFLOP/s and 4096 x 4096 x 8192 at 1850
// (cuBLAS 2000 and 2010; without the epilogue's stores 1945 and 1967), under the power cap of a
// long run less; 128-wide tiles take 300 cycles for half of the products.  What the
// products wait for is the last round of tiles and its epilogue.
//
// Either operand may be K-major (rows of K, as A[M][K] lies) or MN-major (A^T lies [K][M]): the
// tensor core reads both, so no operand is ever transposed in memory.
//
// Where tiles alone are fewer than pairs, K is cut into `splits` parts whose fp32 partial
// sums go to a buffer and are joined, in their order, by k_join with the same epilogue.
//
// The tensor cores add 16 products and the sum so far at a time, each cut off (not rounded) at 2^-25 of the
// binade of the largest, and cut the result off at 2^-23: on average up to 16 / 8 + 3 / 8 = 2.4 of a sum's last
// places, 4.8 at most.  Where the terms have one sign the sum comes out low by up to 6.6e-9 K of
// itself (measured for values in 0.5 .. 1.5: 1.9e-9 K at 4096, 4.0e-9 K at 16384; of either sign, 1e-9 K
// at 2048).  Where the result is kept in fp32 and K is long, `segs` accumulators of a tile take a part of K each
// and the epilogue adds them; a K too long for those is cut in parts.
//
// Every wait is bounded (mbar_wait_bounded).  A wait that gives up is counted in
// g_product_timeouts and told to both CTAs of the pair, whose roles leave their loops; once all
// of them have, the copies and products that either CTA started are waited for (again bounded), and
// only then is the tensor memory freed and the shared memory left.
#pragma once

#include <cuda_fp16.h>

#include <mutex>

#include "mma.cuh"
#include "model.cuh"

namespace dps {

constexpr int kProductThreads = 384;
constexpr int kTileM = 256;
constexpr int kBlockK = 64;
constexpr int kPairs = 76;             // CTA pairs of the whole GPU: 152 SMs
constexpr uint64_t kProductWaitNs = 2000000000ull;

static __device__ unsigned long long g_product_timeouts;

struct ProductArgs {
  int32_t M, N, K;
  int32_t mt, nt;          // tiles
  int32_t batch, splits, kblocks;
  int32_t a_step, b_step;  // 0: one matrix for the whole batch
  int32_t bf16;
  int32_t segs, bufs;      // accumulators of a tile, and of how many tiles at once: segs * bufs * BN columns
  int32_t per, units;      // tiles of a matrix, units in all
  float* partial;          // [splits][batch][M][N], or [splits][batch][N][M] where the epilogue swaps
};

// Element (i, j) of a warp's 32 x 32 block in shared memory: groups of four change places within the
// row by its number, so that neither rows nor columns of lanes meet a bank twice.
__device__ __forceinline__ int block_place(int i, int j) { return i * 32 + ((((j >> 2) ^ i) & 7) << 2 | (j & 3)); }
__device__ __forceinline__ float block_at(const float* block, int i, int j) { return block[block_place(i, j)]; }
__device__ __forceinline__ float4* block_four(float* block, int i, int four) {
  return reinterpret_cast<float4*>(block + i * 32 + (((four ^ i) & 7) << 2));
}

template <int BN>
struct ProductSmem {
  static constexpr int kABytes = kTileM / 2 * kBlockK * 2;
  static constexpr int kBBytes = BN / 2 * kBlockK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kTurnBytes = 8 * 32 * 32 * 4;   // eight warps' blocks
  static constexpr int kBytes = kStages * kStageBytes + kTurnBytes + 1024 /* swizzle atoms start on 1024 */ + 256 /* barriers */;
};

// 32-byte stores, on 32-byte boundaries.
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void put_f8(float* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
  st_v8(p, w);
}

__device__ __forceinline__ int cut32(int n, int by) { return (n + by - 1) / by; }

struct Tile {
  int b, i, j, split;
};

// Tiles of a symmetric D: those that touch its lower half.  Others: panels of 16 rows of tiles,
// down then across, so that the pairs at work share rows and columns in L2 (4096 x 4096 x 8192: 146 us
// in panels of 8, 141 of 16).  (32-bit divisions: the
// 64-bit ones of a tile cost the roles that wait on each other a microsecond.)
template <int BN, bool SYM>
__device__ __forceinline__ Tile unit_tile(const ProductArgs& g, int32_t u) {
  Tile t;
  uint32_t v = static_cast<uint32_t>(u);
  t.split = 0;
  if (g.splits > 1) {
    t.split = static_cast<int>(v % static_cast<uint32_t>(g.splits));
    v /= static_cast<uint32_t>(g.splits);
  }
  const uint32_t per = static_cast<uint32_t>(g.per);
  t.b = static_cast<int>(v / per);
  v -= static_cast<uint32_t>(t.b) * per;
  if (SYM) {
    constexpr int R = kTileM / BN;
    const int w = static_cast<int>(v) / R;
    int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(w) + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > w) --i;
    while ((i + 1) * (i + 2) / 2 <= w) ++i;
    t.i = i;
    t.j = static_cast<int>(v) - i * (i + 1) / 2 * R;
  } else {
    constexpr uint32_t G = 16;
    const uint32_t nt = static_cast<uint32_t>(g.nt), panel = v / (G * nt), i0 = panel * G;
    const uint32_t rows = static_cast<uint32_t>(g.mt) - i0 < G ? static_cast<uint32_t>(g.mt) - i0 : G;
    v -= i0 * nt;
    const uint32_t j = rows == G ? v / G : v / rows;
    t.i = static_cast<int>(i0 + v - j * rows);
    t.j = static_cast<int>(j);
  }
  return t;
}
// The blocks of K of a part: [first, last).
__device__ __forceinline__ int part_begin(const ProductArgs& g, int split) {
  return g.splits == 1 ? (split ? g.kblocks : 0)
                       : static_cast<int>(static_cast<uint32_t>(split) * static_cast<uint64_t>(static_cast<uint32_t>(g.kblocks)) /
                                          static_cast<uint32_t>(g.splits));
}

// Where D goes.  A warp's block of 32 x 32 sums, a row to a lane as tensor memory gives it, goes through
// shared memory so that four lanes hold a row's 32 columns, eight each: a store or load then touches
// eight rows instead of 32 (with a row to a lane the epilogue of a Newton-Schulz iterate took longer
// than the tile's products).  An epilogue has, for eight columns n .. n + 7 of row m of batch b:
//   Pre, fetch(b, m, n, pre)   the loads that apply needs, issued a block ahead (the first before the
//                              tile's sums are done), where ahead(valid) says so
//   Cols, fetch_cols(b, n, cols)   the same for what the columns alone decide
//   apply(b, m, n, v, pre, cols)   stores them, and leaves what it stored in v; called where whole(valid):
//                              the block's columns, `valid` of 32, are stored in whole vectors
//   apply_rows(b, m0, rows, n, block, lane)   otherwise: column n of rows m0 .. from block_at(block, i, lane),
//                              after before(v, pre) where kBefore
//   mirror(b, n, m, v)         where kMirror: the other half of a symmetric D, out[n][m .. m + 7]
//   join(b, m, n, v, valid)    any eight columns, of which `valid` are inside, where kJoins: K may be cut in parts
//   live()                     whether this tile is to be stored at all, where kAsks (with a shuffle of its own for
//                              every epilogue it cost a small product 0.5 us)
//   gave_up()                  is told of a wait that gave up
// and kSwap: D is the transpose of what it stores, apply_cols(b, m, n0, valid, block, lane) stores column m.
//
// A launch may hold G products of different shapes, their units one after the other: tiles of all of them
// fill the last round of each.  AMN, BMN: how the operands lie, or kAsked for each product its own.
constexpr int kAsked = 2;
template <class Epi>
struct Problem {
  CUtensorMap ta, tb;
  ProductArgs g;
  int32_t first;           // unit
  int32_t a_mn, b_mn;
  Epi epi;
};
template <class Epi, int G>
struct Problems {
  Problem<Epi> p[G];
  int32_t n, units;
  __device__ __forceinline__ const Problem<Epi>& of(int32_t u) const {
    int i = 0;
    if (G > 1)
      while (i + 1 < n && u >= p[i + 1].first) ++i;
    return p[i];
  }
};

// After a wait that gave up and a barrier of the pair: waits for the copies and products in flight.  (Out of
// line: in the kernel its instructions cost a small product 0.1 us.)
template <int STAGES>
__device__ __noinline__ void drain(int warp, uint32_t rank, uint64_t* drained, uint64_t* full, const uint32_t* copied) {
  if (warp == 1) {
    if (elect_one()) {   // the thread that issued the products
      if (rank == 0) mma_commit_pair(drained);
      mbar_wait_bounded(drained, 0);
    }
    __syncwarp();
  } else if (warp == 0 && rank == 0) {
    if (elect_one()) {   // a stage that only one CTA's copies took never fills: its wait ends by its limit
      const uint32_t it = copied[0] > copied[1] ? copied[0] : copied[1];
      for (uint32_t n = it < STAGES ? it : STAGES; n > 0; --n)
        mbar_wait_bounded(full + (it - n) % STAGES, ((it - n) / STAGES) & 1);
    }
    __syncwarp();
  }
}

template <int BN, int AMN, int BMN, bool SYM, class Epi, int G>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
k_product(const __grid_constant__ Problems<Epi, G> ps) {
  using S = ProductSmem<BN>;
  static_assert(BMN == 0 || BN >= 128, "an MN-major half of B is whole boxes of 64");
  static_assert(!SYM || kTileM % BN == 0, "mirrored blocks are whole tiles");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  float* turn = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kStages * S::kStageBytes + S::kTurnBytes);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile uint32_t* gave_up = tmem_slot + 1;   // the same in both CTAs once their roles have left
  uint32_t* copied = tmem_slot + 2;             // blocks of K that each CTA's copies took (in the first CTA)

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init_n(full + s, 1);
      mbar_init_n(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init_n(acc_full + s, 1);
      mbar_init_n(acc_empty + s, 16);   // eight warps of each CTA
    }
    mbar_init_n(drained, 1);
    *gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < (G > 1 ? ps.n : 1); ++i) {
      tma_prefetch_map(&ps.p[i].ta);
      tma_prefetch_map(&ps.p[i].tb);
    }
  }
  if (warp == 2) tmem_alloc(tmem_slot);
  tmem_fence_before();
  __syncthreads();
  cluster_sync_all();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_predecessor();

  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*gave_up == 0 && mbar_wait_bounded(bar, parity, kProductWaitNs)) return true;
    if (*gave_up == 0) {
      *gave_up = 1;
      st_cluster(peer_addr(tmem_slot + 1, rank ^ 1), 1);
      atomicAdd(&g_product_timeouts, 1ull);
      ps.p[0].epi.gave_up();
    }
    return false;
  };
  const int32_t u0 = blockIdx.x / 2, du = gridDim.x / 2;

  if (warp == 0) {
    if (elect_one()) {   // copies
      asm volatile("fence.proxy.async;" ::: "memory");   // the predecessor's plain stores, read by TMA
      uint32_t it = 0;
      bool ok = true;
      for (int32_t u = u0; u < ps.units && ok; u += du) {
        const Problem<Epi>& problem = ps.of(u);
        const ProductArgs& g = problem.g;
        const CUtensorMap &ta = problem.ta, &tb = problem.tb;
        const bool a_mn = AMN == kAsked ? problem.a_mn : AMN, b_mn = BMN == kAsked ? problem.b_mn : BMN;
        const Tile t = unit_tile<BN, SYM>(g, u - problem.first);
        const int k0 = part_begin(g, t.split), k1 = part_begin(g, t.split + 1);
        const int m = t.i * kTileM + static_cast<int>(rank) * (kTileM / 2);
        const int n = t.j * BN + static_cast<int>(rank) * (BN / 2);
        for (int k = k0; k < k1; ++k, ++it) {
          const uint32_t s = it % S::kStages;
          if (it >= S::kStages && !(ok = wait(empty + s, (it / S::kStages - 1) & 1))) break;
          uint8_t* a = smem + s * S::kStageBytes;
          uint8_t* b = a + S::kABytes;
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * S::kStageBytes);
          const uint32_t bar = peer_addr(full + s, 0);
          if (a_mn) {
#pragma unroll
            for (int h = 0; h < kTileM / 2; h += 64)
              tma_load3(a + h * 128, &ta, bar, m + h, k * kBlockK, t.b * g.a_step);
          } else {
            tma_load3(a, &ta, bar, k * kBlockK, m, t.b * g.a_step);
          }
          if (b_mn) {
#pragma unroll
            for (int h = 0; h < BN / 2; h += 64) tma_load3(b + h * 128, &tb, bar, n + h, k * kBlockK, t.b * g.b_step);
          } else {
            tma_load3(b, &tb, bar, k * kBlockK, n, t.b * g.b_step);
          }
        }
      }
      st_cluster(peer_addr(copied + rank, 0), it);
      for (uint32_t n = it < S::kStages ? it : S::kStages; n > 0 && ok; --n)   // no arrival may find this CTA gone
        ok = wait(empty + (it - n) % S::kStages, ((it - n) / S::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {   // products
      uint32_t it = 0, tile = 0;
      bool ok = true;
      for (int32_t u = u0; u < ps.units && ok; u += du, ++tile) {
        const Problem<Epi>& problem = ps.of(u);
        const ProductArgs& g = problem.g;
        const bool a_mn = AMN == kAsked ? problem.a_mn : AMN, b_mn = BMN == kAsked ? problem.b_mn : BMN;
        const uint32_t idesc = mma_idesc(g.bf16, a_mn, b_mn, kTileM, BN);
        const int split = g.splits == 1 ? 0 : (u - problem.first) % g.splits;
        const int k0 = part_begin(g, split), k1 = part_begin(g, split + 1);
        const uint32_t buf = tile % g.bufs, use = tile / g.bufs;
        uint32_t d = tmem + buf * g.segs * BN;
        if (use > 0 && !(ok = wait(acc_empty + buf, (use - 1) & 1))) break;
        tmem_fence_after();
        const int per_seg = (k1 - k0 + g.segs - 1) / g.segs;
        int start = k0;
        for (int k = k0; k < k1; ++k, ++it) {
          if (k == start + per_seg) {
            start = k;
            d += BN;
          }
          const uint32_t s = it % S::kStages;
          if (!(ok = wait(full + s, (it / S::kStages) & 1))) break;
          const uint32_t at = smem_addr(smem + s * S::kStageBytes);
          const uint64_t a = smem_desc(at, a_mn), b = smem_desc(at + S::kABytes, b_mn);
          const uint32_t da = (a_mn ? 2048 : 32) >> 4, db = (b_mn ? 2048 : 32) >> 4;
#pragma unroll
          for (int q = 0; q < kBlockK / 16; ++q)   // 16 k: 32 bytes along a row, or 16 rows of 128
            mma_pair(d, a + q * da, b + q * db, idesc, k > start || q > 0);
          mma_commit_pair(empty + s);
        }
        if (!ok) break;
        mma_commit_pair(acc_full + buf);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {   // epilogue: lanes 32 * (warp % 4) .. of the CTA's 128 rows, half of the columns
    const int quad = warp % 4, half = (warp - 4) / 4;
    uint32_t tile = 0;
    for (int32_t u = u0; u < ps.units; u += du, ++tile) {
      const Problem<Epi>& problem = ps.of(u);
      const ProductArgs& g = problem.g;
      const Epi& epi = problem.epi;
      const Tile t = unit_tile<BN, SYM>(g, u - problem.first);
      const uint32_t buf = tile % g.bufs;
      const int m0 = t.i * kTileM + static_cast<int>(rank) * (kTileM / 2) + quad * 32, m = m0 + lane;
      const int c0 = t.j * BN + half * (BN / 2);
      float* block = turn + (warp - 4) * 1024;
      const int row = lane / 4, oct = 8 * (lane % 4);   // rows row, row + 8 .. of a block
      typename Epi::Pre next[4];
      typename Epi::Cols next_cols;
      const auto fetch = [&](int n0) {
        const int valid = g.N - n0 < 32 ? g.N - n0 : 32;
        if ((Epi::kJoins && g.splits > 1) || valid <= 0 || !epi.ahead(valid)) return;
        epi.fetch_cols(t.b, n0 + oct, next_cols);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m0 + row + 8 * i < g.M) epi.fetch(t.b, m0 + row + 8 * i, n0 + oct, next[i]);
      };
      fetch(c0);
      enum { kGaveUp, kStore, kSkip };
      int state = kStore;
      if (lane == 0) {
        if (!wait(acc_full + buf, (tile / g.bufs) & 1)) state = kGaveUp;
        if constexpr (Epi::kAsks)
          if (state == kStore && !epi.live()) state = kSkip;
      }
      state = __shfl_sync(0xffffffffu, state, 0);
      if (state == kGaveUp) break;
      tmem_fence_after();
      if (state == kStore && m0 < g.M) {
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
          const int n0 = c0 + c;
          const int valid = g.N - n0 < 32 ? g.N - n0 : 32;
          if (valid <= 0) break;
          typename Epi::Pre pre[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pre[i] = next[i];
          const typename Epi::Cols cols = next_cols;
          if (c + 32 < BN / 2) fetch(n0 + 32);
          float v[32];
          const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * g.segs * BN + half * (BN / 2) + c;
          tmem_ld32(at, v);
          if (BN <= 128 && g.segs > 1) {
            const int blocks = part_begin(g, t.split + 1) - part_begin(g, t.split);
            const int used = cut32(blocks, cut32(blocks, g.segs));   // the last segments may be empty
            for (int s = 1; s < used; ++s) {
              float w[32];
              tmem_ld32(at + s * BN, w);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += w[j];
            }
          }
          if (!Epi::kJoins || g.splits == 1) {
            __syncwarp();   // the block before this one is stored
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *block_four(block, lane, j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            __syncwarp();
            if constexpr (Epi::kSwap) {
              if (m < g.M) epi.apply_cols(t.b, m, n0, valid, block, lane);
            } else {
              const bool whole = epi.whole(valid);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = row + 8 * i;
                if (m0 + r >= g.M || !(whole || Epi::kBefore)) continue;
                float4 *p = block_four(block, r, oct / 4), *q = block_four(block, r, oct / 4 + 1);
                const float4 lo = *p, hi = *q;
                float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                if (whole)
                  epi.apply(t.b, m0 + r, n0 + oct, f, pre[i], cols);
                else
                  epi.before(f, pre[i]);
                if (Epi::kMirror || !whole) {
                  *p = make_float4(f[0], f[1], f[2], f[3]);
                  *q = make_float4(f[4], f[5], f[6], f[7]);
                }
              }
              if (Epi::kMirror && t.i > n0 / kTileM) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int r = row + 8 * i;
                  if (r >= valid || m0 + oct >= g.M) continue;
                  float f[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) f[k] = block_at(block, oct + k, r);
                  epi.mirror(t.b, n0 + r, m0 + oct, f);
                }
              }
              if (!whole) {
                __syncwarp();
                if (lane < valid) epi.apply_rows(t.b, m0, g.M - m0 < 32 ? g.M - m0 : 32, n0 + lane, block, lane);
              }
            }
            continue;
          }
          if (m >= g.M) continue;
          if (Epi::kSwap) {
            float* p = g.partial + ((int64_t{t.split} * g.batch + t.b) * g.N + n0) * g.M + m;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < valid) p[int64_t{j} * g.M] = v[j];
          } else {
            float* p = g.partial + ((int64_t{t.split} * g.batch + t.b) * g.M + m) * g.N + n0;
            if (valid == 32 && g.N % 8 == 0) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) put_f8(p + j, v + j);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < valid) p[j] = v[j];
            }
          }
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_addr(acc_empty + buf, 0));
    }
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync_all();   // the other CTA's products and arrivals touch this one's memory
  if (*gave_up) {       // so do those that nobody waited for
    drain<S::kStages>(warp, rank, drained, full, copied);
    __syncthreads();
    cluster_sync_all();
  }
  tmem_fence_after();
  if (warp == 2) tmem_free(tmem);
}

// Sums the parts of each element in their order and hands eight at a time to the epilogue.
constexpr int kJoinThreads = 256;
template <class Epi>
__global__ void __launch_bounds__(kJoinThreads)
k_join(const float* partial, int rows, int cols, int batch, int splits, const Epi epi) {
  wait_for_predecessor();
  const int per = (cols + 7) / 8;
  const int64_t n = int64_t{batch} * rows * per;
  const int64_t step = int64_t{batch} * rows * cols;
  for (int64_t x = int64_t{blockIdx.x} * kJoinThreads + threadIdx.x; x < n; x += int64_t{gridDim.x} * kJoinThreads) {
    const int64_t row = x / per;
    const int n0 = static_cast<int>(x - row * per) * 8;
    const int valid = cols - n0 < 8 ? cols - n0 : 8;
    const float* p = partial + row * cols + n0;
    float v[8] = {};
    if (valid == 8 && cols % 4 == 0) {
      for (int s = 0; s < splits; ++s, p += step) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
    } else {
      for (int s = 0; s < splits; ++s, p += step)
        for (int j = 0; j < 8; ++j)
          if (j < valid) v[j] += p[j];
    }
    epi.join(static_cast<int>(row / rows), static_cast<int>(row % rows), n0, v, valid);
  }
}

// ---- host ----
// A 16-bit operand: [batch][outer][inner], inner contiguous; strides in elements, multiples of
// eight (bs 0: one matrix for the whole batch), data on a 16-byte boundary.
struct Operand {
  const void* p;
  int64_t inner, outer, stride, bs;
};

int encode_map(CUtensorMap* map, const Operand& o, int batch, bool bf16, int box_inner, int box_outer);

inline int64_t cut(int64_t n, int64_t by) { return (n + by - 1) / by; }

// Accumulators of a tile whose result is kept in fp32: 4096 of K (2.7e-5 cut off at most where all terms have one
// sign, 8e-6 measured) each, up to four.
inline int sum_segments(int64_t K) { return K <= 4096 ? 1 : K <= 8192 ? 2 : 4; }
// Parts of a K that is longer than that, or where the result is kept in 16 bits longer than 65536 (4.3e-4, a
// quarter of a bf16 rounding).
inline int least_parts(int64_t K, bool f32) { return static_cast<int>(cut(K, f32 ? 4 * 4096 : 16 * 4096)); }

// How a batch of products is cut: the width of its tiles and the parts of K, by what each way
// takes in cycles.  A block of K takes a pair 512 cycles of a tile 256 wide and 300 of a
// narrower one (A's rows cost the same: 16 tokens by 2048 x 2048 take 12.0 us whole, 9.3 in four parts); a tile's epilogue, where the next tile's products do not
// hide it, 12 a column; joining, a launch and the parts' bytes at half the copy rate.
struct ProductCut {
  int bn, splits;
};
inline double product_cycles(int bn, int splits, int64_t tiles, int64_t K, double values) {
  const double per = bn == 256 ? 512 : 300;
  const double waves = static_cast<double>(cut(tiles * splits, kPairs));
  const double join = splits > 1 ? 5000 + 8.0 * splits * values / 1750 : 0;
  return waves * static_cast<double>(cut(cut(K, kBlockK), splits)) * per + 12.0 * bn + join;
}
// tiles(bn): how many; values: of the whole result; fewest: parts that K needs whatever they take;
// whole: no more than those.
template <class Tiles>
ProductCut cut_product_of(Tiles&& tiles, int64_t K, double values, int widest, int narrowest, int fewest = 1,
                          bool whole = false) {
  ProductCut best{widest, fewest};
  double least = 1e300;
  for (int bn = widest; bn >= narrowest; bn /= 2) {
    const int64_t n = tiles(bn), blocks = cut(K, kBlockK);
    // parts of at least two blocks, as many as fill the GPU once or twice
    const int64_t most = whole || n >= kPairs ? 1 : 2 * kPairs / n < blocks / 2 ? 2 * kPairs / n : blocks / 2;
    for (int s = fewest; s == fewest || s <= most; ++s) {
      const double c = product_cycles(bn, s, n, K, values);
      if (c < 0.97 * least) {   // the wider tile and the fewer parts unless it pays
        least = c;
        best = {bn, s};
      }
    }
  }
  return best;
}

template <class K>
int resident_pairs(K kernel, int smem) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const auto key = std::make_pair(reinterpret_cast<const void*>(kernel), dev);
  std::lock_guard<std::mutex> l(mu);
  auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * kPairs);
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  cache[key] = n;
  return n;
}

// D = A B^T over the batch.  a: [M][K], or [K][M] where AMN; b likewise with N.  splits > 1
// needs `partial` (splits * batch * M * N fp32).  long_sums: the result is kept in fp32 (BN <= 128 then
// takes more accumulators for long K).
template <int BN, bool SYM, class Epi>
int fill_problem(Problem<Epi>* p, const Operand& a, bool a_mn, const Operand& b, bool b_mn, int64_t M, int64_t N, int64_t K,
                 int batch, bool bf16, int splits, float* partial, const Epi& epi, bool long_sums) {
  ProductArgs& g = p->g;
  g.M = static_cast<int32_t>(M);
  g.N = static_cast<int32_t>(N);
  g.K = static_cast<int32_t>(K);
  g.mt = static_cast<int32_t>(cut(M, kTileM));
  g.nt = static_cast<int32_t>(cut(N, BN));
  g.batch = batch;
  g.splits = splits;
  g.kblocks = static_cast<int32_t>(cut(K, kBlockK));
  g.a_step = a.bs ? 1 : 0;
  g.b_step = b.bs ? 1 : 0;
  g.bf16 = bf16;
  g.segs = BN <= 128 && long_sums ? sum_segments(cut(K, splits)) : 1;
  g.bufs = g.segs == 4 ? 1 : 2;
  const int64_t per = SYM ? int64_t{g.mt} * (g.mt + 1) / 2 * (kTileM / BN) : int64_t{g.mt} * g.nt;
  if (per * batch * splits > 0x3fff0000) return cudaErrorInvalidValue;   // room for sums, and a stride past the last
  g.per = static_cast<int32_t>(per);
  g.units = static_cast<int32_t>(per * batch * splits);
  g.partial = partial;
  p->first = 0;
  p->a_mn = a_mn;
  p->b_mn = b_mn;
  p->epi = epi;
  const int e = a_mn ? encode_map(&p->ta, a, batch, bf16, 64, kBlockK)
                     : encode_map(&p->ta, a, batch, bf16, kBlockK, kTileM / 2);
  if (e) return e;
  return b_mn ? encode_map(&p->tb, b, batch, bf16, 64, kBlockK) : encode_map(&p->tb, b, batch, bf16, kBlockK, BN / 2);
}

// The products of `ps`, whose units follow each other.
template <int BN, int AMN, int BMN, bool SYM, class Epi, int G>
int launch_problems(Problems<Epi, G>& ps, void* stream) {
  using S = ProductSmem<BN>;
  int64_t units = 0;
  for (int i = 0; i < ps.n; ++i) {
    ps.p[i].first = static_cast<int32_t>(units);
    units += ps.p[i].g.units;
    if (units > 0x7fff0000) return cudaErrorInvalidValue;
  }
  ps.units = static_cast<int32_t>(units);
  const auto kernel = k_product<BN, AMN, BMN, SYM, Epi, G>;
  const cudaError_t ce = ensure_dyn_smem(kernel, S::kBytes);
  if (ce != cudaSuccess) return static_cast<int>(ce);
  const int pairs = resident_pairs(kernel, S::kBytes);
  if (pairs <= 0) {
    const cudaError_t last = cudaGetLastError();
    return static_cast<int>(last != cudaSuccess ? last : cudaErrorLaunchOutOfResources);
  }
  const int64_t grid = 2 * (units < pairs ? units : pairs);
  return launch_g(kernel, dim3(static_cast<unsigned>(grid)), kProductThreads, S::kBytes, stream, ps);
}

template <class Epi>
int join_parts(int64_t M, int64_t N, int batch, int splits, const float* partial, const Epi& epi, void* stream) {
  const int rows = static_cast<int>(Epi::kSwap ? N : M), cols = static_cast<int>(Epi::kSwap ? M : N);
  const int64_t want = cut(int64_t{batch} * rows * cut(cols, 8), kJoinThreads);
  const typename Epi::Straight straight(epi);
  return launch_g(k_join<typename Epi::Straight>, dim3(static_cast<unsigned>(want < 4096 ? want : 4096)), kJoinThreads, 0,
                  stream, partial, rows, cols, batch, splits, straight);
}

template <int BN, bool AMN, bool BMN, bool SYM, class Epi>
int launch_product(const Operand& a, const Operand& b, int64_t M, int64_t N, int64_t K, int batch, bool bf16,
                   int splits, float* partial, const Epi& epi, void* stream, bool long_sums = false) {
  Problems<Epi, 1> ps;
  ps.n = 1;
  int e = fill_problem<BN, SYM>(ps.p, a, AMN, b, BMN, M, N, K, batch, bf16, splits, partial, epi, long_sums);
  if (!e) e = launch_problems<BN, AMN, BMN, SYM>(ps, stream);
  if (e || splits == 1) return e;
  if constexpr (!Epi::kJoins) return cudaErrorInvalidValue;
  else return join_parts(M, N, batch, splits, partial, epi, stream);
}

}  // namespace dps
