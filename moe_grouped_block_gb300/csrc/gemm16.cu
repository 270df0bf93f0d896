// gemm16.cu -- grouped products with 16-bit operands (bf16 or fp16):
//   fprop  C[off_g+i, n] = alpha_g * sum_k A[off_g+i, k] B[g, n, k] + beta_g * C
//   dgrad  C[off_g+i, k] = alpha_g * sum_n A[off_g+i, n] B[g, n, k] + beta_g * C
//   wgrad  C[g, n, k]    = alpha_g * sum_{i in g} A[off_g+i, n] B[off_g+i, k] + beta_g * C
// Group g owns rows off_g .. off_g + M_g - 1 (any M_g >= 0, read on the device).
//
// Every mode is C = R Q^T with R giving the rows of C (the operand A of the
// interface) and Q its columns (B).  A 2-CTA cluster computes units of up to
// 256 rows times 256 columns with the cta_group::2 MMA, transposed: Q is the
// MMA's 256-row operand (128 rows a CTA) and R its other one, whose width is
// any multiple of 32.  So the ragged side costs multiples of 32 rows, not of
// the tile -- with 64 groups of some 500 rows, whole 256-row tiles computed
// 1.7 times the rows there are -- a few rows are one narrow MMA beside the
// weights' stream, and an accumulator lane is a column of C, so that a warp
// stores 32 neighbouring columns of a row at any alignment of C.
//
// Warp 0 loads (TMA), warp 1 of the even CTA issues the MMAs, warps 2-9 are
// the epilogue.  Two 256-column accumulators fill tensor memory, so that the
// epilogue of a unit runs under the MMAs of the next one.  The clusters are
// persistent and walk the units in a static order derived from the group
// sizes on the device.
//
// Where there are few units and a long contraction, clusters of 4 or 8 CTAs take
// one unit each and their pairs a part of its contraction.  They join the parts
// in shared memory, each pair adding and storing some of the rows.
//
// Neither operand is transposed in memory: where the contraction runs along
// rows (Q of dgrad, both of wgrad) the tile is loaded as 64-row boxes of 64
// columns and the MMA reads it MN-major.
//
// What bounds it.  With a few rows, the weights' bytes: 16 rows through 7 of 8
// experts of 14336 x 4096, 126 us at 6.5 TB/s of the 6.78 that a copy reaches.
// With many, the tensor cores and the power they draw: 16384 rows through 8 such
// experts in 1.03 ms when run for milliseconds (1.87 PFLOP/s; the tensor pipe is
// active 92 % of the time), in 1.19 ms when run for seconds, at 1.4 kW and some
// 1.4 GHz.  dgrad of 32768 rows over 63 experts of 1408 x 2048: 138-150 us, 158-162
// us when run for seconds; its narrower units (210 rows on average) cost 509 cycles
// a K block where 420 multiply.  wgrad of the 8 experts into fp32: 1.16 ms, 600 cycles
// a K block against 494 without the 1.9 GB it stores: with both operands MN-major,
// stores and operand reads meet in shared memory.
//
// Contraction tails.  Past N or K the copies fill zeros (for the weights the
// tensor map has the expert as its third dimension, so that a box never runs
// into the next expert).  Only wgrad's contraction ends at a device-side
// number: the rows of the next group that share the last 16-row MMA step are
// zeroed in shared memory, in both operands (a zero against a NaN would not
// be zero), by warp 10 while earlier stages are multiplied.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

struct Gemm16Params {
  const int64_t* group_ws;
  const float* alpha;
  const float* beta;
  void* C;
  int32_t* status;
  int64_t ldc;
  int32_t M_cap, N, K;
  int32_t out_cols;  // columns of C: N for fprop, K for dgrad and wgrad
  int32_t G;
  int32_t out_type;     // mxg_dtype_t
  uint32_t idesc;       // operand types and majors, M = 256; N is added per unit
  int32_t tile_rows;    // rows of C per unit: a multiple of 32, at most 256
  int32_t tile_cols;    // columns of C per unit: 256 or 128
  int32_t col_units;    // units side by side
  uint32_t w_shape;     // unit_shape of dW's rows
  int32_t stages;       // pipeline stages, ...
  int32_t q_bytes;      // ... each half the unit's columns of Q ...
  int32_t stage_bytes;  // ... and half its rows of R
  int32_t splits;       // pairs of CTAs that share a unit's contraction: 1, 2 or 4
};

// The rows of a group (or of dW_g) in units of equal shares: a narrow last unit
// would stream its weights for few products.  `tiles` of them, `share` rows each, a
// multiple of 32; packed into a word.
__host__ __device__ __forceinline__ uint32_t unit_shape(uint32_t rows, uint32_t tile_rows) {
  const uint32_t tiles = (rows + tile_rows - 1) / tile_rows;
  const uint32_t share = tiles == 0 ? 0 : ((rows + tiles - 1) / tiles + 31) / 32;  // <= 8
  return tiles << 4 | share;
}

// Row offsets of the groups, the shape of their units and their first ones, by
// one warp: negative sizes count as 0 and rows past M_cap are dropped, so that no
// access leaves the operands.  A unit is a share of a group's rows times one of
// `col_units` column ranges.  32-bit sums that stop at one row past the capacity:
// with 64-bit ones and divisions a call took 0.5 us longer.
__device__ __forceinline__ void group_tables16(const int64_t* group_ws, int G, uint32_t M_cap,
                                               uint32_t tile_rows, uint32_t col_units,
                                               int32_t* row_off, int32_t* unit_off,
                                               uint32_t* shape, int32_t* status) {
  const uint32_t lane = lane_id(), most = M_cap + 1;
  uint32_t carry_rows = 0, carry_units = 0;
  bool neg = false, over = false;
  for (int base = 0; base < G; base += 32) {
    const int g = base + static_cast<int>(lane);
    const int64_t size = g < G ? group_ws[g] : 0;
    neg |= size < 0;
    const uint32_t s = size < 0 ? 0u : size > M_cap ? most : static_cast<uint32_t>(size);
    uint32_t incl = s;  // all terms are at most `most`, which is below 2^31 + 1
    auto add = [&](uint32_t a, uint32_t b) { return a > most - b ? most : a + b; };
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl = add(incl, u);
    }
    incl = add(incl, carry_rows);
    uint32_t excl = __shfl_up_sync(0xFFFFFFFFu, incl, 1);
    if (lane == 0) excl = carry_rows;
    const uint32_t before = min(excl, M_cap), after = min(incl, M_cap);
    over |= incl > M_cap && s > 0;
    const uint32_t word = unit_shape(after - before, tile_rows);
    uint32_t units = (word >> 4) * col_units;
    const uint32_t own = units;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, units, d);
      if (lane >= d) units += u;
    }
    if (g < G) {
      row_off[g] = static_cast<int32_t>(before);
      unit_off[g] = static_cast<int32_t>(carry_units + units - own);
      shape[g] = word;
    }
    carry_rows = __shfl_sync(0xFFFFFFFFu, incl, 31);
    carry_units += __shfl_sync(0xFFFFFFFFu, units, 31);
  }
  if (lane == 0) {
    row_off[G] = static_cast<int32_t>(min(carry_rows, M_cap));
    unit_off[G] = static_cast<int32_t>(carry_units);
  }
  neg = __any_sync(0xFFFFFFFFu, neg);
  over = __any_sync(0xFFFFFFFFu, over);
  if ((neg || over) && lane == 0 && blockIdx.x == 0)
    status_set(status, (neg ? MXG_DEV_NEG_SIZE : 0) | (over ? MXG_DEV_SUM_OVER_CAPACITY : 0));
}

// Work unit u: `rows` rows of C from i0 on, p.tile_cols columns from j0 on.
struct Unit16 {
  int32_t g;
  int32_t row0;   // first row of the group in the ragged operands
  int32_t i0, j0; // first row (within the group, or of dW_g) and column of C
  int32_t rows;   // rows of the unit
  int32_t n_mma;  // the same, rounded up to 32: the MMAs' width
  int32_t k0;     // this pair's share of the contraction: its start ...
  int32_t kdim;   // ... and length
};

template <int MODE, bool SPLIT>
__device__ __forceinline__ Unit16 map_unit16(int64_t u, const Gemm16Params& p,
                                             const int32_t* row_off, const int32_t* unit_off,
                                             const uint32_t* shape, int32_t pair) {
  Unit16 t;
  const uint32_t cu = static_cast<uint32_t>(p.col_units);
  uint32_t i, j, word;
  int32_t total;  // rows of C in this group
  if constexpr (MODE == 1) {
    word = p.w_shape;
    const uint32_t per = (word >> 4) * cu;
    t.g = static_cast<int32_t>(static_cast<uint32_t>(u) / per);
    const uint32_t local = static_cast<uint32_t>(u) - t.g * per;
    i = local / cu;
    j = local - i * cu;
    total = p.N;
    t.row0 = row_off[t.g];
    t.kdim = row_off[t.g + 1] - t.row0;
  } else {
    int lo = 0, hi = p.G;  // largest g with unit_off[g] <= u: halving, then 32 at once
    while (hi - lo > 32) {
      const int mid = (lo + hi) >> 1;
      if (unit_off[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    const int at = lo + static_cast<int>(lane_id());
    lo += __popc(__ballot_sync(0xFFFFFFFFu, at < hi && unit_off[min(at, p.G)] <= u)) - 1;
    t.g = lo;
    t.row0 = row_off[lo];
    t.kdim = MODE == 0 ? p.K : p.N;
    total = row_off[lo + 1] - t.row0;
    word = shape[lo];
    const uint32_t tiles = word >> 4;
    const uint32_t local = static_cast<uint32_t>(u) - unit_off[lo];
    // column unit, then row unit, so that the clusters in flight share weight
    // tiles and the group's rows stay in L2; where those rows are more than an
    // L2 budget, blocks of column units that fit it, each walked row unit by
    // row unit
    j = local / tiles;
    i = local - j * tiles;
    constexpr int64_t kL2Budget = 32ll << 20;
    if (static_cast<int64_t>(total) * t.kdim * 2 > kL2Budget) {
      int64_t cb = kL2Budget / (static_cast<int64_t>(p.tile_cols) * t.kdim * 2);
      cb = cb < 1 ? 1 : (cb > cu ? cu : cb);
      const uint32_t b = static_cast<uint32_t>(cb), blk = local / (tiles * b);
      const uint32_t width = (blk + 1) * b <= cu ? b : cu - blk * b;
      const uint32_t rem = local - blk * tiles * b;
      i = rem / width;
      j = blk * b + (rem - i * width);
    }
  }
  const int32_t share = static_cast<int32_t>(word & 15u) * 32;
  t.i0 = static_cast<int32_t>(i) * share;
  t.j0 = static_cast<int32_t>(j) * p.tile_cols;
  t.rows = max(0, min(share, total - t.i0));
  t.n_mma = max(32, (t.rows + 31) & ~31);
  t.k0 = 0;
  if constexpr (SPLIT) {  // whole K blocks each
    const int32_t blocks = (t.kdim + 63) / 64;
    t.k0 = blocks * pair / p.splits * 64;
    t.kdim = min(t.kdim, blocks * (pair + 1) / p.splits * 64) - t.k0;
  }
  return t;
}

// One column (of this lane) and up to 32 rows of C: alpha * acc + beta * old.
// The whole chunk without beta is straight-line code: with its two tests per
// row in the way, a 256 x 256 unit's epilogue took 10 k cycles, as long as the
// MMAs of a 1408-long contraction.  With beta each row waits for its old value in
// turn: wgrad of 16384 rows, 8 experts of 14336 x 4096, into fp32 takes 1.09 ms
// without beta and 6.5 ms with it.
template <typename T>
__device__ __forceinline__ void store_column16(T* dst, int64_t ldc, const float (&acc)[32],
                                               int rows, float alpha, float beta) {
  if (rows >= 32 && beta == 0.0f) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      *dst = from_f32<T>(alpha * acc[e]);
      dst += ldc;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    if (e < rows) {
      float v = alpha * acc[e];
      if (beta != 0.0f) v += beta * to_f32(*dst);
      *dst = from_f32<T>(v);
    }
    dst += ldc;
  }
}

// Bounded wait used only while tearing down: ignores the abort flag.
__device__ __forceinline__ void drain16(uint32_t bar, uint32_t parity, int32_t* status) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitTimeoutNs) {
      status_set(status, MXG_DEV_TIMEOUT);
      return;
    }
  }
}

struct Pair16 {
  static constexpr int kMaxStages = 12;
  static constexpr int kBK = 64;                 // contraction elements per stage
  static constexpr int kMmas = kBK / 16;
  static constexpr int kEpiWarps = 8;
  static constexpr int kMaskWarp = 2 + kEpiWarps;
  static constexpr int threads(int mode) { return 32 * (kMaskWarp + (mode == 1 ? 1 : 0)); }
  // full[S], empty[S], land[S], odd_masked[S], tfull[2], tempty[2],
  // info_full[2], info_empty[2], drain; two unit words; TMEM base, abort flag
  static constexpr int kBars = 4 * kMaxStages + 9;
  static constexpr int kBarBytes = 8 * (kBars + 2) + 16;
  // the barriers and tables lie before the stages
  static constexpr int kSmemMax = 227 * 1024;
  static int header_bytes(int G) { return (kBarBytes + 12 * (G + 1) + 1023) / 1024 * 1024; }
};

// Descriptor of a K-major tile (rows of 128 bytes, 128-byte swizzle), or of an
// MN-major one: chunks of 64 rows of 128 bytes (64 values along M or N a row),
// 8192 bytes apart, 8-row groups 1024 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc16(uint32_t saddr) {
  return MN ? smem_desc(saddr, 8192, 1024, 2) : smem_desc(saddr, 16, 1024, 2);
}
// 16 elements further along the contraction, in descriptor units of 16 bytes
template <bool MN>
constexpr uint32_t kStep16 = MN ? 2048 / 16 : 32 / 16;

// SEG: K blocks that are summed in tensor memory at a time, 0 for all of them.
// The tensor cores add to an accumulator by truncation, so a sum over k elements
// comes out some 0.7 k / 16 2^-24 too small (measured: 9e-6 over 8192, 3.8e-5 over
// 32768): nothing beside the rounding of a 16-bit output, but more than an fp32
// one should lose.  For those the epilogue warps take the accumulator over after
// every SEG blocks and add it up in registers, rounding to nearest: 4.9e-7 over
// 32768 with 8 blocks (512 elements).  wgrad of 8 experts of 14336 x 4096, 16381
// rows, into fp32: 1156 us so, 1160 us without; with 6 blocks 1204 us, with 4,
// where the MMAs catch up with the epilogue's stores, 1269 us.
template <int MODE, int SEG, bool SPLIT>
__global__ void __launch_bounds__(Pair16::threads(MODE), 1)
    gemm16_pair_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_r, const Gemm16Params p) {
  using Cfg = Pair16;
  constexpr int S = Cfg::kMaxStages, BK = Cfg::kBK;
  constexpr bool Q_MN = MODE != 0, R_MN = MODE == 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint64_t* info_word = bars + Cfg::kBars;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(info_word + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_s + 1);
  int32_t* row_off = reinterpret_cast<int32_t*>(smem + Cfg::kBarBytes);
  int32_t* unit_off = row_off + (p.G + 1);
  uint32_t* shape = reinterpret_cast<uint32_t*>(unit_off + (p.G + 1));

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t stage0 = smem_u32(smem) + ((Cfg::kBarBytes + 12 * (p.G + 1) + 1023) & ~1023);
  const uint32_t stages = p.stages, stage_bytes = p.stage_bytes, q_bytes = p.q_bytes;
  // of a pair, its place in the pair and the cluster's rank of its even CTA
  const uint32_t rank = cluster_ctarank() & 1u, even = SPLIT ? cluster_ctarank() & ~1u : 0u;
  const int32_t pair = static_cast<int32_t>(even >> 1);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto full_bar = [&](int s) { return bar(s); };
  auto empty_bar = [&](int s) { return bar(S + s); };
  auto land_bar = [&](int s) { return bar(2 * S + s); };
  auto odd_bar = [&](int s) { return bar(3 * S + s); };
  auto tfull_bar = [&](int a) { return bar(4 * S + a); };
  auto tempty_bar = [&](int a) { return bar(4 * S + 2 + a); };
  auto info_full_bar = [&](int i) { return bar(4 * S + 4 + i); };
  auto info_empty_bar = [&](int i) { return bar(4 * S + 6 + i); };
  const uint32_t drain_bar = bar(4 * S + 8);

  // ------------------------------------------------------------ set-up
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);   // even CTA: its producer's (or mask warp's) arrival + bytes
      mbar_init(empty_bar(s), 1);  // the pair's MMA commit
      mbar_init(land_bar(s), 1);   // a masked stage: this CTA's own bytes
      mbar_init(odd_bar(s), 1);    // even CTA: the odd CTA has masked its part
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * Cfg::kEpiWarps);  // even CTA: both CTAs' epilogue warps
      mbar_init(info_full_bar(i), 1);
      mbar_init(info_empty_bar(i), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(tmem_base_s), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_r);
  }
  __syncwarp();
  cluster_arrive();  // the barriers are there for the cluster's other CTAs
  // from here on memory is read: what came before on the stream is done
  grid_launch_dependents();
  grid_wait_for_previous();
  if (warp == 1)
    group_tables16(p.group_ws, p.G, static_cast<uint32_t>(p.M_cap),
                   static_cast<uint32_t>(p.tile_rows), static_cast<uint32_t>(p.col_units), row_off,
                   unit_off, shape, p.status);
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the even CTA's barriers exist before the odd CTA's copies signal them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_s;
  const uint32_t cluster_ctas = SPLIT ? 2 * static_cast<uint32_t>(p.splits) : 2u;
  const int64_t unit0 = blockIdx.x / cluster_ctas, ustride = gridDim.x / cluster_ctas;
  const int64_t total =
      MODE == 1 ? static_cast<int64_t>(p.G) * (p.w_shape >> 4) * p.col_units
                : unit_off[p.G];

  // ------------------------------------------------------------ producers (both CTAs)
  if (warp == 0) {
    const uint32_t leader = elect_leader();
    uint32_t stage = 0, phase = 0, issued = 0, parity = 0, tail_issued = 0, tail_parity = 0;
    // MN-major: a second chunk of 64
    const bool two_q = q_bytes > 8192, two_r = stage_bytes - q_bytes > 8192;
    bool ok = true;
    for (int64_t u = unit0, n = 0; ok && u < total; u += ustride, ++n) {
      const Unit16 t = map_unit16<MODE, SPLIT>(u, p, row_off, unit_off, shape, pair);
      const int32_t kb_count = (t.kdim + BK - 1) / BK;
      const int32_t last = t.kdim - (kb_count - 1) * BK;  // elements of the last block
      if (rank == 0) {
        // the unit's shape, for the MMA warp
        const int slot = static_cast<int>(n & 1), par = static_cast<int>((n >> 1) & 1);
        if (!mbar_wait_warp(info_empty_bar(slot), par ^ 1, abort_flag, p.status)) break;
        if (leader)
          info_word[slot] = static_cast<uint64_t>(static_cast<uint32_t>(kb_count)) |
                            (static_cast<uint64_t>((last + 15) / 16) << 32) |
                            (static_cast<uint64_t>(t.n_mma) << 40);
        mbar_arrive_if(info_full_bar(slot), leader);
      }
      const int32_t q_at = t.j0 + p.tile_cols / 2 * static_cast<int32_t>(rank);
      const int32_t r_at = t.i0 + (t.n_mma / 2) * static_cast<int32_t>(rank);
      for (int32_t kb = 0; kb < kb_count; ++kb) {
        if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const uint32_t sq = stage0 + stage * stage_bytes, sr = sq + q_bytes;
        const int32_t k0 = t.k0 + kb * BK;
        if (MODE == 1 && kb + 1 == kb_count && (last & 15) != 0) {
          // rows of the next group in the last MMA step: this CTA's bytes
          // land on its own barrier, and its mask warp passes them on
          const uint32_t lb = land_bar(stage);
          mbar_arrive_expect_tx_if(lb, stage_bytes, leader);
          tma_load_2d_if(sq, &tmap_q, lb, q_at, t.row0 + k0, leader);
          if (two_q) tma_load_2d_if(sq + 8192, &tmap_q, lb, q_at + 64, t.row0 + k0, leader);
          tma_load_2d_if(sr, &tmap_r, lb, r_at, t.row0 + k0, leader);
          if (two_r) tma_load_2d_if(sr + 8192, &tmap_r, lb, r_at + 64, t.row0 + k0, leader);
          tail_issued |= 1u << stage;
          tail_parity ^= 1u << stage;
        } else {
          if (rank == 0) mbar_arrive_expect_tx_if(full_bar(stage), 2 * stage_bytes, leader);
          const uint32_t fb = mapa_shared(full_bar(stage), even);
          if constexpr (MODE == 0) {
            tma_load_3d_pair_if(sq, &tmap_q, fb, k0, q_at, t.g, leader);
          } else if constexpr (MODE == 2) {
            tma_load_3d_pair_if(sq, &tmap_q, fb, q_at, k0, t.g, leader);
            if (two_q) tma_load_3d_pair_if(sq + 8192, &tmap_q, fb, q_at + 64, k0, t.g, leader);
          } else {
            tma_load_2d_pair_if(sq, &tmap_q, fb, q_at, t.row0 + k0, leader);
            if (two_q)
              tma_load_2d_pair_if(sq + 8192, &tmap_q, fb, q_at + 64, t.row0 + k0, leader);
          }
          if constexpr (MODE == 1) {
            tma_load_2d_pair_if(sr, &tmap_r, fb, r_at, t.row0 + k0, leader);
            if (two_r) tma_load_2d_pair_if(sr + 8192, &tmap_r, fb, r_at + 64, t.row0 + k0, leader);
          } else {
            tma_load_2d_pair_if(sr, &tmap_r, fb, k0, t.row0 + r_at, leader);
          }
        }
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy has landed before the CTAs may exit: the even CTA's full
    // barriers count both CTAs' bytes; masked stages count their own
    for (int s = 0; s < S; ++s) {
      if (rank == 0 && (issued >> s & 1u)) drain16(full_bar(s), (parity >> s) & 1u, p.status);
      if (tail_issued >> s & 1u) drain16(land_bar(s), (~tail_parity >> s) & 1u, p.status);
    }
  }
  // ------------------------------------------------------------ MMA issuer (even CTA)
  else if (warp == 1) {
    if (rank == 0) {
      const uint32_t leader = elect_leader();
      const uint16_t pair_mask = static_cast<uint16_t>(0x3u << even);
      uint32_t stage = 0, phase = 0, seg = 0;  // seg: accumulators filled so far
      bool ok = true;
      int64_t n = 0;
      for (int64_t u = unit0; ok && u < total; u += ustride, ++n) {
        const int slot = static_cast<int>(n & 1);
        if (!mbar_wait_warp(info_full_bar(slot), static_cast<uint32_t>((n >> 1) & 1), abort_flag,
                            p.status))
          break;
        const uint64_t info = info_word[slot];
        __syncwarp();  // every lane has read the word
        mbar_arrive_if(info_empty_bar(slot), leader);
        const int32_t kb_count = static_cast<int32_t>(info & 0xFFFFFFFFu);
        const int last_mmas = static_cast<int>((info >> 32) & 0xFFu);
        const uint32_t n_mma = static_cast<uint32_t>(info >> 40);
        const uint32_t idesc = p.idesc | ((n_mma >> 3) << 17);
        int32_t kb = 0;
        do {
          // the accumulator has been read out since it was last filled
          const uint32_t acc = seg & 1u;
          if (!mbar_wait_warp<true>(tempty_bar(acc), ((seg >> 1) & 1u) ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + 256u * acc;
          const int32_t kb0 = kb, kb1 = SEG != 0 ? min(kb_count, kb + SEG) : kb_count;
          for (; kb < kb1; ++kb) {
            if (!mbar_wait_warp(full_bar(stage), phase, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sq = stage0 + stage * stage_bytes, sr = sq + q_bytes;
            const uint64_t qd = tile_desc16<Q_MN>(sq), rd = tile_desc16<R_MN>(sr);
            const int nmma = kb + 1 == kb_count ? last_mmas : Cfg::kMmas;
#pragma unroll
            for (int kk = 0; kk < Cfg::kMmas; ++kk) {
              if (kk >= nmma) break;
              tc_mma_f16_pair_if(d, qd + kk * kStep16<Q_MN>, rd + kk * kStep16<R_MN>, idesc,
                                 (kb > kb0 || kk > 0) ? 1u : 0u, leader);
            }
            tc_commit_pair_mc_if(empty_bar(stage), pair_mask, leader);
            if (++stage == stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit_pair_mc_if(tfull_bar(acc), pair_mask, leader);
          ++seg;
        } while (kb < kb_count);
      }
      if (leader) tc_commit_pair(drain_bar);
      __syncwarp();
      drain16(drain_bar, 0, p.status);
    }
  }
  // ------------------------------------------------------------ mask warp (wgrad, both CTAs)
  else if (MODE == 1 && warp == Cfg::kMaskWarp) {
    uint32_t stage = 0, used = 0;  // used: parity of each stage's masked uses so far
    for (int64_t u = unit0; u < total; u += ustride) {
      const Unit16 t = map_unit16<MODE, SPLIT>(u, p, row_off, unit_off, shape, pair);
      const int32_t kb_count = (t.kdim + BK - 1) / BK;
      if (kb_count == 0) continue;
      const int32_t last = t.kdim - (kb_count - 1) * BK;
      stage = (stage + static_cast<uint32_t>(kb_count - 1)) % stages;
      if ((last & 15) != 0) {
        const uint32_t par = (used >> stage) & 1u;
        if (!mbar_wait_warp(land_bar(stage), par, abort_flag, p.status)) break;
        // rows last .. end of the 16: whole 128-byte rows, which the swizzle
        // permutes only within themselves
        const uint32_t bytes = static_cast<uint32_t>(((last + 15) & ~15) - last) * 128u;
        const uint32_t at = stage0 + stage * stage_bytes + static_cast<uint32_t>(last) * 128u;
        for (uint32_t o = lane * 16; o < bytes; o += 512)
          for (uint32_t c = 0; c < stage_bytes; c += 8192) st_shared_v4(at + c + o, 0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
        if (rank == 0) {
          if (!mbar_wait_warp<true>(odd_bar(stage), par, abort_flag, p.status)) break;
          if (lane == 0) mbar_arrive(full_bar(stage));
        } else if (lane == 0) {
          mbar_arrive_cluster(mapa_shared(odd_bar(stage), even));
        }
        used ^= 1u << stage;
      }
      stage = (stage + 1) % stages;
    }
  }
  // ------------------------------------------------------------ epilogue (both CTAs)
  else {
    // lane quarter = 32 columns of C, every other chunk of 32 rows
    const uint32_t quarter = warp & 3u, half = (warp - 2) >> 2;
    uint32_t seg = 0;
    bool ok = true, joined = !SPLIT;
    for (int64_t u = unit0; ok && u < total; u += ustride) {
      const Unit16 t = map_unit16<MODE, SPLIT>(u, p, row_off, unit_off, shape, pair);
      const bool has_k = t.kdim > 0;
      const float alpha = p.alpha ? p.alpha[t.g] : 1.0f;
      const float beta = p.beta ? p.beta[t.g] : 0.0f;
      const int32_t lane_col = static_cast<int32_t>(32 * quarter + lane);
      const int32_t col = t.j0 + p.tile_cols / 2 * static_cast<int32_t>(rank) + lane_col;
      const int64_t row =
          (MODE == 1 ? static_cast<int64_t>(t.g) * p.N : static_cast<int64_t>(t.row0)) + t.i0;
      const bool in = lane_col < p.tile_cols / 2 && col < p.out_cols;
      const int32_t c0 = 32 * static_cast<int32_t>(half);
      auto store = [&](int32_t c, const float(&v)[32]) {
        if (!in) return;
        const int64_t at = (row + c) * p.ldc + col;
        if (SEG != 0 || p.out_type == MXG_F32)
          store_column16(static_cast<float*>(p.C) + at, p.ldc, v, t.rows - c, alpha, beta);
        else if (p.out_type == MXG_BF16)
          store_column16(static_cast<Bf16*>(p.C) + at, p.ldc, v, t.rows - c, alpha, beta);
        else
          store_column16(static_cast<F16*>(p.C) + at, p.ldc, v, t.rows - c, alpha, beta);
      };
      // the next accumulator, and the word that it may be filled again.  That
      // arrival is relaxed: a release would wait for the stores
      auto take = [&] {
        const uint32_t acc = seg & 1u;
        if (!mbar_wait_warp(tfull_bar(acc), (seg >> 1) & 1u, abort_flag, p.status)) return false;
        tc_fence_after();
        return true;
      };
      auto give = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(seg & 1u), even));
        ++seg;
      };
      const uint32_t lanes = tmem_base + ((32u * quarter) << 16);
      // Pairs that share the contraction: chunk m (of this warp's four) of the
      // sums is wanted by pair m % splits.  The others put theirs into the
      // stages of that pair's CTA, once no pair copies or multiplies any more
      // (a cluster has one unit only), and it adds them in the pairs' order.
      auto join = [&](auto&& chunk) {
        const int32_t S = p.splits, per = 4 / S;
        auto place = [&](int32_t from, int32_t m) {
          return stage0 + static_cast<uint32_t>(((from * per + m / S) * 2 + static_cast<int32_t>(half)) * 32 * 128 +
                                                lane_col) * 4u;
        };
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int32_t m = 0; m < 4; ++m) {
          const int32_t to = m & (S - 1);
          if (c0 + 64 * m >= t.rows || to == pair) continue;
          float v[32];
          chunk(m, v);
          const uint32_t dst = mapa_shared(place(pair < to ? pair : pair - 1, m), 2 * to + rank);
#pragma unroll
          for (int e = 0; e < 32; ++e) st_cluster_f32(dst + e * 512, v[e]);
        }
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int32_t m = 0; m < 4; ++m) {
          if (c0 + 64 * m >= t.rows || (m & (S - 1)) != pair) continue;
          float v[32];
          chunk(m, v);
          for (int32_t from = 0; from < S - 1; ++from) {
            const uint32_t src = place(from, m);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] += ld_shared_f32(src + e * 512);
          }
          store(c0 + 64 * m, v);
          __syncwarp();
        }
        joined = true;
      };
      if constexpr (SEG == 0) {
        if (!(ok = take())) break;
        const uint32_t taddr = lanes + 256u * (seg & 1u);
        auto read = [&](int32_t c, float(&v)[32]) {
          if (has_k) {
            uint32_t w[32];
            tmem_ld32(taddr + static_cast<uint32_t>(c), w);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(w[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.0f;
          }
        };
        if constexpr (SPLIT) {
          join([&](int32_t m, float(&v)[32]) { read(c0 + 64 * m, v); });
        } else {
          for (int32_t c = c0; c < t.rows; c += 64) {
            float v[32];
            read(c, v);
            store(c, v);
            __syncwarp();
          }
        }
        give();
      } else {
        float v[4][32];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[m][e] = 0.0f;
        int32_t k = 0;
        do {
          if (!(ok = take())) break;
          const uint32_t taddr = lanes + 256u * (seg & 1u) + static_cast<uint32_t>(c0);
          if (has_k) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              if (c0 + 64 * m < t.rows) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t w[16];
                  tmem_ld16(taddr + 64 * m + 16 * h, w);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[m][16 * h + e] += __uint_as_float(w[e]);
                }
              }
            }
          }
          give();
          k += SEG * BK;
        } while (k < t.kdim);
        if (!ok) break;
        if constexpr (SPLIT) {
          join([&](int32_t m, float(&w)[32]) {
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = v[m][e];
          });
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (c0 + 64 * m < t.rows) store(c0 + 64 * m, v[m]);
          __syncwarp();
        }
      }
    }
    if (!joined) {  // no unit, or given up
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  }
  if (SPLIT && (warp < 2 || warp == Cfg::kMaskWarp)) {  // the epilogues' join
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no copy, commit or remote arrival still targets either CTA
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

namespace {

constexpr int kMaxDev16 = 64;
constexpr int kSeg16 = 8;  // K blocks an fp32 output's sum stays in tensor memory

// Clusters of 2 * splits CTAs that the device holds at once (-1: none of more
// than a pair), asked once per device, with all the shared memory there is.
int pair_clusters(int splits, int num_sms) {
  static std::atomic<int> known[3][kMaxDev16];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev16) return 0;
  std::atomic<int>& slot = known[splits >> 1][dev];
  int c = slot.load(std::memory_order_relaxed);
  if (c != 0) return c;
  auto kern = gemm16_pair_kernel<1, kSeg16, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pair16::kSmemMax) !=
      cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / (2 * splits) * 2 * splits));
  cfg.blockDim = dim3(Pair16::threads(1));
  cfg.dynamicSmemBytes = Pair16::kSmemMax;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess || c < 1)
    c = splits == 1 ? num_sms / 2 : -1;
  slot.store(c, std::memory_order_relaxed);
  return c;
}

template <int MODE, int SEG, bool SPLIT>
cudaError_t launch_pair16(const CUtensorMap& tq, const CUtensorMap& tr, const Gemm16Params& p,
                          int smem, int64_t max_units, int num_sms, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDev16];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev16)
    return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(gemm16_pair_kernel<MODE, SEG, SPLIT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Pair16::kSmemMax);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  const int clusters = pair_clusters(p.splits, num_sms);
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  const int64_t n = max_units < clusters ? max_units : clusters;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * p.splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  // set up beside the kernel before it, where that one allows it
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.splits * n));
  cfg.blockDim = dim3(Pair16::threads(MODE));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm16_pair_kernel<MODE, SEG, SPLIT>, tq, tr, p);
}

// A ragged matrix [rows, cols] of 16-bit elements, boxes of 64 columns.
bool ragged_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld,
                uint32_t box_rows) {
  return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, static_cast<uint64_t>(cols),
                      static_cast<uint64_t>(rows < 1 ? 1 : rows), static_cast<uint64_t>(ld) * 2, 64,
                      box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t launch_grouped_gemm16(int in_f16, int mode, const void* A, int64_t lda, const void* B,
                                  int64_t ldb, const int64_t* group_ws, int G, int64_t M_cap,
                                  int64_t N, int64_t K, const float* alpha, const float* beta,
                                  void* C, int64_t ldc, int out_type, int32_t* status, int num_sms,
                                  cudaStream_t stream) {
  Gemm16Params p;
  p.group_ws = group_ws;
  p.alpha = alpha;
  p.beta = beta;
  p.C = C;
  p.status = status;
  p.ldc = ldc;
  p.M_cap = static_cast<int32_t>(M_cap);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.out_cols = mode == 0 ? p.N : p.K;
  p.G = G;
  p.out_type = out_type;
  // FP32 accumulation (bit 4), operand types (bits 7 and 10: 0 fp16, 1 bf16),
  // MN-major Q and R (bits 15 and 16), M = 256 (bit 24)
  p.idesc = (1u << 4) | (in_f16 ? 0u : (1u << 7) | (1u << 10)) | (mode != 0 ? 1u << 15 : 0u) |
            (mode == 1 ? 1u << 16 : 0u) | ((256u >> 4) << 24);
  // Units of 256 x 256, or as many rows as there can be; while twice as many
  // still find a cluster each, their longer side is halved, down to 64 rows and
  // 128 columns (one row through 4096 x 4096 unshared: 23 us in 16 units, 20 us in
  // 32; in 64 of 64 columns 25 us).  The MMA always runs on 256 columns; the lanes of
  // those that a unit does not have are not read.  What small units leave free of
  // a stage goes to more stages, i.e. more of the operands in flight.
  const int64_t c_rows = mode == 1 ? N : M_cap;
  p.tile_rows = c_rows >= 256 ? 256 : static_cast<int32_t>((c_rows + 31) / 32 * 32);
  p.tile_cols = 256;
  // an upper bound: the sizes are on the device
  const int64_t live = M_cap < G ? M_cap : G;
  auto count = [&] {
    const int64_t cu = (p.out_cols + p.tile_cols - 1) / p.tile_cols;
    return mode == 1 ? G * ((N + p.tile_rows - 1) / p.tile_rows) * cu
                     : (M_cap + live * (p.tile_rows - 1)) / p.tile_rows * cu;
  };
  // Where units are few and the contraction is long, 4 or 2 pairs share a unit's
  // -- as many as leave each cluster one unit at most, and each pair 8 K blocks of
  // 64, or 16 where it has more than 64 rows to join (one row through 4096 x 4096:
  // 14.7 us by two pairs, 19.4 us by one; through 1024 x 4096: 10.3 us by four,
  // 12.8 us by two, 17.9 us by one; 16 rows through 1024 x 2048: 8.7, 9.7 and
  // 11.8 us; wgrad of 512 x 512 over 2048 rows: 12.5 us by four, 10.8 us by two,
  // 11.8 us by one; 128 rows through 1024 x 1024: 8.2 us by two, 7.7 us by one).
  // The length of wgrad's is known on average only.
  const int64_t k_avg = mode == 0 ? K : mode == 2 ? N : live > 0 ? M_cap / live : 0;
  p.splits = 1;
  for (int s = 4; s > 1 && p.splits == 1; s /= 2)
    if ((k_avg + 63) / 64 >= s * (p.tile_rows <= 64 ? 8 : 16) &&
        count() <= pair_clusters(s, num_sms))
      p.splits = s;
  const int most = p.splits == 1 ? num_sms / 2 : pair_clusters(p.splits, num_sms);
  while (count() * 2 <= most && (p.tile_cols > 128 || p.tile_rows > 64)) {
    if (p.tile_cols > 128 && (p.tile_cols >= p.tile_rows || p.tile_rows <= 64))
      p.tile_cols /= 2;
    else
      p.tile_rows = (p.tile_rows / 2 + 31) / 32 * 32;
  }
  p.col_units = (p.out_cols + p.tile_cols - 1) / p.tile_cols;
  p.w_shape = unit_shape(static_cast<uint32_t>(N), static_cast<uint32_t>(p.tile_rows));
  p.q_bytes = p.tile_cols / 2 * 128;
  const int r_bytes = mode == 1 ? (p.tile_rows > 128 ? 16384 : 8192) : p.tile_rows / 2 * 128;
  p.stage_bytes = p.q_bytes + r_bytes;
  const int header = Pair16::header_bytes(G) + 1024;
  p.stages = (Pair16::kSmemMax - header) / p.stage_bytes;
  if (p.stages > Pair16::kMaxStages) p.stages = Pair16::kMaxStages;
  // the MMA reads 16 KB from each tile of Q on, however many columns are in it
  int smem = header + (p.stages - 1) * p.stage_bytes + std::max(p.stage_bytes, 16384);
  // the sums of the other pairs: 32 rows of 128 columns eight times over, less its own share
  if (p.splits > 1) smem = std::max(smem, header + (p.splits - 1) * (8 / p.splits) * 16384);

  // without rows no copy is made: any aligned address serves the tensor maps
  if (M_cap == 0) A = B = reinterpret_cast<const void*>(uintptr_t{1} << 20);
  CUtensorMap tq, tr;
  const int64_t r_cols = mode == 0 ? K : N;
  if (!ragged_map(&tr, A, r_cols, M_cap, lda,
                  mode == 1 ? 64u : static_cast<uint32_t>(p.tile_rows / 2)))
    return cudaErrorInvalidValue;
  if (mode == 1) {
    if (!ragged_map(&tq, B, K, M_cap, ldb, 64)) return cudaErrorInvalidValue;
  } else {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N),
                              static_cast<uint64_t>(G)};
    const uint64_t strides[2] = {static_cast<uint64_t>(ldb) * 2, static_cast<uint64_t>(N * ldb) * 2};
    const uint32_t box[3] = {64, mode == 0 ? static_cast<uint32_t>(p.tile_cols / 2) : 64u, 1};
    if (!make_tmap_3d_swizzled(&tq, B, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  const int64_t units = count();
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  auto launch = [&](auto seg, auto split) {
    constexpr int SEG = decltype(seg)::value;
    constexpr bool SPLIT = decltype(split)::value;
    if (mode == 0) return launch_pair16<0, SEG, SPLIT>(tq, tr, p, smem, units, num_sms, stream);
    if (mode == 1) return launch_pair16<1, SEG, SPLIT>(tq, tr, p, smem, units, num_sms, stream);
    return launch_pair16<2, SEG, SPLIT>(tq, tr, p, smem, units, num_sms, stream);
  };
  using Whole = std::integral_constant<int, 0>;
  using Parts = std::integral_constant<int, kSeg16>;
  if (out_type == MXG_F32)
    return p.splits > 1 ? launch(Parts{}, std::true_type{}) : launch(Parts{}, std::false_type{});
  return p.splits > 1 ? launch(Whole{}, std::true_type{}) : launch(Whole{}, std::false_type{});
}

}  // namespace mxg
