// gemm16.cu -- grouped products with 16-bit operands (bf16 or fp16):
//   fprop  C[off_g+i, n] = alpha_g * sum_k A[off_g+i, k] B[g, n, k] + beta_g * C
//   dgrad  C[off_g+i, k] = alpha_g * sum_n A[off_g+i, n] B[g, n, k] + beta_g * C
//   wgrad  C[g, n, k]    = alpha_g * sum_{i in g} A[off_g+i, n] B[off_g+i, k] + beta_g * C
// Group g owns rows off_g .. off_g + M_g - 1 (any M_g >= 0, read on the device).
//
// A 2-CTA cluster computes 256 x 256 output units with the cta_group::2 MMA;
// CTA r holds 128 rows of the unit's A tile and half of its B tile.  Warp 0
// loads (TMA), warp 1 of the even CTA issues the MMAs, warps 2-9 are the
// epilogue (one TMEM lane quarter and 128 columns each).  The two 256-column
// accumulators fill tensor memory, so that the epilogue of a unit runs under
// the MMAs of the next one.  The clusters are persistent and walk the units
// in a static order derived from the group sizes on the device.
//
// Neither operand is transposed in memory: where the contraction runs along
// rows (B of dgrad, both of wgrad) the tile is loaded as 64-row boxes of 64
// columns and the MMA reads it MN-major.
//
// Contraction tails.  Past N or K the copies fill zeros (for the weights the
// tensor map has the expert as its third dimension, so that a box never runs
// into the next expert).  Only wgrad's contraction ends at a device-side
// number: the rows of the next group that share the last 16-row MMA step are
// zeroed in shared memory, in A and in B (a zero against their NaN would not
// be zero), by warp 10 while earlier stages are multiplied.
#include <atomic>

#include "elem.cuh"
#include "mxg_host.h"

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
  int32_t out_type;  // mxg_dtype_t
  uint32_t idesc;    // operand types and majors (M and N are added per unit)
  int32_t c_vec;     // bytes of the widest aligned access to rows of C: 32, 16 or 0
};

// Row offsets of the groups and their first units, by one warp: negative
// sizes count as 0 and rows past M_cap are dropped, so that no access leaves
// the operands.  A unit is `rows_per_unit` rows of a group times one of
// `col_units` column ranges.
__device__ __forceinline__ void group_tables16(const int64_t* group_ws, int G, int64_t M_cap,
                                               int rows_per_unit, int64_t col_units,
                                               int32_t* row_off, int32_t* unit_off,
                                               int32_t* status) {
  const uint32_t lane = lane_id();
  int64_t carry_rows = 0, carry_units = 0;
  int32_t bits = 0;
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= static_cast<uint32_t>(d)) v += u;
    }
    return v;
  };
  for (int base = 0; base < G; base += 32) {
    const int g = base + static_cast<int>(lane);
    int64_t s = 0;
    if (g < G) {
      s = group_ws[g];
      if (s < 0) {
        s = 0;
        bits |= MXG_DEV_NEG_SIZE;
      }
      if (s > M_cap) s = M_cap + 1;  // keeps the sum small, still past the capacity
    }
    const int64_t incl = scan(s);
    const int64_t before = min(carry_rows + incl - s, M_cap);
    const int64_t after = min(carry_rows + incl, M_cap);
    if (carry_rows + incl > M_cap && s > 0) bits |= MXG_DEV_SUM_OVER_CAPACITY;
    const int64_t units = (after - before + rows_per_unit - 1) / rows_per_unit * col_units;
    const int64_t uincl = scan(units);
    if (g < G) {
      row_off[g] = static_cast<int32_t>(before);
      unit_off[g] = static_cast<int32_t>(carry_units + uincl - units);
    }
    carry_rows += __shfl_sync(0xFFFFFFFFu, incl, 31);
    carry_units += __shfl_sync(0xFFFFFFFFu, uincl, 31);
  }
  if (lane == 0) {
    row_off[G] = static_cast<int32_t>(min(carry_rows, M_cap));
    unit_off[G] = static_cast<int32_t>(carry_units);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) bits |= __shfl_xor_sync(0xFFFFFFFFu, bits, d);
  if (lane == 0 && blockIdx.x == 0) status_set(status, bits);
}

// Work unit u of the pair kernel: 256 rows times 256 columns of C.
struct Unit16 {
  int32_t g;
  int32_t row0;       // first row of the group in the ragged operands
  int32_t i0, j0;     // first row (within the group, or of dW_g) and column of C
  int32_t rows_left;  // rows of C from i0 on that belong to the group / dW_g
  int32_t kdim;       // contraction length
  int32_t n_mma;      // columns the MMAs compute: 256, fewer in the last column unit
};

constexpr int kTile16 = 256;

template <int MODE>
__device__ __forceinline__ Unit16 map_unit16(int64_t u, const Gemm16Params& p,
                                             const int32_t* row_off, const int32_t* unit_off) {
  Unit16 t;
  const int32_t cu = (p.out_cols + kTile16 - 1) / kTile16;
  if constexpr (MODE == 1) {
    const uint32_t per = static_cast<uint32_t>((p.N + kTile16 - 1) / kTile16) * cu;
    t.g = static_cast<int32_t>(static_cast<uint32_t>(u) / per);
    const uint32_t local = static_cast<uint32_t>(u) - t.g * per;
    const uint32_t iu = local / cu;
    t.i0 = static_cast<int32_t>(iu) * kTile16;
    t.j0 = static_cast<int32_t>(local - iu * cu) * kTile16;
    t.rows_left = p.N - t.i0;
    t.row0 = row_off[t.g];
    t.kdim = row_off[t.g + 1] - t.row0;
  } else {
    int lo = 0, hi = p.G;  // largest g with unit_off[g] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (unit_off[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    t.g = lo;
    t.row0 = row_off[lo];
    t.kdim = MODE == 0 ? p.K : p.N;
    const int32_t rows = row_off[lo + 1] - t.row0;
    const uint32_t ru = static_cast<uint32_t>((rows + kTile16 - 1) / kTile16);
    const uint32_t local = static_cast<uint32_t>(u) - unit_off[lo];
    // column unit, then row unit, so that the clusters in flight share weight
    // tiles and the group's rows stay in L2; where those rows are more than an
    // L2 budget, blocks of column units that fit it, each walked row unit by
    // row unit
    uint32_t j = local / ru, i = local - j * ru;
    constexpr int64_t kL2Budget = 32ll << 20;
    if (static_cast<int64_t>(rows) * t.kdim * 2 > kL2Budget) {
      int64_t cb = kL2Budget / (static_cast<int64_t>(kTile16) * t.kdim * 2);
      cb = cb < 1 ? 1 : (cb > cu ? cu : cb);
      const uint32_t b = static_cast<uint32_t>(cb), blk = local / (ru * b);
      const uint32_t width = (blk + 1) * b <= static_cast<uint32_t>(cu) ? b : cu - blk * b;
      const uint32_t rem = local - blk * ru * b;
      i = rem / width;
      j = blk * b + (rem - i * width);
    }
    t.i0 = static_cast<int32_t>(i) * kTile16;
    t.j0 = static_cast<int32_t>(j) * kTile16;
    t.rows_left = rows - t.i0;
  }
  const int32_t left = p.out_cols - t.j0;
  t.n_mma = left >= kTile16 ? kTile16 : (left + 31) / 32 * 32;
  return t;
}

// 16 columns of one output row: alpha * acc + beta * old, stored as the output
// type.  `n`: columns of the 16 that exist.
template <typename T>
__device__ __forceinline__ void store_cols16(T* dst, const uint32_t* acc, int n, int vec, bool has_k,
                                             float alpha, float beta) {
  float f[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) f[e] = has_k ? alpha * __uint_as_float(acc[e]) : 0.0f;
  if (n >= 16 && vec != 0) {
    if (beta != 0.0f) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o[8];
        unpack8<T>(load8<T>(dst + 8 * h), o);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * h + e] += beta * o[e];
      }
    }
    if (vec == 32) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(f[8 * h + e]);
          st_global_32B(dst + 8 * h, w);
        }
      } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack2<T>(f[2 * e], f[2 * e + 1]);
        st_global_32B(dst, w);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f[8 * h + e];
        store8<T>(dst + 8 * h, o);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < n) {
      float v = f[e];
      if (beta != 0.0f) v += beta * to_f32(dst[e]);
      dst[e] = from_f32<T>(v);
    }
}

__device__ __forceinline__ void store_row16(const Gemm16Params& p, int64_t row, int32_t col,
                                            const uint32_t* acc, bool has_k, float alpha,
                                            float beta) {
  const int n = p.out_cols - col;
  if (n <= 0) return;
  const int64_t at = row * p.ldc + col;
  if (p.out_type == MXG_F32)
    store_cols16(static_cast<float*>(p.C) + at, acc, n, p.c_vec, has_k, alpha, beta);
  else if (p.out_type == MXG_BF16)
    store_cols16(static_cast<Bf16*>(p.C) + at, acc, n, p.c_vec, has_k, alpha, beta);
  else
    store_cols16(static_cast<F16*>(p.C) + at, acc, n, p.c_vec, has_k, alpha, beta);
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
  static constexpr int kStages = 6;
  static constexpr int kBK = 64;                   // contraction elements per stage
  static constexpr int kOperand = 128 * kBK * 2;   // bytes of A, and of B, per CTA and stage
  static constexpr int kStageBytes = 2 * kOperand;
  static constexpr int kMmas = kBK / 16;
  static constexpr int kEpiWarps = 8;
  static constexpr int kMaskWarp = 2 + kEpiWarps;
  static constexpr int threads(int mode) { return 32 * (kMaskWarp + (mode == 1 ? 1 : 0)); }
  // full[S], empty[S], land[S], odd_masked[S], tfull[2], tempty[2],
  // info_full[2], info_empty[2], drain; two unit words; TMEM base, abort flag
  static constexpr int kBars = 4 * kStages + 9;
  static constexpr int kBarBytes = 8 * (kBars + 2) + 16;
  static size_t smem_bytes(int G) {
    return 1024 + static_cast<size_t>(kStages) * kStageBytes + kBarBytes + 8 * (G + 1);
  }
};

// Descriptor of a 128-row K-major tile (rows of 128 bytes, 128-byte swizzle),
// or of an MN-major one: chunks of 64 rows of 128 bytes (64 values along M or
// N a row), 8192 bytes apart, 8-row groups 1024 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc16(uint32_t saddr) {
  return MN ? smem_desc(saddr, 8192, 1024, 2) : smem_desc(saddr, 16, 1024, 2);
}
// 16 elements further along the contraction, in descriptor units of 16 bytes
template <bool MN>
constexpr uint32_t kStep16 = MN ? 2048 / 16 : 32 / 16;

template <int MODE>
__global__ void __launch_bounds__(Pair16::threads(MODE), 1)
    gemm16_pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                       const __grid_constant__ CUtensorMap tmap_b, const Gemm16Params p) {
  using Cfg = Pair16;
  constexpr int S = Cfg::kStages, BK = Cfg::kBK;
  constexpr bool A_MN = MODE == 1, B_MN = MODE != 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Cfg::kStageBytes);
  uint64_t* info_word = bars + Cfg::kBars;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(info_word + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_s + 1);
  int32_t* row_off = reinterpret_cast<int32_t*>(smem + S * Cfg::kStageBytes + Cfg::kBarBytes);
  int32_t* unit_off = row_off + (p.G + 1);

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t rank = cluster_ctarank();
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
  if (warp == 1)
    group_tables16(p.group_ws, p.G, p.M_cap, kTile16, (p.out_cols + kTile16 - 1) / kTile16,
                   row_off, unit_off, p.status);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the even CTA's barriers exist before the odd CTA's copies signal them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_s;
  const int64_t unit0 = blockIdx.x >> 1, ustride = gridDim.x >> 1;
  const int64_t total =
      MODE == 1 ? static_cast<int64_t>(p.G) * ((p.N + kTile16 - 1) / kTile16) *
                      ((p.out_cols + kTile16 - 1) / kTile16)
                : unit_off[p.G];

  // ------------------------------------------------------------ producers (both CTAs)
  if (warp == 0) {
    {
      const uint32_t leader = elect_leader();
      prefetch_tmap(&tmap_a);
      prefetch_tmap(&tmap_b);
      uint32_t stage = 0, phase = 0, issued = 0, parity = 0, tail_issued = 0, tail_parity = 0;
      bool ok = true;
      for (int64_t u = unit0, n = 0; ok && u < total; u += ustride, ++n) {
        const Unit16 t = map_unit16<MODE>(u, p, row_off, unit_off);
        const int32_t kb_count = (t.kdim + BK - 1) / BK;
        const int32_t last = t.kdim - (kb_count - 1) * BK;  // elements of the last block
        if (rank == 0) {
          // the unit's shape, for the MMA thread
          const int slot = static_cast<int>(n & 1), par = static_cast<int>((n >> 1) & 1);
          if (!mbar_wait_warp(info_empty_bar(slot), par ^ 1, abort_flag, p.status)) break;
          if (leader)
            info_word[slot] = static_cast<uint64_t>(static_cast<uint32_t>(kb_count)) |
                              (static_cast<uint64_t>((last + 15) / 16) << 32) |
                              (static_cast<uint64_t>(t.n_mma) << 40);
          mbar_arrive_if(info_full_bar(slot), leader);
        }
        const int32_t b_at = t.j0 + (t.n_mma / 2) * static_cast<int32_t>(rank);
        const int32_t a_at = t.i0 + 128 * static_cast<int32_t>(rank);
        for (int32_t kb = 0; kb < kb_count; ++kb) {
          if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_base + stage * Cfg::kStageBytes, sb = sa + Cfg::kOperand;
          const int32_t k0 = kb * BK;
          if (MODE == 1 && kb + 1 == kb_count && (last & 15) != 0) {
            // rows of the next group in the last MMA step: this CTA's bytes
            // land on its own barrier, and its mask warp passes them on
            mbar_arrive_expect_tx_if(land_bar(stage), Cfg::kStageBytes, leader);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tma_load_2d_if(sa + 8192 * c, &tmap_a, land_bar(stage), a_at + 64 * c, t.row0 + k0, leader);
              tma_load_2d_if(sb + 8192 * c, &tmap_b, land_bar(stage), b_at + 64 * c, t.row0 + k0, leader);
            }
            tail_issued |= 1u << stage;
            tail_parity ^= 1u << stage;
          } else {
            if (rank == 0) mbar_arrive_expect_tx_if(full_bar(stage), 2 * Cfg::kStageBytes, leader);
            const uint32_t fb = mapa_shared(full_bar(stage), 0);
            if constexpr (A_MN) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                tma_load_2d_pair_if(sa + 8192 * c, &tmap_a, fb, a_at + 64 * c, t.row0 + k0, leader);
            } else {
              tma_load_2d_pair_if(sa, &tmap_a, fb, k0, t.row0 + a_at, leader);
            }
            if constexpr (MODE == 0) {
              tma_load_3d_pair_if(sb, &tmap_b, fb, k0, b_at, t.g, leader);
            } else {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if constexpr (MODE == 2)
                  tma_load_3d_pair_if(sb + 8192 * c, &tmap_b, fb, b_at + 64 * c, k0, t.g, leader);
                else
                  tma_load_2d_pair_if(sb + 8192 * c, &tmap_b, fb, b_at + 64 * c, t.row0 + k0, leader);
              }
            }
          }
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
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
  }
  // ------------------------------------------------------------ MMA issuer (even CTA)
  else if (warp == 1) {
    if (rank == 0) {
      const uint32_t leader = elect_leader();
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int64_t n = 0;
      for (int64_t u = unit0; ok && u < total; u += ustride, ++n) {
        const int slot = static_cast<int>(n & 1);
        const uint32_t par = static_cast<uint32_t>((n >> 1) & 1);
        if (!mbar_wait_warp(info_full_bar(slot), par, abort_flag, p.status)) break;
        const uint64_t info = info_word[slot];
        __syncwarp();  // every lane has read the word
        mbar_arrive_if(info_empty_bar(slot), leader);
        const int32_t kb_count = static_cast<int32_t>(info & 0xFFFFFFFFu);
        const int last_mmas = static_cast<int>((info >> 32) & 0xFFu);
        const uint32_t n_mma = static_cast<uint32_t>(info >> 40);
        const uint32_t idesc = p.idesc | ((n_mma >> 3) << 17);
        // the accumulator's previous unit has been read out
        if (!mbar_wait_warp<true>(tempty_bar(slot), par ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + 256u * slot;
        for (int32_t kb = 0; kb < kb_count; ++kb) {
          if (!mbar_wait_warp(full_bar(stage), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_base + stage * Cfg::kStageBytes, sb = sa + Cfg::kOperand;
          const uint64_t ad = tile_desc16<A_MN>(sa), bd = tile_desc16<B_MN>(sb);
          const int nmma = kb + 1 == kb_count ? last_mmas : Cfg::kMmas;
#pragma unroll
          for (int kk = 0; kk < Cfg::kMmas; ++kk) {
            if (kk >= nmma) break;
            tc_mma_f16_pair_if(d, ad + kk * kStep16<A_MN>, bd + kk * kStep16<B_MN>, idesc,
                               (kb > 0 || kk > 0) ? 1u : 0u, leader);
          }
          tc_commit_pair_mc_if(empty_bar(stage), 0x3, leader);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_mc_if(tfull_bar(slot), 0x3, leader);
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
      const Unit16 t = map_unit16<MODE>(u, p, row_off, unit_off);
      const int32_t kb_count = (t.kdim + BK - 1) / BK;
      if (kb_count == 0) continue;
      const int32_t last = t.kdim - (kb_count - 1) * BK;
      stage = (stage + static_cast<uint32_t>(kb_count - 1)) % S;
      if ((last & 15) != 0) {
        const uint32_t par = (used >> stage) & 1u;
        if (!mbar_wait_warp(land_bar(stage), par, abort_flag, p.status)) break;
        // rows last .. end of the 16: whole 128-byte rows, which the swizzle
        // permutes only within themselves
        const uint32_t bytes = static_cast<uint32_t>(((last + 15) & ~15) - last) * 128u;
        const uint32_t at = smem_base + stage * Cfg::kStageBytes + static_cast<uint32_t>(last) * 128u;
        for (uint32_t o = lane * 16; o < bytes; o += 512)
#pragma unroll
          for (uint32_t c = 0; c < 4; ++c) st_shared_v4(at + 8192 * c + o, 0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
        if (rank == 0) {
          if (!mbar_wait_warp<true>(odd_bar(stage), par, abort_flag, p.status)) break;
          if (lane == 0) mbar_arrive(full_bar(stage));
        } else if (lane == 0) {
          mbar_arrive_cluster(mapa_shared(odd_bar(stage), 0));
        }
        used ^= 1u << stage;
      }
      stage = (stage + 1) % S;
    }
  }
  // ------------------------------------------------------------ epilogue (both CTAs)
  else {
    const uint32_t ew = warp - 2;
    const uint32_t quarter = warp & 3u;  // TMEM lanes 32 * quarter .. + 31
    const uint32_t col0 = 128u * (ew >> 2);
    int64_t n = 0;
    for (int64_t u = unit0; u < total; u += ustride, ++n) {
      const Unit16 t = map_unit16<MODE>(u, p, row_off, unit_off);
      const int slot = static_cast<int>(n & 1);
      const bool has_k = t.kdim > 0;
      const float alpha = p.alpha ? p.alpha[t.g] : 1.0f;
      const float beta = p.beta ? p.beta[t.g] : 0.0f;
      if (!mbar_wait_warp(tfull_bar(slot), static_cast<uint32_t>((n >> 1) & 1), abort_flag, p.status))
        break;
      tc_fence_after();
      uint32_t v[4][32];
      if (has_k) {
        const uint32_t taddr = tmem_base + ((32u * quarter) << 16) + 256u * slot + col0;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(taddr + 32 * c, v[c]);
        tmem_ld_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar(slot), 0));
      const int32_t r = static_cast<int32_t>(128 * rank + 32 * quarter + lane);
      if (r < t.rows_left) {
        const int64_t row = (MODE == 1 ? static_cast<int64_t>(t.g) * p.N : t.row0) + t.i0 + r;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          store_row16(p, row, t.j0 + static_cast<int32_t>(col0) + 16 * k, &v[k >> 1][16 * (k & 1)],
                      has_k, alpha, beta);
      }
    }
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

// Clusters of the pair kernel that the device holds at once, asked once per
// device (with the shared memory of the largest group table).
template <int MODE>
int pair_clusters(int num_sms) {
  static std::atomic<int> known[kMaxDev16];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev16) return 0;
  int c = known[dev].load(std::memory_order_relaxed);
  if (c != 0) return c;
  auto kern = gemm16_pair_kernel<MODE>;
  const int smem = static_cast<int>(Pair16::smem_bytes(1024));
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
  cfg.blockDim = dim3(Pair16::threads(MODE));
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess || c < 1) c = num_sms / 2;
  known[dev].store(c, std::memory_order_relaxed);
  return c;
}

template <int MODE>
cudaError_t launch_pair16(const CUtensorMap& ta, const CUtensorMap& tb, const Gemm16Params& p,
                          int64_t max_units, int num_sms, cudaStream_t stream) {
  const int clusters = pair_clusters<MODE>(num_sms);
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  const int64_t n = max_units < clusters ? max_units : clusters;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * n));
  cfg.blockDim = dim3(Pair16::threads(MODE));
  cfg.dynamicSmemBytes = Pair16::smem_bytes(p.G);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm16_pair_kernel<MODE>, ta, tb, p);
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
  // MN-major operands (bits 15 and 16), M = 256 (bit 24)
  p.idesc = (1u << 4) | (in_f16 ? 0u : (1u << 7) | (1u << 10)) | (mode == 1 ? 1u << 15 : 0u) |
            (mode != 0 ? 1u << 16 : 0u) | ((256u >> 4) << 24);
  const int64_t size = out_type == MXG_F32 ? 4 : 2;
  const uintptr_t c_at = reinterpret_cast<uintptr_t>(C) | static_cast<uintptr_t>(ldc * size);
  p.c_vec = (c_at & 31u) == 0 ? 32 : ((c_at & 15u) == 0 ? 16 : 0);

  // without rows no copy is made: any aligned address serves the tensor maps
  if (M_cap == 0) {
    A = group_ws;
    B = mode == 1 ? group_ws : B;
  }
  CUtensorMap ta, tb;
  const int64_t a_cols = mode == 0 ? K : N;
  if (!ragged_map(&ta, A, a_cols, M_cap, lda, mode == 1 ? 64 : 128)) return cudaErrorInvalidValue;
  if (mode == 1) {
    if (!ragged_map(&tb, B, K, M_cap, ldb, 64)) return cudaErrorInvalidValue;
  } else {
    const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N),
                              static_cast<uint64_t>(G)};
    const uint64_t strides[2] = {static_cast<uint64_t>(ldb) * 2, static_cast<uint64_t>(N * ldb) * 2};
    const uint32_t box[3] = {64, mode == 0 ? 128u : 64u, 1};
    if (!make_tmap_3d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT16, B, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const int64_t cu = (p.out_cols + kTile16 - 1) / kTile16;
  // an upper bound: the sizes are on the device
  const int64_t live = M_cap < G ? M_cap : G;
  const int64_t units = mode == 1 ? G * ((N + kTile16 - 1) / kTile16) * cu
                                  : ((M_cap + live * (kTile16 - 1)) / kTile16) * cu;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  if (mode == 0) return launch_pair16<0>(ta, tb, p, units, num_sms, stream);
  if (mode == 1) return launch_pair16<1>(ta, tb, p, units, num_sms, stream);
  return launch_pair16<2>(ta, tb, p, units, num_sms, stream);
}

}  // namespace mxg
