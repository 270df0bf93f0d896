// gemm16.cu -- grouped products with 16-bit operands (bf16 or fp16):
//   fprop  C[off_g+i, n] = alpha_g * sum_k A[off_g+i, k] B[g, n, k] + beta_g * C
//   dgrad  C[off_g+i, k] = alpha_g * sum_n A[off_g+i, n] B[g, n, k] + beta_g * C
//   wgrad  C[g, n, k]    = alpha_g * sum_{i in g} A[off_g+i, n] B[off_g+i, k] + beta_g * C
// Group g owns rows off_g .. off_g + M_g - 1 (any M_g >= 0, read on the device).
//
// Simple form: 64 x 64 output tiles, 16 steps of the contraction at a time
// through shared memory, fp32 fused multiply-adds.
#include "elem.cuh"
#include "mxg_host.h"

namespace mxg {

struct Gemm16Params {
  const uint16_t* A;
  const uint16_t* B;
  const int64_t* group_ws;
  const float* alpha;
  const float* beta;
  void* C;
  int32_t* status;
  int64_t M_cap, N, K, lda, ldb, ldc;
  int G, mode, in_f16, out_type;
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

__device__ __forceinline__ float ld16(const uint16_t* p, int f16) {
  return f16 ? to_f32(F16{*p}) : to_f32(Bf16{*p});
}

__global__ void __launch_bounds__(256) gemm16_simple_kernel(const Gemm16Params p) {
  extern __shared__ int32_t tab[];
  int32_t* row_off = tab;
  int32_t* unit_off = tab + p.G + 1;
  __shared__ float as[16][65], bs[16][65];
  const int64_t out_cols = p.mode == 0 ? p.N : p.K;
  const int64_t ct = (out_cols + 63) / 64;
  if (threadIdx.x < 32)
    group_tables16(p.group_ws, p.G, p.M_cap, 64, ct, row_off, unit_off, p.status);
  __syncthreads();
  const int64_t nt = (p.N + 63) / 64;
  const int64_t total = p.mode == 1 ? p.G * nt * ct : unit_off[p.G];
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    int g;
    int64_t i0, j0, rows, kdim;         // tile origin, output rows of the group, contraction
    int64_t a_i, a_k, b_j, b_k, ab, bb;  // element strides and bases
    int64_t c_row;
    if (p.mode != 1) {
      int lo = 0, hi = p.G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (unit_off[mid] <= u) lo = mid; else hi = mid;
      }
      g = lo;
      const int64_t local = u - unit_off[g];
      i0 = local / ct * 64;
      j0 = local % ct * 64;
      rows = row_off[g + 1] - row_off[g];
      kdim = p.mode == 0 ? p.K : p.N;
      ab = row_off[g] * p.lda;
      a_i = p.lda;
      a_k = 1;
      bb = static_cast<int64_t>(g) * p.N * p.ldb;
      b_j = p.mode == 0 ? p.ldb : 1;
      b_k = p.mode == 0 ? 1 : p.ldb;
      c_row = row_off[g];
    } else {
      g = static_cast<int>(u / (nt * ct));
      const int64_t local = u % (nt * ct);
      i0 = local / ct * 64;
      j0 = local % ct * 64;
      rows = p.N;
      kdim = row_off[g + 1] - row_off[g];
      ab = row_off[g] * p.lda;
      a_i = 1;
      a_k = p.lda;
      bb = row_off[g] * p.ldb;
      b_j = 1;
      b_k = p.ldb;
      c_row = static_cast<int64_t>(g) * p.N;
    }
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < kdim; k0 += 16) {
      for (int e = threadIdx.x; e < 1024; e += 256) {
        const int ka = a_k == 1 ? e % 16 : e / 64, ia = a_k == 1 ? e / 16 : e % 64;
        const int kb = b_k == 1 ? e % 16 : e / 64, jb = b_k == 1 ? e / 16 : e % 64;
        as[ka][ia] = (i0 + ia < rows && k0 + ka < kdim)
                         ? ld16(p.A + ab + (i0 + ia) * a_i + (k0 + ka) * a_k, p.in_f16) : 0.0f;
        bs[kb][jb] = (j0 + jb < out_cols && k0 + kb < kdim)
                         ? ld16(p.B + bb + (j0 + jb) * b_j + (k0 + kb) * b_k, p.in_f16) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty + 16 * i] * bs[k][tx + 16 * j];
      __syncthreads();
    }
    const float al = p.alpha ? p.alpha[g] : 1.0f, be = p.beta ? p.beta[g] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
        if (r >= rows || c >= out_cols) continue;
        const int64_t at = (c_row + r) * p.ldc + c;
        float v = al * acc[i][j];
        if (p.out_type == MXG_F32) {
          float* o = static_cast<float*>(p.C) + at;
          if (be != 0.0f) v += be * *o;
          *o = v;
        } else if (p.out_type == MXG_BF16) {
          Bf16* o = static_cast<Bf16*>(p.C) + at;
          if (be != 0.0f) v += be * to_f32(*o);
          *o = from_f32<Bf16>(v);
        } else {
          F16* o = static_cast<F16*>(p.C) + at;
          if (be != 0.0f) v += be * to_f32(*o);
          *o = from_f32<F16>(v);
        }
      }
  }
}

cudaError_t launch_grouped_gemm16(int in_f16, int mode, const void* A, int64_t lda, const void* B,
                                  int64_t ldb, const int64_t* group_ws, int G, int64_t M_cap,
                                  int64_t N, int64_t K, const float* alpha, const float* beta,
                                  void* C, int64_t ldc, int out_type, int32_t* status, int num_sms,
                                  cudaStream_t stream) {
  Gemm16Params p{static_cast<const uint16_t*>(A), static_cast<const uint16_t*>(B), group_ws, alpha,
                 beta, C, status, M_cap, N, K, lda, ldb, ldc, G, mode, in_f16, out_type};
  gemm16_simple_kernel<<<num_sms * 4, 256, 8 * (G + 1), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mxg
