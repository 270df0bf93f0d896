// block_norm.cu -- the norms on both sides of a residual block, fused with the
// block's gate and residual scale (root-mean-square norms over `cols`):
//   after  : x' = x + s * gate . (y * ry . w_post),   ry = 1 / sqrt(mean(y^2) + eps)
//   before : n  = x' * rx . w_pre,                    rx = 1 / sqrt(mean(x'^2) + eps)
// and their gradients.  With xh = x' rx, yh = y ry, v = s * gate, and the
// gradients dx' and dn given:
//   a = dn . w_pre,  t = dx' + rx (a - xh mean(a . xh)),  dx = t
//   b = t . v . w_post,  dy = ry (b - yh mean(b . yh))
//   dw_pre = sum_rows dn . xh,  dw_post = sum_rows t . v . yh
//   dgate = s t . yh . w_post, summed over the axes the gate is broadcast along
// Every sum is fp32; n is formed from x' before x' is rounded to its type.
//
// One CTA owns a row and keeps it in registers, so each input is read once and
// each output written once: the memory bandwidth is the bound.
#include "elem.cuh"
#include "mxg_host.h"

namespace mxg {

constexpr int kNormMaxBlocks = 304;  // CTAs of the backward kernel: partial sums per column

template <typename T, bool VEC>
struct RowIo {
  // element index of (chunk it, slot e) of thread tid among nt threads
  static __device__ __forceinline__ int64_t index(int it, int e, int tid, int nt) {
    return VEC ? (static_cast<int64_t>(it) * nt + tid) * 8 + e
               : (static_cast<int64_t>(it) * 8 + e) * nt + tid;
  }
  static __device__ __forceinline__ void load(const T* row, int64_t cols, int it, int tid, int nt,
                                              float (&f)[8]) {
    if constexpr (VEC) {
      const int64_t c = index(it, 0, tid, nt);
      if (c < cols) {
        unpack8<T>(load8<T>(row + c), f);
        return;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.0f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t c = index(it, e, tid, nt);
        f[e] = c < cols ? to_f32(row[c]) : 0.0f;
      }
    }
  }
  static __device__ __forceinline__ void store(T* row, int64_t cols, int it, int tid, int nt,
                                               const float (&f)[8]) {
    if constexpr (VEC) {
      const int64_t c = index(it, 0, tid, nt);
      if (c < cols) store8<T>(row + c, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t c = index(it, e, tid, nt);
        if (c < cols) row[c] = from_f32<T>(f[e]);
      }
    }
  }
};

// Sums of NV values over the CTA, in a fixed order; `buf` holds 32 * NV floats
// and is not written again before another block_sum (on another buffer) has
// passed.
template <int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float* buf) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[i * 32 + w] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = lane < warps ? buf[i * 32 + lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  }
}

template <typename T, typename R, bool VEC, int ITER>
__global__ void __launch_bounds__(1024) block_norm_kernel(const mxg_block_norm_t p) {
  __shared__ float red[2][32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const float inv = 1.0f / static_cast<float>(p.cols);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float x[ITER][8];
#pragma unroll
    for (int it = 0; it < ITER; ++it)
      RowIo<R, VEC>::load(static_cast<const R*>(p.x) + row * p.ldx, p.cols, it, tid, nt, x[it]);
    if (p.y != nullptr) {
      float y[ITER][8], s[1] = {0.0f};
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        RowIo<T, VEC>::load(static_cast<const T*>(p.y) + row * p.ldy, p.cols, it, tid, nt, y[it]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += y[it][e] * y[it][e];
      }
      block_sum(s, red[0]);
      float r = rsqrtf(s[0] * inv + p.eps) * p.res_scale;
      if (p.gate_mode == MXG_GATE_ROW) r *= static_cast<const float*>(p.gate)[row];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        float w[8];
        if (p.w_post != nullptr) {
          RowIo<T, VEC>::load(static_cast<const T*>(p.w_post), p.cols, it, tid, nt, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[it][e] *= w[e];
        }
        if (p.gate_mode >= MXG_GATE_COL) {
          RowIo<T, VEC>::load(static_cast<const T*>(p.gate) +
                                  (p.gate_mode == MXG_GATE_FULL ? row * p.ldg : 0),
                              p.cols, it, tid, nt, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[it][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[it][e] += r * y[it][e];
        RowIo<R, VEC>::store(static_cast<R*>(p.x_out) + row * p.ldxo, p.cols, it, tid, nt, x[it]);
      }
    }
    if (p.n_out != nullptr) {
      float s[1] = {0.0f};
#pragma unroll
      for (int it = 0; it < ITER; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += x[it][e] * x[it][e];
      block_sum(s, red[1]);
      const float r = rsqrtf(s[0] * inv + p.eps);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        float w[8];
        if (p.w_pre != nullptr) {
          RowIo<T, VEC>::load(static_cast<const T*>(p.w_pre), p.cols, it, tid, nt, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[it][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[it][e] *= r;
        RowIo<T, VEC>::store(static_cast<T*>(p.n_out) + row * p.ldn, p.cols, it, tid, nt, x[it]);
      }
    }
    if (p.y == nullptr || p.n_out == nullptr) __syncthreads();  // one buffer in use: order its reuse
  }
}

// Backward.  Column sums of this CTA's rows go to the workspace
// [block][2][cols]: S0 = sum dn . xh, S1 = sum t . u . yh with u the gate where
// it varies over rows (row, full) and 1 otherwise; the finish kernel applies
// what is constant down a column.
template <typename T, typename R, bool VEC, int ITER>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(const mxg_block_norm_grad_t p,
                                                              float* ws) {
  __shared__ float red[2][96];
  const int tid = threadIdx.x, nt = blockDim.x;
  const float inv = 1.0f / static_cast<float>(p.cols);
  const bool has_y = p.y != nullptr, has_n = p.dn != nullptr;
  float s0[ITER][8] = {}, s1[ITER][8] = {};
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float t[ITER][8], y[ITER][8], v[3] = {0.0f, 0.0f, 0.0f};
    float x[ITER][8], a[ITER][8];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[it][e] = y[it][e] = 0.0f;
      if (p.dx_out != nullptr)
        RowIo<R, VEC>::load(static_cast<const R*>(p.dx_out) + row * p.lddxo, p.cols, it, tid, nt,
                            t[it]);
      if (has_y) {
        RowIo<T, VEC>::load(static_cast<const T*>(p.y) + row * p.ldy, p.cols, it, tid, nt, y[it]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[2] += y[it][e] * y[it][e];
      }
      if (has_n) {
        RowIo<R, VEC>::load(static_cast<const R*>(p.x) + row * p.ldx, p.cols, it, tid, nt, x[it]);
        RowIo<T, VEC>::load(static_cast<const T*>(p.dn) + row * p.lddn, p.cols, it, tid, nt, a[it]);
        float w[8];
        if (p.w_pre != nullptr)
          RowIo<T, VEC>::load(static_cast<const T*>(p.w_pre), p.cols, it, tid, nt, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[0] += x[it][e] * x[it][e];
          v[1] += (p.w_pre != nullptr ? a[it][e] * w[e] : a[it][e]) * x[it][e];
        }
      }
    }
    block_sum(v, red[0]);
    const float ry = rsqrtf(v[2] * inv + p.eps);
    if (has_n) {
      const float rx = rsqrtf(v[0] * inv + p.eps);
      const float c = v[1] * inv * rx;  // mean(a . xh)
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        float w[8];
        if (p.w_pre != nullptr)
          RowIo<T, VEC>::load(static_cast<const T*>(p.w_pre), p.cols, it, tid, nt, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = x[it][e] * rx;
          s0[it][e] += a[it][e] * xh;
          const float aw = p.w_pre != nullptr ? a[it][e] * w[e] : a[it][e];
          t[it][e] += rx * (aw - xh * c);
        }
      }
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it)
      RowIo<R, VEC>::store(static_cast<R*>(p.dx) + row * p.lddx, p.cols, it, tid, nt, t[it]);
    if (has_y) {
      // b = t . w_post . (gate where it varies along the row); the rest of v
      // is the factor f of the whole row
      float f = p.res_scale;
      const float gr =
          p.gate_mode == MXG_GATE_ROW ? static_cast<const float*>(p.gate)[row] : 1.0f;
      f *= gr;
      float q[1] = {0.0f};
      float b[ITER][8];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        float w[8], gt[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[it][e] = t[it][e];
        if (p.w_post != nullptr) {
          RowIo<T, VEC>::load(static_cast<const T*>(p.w_post), p.cols, it, tid, nt, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) b[it][e] *= w[e];
        }
        if (p.gate_mode >= MXG_GATE_COL) {
          RowIo<T, VEC>::load(static_cast<const T*>(p.gate) +
                                  (p.gate_mode == MXG_GATE_FULL ? row * p.ldg : 0),
                              p.cols, it, tid, nt, gt);
          if (p.gate_mode == MXG_GATE_FULL) {
            if (p.dgate != nullptr) {
              float dg[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) dg[e] = p.res_scale * b[it][e] * (y[it][e] * ry);
              RowIo<T, VEC>::store(static_cast<T*>(p.dgate) + row * p.lddg, p.cols, it, tid, nt,
                                   dg);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) t[it][e] *= gt[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) b[it][e] *= gt[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          q[0] += b[it][e] * y[it][e];
          s1[it][e] += t[it][e] * gr * (y[it][e] * ry);
        }
      }
      block_sum(q, red[1]);
      if (p.gate_mode == MXG_GATE_ROW && p.dgate != nullptr && tid == 0)
        static_cast<float*>(p.dgate)[row] = p.res_scale * ry * q[0];
      const float m = q[0] * inv * ry;  // mean(b . yh) / f
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[it][e] = f * ry * (b[it][e] - y[it][e] * ry * m);
        RowIo<T, VEC>::store(static_cast<T*>(p.dy) + row * p.lddy, p.cols, it, tid, nt, b[it]);
      }
    } else {
      __syncthreads();
    }
  }
  float* out = ws + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
#pragma unroll
  for (int it = 0; it < ITER; ++it)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = RowIo<T, VEC>::index(it, e, tid, nt);
      if (c < p.cols) {
        out[c] = s0[it][e];
        out[p.cols + c] = s1[it][e];
      }
    }
}

// Column sums of `blocks` partial rows, in a fixed order: 32 columns a CTA,
// 8 threads a column.
template <typename T>
__global__ void __launch_bounds__(256) block_norm_bwd_finish_kernel(const mxg_block_norm_grad_t p,
                                                                    const float* ws, int blocks) {
  __shared__ float part[2][8][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float a0 = 0.0f, a1 = 0.0f;
  if (c < p.cols)
    for (int b = slice; b < blocks; b += 8) {
      a0 += ws[static_cast<int64_t>(b) * 2 * p.cols + c];
      a1 += ws[static_cast<int64_t>(b) * 2 * p.cols + p.cols + c];
    }
  part[0][slice][lane] = a0;
  part[1][slice][lane] = a1;
  __syncthreads();
  if (slice != 0 || c >= p.cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    a0 += part[0][i][lane];
    a1 += part[1][i][lane];
  }
  if (p.dw_pre != nullptr) p.dw_pre[c] = a0;
  a1 *= p.res_scale;
  const bool col = p.gate_mode == MXG_GATE_COL;
  if (p.dw_post != nullptr)
    p.dw_post[c] = col ? a1 * to_f32(static_cast<const T*>(p.gate)[c]) : a1;
  if (col && p.dgate != nullptr)
    static_cast<float*>(p.dgate)[c] =
        p.w_post != nullptr ? a1 * to_f32(static_cast<const T*>(p.w_post)[c]) : a1;
}

namespace {

bool aligned_rows(const void* p, int64_t ld, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * static_cast<int64_t>(size)) % 16 == 0;
}

template <typename T, typename R>
cudaError_t norm_forward(const mxg_block_norm_t& p, int num_sms, cudaStream_t stream) {
  const bool full = p.gate_mode == MXG_GATE_FULL;
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, sizeof(R)) &&
                   aligned_rows(p.y, p.ldy, sizeof(T)) && aligned_rows(p.x_out, p.ldxo, sizeof(R)) &&
                   aligned_rows(p.n_out, p.ldn, sizeof(T)) && aligned_rows(p.w_post, 0, sizeof(T)) &&
                   aligned_rows(p.w_pre, 0, sizeof(T)) &&
                   (p.gate_mode < MXG_GATE_COL || aligned_rows(p.gate, full ? p.ldg : 0, sizeof(T)));
  const int iter = p.cols > 8192 ? 2 : 1;
  const int64_t per = 8 * iter;
  const int nt = static_cast<int>(((p.cols + per - 1) / per + 31) / 32 * 32);
  int64_t grid = static_cast<int64_t>(num_sms) * (2048 / nt);
  if (grid > p.rows) grid = p.rows;
  const dim3 g(static_cast<unsigned>(grid));
  if (vec && iter == 1) block_norm_kernel<T, R, true, 1><<<g, nt, 0, stream>>>(p);
  else if (vec) block_norm_kernel<T, R, true, 2><<<g, nt, 0, stream>>>(p);
  else if (iter == 1) block_norm_kernel<T, R, false, 1><<<g, nt, 0, stream>>>(p);
  else block_norm_kernel<T, R, false, 2><<<g, nt, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, typename R>
cudaError_t norm_backward(const mxg_block_norm_grad_t& p, float* ws, int num_sms,
                          cudaStream_t stream) {
  const bool full = p.gate_mode == MXG_GATE_FULL;
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, sizeof(R)) &&
                   aligned_rows(p.y, p.ldy, sizeof(T)) &&
                   aligned_rows(p.dx_out, p.lddxo, sizeof(R)) &&
                   aligned_rows(p.dn, p.lddn, sizeof(T)) && aligned_rows(p.dx, p.lddx, sizeof(R)) &&
                   aligned_rows(p.dy, p.lddy, sizeof(T)) && aligned_rows(p.w_post, 0, sizeof(T)) &&
                   aligned_rows(p.w_pre, 0, sizeof(T)) &&
                   (p.gate_mode < MXG_GATE_COL || aligned_rows(p.gate, full ? p.ldg : 0, sizeof(T))) &&
                   (!full || aligned_rows(p.dgate, p.lddg, sizeof(T)));
  const int iter = p.cols > 8192 ? 2 : 1;
  const int64_t per = 8 * iter;
  const int nt = static_cast<int>(((p.cols + per - 1) / per + 31) / 32 * 32);
  int64_t grid = 2 * num_sms;
  if (grid > kNormMaxBlocks) grid = kNormMaxBlocks;
  if (grid > p.rows) grid = p.rows;
  const dim3 g(static_cast<unsigned>(grid));
  if (grid > 0) {
    if (vec && iter == 1) block_norm_bwd_kernel<T, R, true, 1><<<g, nt, 0, stream>>>(p, ws);
    else if (vec) block_norm_bwd_kernel<T, R, true, 2><<<g, nt, 0, stream>>>(p, ws);
    else if (iter == 1) block_norm_bwd_kernel<T, R, false, 1><<<g, nt, 0, stream>>>(p, ws);
    else block_norm_bwd_kernel<T, R, false, 2><<<g, nt, 0, stream>>>(p, ws);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  block_norm_bwd_finish_kernel<T><<<static_cast<unsigned>((p.cols + 31) / 32), 256, 0, stream>>>(
      p, ws, static_cast<int>(grid));
  return cudaGetLastError();
}

}  // namespace

int64_t block_norm_ws_bytes(int64_t rows, int64_t cols) {
  return (rows < kNormMaxBlocks ? rows : kNormMaxBlocks) * 2 * cols * 4;
}

cudaError_t launch_block_norm(const mxg_block_norm_t& p, int num_sms, cudaStream_t stream) {
  if (p.dtype == MXG_F32) return norm_forward<float, float>(p, num_sms, stream);
  if (p.dtype == MXG_BF16)
    return p.res_dtype == MXG_F32 ? norm_forward<Bf16, float>(p, num_sms, stream)
                                  : norm_forward<Bf16, Bf16>(p, num_sms, stream);
  return p.res_dtype == MXG_F32 ? norm_forward<F16, float>(p, num_sms, stream)
                                : norm_forward<F16, F16>(p, num_sms, stream);
}

cudaError_t launch_block_norm_backward(const mxg_block_norm_grad_t& p, float* ws, int num_sms,
                                       cudaStream_t stream) {
  if (p.dtype == MXG_F32) return norm_backward<float, float>(p, ws, num_sms, stream);
  if (p.dtype == MXG_BF16)
    return p.res_dtype == MXG_F32 ? norm_backward<Bf16, float>(p, ws, num_sms, stream)
                                  : norm_backward<Bf16, Bf16>(p, ws, num_sms, stream);
  return p.res_dtype == MXG_F32 ? norm_backward<F16, float>(p, ws, num_sms, stream)
                                : norm_backward<F16, F16>(p, ws, num_sms, stream);
}

}  // namespace mxg
