// block_norm.cu -- the norms on both sides of a residual block, fused with the
// block's gate and residual scale (root-mean-square norms over `cols`):
//   after  : x' = x + s * gate . (y * ry . w_post),   ry = 1 / sqrt(mean(y^2) + eps)
//   before : n  = x' * rx . w_pre,                    rx = 1 / sqrt(mean(x'^2) + eps)
// Sums are fp32; n is formed from x' before x' is rounded to its type.
//
// Each input is read once and each output written once (rows.cuh), so the
// memory bandwidth is the bound; the row stays in registers between the two
// reductions.
#include "rows.cuh"

namespace mxg {

template <typename T, typename R, bool VEC, int ITER, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const mxg_block_norm_t p, int team,
                                                          int depth) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32];
  const int nt = blockDim.x, teams = nt / team;
  const int lane = threadIdx.x % team, cols = static_cast<int>(p.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  const bool has_y = p.y != nullptr, has_n = p.n_out != nullptr;
  const bool full = p.gate_mode == MXG_GATE_FULL;
  const int r_bytes = kHalves<R> * nt * 16, t_bytes = kHalves<T> * nt * 16;
  const int at_g = r_bytes + t_bytes;
  const int chunk_bytes = r_bytes + (has_y ? t_bytes : 0) + (full ? t_bytes : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t base0 = static_cast<int64_t>(blockIdx.x) * teams;
  const int team_id = threadIdx.x / team;
  uint8_t* mine = ring + threadIdx.x * 16;

  auto slot_at = [&](int slot, int it) { return mine + (slot * ITER + it) * chunk_bytes; };
  auto fill = [&](int64_t base, int slot) {
    const int64_t row = base + team_id;
    const int limit = row < p.rows ? cols : 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      uint8_t* at = slot_at(slot, it);
      ring_fill<R, VEC>(at, static_cast<const R*>(p.x) + row * p.ldx, limit, it, lane, team, nt);
      if (has_y)
        ring_fill<T, VEC>(at + r_bytes, static_cast<const T*>(p.y) + row * p.ldy, limit, it, lane,
                          team, nt);
      if (full)
        ring_fill<T, VEC>(at + at_g, static_cast<const T*>(p.gate) + row * p.ldg, limit, it, lane,
                          team, nt);
    }
    if (VEC) cp_async_commit();
  };
  for (int d = 0; d < depth - 1; ++d) fill(base0 + d * step, d);
  const Weight<T, VEC, ITER> w_post(has_y ? p.w_post : nullptr, cols, lane, team);
  const Weight<T, VEC, ITER> g_col(p.gate_mode == MXG_GATE_COL ? p.gate : nullptr, cols, lane, team);
  const Weight<T, VEC, ITER> w_pre(has_n ? p.w_pre : nullptr, cols, lane, team);

  int slot = 0;
  for (int64_t base = base0; base < p.rows; base += step) {
    const int64_t row = base + team_id;
    const bool live = row < p.rows;
    const int limit = live ? cols : 0;  // a team past the last row loads and stores nothing
    const int ahead = slot + depth - 1 >= depth ? slot - 1 : slot + depth - 1;
    fill(base + (depth - 1) * step, ahead);
    if (VEC) cp_async_wait(depth - 1);

    F2 x[ITER][4];
#pragma unroll
    for (int it = 0; it < ITER; ++it)
      ring_read<R, VEC>(slot_at(slot, it), limit, it, lane, team, nt, x[it]);
    if (has_y) {
      F2 y[ITER][4], q = 0;
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        ring_read<T, VEC>(slot_at(slot, it) + r_bytes, limit, it, lane, team, nt, y[it]);
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(y[it][i], y[it][i], q);
      }
      float s[1] = {sum2(q)};
      team_sum(s, red[0], team);
      float r = rsqrtf(s[0] * inv + p.eps) * p.res_scale;
      if (p.gate_mode == MXG_GATE_ROW && live) r *= static_cast<const float*>(p.gate)[row];
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        w_post.apply(it, y[it]);
        g_col.apply(it, y[it]);
        if (full) {
          F2 g[4];
          ring_read<T, VEC>(slot_at(slot, it) + at_g, limit, it, lane, team, nt, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[it][i] = mul2(y[it][i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[it][i] = fma2(y[it][i], f2(r), x[it][i]);
        RowIo<R, VEC>::store(static_cast<R*>(p.x_out) + row * p.ldxo, limit, it, lane, team, x[it]);
      }
    }
    if (has_n) {
      F2 q = 0;
#pragma unroll
      for (int it = 0; it < ITER; ++it)
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(x[it][i], x[it][i], q);
      float s[1] = {sum2(q)};
      team_sum(s, red[1], team);
      const float r = rsqrtf(s[0] * inv + p.eps);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        w_pre.apply(it, x[it]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[it][i] = mul2(x[it][i], f2(r));
        RowIo<T, VEC>::store(static_cast<T*>(p.n_out) + row * p.ldn, limit, it, lane, team, x[it]);
      }
    }
    // one buffer in use: order its reuse
    if (team > 32 && !(has_y && has_n)) __syncthreads();
    if (++slot >= depth) slot = 0;
  }
}

namespace {

template <typename T, typename R, bool VEC>
cudaError_t forward_rows(const mxg_block_norm_t& p, const RowShape& r, int64_t grid, int smem,
                         int depth, cudaStream_t stream) {
  if (r.iter == 1)
    return launch_rows(block_norm_kernel<T, R, VEC, 1, 256>, grid, r.threads, smem, stream, p,
                       r.team, depth);
  if (r.threads <= 512)
    return launch_rows(block_norm_kernel<T, R, VEC, 2, 512>, grid, r.threads, smem, stream, p,
                       r.team, depth);
  return launch_rows(block_norm_kernel<T, R, VEC, 2, 1024>, grid, r.threads, smem, stream, p,
                     r.team, depth);
}

template <typename T, typename R>
cudaError_t norm_forward(const mxg_block_norm_t& p, int num_sms, cudaStream_t stream) {
  const bool full = p.gate_mode == MXG_GATE_FULL;
  const bool vec = p.cols % 8 == 0 && aligned_rows(p.x, p.ldx, sizeof(R)) &&
                   aligned_rows(p.y, p.ldy, sizeof(T)) && aligned_rows(p.x_out, p.ldxo, sizeof(R)) &&
                   aligned_rows(p.n_out, p.ldn, sizeof(T)) && aligned_rows(p.w_post, 0, sizeof(T)) &&
                   aligned_rows(p.w_pre, 0, sizeof(T)) &&
                   (p.gate_mode < MXG_GATE_COL || aligned_rows(p.gate, full ? p.ldg : 0, sizeof(T)));
  const RowShape r = row_shape(p.cols, 256);
  const int ctas = std::max(1, std::min(8, 768 / r.threads));  // per SM
  const int64_t teams = r.threads / r.team;
  const int64_t grid =
      std::min<int64_t>((p.rows + teams - 1) / teams, static_cast<int64_t>(num_sms) * ctas);
  // at most 192 KB a slot: 16384 columns of three fp32 inputs
  const int slot = r.threads * 8 * r.iter *
                   static_cast<int>(sizeof(R) + (p.y ? sizeof(T) : 0) + (full ? sizeof(T) : 0));
  const int depth = std::max(1, std::min(vec ? 4 : 2, kRowSmem / ctas / slot));
  if (vec) return forward_rows<T, R, true>(p, r, grid, slot * depth, depth, stream);
  return forward_rows<T, R, false>(p, r, grid, slot * depth, depth, stream);
}

}  // namespace

cudaError_t launch_block_norm(const mxg_block_norm_t& p, int num_sms, cudaStream_t stream) {
  if (p.dtype == MXG_F32) return norm_forward<float, float>(p, num_sms, stream);
  if (p.dtype == MXG_BF16)
    return p.res_dtype == MXG_F32 ? norm_forward<Bf16, float>(p, num_sms, stream)
                                  : norm_forward<Bf16, Bf16>(p, num_sms, stream);
  return p.res_dtype == MXG_F32 ? norm_forward<F16, float>(p, num_sms, stream)
                                : norm_forward<F16, F16>(p, num_sms, stream);
}

}  // namespace mxg
