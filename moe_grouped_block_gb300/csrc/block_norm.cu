// block_norm.cu -- the norms on both sides of a residual block, fused with the
// block's gate and residual scale (root-mean-square norms over `cols`):
//   after  : x' = x + s * gate . (y * ry . w_post),   ry = 1 / sqrt(mean(y^2) + eps)
//   before : n  = x' * rx . w_pre,                    rx = 1 / sqrt(mean(x'^2) + eps)
// Sums are fp32; n is formed from x' before x' is rounded to its type.
//
// Each input is read once and each output written once (rows.cuh), so the
// memory bandwidth is the bound; the row stays in registers between the two
// reductions.  16384 x 4096 in bf16: 93 us, 5.8 TB/s of the 6.78 that a copy
// reaches.  One row: 4 us, of which the two reductions take the most.
#include "rows.cuh"

namespace mxg {

// COMMON: both parts and no full gate, known when compiled -- with these left to
// run time, a row costs a thread some 200 instructions beside the arithmetic on
// its 8 or 16 columns, a third of all.
template <typename T, typename R, bool VEC, int ITER, int MAXT, bool COMMON>
__global__ void __launch_bounds__(MAXT, 1) block_norm_kernel(const mxg_block_norm_t p, int team,
                                                          int depth) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32];
  const int nt = blockDim.x, teams = nt / team;
  const int lane = threadIdx.x % team, team_id = threadIdx.x / team;
  const int cols = static_cast<int>(p.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  const bool has_y = COMMON || p.y != nullptr, has_n = COMMON || p.n_out != nullptr;
  const bool full = !COMMON && p.gate_mode == MXG_GATE_FULL;
  const int r_bytes = kHalves<R> * nt * 16, t_bytes = kHalves<T> * nt * 16;
  const int at_g = r_bytes + t_bytes;
  const int chunk_bytes = r_bytes + (has_y ? t_bytes : 0) + (full ? t_bytes : 0);
  const int slot_bytes = ITER * chunk_bytes, ring_bytes = depth * slot_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + ring_bytes;
  if (VEC) ring_clear(mine, ring_bytes, nt);
  const int c0 = RowIo<T, VEC>::col(0, 0, lane, team);
  const int dc = RowIo<T, VEC>::col(1, 0, lane, team) - c0;  // from one chunk to the next

  int64_t f_row = static_cast<int64_t>(blockIdx.x) * teams + team_id;  // the row filled next
  uint32_t f_at = mine;                                                // and where to
  const R* x = static_cast<const R*>(p.x) + f_row * p.ldx + c0;
  const T* y = static_cast<const T*>(p.y) + f_row * p.ldy + c0;
  R* x_out = static_cast<R*>(p.x_out) + f_row * p.ldxo;
  T* n_out = static_cast<T*>(p.n_out) + f_row * p.ldn;
  const int64_t dx = step * p.ldx, dy = step * p.ldy, dxo = step * p.ldxo, dn = step * p.ldn;
  auto fill = [&] {
    if (f_row < p.rows) {
      const T* g = static_cast<const T*>(p.gate) + f_row * p.ldg + c0;
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const uint32_t at = f_at + it * chunk_bytes;
        const bool in = c0 + it * dc < cols;
        ring_fill<R, VEC>(at, x + it * dc, in, cols, it, lane, team, nt);
        if (has_y) ring_fill<T, VEC>(at + r_bytes, y + it * dc, in, cols, it, lane, team, nt);
        if (full) ring_fill<T, VEC>(at + at_g, g + it * dc, in, cols, it, lane, team, nt);
      }
    } else {
      ring_clear(f_at, slot_bytes, nt);  // a team past the last row adds nothing
    }
    if (VEC) cp_async_commit();
    f_row += step;
    x += dx;
    y += dy;
    if ((f_at += slot_bytes) == end) f_at = mine;
  };
  int64_t row = f_row;
  for (int d = 0; d < depth - 1; ++d) fill();
  using W = Weight<T, VEC, ITER, MAXT <= 512>;
  const W w_post(p.w_post, 0, cols, lane, team);
  const W g_col(p.gate_mode == MXG_GATE_COL ? p.gate : nullptr, 0, cols, lane, team);
  const W w_pre(p.w_pre, 0, cols, lane, team);

  // a row's gate is asked for a row ahead: its latency is that of memory
  const bool g_row = p.gate_mode == MXG_GATE_ROW;
  auto row_gate = [&](int64_t r) {
    return g_row && r < p.rows ? static_cast<const float*>(p.gate)[r] : 1.0f;
  };
  float gr = row_gate(row);
  uint32_t at0 = mine;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams; base < p.rows; base += step) {
    const int limit = row < p.rows ? cols : 0;  // a team past the last row stores nothing
    fill();
    if (VEC) cp_async_wait(depth - 1);
    const float gr_next = row_gate(row + step);

    F2 s[ITER][4];  // the stream
#pragma unroll
    for (int it = 0; it < ITER; ++it) ring_read<R>(at0 + it * chunk_bytes, nt, s[it]);
    if (has_y) {
      F2 b[ITER][4], q = 0;  // the block's output
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        ring_read<T>(at0 + it * chunk_bytes + r_bytes, nt, b[it]);
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(b[it][i], b[it][i], q);
      }
      const float r = rsqrtf(team_sum(sum2(q), red[0], team) * inv + p.eps) * p.res_scale * gr;
      const F2 r2 = f2(r);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        w_post.apply(it, b[it]);
        if (p.gate_mode == MXG_GATE_COL) g_col.apply(it, b[it]);
        if (full) {
          F2 g[4];
          ring_read<T>(at0 + it * chunk_bytes + at_g, nt, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) b[it][i] = mul2(b[it][i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[it][i] = fma2(b[it][i], r2, s[it][i]);
        RowIo<R, VEC>::store(x_out, limit, it, lane, team, s[it]);
      }
    }
    if (has_n) {
      F2 q = 0;
#pragma unroll
      for (int it = 0; it < ITER; ++it)
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(s[it][i], s[it][i], q);
      const F2 r2 = f2(rsqrtf(team_sum(sum2(q), red[1], team) * inv + p.eps));
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        w_pre.apply(it, s[it]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[it][i] = mul2(s[it][i], r2);
        RowIo<T, VEC>::store(n_out, limit, it, lane, team, s[it]);
      }
    }
    // one buffer in use: order its reuse
    if (team > 32 && !(has_y && has_n)) __syncthreads();
    gr = gr_next;
    row += step;
    x_out += dxo;
    n_out += dn;
    if ((at0 += slot_bytes) == end) at0 = mine;
  }
}

namespace {

// up to 98 registers a thread at 8 columns, 115 at 16 (64 in CTAs of 1024)
constexpr RowLimits kFwdLimits = {256, {256, 1024}, {640, 512}, 1 << 30};
static_assert(kFwdLimits.split_at >= kMaxRowCols, "the forward kernel's rows are not shared");

template <typename T, typename R, bool VEC, bool COMMON>
cudaError_t forward_rows(const mxg_block_norm_t& p, const RowShape& r, int64_t grid, int smem,
                         int depth, cudaStream_t stream) {
  if (r.iter == 1)
    return launch_rows<block_norm_kernel<T, R, VEC, 1, 256, COMMON>>(r, grid, smem, stream, p,
                       r.team, depth);
  if (r.threads <= 512)
    return launch_rows<block_norm_kernel<T, R, VEC, 2, 512, COMMON>>(r, grid, smem, stream, p,
                       r.team, depth);
  return launch_rows<block_norm_kernel<T, R, VEC, 2, 1024, COMMON>>(r, grid, smem, stream, p,
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
  const RowShape r = row_shape(p.cols, kFwdLimits);
  // twice as many CTAs as an SM holds where that is more than one, so that the
  // slower SMs end up with fewer (16384 x 4096: 92 us, 96 us with one wave; 4096
  // x 8192, one CTA an SM: 97 us with two, 95 us with one)
  const int ctas = row_ctas(r, kFwdLimits, 16);
  const int waves = ctas > 1 ? 2 : 1;
  const int64_t teams = r.threads / r.team;
  const int64_t grid = std::min<int64_t>((p.rows + teams - 1) / teams,
                                         static_cast<int64_t>(num_sms) * ctas * waves);
  // at most 192 KB a slot: 16384 columns of three fp32 inputs
  const int slot = r.threads * 8 * r.iter *
                   static_cast<int>(sizeof(R) + (p.y ? sizeof(T) : 0) + (full ? sizeof(T) : 0));
  const int64_t each = (p.rows + grid * teams - 1) / (grid * teams);  // rows a team walks
  const int depth = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({vec ? 4 : 2, kRowSmem / ctas / slot, each})));
  const bool common = p.y != nullptr && p.n_out != nullptr && !full;
  if (!vec)
    return common ? forward_rows<T, R, false, true>(p, r, grid, slot * depth, depth, stream)
                  : forward_rows<T, R, false, false>(p, r, grid, slot * depth, depth, stream);
  return common ? forward_rows<T, R, true, true>(p, r, grid, slot * depth, depth, stream)
                : forward_rows<T, R, true, false>(p, r, grid, slot * depth, depth, stream);
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
