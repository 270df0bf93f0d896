// block_norm_bwd.cu -- the gradients of the norms around a residual block
// (block_norm.cu).  With xh = x' rx, yh = y ry, v = s * gate, and the gradients
// dx' and dn given:
//   a = dn . w_pre,  t = dx' + rx (a - xh mean(a . xh)),  dx = t
//   b = t . v . w_post,  dy = ry (b - yh mean(b . yh))
//   dw_pre = sum_rows dn . xh,  dw_post = sum_rows t . v . yh
//   dgate = s t . yh . w_post, summed over the axes the gate is broadcast along
// rx and ry are made again from x' and y, which are read anyway.
//
// One pass over the rows (rows.cuh).  Two reductions make a row: rx, ry and
// mean(a . xh), then mean(b . yh).  The first is taken a row ahead, together with
// the second one of the row before, so that a row costs one barrier.  The
// column sums of a CTA's rows stay in registers and leave one partial row per
// CTA; a second kernel adds those in a fixed order.
//
// Memory is the bound: 16384 x 4096 in bf16 takes 137 us, 5.9 TB/s of the 6.78
// that a copy reaches, the second kernel's 7 us among them.  2777 x 7168 beside an
// fp32 stream: 88 us, 4.1 TB/s -- one CTA an SM, whose ring holds two rows, and a
// barrier every row.
//
// Rows of more than 8192 columns are shared by two CTAs, whose warps post their
// sums to each other: one of 1024 threads would leave 64 registers a thread, and
// spilled 400 bytes (4096 x 16384: 346 us so, 207 us shared).
#include "rows.cuh"

namespace mxg {

// CTAs of the backward kernel: as many partial rows as the workspace has room
// for.  160 bounds the SM count; a thread takes some 120 registers.
constexpr int kNormMaxSms = 160;
constexpr RowLimits kBwdLimits = {128, {512, 512}, {512, 512}, 8192};
// A shared row runs the kernel of 16 columns a thread, and its ring is sized by the
// columns a thread that row_shape gives: 16 wherever a CTA's part is not narrow.
static_assert(kBwdLimits.split_at >= 2 * kNarrowCols, "a shared row has 16 columns a thread");

// Column sums of this CTA's rows go to the workspace [block][2][cols]:
// S0 = sum dn . xh, S1 = sum t . u . yh with u the gate where it varies over
// rows (row, full) and 1 otherwise; the finish kernel applies what is constant
// down a column.
// lean: dx' and a full gate do not come through the ring (rows so wide that it
// would not hold two of them).
// COMMON: all inputs, no full gate and not lean, known when compiled.
template <typename T, typename R, bool VEC, int ITER, int SPLIT, bool COMMON>
__global__ void __launch_bounds__(512, 1) block_norm_bwd_kernel(const mxg_block_norm_grad_t p,
                                                              float* ws, int team, int depth,
                                                              bool is_lean) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[3][128];
  const int nt = blockDim.x, teams = nt / team;
  const int lane = threadIdx.x % team, team_id = threadIdx.x / team;
  // this CTA's columns: cols of them from off on
  const int64_t off = SPLIT == 1 ? 0 : cluster_ctarank() * cols_per_cta(p.cols, SPLIT);
  const int cols = static_cast<int>(SPLIT == 1 ? p.cols
                                               : min(p.cols - off, cols_per_cta(p.cols, SPLIT)));
  const float inv = 1.0f / static_cast<float>(p.cols);
  const int64_t block = blockIdx.x / SPLIT;
  const bool has_y = COMMON || p.y != nullptr, has_n = COMMON || p.dn != nullptr;
  const bool has_x = COMMON || p.dx_out != nullptr;
  const bool full = !COMMON && p.gate_mode == MXG_GATE_FULL, lean = !COMMON && is_lean;
  const int r_bytes = kHalves<R> * nt * 16, t_bytes = kHalves<T> * nt * 16;
  // places of x', dn, y, dx' and the gate in a chunk
  const int at_n = has_n ? r_bytes : 0, at_y = at_n + (has_n ? t_bytes : 0);
  const int at_x = at_y + (has_y ? t_bytes : 0), at_g = at_x + (has_x && !lean ? r_bytes : 0);
  const int chunk_bytes = at_g + (full && !lean ? t_bytes : 0);
  const int slot_bytes = ITER * chunk_bytes, ring_bytes = depth * slot_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x / SPLIT) * teams;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + ring_bytes;
  if (VEC) ring_clear(mine, ring_bytes, nt);
  grid_launch_dependents();
  const int c0 = RowIo<T, VEC>::col(0, 0, lane, team);
  const int dc = RowIo<T, VEC>::col(1, 0, lane, team) - c0;  // from one chunk to the next

  int64_t f_row = block * teams + team_id;  // the row filled next
  const R* x = static_cast<const R*>(p.x) + f_row * p.ldx + off + c0;
  const T* n = static_cast<const T*>(p.dn) + f_row * p.lddn + off + c0;
  const T* y = static_cast<const T*>(p.y) + f_row * p.ldy + off + c0;
  const R* d = static_cast<const R*>(p.dx_out) + f_row * p.lddxo + off + c0;
  R* dx = static_cast<R*>(p.dx) + f_row * p.lddx + off;
  T* dy = static_cast<T*>(p.dy) + f_row * p.lddy + off;
  // One row into the slot at `to`, in two parts: what is read until t is made,
  // and what is read after that.  EARLY: a thread refills its own pieces of a
  // slot as soon as it has read them, so that a ring of two rows still has one in
  // flight (2777 x 7168, fp32 stream: 97 us without, 87 us with it); where the
  // ring holds four rows, the slot of the row before is refilled at once (16384 x
  // 4096: 138 us, against 145 us).
  constexpr bool EARLY = ITER == 2;
  auto fill_early = [&](uint32_t to) {
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const uint32_t at = to + it * chunk_bytes;
      if (f_row >= p.rows) {  // a team past the last row adds nothing
        ring_clear(at, EARLY ? at_y : at_x, nt);
        ring_clear(at + at_x, chunk_bytes - at_x, nt);
        continue;
      }
      const int o = it * dc;
      const bool in = c0 + o < cols;
      if (has_n) {
        ring_fill<R, VEC>(at, x + o, in, cols, it, lane, team, nt);
        ring_fill<T, VEC>(at + at_n, n + o, in, cols, it, lane, team, nt);
      }
      if (!EARLY && has_y) ring_fill<T, VEC>(at + at_y, y + o, in, cols, it, lane, team, nt);
      if (has_x && !lean) ring_fill<R, VEC>(at + at_x, d + o, in, cols, it, lane, team, nt);
      if (full && !lean)
        ring_fill<T, VEC>(at + at_g, static_cast<const T*>(p.gate) + f_row * p.ldg + off + c0 + o, in,
                          cols, it, lane, team, nt);
    }
  };
  auto fill_late = [&](uint32_t to) {
    if (EARLY && has_y)
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        const uint32_t at = to + it * chunk_bytes + at_y;
        if (f_row < p.rows)
          ring_fill<T, VEC>(at, y + it * dc, c0 + it * dc < cols, cols, it, lane, team, nt);
        else
          ring_clear(at, t_bytes, nt);
      }
    if (VEC) cp_async_commit();
    f_row += step;
    x += step * p.ldx;
    n += step * p.lddn;
    y += step * p.ldy;
    d += step * p.lddxo;
  };
  int64_t row = f_row;
  uint32_t f_at = mine;  // the slot filled next, unless EARLY
  for (int i = 0; i < (EARLY ? depth : depth - 1); ++i, f_at += slot_bytes) {
    fill_early(mine + i * slot_bytes);
    fill_late(mine + i * slot_bytes);
  }

  if (SPLIT > 1) cluster_sync();  // both are there before one writes to the other
  using W = Weight<T, VEC, ITER>;
  const W w_pre(p.w_pre, off, cols, lane, team);
  F2 wg[ITER][4];  // w_post times a gate per channel, in fp32
  {
    const W w_post(p.w_post, off, cols, lane, team);
    const W g_col(p.gate_mode == MXG_GATE_COL ? p.gate : nullptr, off, cols, lane, team);
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wg[it][i] = f2(1.0f);
      w_post.apply(it, wg[it]);
      g_col.apply(it, wg[it]);
    }
  }
  auto times_wg = [&](int it, F2(&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], wg[it][i]);
  };

  // this thread's share of sum x'^2, sum a . x' and sum y^2 of the row at `at0`
  auto row_sums = [&](uint32_t at0, float(&v)[4]) {
    F2 v1 = 0, v2 = 0, v3 = 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const uint32_t at = at0 + it * chunk_bytes;
      if (has_n) {
        F2 x[4], a[4];
        ring_read<R>(at, nt, x);
        ring_read<T>(at + at_n, nt, a);
        w_pre.apply(it, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v1 = fma2(x[i], x[i], v1);
          v2 = fma2(a[i], x[i], v2);
        }
      }
      if (has_y) {
        F2 y[4];
        ring_read<T>(at + at_y, nt, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) v3 = fma2(y[i], y[i], v3);
      }
    }
    v[1] = sum2(v1);
    v[2] = sum2(v2);
    v[3] = sum2(v3);
  };

  F2 s0[ITER][4] = {}, s1[ITER][4] = {};
  uint32_t at0 = mine;
  const bool ahead = depth > 1;  // the ring holds the next row too
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (ahead) {
    if (VEC) cp_async_wait(EARLY ? depth - 1 : depth - 2);
    row_sums(at0, v);
    team_sum4<SPLIT>(v, red[2], team);
  }
  // a row's gate is asked for a row ahead: its latency is that of memory
  const bool g_row = p.gate_mode == MXG_GATE_ROW;
  auto row_gate = [&](int64_t r) {
    return g_row && r < p.rows ? static_cast<const float*>(p.gate)[r] : 1.0f;
  };
  float gr = row_gate(row);
  int parity = 0;
  for (int64_t base = block * teams; base < p.rows; base += step) {
    const int limit = row < p.rows ? cols : 0;
    const uint32_t next = at0 + slot_bytes == end ? mine : at0 + slot_bytes;
    if (!EARLY) {
      fill_early(f_at);
      fill_late(f_at);
      if ((f_at += slot_bytes) == end) f_at = mine;
    }
    if (!ahead) {
      if (VEC) cp_async_wait(0);
      row_sums(at0, v);
      team_sum4<SPLIT>(v, red[2], team);
    }
    const float rx = rsqrtf(v[1] * inv + p.eps), ry = rsqrtf(v[3] * inv + p.eps);
    const float c = v[2] * inv * rx;  // mean(a . xh)

    // ---- t, its column sums, and the sum for dy
    const float gr_next = row_gate(row + step);
    const F2 rx2 = f2(rx), k2 = f2(-rx * rx * c), gy2 = f2(gr * ry);
    F2 t[ITER][4], q2 = 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const uint32_t at = at0 + it * chunk_bytes;
      if (!has_x)
        zero4(t[it]);
      else if (lean)
        unpack8<R>(RowIo<R, VEC>::load(static_cast<const R*>(p.dx_out) + row * p.lddxo + off, limit, it,
                                       lane, team),
                   t[it]);
      else
        ring_read<R>(at + at_x, nt, t[it]);
      if (has_n) {
        F2 x[4], a[4];
        ring_read<R>(at, nt, x);
        ring_read<T>(at + at_n, nt, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) s0[it][i] = fma2(mul2(a[i], x[i]), rx2, s0[it][i]);
        w_pre.apply(it, a);
        // rx (a - xh c) = rx a - (rx rx c) x'
#pragma unroll
        for (int i = 0; i < 4; ++i) t[it][i] = fma2(x[i], k2, fma2(a[i], rx2, t[it][i]));
      }
      RowIo<R, VEC>::store(dx, limit, it, lane, team, t[it]);
      if (has_y) {
        F2 y[4];
        ring_read<T>(at + at_y, nt, y);
        if (full) {
          F2 g[4];
          if (lean)
            unpack8<T>(RowIo<T, VEC>::load(static_cast<const T*>(p.gate) + row * p.ldg + off, limit, it,
                                           lane, team),
                       g);
          else
            ring_read<T>(at + at_g, nt, g);
          if (p.dgate != nullptr) {
            F2 dg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) dg[i] = mul2(t[it][i], mul2(y[i], f2(p.res_scale * ry)));
            times_wg(it, dg);
            RowIo<T, VEC>::store(static_cast<T*>(p.dgate) + row * p.lddg + off, limit, it, lane, team,
                                 dg);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) t[it][i] = mul2(t[it][i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s1[it][i] = fma2(mul2(t[it][i], y[i]), gy2, s1[it][i]);
        times_wg(it, t[it]);  // b but for the factor of the whole row
#pragma unroll
        for (int i = 0; i < 4; ++i) q2 = fma2(t[it][i], y[i], q2);
      }
    }
    v[0] = sum2(q2);
    if (EARLY) fill_early(at0);
    if (ahead) {
      if (VEC) cp_async_wait(depth - 2);
      row_sums(next, v);
    }
    team_sum4<SPLIT>(v, red[parity], team);
    parity ^= 1;
    if (has_y) {
      if (g_row && p.dgate != nullptr && lane == 0 && off == 0 && limit != 0)
        static_cast<float*>(p.dgate)[row] = p.res_scale * ry * v[0];
      // dy = fr (b - y ry m) with m = mean(b . yh)
      const float fr = p.res_scale * gr * ry, m = v[0] * inv * ry;
      const F2 fr2 = f2(fr), my2 = f2(-fr * ry * m);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        F2 y[4];
        ring_read<T>(at0 + it * chunk_bytes + at_y, nt, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[it][i] = fma2(y[i], my2, mul2(t[it][i], fr2));
        RowIo<T, VEC>::store(dy, limit, it, lane, team, t[it]);
      }
    }
    if (EARLY) fill_late(at0);
    gr = gr_next;
    row += step;
    dx += step * p.lddx;
    dy += step * p.lddy;
    at0 = next;
  }

  // ---- this CTA's part of a partial row
  const int64_t total = p.cols;
  float* out = ws + block * 2 * total + off;
  if (teams > 1) {  // several teams: their sums meet in shared memory (the ring is done with)
    if (VEC) cp_async_wait(0);
    __syncthreads();
    out = reinterpret_cast<float*>(ring) + team_id * 2 * total;
  }
#pragma unroll
  for (int it = 0; it < ITER; ++it)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = RowIo<T, VEC>::col(it, e, lane, team);
      if (at < cols) {
        out[at] = e & 1 ? f2_hi(s0[it][e >> 1]) : f2_lo(s0[it][e >> 1]);
        out[total + at] = e & 1 ? f2_hi(s1[it][e >> 1]) : f2_lo(s1[it][e >> 1]);
      }
    }
  if (teams > 1) {
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(ring);
    out = ws + block * 2 * total;
    for (int i = threadIdx.x; i < 2 * cols; i += nt) {
      float s = 0.0f;
      for (int k = 0; k < teams; ++k) s += sums[k * 2 * cols + i];
      out[i] = s;
    }
  }
}

// Column sums of `blocks` partial rows, in a fixed order: 32 columns a CTA,
// kSlices threads a column.
constexpr int kSlices = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kSlices)
    block_norm_bwd_finish_kernel(const mxg_block_norm_grad_t p, const float* ws, int blocks) {
  __shared__ float part[2][kSlices][32];
  grid_wait_for_previous();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int cols = static_cast<int>(p.cols), c = blockIdx.x * 32 + lane;
  float a0 = 0.0f, a1 = 0.0f;
  if (c < cols) {
    const float* at = ws + c;
#pragma unroll 4
    for (int b = slice; b < blocks; b += kSlices) {
      a0 += at[static_cast<int64_t>(b) * 2 * cols];
      a1 += at[static_cast<int64_t>(b) * 2 * cols + cols];
    }
  }
  part[0][slice][lane] = a0;
  part[1][slice][lane] = a1;
  __syncthreads();
  if (slice != 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < kSlices; ++i) {
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

template <typename T, typename R, bool VEC, bool COMMON>
cudaError_t backward_rows(const mxg_block_norm_grad_t& p, float* ws, const RowShape& r,
                          int64_t grid, int smem, int depth, bool lean, cudaStream_t stream) {
  if (r.split > 1)
    return launch_rows<block_norm_bwd_kernel<T, R, VEC, 2, 2, COMMON>>(r, grid, smem, stream, p, ws,
                       r.team, depth, lean);
  if (r.iter == 1)
    return launch_rows<block_norm_bwd_kernel<T, R, VEC, 1, 1, COMMON>>(r, grid, smem, stream, p, ws,
                       r.team, depth, lean);
  return launch_rows<block_norm_bwd_kernel<T, R, VEC, 2, 1, COMMON>>(r, grid, smem, stream, p, ws,
                     r.team, depth, lean);
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
  const RowShape r = row_shape(p.cols, kBwdLimits);
  const int ctas = row_ctas(r, kBwdLimits, 8);
  const int64_t teams = r.threads / r.team;
  const int64_t grid = std::min<int64_t>((p.rows + teams - 1) / teams,
                                         static_cast<int64_t>(std::min(num_sms, kNormMaxSms) / r.split) * ctas);
  if (grid > 0) {
    const int chunk = r.threads * 8 * r.iter;
    const int core = static_cast<int>((p.dn ? sizeof(R) + sizeof(T) : 0) + (p.y ? sizeof(T) : 0));
    const int rest = static_cast<int>((p.dx_out ? sizeof(R) : 0) + (full ? sizeof(T) : 0));
    // without dx' and a full gate where the ring could not hold two rows else;
    // the rest is at most 192 KB a row
    const bool lean = chunk * (core + rest) * 2 > kRowSmem && core > 0;
    const int slot = chunk * (core + (lean ? 0 : rest));
    const int64_t each = (p.rows + grid * teams - 1) / (grid * teams);  // rows a team walks
    const int depth = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>({vec ? 4 : 2, kRowSmem / ctas / slot, each})));
    // narrow rows: the teams' column sums meet where the ring was
    const int sums = teams > 1 ? static_cast<int>(teams * 2 * p.cols * sizeof(float)) : 0;
    const int smem = std::max(slot * depth, sums);
    // (16 odd columns a thread spill less with the general code)
    const bool common = p.y && p.dn && p.dx_out && !full && !lean && (vec || r.iter == 1);
    const cudaError_t e =
        vec ? (common ? backward_rows<T, R, true, true>(p, ws, r, grid, smem, depth, lean, stream)
                      : backward_rows<T, R, true, false>(p, ws, r, grid, smem, depth, lean, stream))
            : (common ? backward_rows<T, R, false, true>(p, ws, r, grid, smem, depth, lean, stream)
                      : backward_rows<T, R, false, false>(p, ws, r, grid, smem, depth, lean, stream));
    if (e != cudaSuccess) return e;
  }
  return launch_after(grid > 0, block_norm_bwd_finish_kernel<T>,
                      static_cast<unsigned>((p.cols + 31) / 32), 32 * kSlices, 0, stream, p,
                      static_cast<const float*>(ws), static_cast<int>(grid));
}

}  // namespace

int64_t block_norm_ws_bytes(int64_t rows, int64_t cols) {
  const RowShape r = row_shape(cols, kBwdLimits);
  return std::min<int64_t>(rows, static_cast<int64_t>(kNormMaxSms) * row_ctas(r, kBwdLimits, 8)) * 2 * cols * 4;
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
