// block_norm_bwd.cu -- the gradients of the norms around a residual block
// (block_norm.cu).  With xh = x' rx, yh = y ry, v = s * gate, and the gradients
// dx' and dn given:
//   a = dn . w_pre,  t = dx' + rx (a - xh mean(a . xh)),  dx = t
//   b = t . v . w_post,  dy = ry (b - yh mean(b . yh))
//   dw_pre = sum_rows dn . xh,  dw_post = sum_rows t . v . yh
//   dgate = s t . yh . w_post, summed over the axes the gate is broadcast along
// rx and ry are made again from x' and y, which are read anyway.
//
// One pass over the rows (rows.cuh): a first reduction gives rx, ry and
// mean(a . xh), a second one mean(b . yh).  The column sums of a CTA's rows stay
// in registers and leave one partial row per CTA; a second kernel adds those in
// a fixed order.
#include "rows.cuh"

namespace mxg {

// CTAs of the backward kernel: as many partial rows as the workspace has room
// for.  160 bounds the SM count; a thread takes some 120 registers.
constexpr int kNormMaxSms = 160;
constexpr int kBwdCta = 128;  // CTA size of the narrow rows

static int bwd_ctas(const RowShape& r) { return std::max(1, std::min(8, 512 / r.threads)); }

// Column sums of this CTA's rows go to the workspace [block][2][cols]:
// S0 = sum dn . xh, S1 = sum t . u . yh with u the gate where it varies over
// rows (row, full) and 1 otherwise; the finish kernel applies what is constant
// down a column.
// lean: dx' and a full gate do not come through the ring (rows so wide that it
// would not hold them).
template <typename T, typename R, bool VEC, int ITER, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_bwd_kernel(const mxg_block_norm_grad_t p,
                                                              float* ws, int team, int depth,
                                                              bool lean) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][96];
  const int nt = blockDim.x, teams = nt / team;
  const int lane = threadIdx.x % team, cols = static_cast<int>(p.cols);
  const float inv = 1.0f / static_cast<float>(cols);
  const bool has_y = p.y != nullptr, has_n = p.dn != nullptr, has_x = p.dx_out != nullptr;
  const bool full = p.gate_mode == MXG_GATE_FULL;
  const int r_bytes = kHalves<R> * nt * 16, t_bytes = kHalves<T> * nt * 16;
  // places of x', dn, y, dx' and the gate in a chunk
  const int at_n = has_n ? r_bytes : 0, at_y = at_n + (has_n ? t_bytes : 0);
  const int at_x = at_y + (has_y ? t_bytes : 0), at_g = at_x + (has_x && !lean ? r_bytes : 0);
  const int chunk_bytes = at_g + (full && !lean ? t_bytes : 0);
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
      if (has_n) {
        ring_fill<R, VEC>(at, static_cast<const R*>(p.x) + row * p.ldx, limit, it, lane, team, nt);
        ring_fill<T, VEC>(at + at_n, static_cast<const T*>(p.dn) + row * p.lddn, limit, it, lane,
                          team, nt);
      }
      if (has_y)
        ring_fill<T, VEC>(at + at_y, static_cast<const T*>(p.y) + row * p.ldy, limit, it, lane,
                          team, nt);
      if (has_x && !lean)
        ring_fill<R, VEC>(at + at_x, static_cast<const R*>(p.dx_out) + row * p.lddxo, limit, it,
                          lane, team, nt);
      if (full && !lean)
        ring_fill<T, VEC>(at + at_g, static_cast<const T*>(p.gate) + row * p.ldg, limit, it, lane,
                          team, nt);
    }
    if (VEC) cp_async_commit();
  };
  for (int d = 0; d < depth - 1; ++d) fill(base0 + d * step, d);

  const Weight<T, VEC, ITER> w_pre(has_n ? p.w_pre : nullptr, cols, lane, team);
  // w_post times a gate per channel, in fp32
  F2 wg[ITER][4];
  {
    const Weight<T, VEC, ITER> w_post(has_y ? p.w_post : nullptr, cols, lane, team);
    const Weight<T, VEC, ITER> g_col(p.gate_mode == MXG_GATE_COL ? p.gate : nullptr, cols, lane,
                                     team);
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wg[it][i] = f2(1.0f);
      w_post.apply(it, wg[it]);
      g_col.apply(it, wg[it]);
    }
  }

  F2 s0[ITER][4] = {}, s1[ITER][4] = {};
  int slot = 0;
  for (int64_t base = base0; base < p.rows; base += step) {
    const int64_t row = base + team_id;
    const bool live = row < p.rows;
    const int limit = live ? cols : 0;
    const int ahead = slot + depth - 1 >= depth ? slot - 1 : slot + depth - 1;
    fill(base + (depth - 1) * step, ahead);
    if (VEC) cp_async_wait(depth - 1);
    auto get_r = [&](int at, int it, F2(&f)[4]) {
      ring_read<R, VEC>(slot_at(slot, it) + at, limit, it, lane, team, nt, f);
    };
    auto get_t = [&](int at, int it, F2(&f)[4]) {
      ring_read<T, VEC>(slot_at(slot, it) + at, limit, it, lane, team, nt, f);
    };
    auto get_gate = [&](int it, F2(&f)[4]) {
      if (lean)
        unpack8<T>(RowIo<T, VEC>::load(static_cast<const T*>(p.gate) + row * p.ldg, limit, it, lane,
                                       team),
                   f);
      else
        get_t(at_g, it, f);
    };

    // ---- the sums that need nothing else
    F2 v0 = 0, v1 = 0, v2 = 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      if (has_n) {
        F2 x[4], a[4];
        get_r(0, it, x);
        get_t(at_n, it, a);
        w_pre.apply(it, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v0 = fma2(x[i], x[i], v0);
          v1 = fma2(a[i], x[i], v1);
        }
      }
      if (has_y) {
        F2 y[4];
        get_t(at_y, it, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) v2 = fma2(y[i], y[i], v2);
      }
    }
    float v[3] = {sum2(v0), sum2(v1), sum2(v2)};
    team_sum(v, red[0], team);
    const float rx = rsqrtf(v[0] * inv + p.eps), ry = rsqrtf(v[2] * inv + p.eps);
    const float c = v[1] * inv * rx;  // mean(a . xh)

    // ---- t, its column sums, and the sum for dy
    const float gr = p.gate_mode == MXG_GATE_ROW && live ? static_cast<const float*>(p.gate)[row]
                                                         : 1.0f;
    F2 t[ITER][4], q2 = 0;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      zero4(t[it]);
      if (has_x) {
        if (lean)
          unpack8<R>(RowIo<R, VEC>::load(static_cast<const R*>(p.dx_out) + row * p.lddxo, limit, it,
                                         lane, team),
                     t[it]);
        else
          get_r(at_x, it, t[it]);
      }
      if (has_n) {
        F2 x[4], a[4];
        get_r(0, it, x);
        get_t(at_n, it, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) s0[it][i] = fma2(mul2(a[i], x[i]), f2(rx), s0[it][i]);
        w_pre.apply(it, a);
        // rx (a - xh c) = rx a - (rx rx c) x'
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[it][i] = fma2(x[i], f2(-rx * rx * c), fma2(a[i], f2(rx), t[it][i]));
      }
      RowIo<R, VEC>::store(static_cast<R*>(p.dx) + row * p.lddx, limit, it, lane, team, t[it]);
      if (has_y) {
        F2 y[4];
        get_t(at_y, it, y);
        if (full) {
          F2 g[4];
          get_gate(it, g);
          if (p.dgate != nullptr) {
            F2 dg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dg[i] = mul2(mul2(t[it][i], wg[it][i]), mul2(y[i], f2(p.res_scale * ry)));
            RowIo<T, VEC>::store(static_cast<T*>(p.dgate) + row * p.lddg, limit, it, lane, team,
                                 dg);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) t[it][i] = mul2(t[it][i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 ty = mul2(t[it][i], y[i]);
          s1[it][i] = fma2(ty, f2(gr * ry), s1[it][i]);
          t[it][i] = mul2(t[it][i], wg[it][i]);  // b but for the factor of the whole row
          q2 = fma2(t[it][i], y[i], q2);
        }
      }
    }
    if (has_y) {
      float q[1] = {sum2(q2)};
      team_sum(q, red[1], team);
      if (p.gate_mode == MXG_GATE_ROW && p.dgate != nullptr && lane == 0 && live)
        static_cast<float*>(p.dgate)[row] = p.res_scale * ry * q[0];
      const float fr = p.res_scale * gr * ry, m = q[0] * inv * ry;  // m: mean(b . yh) / f
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        F2 y[4];
        get_t(at_y, it, y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[it][i] = mul2(fma2(y[i], f2(-ry * m), t[it][i]), f2(fr));
        RowIo<T, VEC>::store(static_cast<T*>(p.dy) + row * p.lddy, limit, it, lane, team, t[it]);
      }
    } else if (team > 32) {
      __syncthreads();
    }
    if (++slot >= depth) slot = 0;
  }

  // ---- this CTA's partial row
  float* out = ws + static_cast<int64_t>(blockIdx.x) * 2 * cols;
  if (teams > 1) {  // several teams: their sums meet in shared memory (the ring is done with)
    if (VEC) cp_async_wait(0);
    __syncthreads();
    out = reinterpret_cast<float*>(ring) + team_id * 2 * cols;
  }
#pragma unroll
  for (int it = 0; it < ITER; ++it)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = RowIo<T, VEC>::col(it, e, lane, team);
      if (at < cols) {
        out[at] = e & 1 ? f2_hi(s0[it][e >> 1]) : f2_lo(s0[it][e >> 1]);
        out[cols + at] = e & 1 ? f2_hi(s1[it][e >> 1]) : f2_lo(s1[it][e >> 1]);
      }
    }
  if (teams > 1) {
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(ring);
    out = ws + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    for (int i = threadIdx.x; i < 2 * cols; i += nt) {
      float s = 0.0f;
      for (int k = 0; k < teams; ++k) s += sums[k * 2 * cols + i];
      out[i] = s;
    }
  }
}

// Column sums of `blocks` partial rows, in a fixed order: 32 columns a CTA,
// kSlices threads a column.
constexpr int kSlices = 16;
template <typename T>
__global__ void __launch_bounds__(32 * kSlices)
    block_norm_bwd_finish_kernel(const mxg_block_norm_grad_t p, const float* ws, int blocks) {
  __shared__ float part[2][kSlices][32];
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

template <typename T, typename R, bool VEC>
cudaError_t backward_rows(const mxg_block_norm_grad_t& p, float* ws, const RowShape& r,
                          int64_t grid, int smem, int depth, bool lean, cudaStream_t stream) {
  if (r.iter == 1)
    return launch_rows(block_norm_bwd_kernel<T, R, VEC, 1, 256>, grid, r.threads, smem, stream, p,
                       ws, r.team, depth, lean);
  if (r.threads <= 512)
    return launch_rows(block_norm_bwd_kernel<T, R, VEC, 2, 512>, grid, r.threads, smem, stream, p,
                       ws, r.team, depth, lean);
  return launch_rows(block_norm_bwd_kernel<T, R, VEC, 2, 1024>, grid, r.threads, smem, stream, p,
                     ws, r.team, depth, lean);
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
  const RowShape r = row_shape(p.cols, kBwdCta);
  const int ctas = bwd_ctas(r);
  const int64_t teams = r.threads / r.team;
  const int64_t grid = std::min<int64_t>((p.rows + teams - 1) / teams,
                                         static_cast<int64_t>(std::min(num_sms, kNormMaxSms)) * ctas);
  if (grid > 0) {
    const int chunk = r.threads * 8 * r.iter;
    const int core = static_cast<int>((p.dn ? sizeof(R) + sizeof(T) : 0) + (p.y ? sizeof(T) : 0));
    const int rest = static_cast<int>((p.dx_out ? sizeof(R) : 0) + (full ? sizeof(T) : 0));
    const bool lean = chunk * (core + rest) > kRowSmem;  // the core is at most 192 KB
    const int slot = chunk * (core + (lean ? 0 : rest));
    const int depth =
        slot == 0 ? 1 : std::max(1, std::min(vec ? 4 : 2, kRowSmem / ctas / slot));
    // narrow rows: the teams' column sums meet where the ring was
    const int sums = teams > 1 ? static_cast<int>(teams * 2 * p.cols * sizeof(float)) : 0;
    const int smem = std::max(slot * depth, sums);
    const cudaError_t e =
        vec ? backward_rows<T, R, true>(p, ws, r, grid, smem, depth, lean, stream)
            : backward_rows<T, R, false>(p, ws, r, grid, smem, depth, lean, stream);
    if (e != cudaSuccess) return e;
  }
  block_norm_bwd_finish_kernel<T>
      <<<static_cast<unsigned>((p.cols + 31) / 32), 32 * kSlices, 0, stream>>>(
          p, ws, static_cast<int>(grid));
  return cudaGetLastError();
}

}  // namespace

int64_t block_norm_ws_bytes(int64_t rows, int64_t cols) {
  const RowShape r = row_shape(cols, kBwdCta);
  return std::min<int64_t>(rows, static_cast<int64_t>(kNormMaxSms) * bwd_ctas(r)) * 2 * cols * 4;
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
