// expert_rows.cu -- rows between the tokens' order and the experts':
//   dispatch         : rows[row_of[t, j]] = tokens[t]
//   combine          : tokens[t] = sum_j weight[t, j] rows[row_of[t, j]]
//   combine backward : rows[row_of[t, j]] = weight[t, j] tokens[t],
//                      dweight[t, j] = sum over the columns of tokens[t] y_rows[row_of[t, j]]
//
// All three go by tokens, so that a token's row is read (or written) once and only the k
// rows beside it are scattered; no row is shared, so nothing is atomic.  Memory is the
// bound: dispatching 8192 tokens of 4096 in bf16 to 2 experts each takes 31.8 us, 6.5 TB/s of the
// 6.78 that a copy reaches.  Rows that do not start on 16 bytes move element by element, at
// 30 to 55 % of that.
#include <algorithm>
#include <atomic>

#include "rows.cuh"

namespace mxg {

constexpr int kRowThreads = 256;

// A lane's piece of a row: BYTES (32, 16, or one element) at a time, as fp32 and back.
template <typename T, int BYTES>
struct Piece {
  static constexpr int kElems = BYTES / static_cast<int>(sizeof(T));
  static_assert(BYTES == 32 || BYTES == 16 || kElems == 1, "pieces of three sizes");
  static constexpr int kWords = BYTES >= 4 ? BYTES / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 32) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7])
                   : "l"(p));  // (volatile: in order with the stores)
    } else if constexpr (BYTES == 16) {
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    } else {
      load_if(p, true);
    }
  }
  // An element, or 0 where `in` is not set; without a branch, so that many can be asked for at once.
  __device__ __forceinline__ void load_if(const T* p, bool in) {
    static_assert(kElems == 1, "of single elements");
    // (the 0 comes before the load: put behind it, it would wait for it)
    if constexpr (sizeof(T) == 4) {
      w[0] = 0;
      asm volatile(
          "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.b32 %0, [%1];\n\t}"
          : "+r"(w[0])
          : "l"(p), "r"(static_cast<int>(in)));
    } else {
      uint16_t v = 0;
      asm volatile(
          "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.b16 %0, [%1];\n\t}"
          : "+h"(v)
          : "l"(p), "r"(static_cast<int>(in)));
      w[0] = v;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 32) {
      st_global_32B(p, w);
    } else if constexpr (BYTES == 16) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (sizeof(T) == 4) {
      *p = __uint_as_float(w[0]);
    } else {
      p->bits = static_cast<uint16_t>(w[0]);
    }
  }
  __device__ __forceinline__ void get(float (&f)[kElems]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (kElems == 1) {
      f[0] = to_f32(T{static_cast<uint16_t>(w[0])});
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) unpack2<T>(w[i], f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[kElems]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (kElems == 1) {
      w[0] = from_f32<T>(f[0]).bits;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
  }
};

// Zeros in the rows between an expert's count and its padded size: item kPadWarps e + i is a warp's
// share of expert e's.
constexpr int kPadWarps = 16;

template <typename T, int BYTES>
__device__ __forceinline__ void zero_padding(const mxg_expert_rows_t& d, int64_t item) {
  const int lane = threadIdx.x & 31;
  const int e = static_cast<int>(item / kPadWarps), part = static_cast<int>(item % kPadWarps);
  // the group's start: the sizes before it
  int64_t start = 0;
  for (int i = lane; i < e; i += 32) {
    const int64_t s = d.group_ws[i];
    start += s > 0 ? min(s, d.rows_capacity) : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) start += __shfl_xor_sync(0xFFFFFFFFu, start, o);
  const int64_t size = min(max(d.group_ws[e], static_cast<int64_t>(0)), d.rows_capacity);
  const int64_t count = max(d.counts[e], 0);
  const int64_t end = min(start + size, d.rows_capacity);
  constexpr int kElems = Piece<T, BYTES>::kElems;
  Piece<T, BYTES> none;
  none.zero();
  for (int64_t r = start + count + part; r < end; r += kPadWarps) {
    T* row = static_cast<T*>(d.rows) + r * d.ldr;
    for (int64_t c = lane * kElems; c < d.cols; c += 32 * kElems) {
      if (c + kElems <= d.cols)
        none.store(row + c);
      else
        for (int64_t i = c; i < d.cols; ++i) row[i] = T{};
    }
  }
}

// A warp's item: a token and `32 * UNROLL` pieces of its columns.
template <typename T, int BYTES, int UNROLL>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const mxg_expert_rows_t d, int slices, int64_t pad_items) {
  constexpr int kElems = Piece<T, BYTES>::kElems;
  const int lane = threadIdx.x & 31;
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  const int64_t items = pad_items + d.n * slices;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
       item < items; item += warps) {
    if (item < pad_items) {
      zero_padding<T, BYTES>(d, item);
      continue;
    }
    const int64_t t = (item - pad_items) / slices;
    const int slice = static_cast<int>((item - pad_items) - t * slices);
    int32_t at = -1;
    if (lane < d.k) at = d.row_of[t * d.k + lane];
    const T* from = static_cast<const T*>(d.tokens) + t * d.ldt;
    const int c0 = (slice * UNROLL * 32 + lane) * kElems;
    Piece<T, BYTES> x[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (c0 + (u * 32 + 1) * kElems <= d.cols) x[u].load(from + c0 + u * 32 * kElems);
    for (int j = 0; j < d.k; ++j) {
      const int64_t r = __shfl_sync(0xFFFFFFFFu, at, j);
      if (r < 0 || r >= d.rows_capacity) continue;
      T* to = static_cast<T*>(d.rows) + r * d.ldr;
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int c = c0 + u * 32 * kElems;
        if (c + kElems <= d.cols)
          x[u].store(to + c);
        else
          for (int i = c; i < d.cols; ++i) to[i] = from[i];
      }
    }
  }
}

// A warp's walk through (token, slice of its columns), all warps of the grid apart.
template <int NT>
struct TokenWalk {
  int64_t t, t_step;
  int slice, slice_step, slices;
  __device__ __forceinline__ TokenWalk(int slices) : slices(slices) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (NT / 32);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (NT / 32) + (threadIdx.x >> 5);
    t = item / slices;
    slice = static_cast<int>(item - t * slices);
    t_step = warps / slices;
    slice_step = static_cast<int>(warps - t_step * slices);
  }
  __device__ __forceinline__ void next() {
    t += t_step;
    slice += slice_step;
    if (slice >= slices) {
      slice -= slices;
      ++t;
    }
  }
};

// Where a lane's row of its token starts (lane j: the j-th), in elements, or -1; and its weight, 0
// where there is none.
__device__ __forceinline__ int64_t row_start(const mxg_expert_rows_t& d, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t at = -1;
  if (t < d.n && lane < d.k) at = d.row_of[t * d.k + lane];
  return at >= 0 && at < d.rows_capacity ? at * d.ldr : -1;
}
__device__ __forceinline__ float row_weight(const mxg_expert_rows_t& d, int64_t t) {
  const int lane = threadIdx.x & 31;
  if (t >= d.n || lane >= d.k) return 0.0f;
  const int32_t at = d.row_of[t * d.k + lane];
  if (at < 0 || at >= d.rows_capacity) return 0.0f;
  return d.weight != nullptr ? d.weight[t * d.k + lane] : 1.0f;
}

// 16 bytes into shared memory past L1; zeros where `in` is not set (`src` is not read).
__device__ __forceinline__ void cp_async_16_or_zeros(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// Sums of rows that start on 16 bytes.  A warp's item is a token and 1 KB of its columns, twice 16
// bytes a lane; a lane's pieces of PER rows are a unit, and every thread has a ring of kDepth units in
// shared memory that asynchronous copies fill ahead of the sums.  No thread reads another's
// pieces, so there is no barrier.  4096 tokens of 8 rows of 2048 in fp16: 25.8 us, 5.9 TB/s; with the
// rows in registers, 4 at a time to leave room for enough warps, 38.6 us; with 16 bytes a lane the
// instructions for a row's place were the bound, at 33.5 us.
constexpr int kRingThreads = 128, kDepth = 4;

template <typename T, int PER>
__global__ void __launch_bounds__(kRingThreads)
    combine_ring_kernel(const mxg_expert_rows_t d, int slices) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kHalf = 16 / static_cast<int>(sizeof(T));  // elements of 16 bytes
  constexpr uint32_t kPitch = kRingThreads * 16;           // from one half piece to the next one's
  constexpr uint32_t kUnit = 2 * PER * kPitch;
  const int lane = threadIdx.x & 31, cols = static_cast<int>(d.cols);
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDepth * kUnit;
  const T* const rows = static_cast<const T*>(d.rows);
  grid_wait_for_previous();
  grid_launch_dependents();

  TokenWalk<kRingThreads> fill(slices), work = fill, fill_next = fill;
  fill_next.next();
  int64_t fill_row = row_start(d, fill.t), fill_then = row_start(d, fill_next.t);
  float work_w = row_weight(d, work.t);
  int fill_j = 0;
  uint32_t fill_at = mine;
  auto fill_unit = [&] {
    if (fill.t < d.n) {
      const int c = (fill.slice * 64 + lane) * kHalf;
      const bool in0 = c + kHalf <= cols, in1 = c + 33 * kHalf <= cols;
      const T* const from = rows + c;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        // (lanes behind the k-th have no row; past 32 there is none to ask)
        const int64_t r = __shfl_sync(0xFFFFFFFFu, fill_row, (fill_j + j) & 31);
        const T* const src = r < 0 ? rows : from + r;
        cp_async_16_or_zeros(fill_at + 2 * j * kPitch, in0 ? src : rows, in0 && r >= 0);
        cp_async_16_or_zeros(fill_at + (2 * j + 1) * kPitch, in1 ? src + 32 * kHalf : rows, in1 && r >= 0);
      }
      fill_j += PER;
      if (fill_j >= d.k) {
        fill_j = 0;
        fill = fill_next;
        fill_row = fill_then;
        fill_next.next();
        fill_then = row_start(d, fill_next.t);
      }
    }
    cp_async_commit();
    if ((fill_at += kUnit) == end) fill_at = mine;
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fill_unit();
  uint32_t at = mine;
  TokenWalk<kRingThreads> then = work;
  for (; work.t < d.n; work = then) {
    const float w_now = work_w;
    then.next();
    work_w = row_weight(d, then.t);
    const int c = (work.slice * 64 + lane) * kHalf;
    F2 acc[kHalf];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) acc[i] = 0;
    for (int j0 = 0; j0 < d.k; j0 += PER) {
      fill_unit();
      cp_async_wait(kDepth - 1);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const F2 w = f2(__shfl_sync(0xFFFFFFFFu, w_now, (j0 + j) & 31));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 q = lds16(at + (2 * j + h) * kPitch);
          const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) {
            float lo, hi;
            if constexpr (sizeof(T) == 4) {
              lo = __uint_as_float(word[2 * i]);
              hi = __uint_as_float(word[2 * i + 1]);
            } else {
              unpack2<T>(word[i], lo, hi);
            }
            acc[h * kHalf / 2 + i] = fma2(w, f2(lo, hi), acc[h * kHalf / 2 + i]);
          }
        }
      }
      if ((at += kUnit) == end) at = mine;
    }
    T* const to = static_cast<T*>(d.tokens) + work.t * d.ldt;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c + (32 * h + 1) * kHalf <= cols) {
        uint32_t word[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4)
            word[i] = __float_as_uint(i & 1 ? f2_hi(acc[h * 2 + i / 2]) : f2_lo(acc[h * 2 + i / 2]));
          else
            word[i] = pack2<T>(f2_lo(acc[h * 4 + i]), f2_hi(acc[h * 4 + i]));
        }
        *reinterpret_cast<uint4*>(to + c + 32 * h * kHalf) =
            make_uint4(word[0], word[1], word[2], word[3]);
      }
    // what is left of a row whose columns do not end on 16 bytes
    if (cols % kHalf != 0) {
      const int64_t row = row_start(d, work.t);
      const int first = cols / kHalf * kHalf;
      const bool last = first == c || first == c + 32 * kHalf;
      for (int i = first; i < cols; ++i) {
        float sum = 0.0f;
        for (int j = 0; j < d.k; ++j) {
          const int64_t r = __shfl_sync(0xFFFFFFFFu, row, j);
          const float w = __shfl_sync(0xFFFFFFFFu, w_now, j);
          if (r >= 0 && last) sum = fmaf(w, to_f32(rows[r + i]), sum);
        }
        if (last) to[i] = from_f32<T>(sum);
      }
    }
  }
}

// Rows of any alignment: kAcross elements a lane, 32 columns apart.
constexpr int kAcross = 4;

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const mxg_expert_rows_t d, int slices) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31, cols = static_cast<int>(d.cols);
  grid_wait_for_previous();
  grid_launch_dependents();
  TokenWalk<kRowThreads> at(slices), then = at;
  int64_t row = row_start(d, at.t);
  float weight = row_weight(d, at.t);
  for (; at.t < d.n; at = then) {
    const int64_t row_now = row;
    const float w_now = weight;
    then.next();
    row = row_start(d, then.t);
    weight = row_weight(d, then.t);
    const int c = at.slice * 32 * kAcross + lane;
    const T* const from = static_cast<const T*>(d.rows) + c;
    float sum[kAcross];
#pragma unroll
    for (int i = 0; i < kAcross; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < d.k; j0 += kAhead) {
      Piece<T, static_cast<int>(sizeof(T))> x[kAhead][kAcross];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        // (lanes behind the k-th have no row)
        const int64_t r = __shfl_sync(0xFFFFFFFFu, row_now, (j0 + j) & 31);
#pragma unroll
        for (int i = 0; i < kAcross; ++i)
          x[j][i].load_if(from + r + 32 * i, r >= 0 && c + 32 * i < cols);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float w = __shfl_sync(0xFFFFFFFFu, w_now, (j0 + j) & 31);
#pragma unroll
        for (int i = 0; i < kAcross; ++i) {
          float f[1];
          x[j][i].get(f);
          sum[i] = fmaf(w, f[0], sum[i]);
        }
      }
    }
    T* const to = static_cast<T*>(d.tokens) + at.t * d.ldt + c;
#pragma unroll
    for (int i = 0; i < kAcross; ++i)
      if (c + 32 * i < cols) to[32 * i] = from_f32<T>(sum[i]);
  }
}

// The gradients of sums of rows, without the weights' or (DOTS, rows of any alignment alone) with them.
// 8192 tokens of 2 rows of 4096 in bf16, rows alone: 37 us, 5.4 TB/s; of 4095, both: 90 us.  A team of
// `team` warps owns a token, KA of its rows at a time and ACROSS pieces of each row a lane; a lane's next
// pieces are asked for before it works on those it has.  Sums over the columns are joined in shared
// memory.  (With the sums tested for when run, registers of both: 41 us for the rows alone.)
template <typename T, int BYTES, int KA, int ACROSS, bool DOTS>
__global__ void __launch_bounds__(kRowThreads)
    combine_backward_kernel(const mxg_expert_rows_t d, int team, int64_t pad_items) {
  using P = Piece<T, BYTES>;
  constexpr int kElems = P::kElems, kSpan = 32 * kElems;
  constexpr int kWarps = kRowThreads / 32;
  static_assert(!DOTS || kElems == 1, "rows on 16 bytes and their weights: by rings");
  __shared__ float part[DOTS ? kWarps : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, teams = kWarps / team;
  const int place = warp % team;  // in the team
  const bool writes = !DOTS || d.rows != nullptr;
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t pad_blocks = (pad_items + kWarps - 1) / kWarps;
  const int64_t token_blocks = (d.n + teams - 1) / teams;
  const int cols = static_cast<int>(d.cols), step = team * kSpan * ACROSS;
  for (int64_t b = blockIdx.x; b < pad_blocks + token_blocks; b += gridDim.x) {
    if (b < pad_blocks) {
      if (b * kWarps + warp < pad_items) zero_padding<T, BYTES>(d, b * kWarps + warp);
      continue;
    }
    const int64_t t = (b - pad_blocks) * teams + warp / team;
    const bool on = t < d.n;
    int32_t at = -1;
    float w = 1.0f, dot_mine = 0.0f;
    if (on && lane < d.k) {
      at = d.row_of[t * d.k + lane];
      if (d.weight != nullptr) w = d.weight[t * d.k + lane];
    }
    if (at >= d.rows_capacity) at = -1;
    const T* dy = static_cast<const T*>(d.tokens) + (on ? t : 0) * d.ldt;
    const T* y_rows = static_cast<const T*>(d.y_rows);
    T* rows = static_cast<T*>(d.rows);
    for (int j0 = 0; j0 < d.k; j0 += KA) {
      float wj[KA], dot[KA];
      int32_t r[KA];
#pragma unroll
      for (int j = 0; j < KA; ++j) {
        const int from = j0 + j < d.k ? j0 + j : 31;
        r[j] = __shfl_sync(0xFFFFFFFFu, at, from);
        wj[j] = __shfl_sync(0xFFFFFFFFu, w, from);
        if (j0 + j >= d.k) r[j] = -1;
        dot[j] = 0.0f;
      }
      struct Pieces {
        P x[ACROSS], y[DOTS ? ACROSS : 1][DOTS ? KA : 1];
      };
      auto fetch = [&](Pieces& p, int c) {
#pragma unroll
        for (int i = 0; i < ACROSS; ++i) {
          const int at_c = c + i * kSpan;
          const bool in = on && at_c + kElems <= cols;
          if constexpr (kElems == 1) {
            p.x[i].load_if(dy + at_c, in);
            if constexpr (DOTS) {
#pragma unroll
              for (int j = 0; j < KA; ++j)
                p.y[i][j].load_if(y_rows + r[j] * d.ldy + at_c, in && r[j] >= 0);
            }
          } else if (in) {
            p.x[i].load(dy + at_c);
          }
        }
      };
      int c = place * kSpan * ACROSS + lane * kElems;
      Pieces now;
      fetch(now, c);
      for (; on && c + kElems <= cols; c += step) {
        Pieces next;
        fetch(next, c + step);
#pragma unroll
        for (int i = 0; i < ACROSS; ++i) {
          if (c + i * kSpan + kElems > cols) continue;
          float g[kElems];
          now.x[i].get(g);
#pragma unroll
          for (int j = 0; j < KA; ++j) {
            if (r[j] < 0) continue;
            float f[kElems];
            if constexpr (DOTS) {
              now.y[i][j].get(f);
#pragma unroll
              for (int e = 0; e < kElems; ++e) dot[j] = fmaf(g[e], f[e], dot[j]);
            }
            if (writes) {
#pragma unroll
              for (int e = 0; e < kElems; ++e) f[e] = wj[j] * g[e];
              P o;
              o.set(f);
              o.store(rows + r[j] * d.ldr + c + i * kSpan);
            }
          }
        }
        now = next;
      }
      // what is left of a row whose columns do not end on a piece: an element a lane
      if (kElems > 1 && on && place == 0 && lane < cols % kElems) {
        const int e = cols / kElems * kElems + lane;
        const float g = to_f32(dy[e]);
#pragma unroll
        for (int j = 0; j < KA; ++j) {
          if (r[j] < 0) continue;
          rows[r[j] * d.ldr + e] = from_f32<T>(wj[j] * g);
        }
      }
      if constexpr (DOTS) {
#pragma unroll
        for (int j = 0; j < KA; ++j) {
          float v = dot[j];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
          if (lane == j0 + j) dot_mine = v;
        }
      }
    }
    if constexpr (DOTS) {
      if (team > 1) {
        part[warp][lane] = dot_mine;
        __syncthreads();
        if (place == 0)
          for (int i = 1; i < team; ++i) dot_mine += part[warp + i][lane];
        __syncthreads();
      }
      if (on && place == 0 && lane < d.k) d.dweight[t * d.k + lane] = dot_mine;
    }
  }
}

// The gradients of sums of rows that start on 16 bytes, with the weights' among them: as the sums,
// through rings, a unit being 1 KB of a token's gradient and of PER of its rows.  A team of `team`
// warps owns a token.  4096 tokens of 8 rows of 2048 in bf16: 53 us, 5.3 TB/s, through registers 62
// us; 8192 tokens of 2 rows of 4096: 54 us, 6.1 TB/s.
constexpr int ring_depth(int per) { return per == 8 ? 3 : 4; }

// A unit's halves for a thread, as pairs.
template <typename T>
__device__ __forceinline__ void ring_values(uint32_t at, uint32_t pitch,
                                            F2 (&f)[16 / sizeof(T)]) {
  constexpr int kPairs = 8 / static_cast<int>(sizeof(T));  // of a half
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q = lds16(at + h * pitch);
    const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float lo, hi;
      if constexpr (sizeof(T) == 4) {
        lo = __uint_as_float(word[2 * i]);
        hi = __uint_as_float(word[2 * i + 1]);
      } else {
        unpack2<T>(word[i], lo, hi);
      }
      f[h * kPairs + i] = f2(lo, hi);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 half_of(const F2* f) {
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4)
      word[i] = __float_as_uint(i & 1 ? f2_hi(f[i / 2]) : f2_lo(f[i / 2]));
    else
      word[i] = pack2<T>(f2_lo(f[i]), f2_hi(f[i]));
  }
  return make_uint4(word[0], word[1], word[2], word[3]);
}

template <typename T, int PER>
__global__ void __launch_bounds__(kRingThreads)
    combine_backward_ring_kernel(const mxg_expert_rows_t d, int team, int slices, int64_t pad_items) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kWarps = kRingThreads / 32, kDeep = ring_depth(PER);
  constexpr int kHalf = 16 / static_cast<int>(sizeof(T)), kPairs = kHalf;  // pairs of both halves
  constexpr uint32_t kPitch = kRingThreads * 16, kUnit = 2 * (1 + PER) * kPitch;
  __shared__ float part[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = static_cast<int>(d.cols);
  grid_wait_for_previous();
  grid_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < pad_items;
       i += static_cast<int64_t>(gridDim.x) * kWarps)
    zero_padding<T, 16>(d, i);
  const int teams = kWarps / team, place = warp % team;
  const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams + warp / team;
  const T* const dy = static_cast<const T*>(d.tokens);
  const T* const y_rows = static_cast<const T*>(d.y_rows);
  T* const rows = static_cast<T*>(d.rows);
  auto row_at = [&](int64_t t) {
    const int32_t at = t < d.n && lane < d.k ? d.row_of[t * d.k + lane] : -1;
    return at < d.rows_capacity ? at : -1;
  };
  auto weight_at = [&](int64_t t) {
    return t < d.n && lane < d.k && d.weight != nullptr ? d.weight[t * d.k + lane] : 1.0f;
  };
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDeep * kUnit;
  int64_t fill_t = first;
  int fill_j = 0, fill_s = place;
  int32_t fill_row = row_at(first), fill_then = row_at(first + step);
  uint32_t fill_at = mine;
  auto fill_unit = [&] {
    if (fill_t < d.n) {
      const int c = (fill_s * 64 + lane) * kHalf;
      const bool in0 = c + kHalf <= cols, in1 = c + 33 * kHalf <= cols;
      const T* const from = dy + fill_t * d.ldt + c;
      cp_async_16_or_zeros(fill_at, in0 ? from : dy, in0);
      cp_async_16_or_zeros(fill_at + kPitch, in1 ? from + 32 * kHalf : dy, in1);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        // (lanes behind the k-th have no row)
        const int32_t r = __shfl_sync(0xFFFFFFFFu, fill_row, (fill_j + j) & 31);
        const T* const src = y_rows + r * d.ldy + c;
        cp_async_16_or_zeros(fill_at + (2 + 2 * j) * kPitch, in0 && r >= 0 ? src : dy, in0 && r >= 0);
        cp_async_16_or_zeros(fill_at + (3 + 2 * j) * kPitch, in1 && r >= 0 ? src + 32 * kHalf : dy,
                             in1 && r >= 0);
      }
      if ((fill_s += team) >= slices) {
        fill_s = place;
        if ((fill_j += PER) >= d.k) {
          fill_j = 0;
          fill_t += step;
          fill_row = fill_then;
          fill_then = row_at(fill_t + step);
        }
      }
    }
    cp_async_commit();
    if ((fill_at += kUnit) == end) fill_at = mine;
  };
#pragma unroll
  for (int i = 0; i < kDeep - 1; ++i) fill_unit();
  uint32_t at = mine;
  int32_t next_row = row_at(first);
  float next_w = weight_at(first);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams, t = first; base < d.n;
       base += step, t += step) {
    const bool on = t < d.n;
    const int32_t row = next_row;
    const float w = next_w;
    next_row = row_at(t + step);
    next_w = weight_at(t + step);
    float dot_mine = 0.0f;
    for (int j0 = 0; on && j0 < d.k; j0 += PER) {
      int32_t r[PER];
      F2 wj[PER], dot[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        r[j] = __shfl_sync(0xFFFFFFFFu, row, (j0 + j) & 31);
        wj[j] = f2(__shfl_sync(0xFFFFFFFFu, w, (j0 + j) & 31));
        dot[j] = 0;
      }
      for (int s = place; s < slices; s += team) {
        fill_unit();
        cp_async_wait(kDeep - 1);
        const int c = (s * 64 + lane) * kHalf;
        const bool in0 = c + kHalf <= cols, in1 = c + 33 * kHalf <= cols;
        F2 g[kPairs];
        ring_values<T>(at, kPitch, g);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          F2 f[kPairs];
          ring_values<T>(at + (2 + 2 * j) * kPitch, kPitch, f);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) dot[j] = fma2(g[i], f[i], dot[j]);
          if (rows != nullptr && r[j] >= 0) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) f[i] = mul2(wj[j], g[i]);
            T* const to = rows + r[j] * d.ldr + c;
            if (in0) *reinterpret_cast<uint4*>(to) = half_of<T>(f);
            if (in1) *reinterpret_cast<uint4*>(to + 32 * kHalf) = half_of<T>(f + kPairs / 2);
          }
        }
        if ((at += kUnit) == end) at = mine;
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float v = r[j] < 0 ? 0.0f : sum2(dot[j]);
        // what is left of a row whose columns do not end on 16 bytes: an element a lane
        if (place == 0 && r[j] >= 0 && lane < cols % kHalf) {
          const int e = cols / kHalf * kHalf + lane;
          const float g = to_f32(dy[t * d.ldt + e]);
          v = fmaf(g, to_f32(y_rows[r[j] * d.ldy + e]), v);
          if (rows != nullptr) rows[r[j] * d.ldr + e] = from_f32<T>(f2_lo(wj[j]) * g);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == j0 + j) dot_mine = v;
      }
    }
    if (team > 1) {
      part[warp][lane] = dot_mine;
      __syncthreads();
      if (place == 0)
        for (int i = 1; i < team; ++i) dot_mine += part[warp + i][lane];
      __syncthreads();
    }
    if (on && place == 0 && lane < d.k) d.dweight[t * d.k + lane] = dot_mine;
  }
}

namespace {

// Bytes of the accesses that every row allows: 32, 16 or an element's.
int piece_bytes(const mxg_expert_rows_t& d, size_t size) {
  uintptr_t all = reinterpret_cast<uintptr_t>(d.tokens) | reinterpret_cast<uintptr_t>(d.rows) |
                  reinterpret_cast<uintptr_t>(d.y_rows) | static_cast<uintptr_t>(d.ldt * size) |
                  (d.rows != nullptr ? static_cast<uintptr_t>(d.ldr * size) : 0) |
                  (d.y_rows != nullptr ? static_cast<uintptr_t>(d.ldy * size) : 0);
  return (all & 31u) == 0 ? 32 : ((all & 15u) == 0 ? 16 : static_cast<int>(size));
}

unsigned grid_for(int64_t warps, int num_sms, int64_t most) {
  const int64_t blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(blocks, num_sms * most)));
}

int64_t slices_of(int64_t cols, int per) { return (cols + per - 1) / per; }

constexpr int kRingSmem = 220 * 1024;  // of an SM's 227 KB

// Allows KERN `smem` bytes, once per device: the limit belongs to the kernel, for all host threads.
template <auto KERN>
cudaError_t allow_smem(int smem) {
  constexpr int kMaxDev = 64;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
  return e;
}

// Units of 1, 2 or 4 rows, whichever holds k in fewest; as many CTAs as an SM has room for.
template <typename T, int PER>
cudaError_t run_combine_ring(const mxg_expert_rows_t& d, int num_sms, cudaStream_t stream) {
  constexpr int kSmem = kDepth * 2 * PER * kRingThreads * 16;
  constexpr int kCtas = std::min(8, kRingSmem / (kSmem + 1024));
  const cudaError_t e = allow_smem<combine_ring_kernel<T, PER>>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t slices = slices_of(d.cols, 32 * 32 / static_cast<int>(sizeof(T)));
  const int64_t blocks = (d.n * slices + kRingThreads / 32 - 1) / (kRingThreads / 32);
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * kCtas));
  return launch_after(true, combine_ring_kernel<T, PER>, grid, kRingThreads, kSmem, stream, d,
                      static_cast<int>(slices));
}

template <typename T, int PER>
cudaError_t run_backward_ring(const mxg_expert_rows_t& d, int64_t pad, int num_sms,
                              cudaStream_t stream) {
  constexpr int kSmem = ring_depth(PER) * 2 * (1 + PER) * kRingThreads * 16;
  constexpr int kCtas = std::min(4, kRingSmem / (kSmem + 2048)), kWarps = kRingThreads / 32;
  const cudaError_t e = allow_smem<combine_backward_ring_kernel<T, PER>>(kSmem);
  if (e != cudaSuccess) return e;
  const int slices = static_cast<int>(slices_of(d.cols, 32 * 32 / static_cast<int>(sizeof(T))));
  // more warps a token where the tokens alone do not fill the device
  const int64_t most = static_cast<int64_t>(num_sms) * kCtas;
  int team = 1;
  while (team < kWarps && 2 * team <= slices && d.n * team < most * kWarps) team *= 2;
  const int64_t warps = std::max(pad, d.n * team);
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>((warps + kWarps - 1) / kWarps, most));
  return launch_after(true, combine_backward_ring_kernel<T, PER>, grid, kRingThreads, kSmem, stream,
                      d, team, slices, pad);
}

template <typename T, int BYTES>
cudaError_t run(const mxg_expert_rows_t& d, int op, int num_sms, cudaStream_t stream) {
  constexpr int kSpan = 32 * Piece<T, BYTES>::kElems;
  const int64_t pad = d.counts != nullptr && d.rows != nullptr
                          ? static_cast<int64_t>(d.experts) * kPadWarps
                          : 0;
  if (op == 0) {
    constexpr int kUnroll = BYTES >= 16 ? 2 : 8;
    const int64_t slices = slices_of(d.cols, kSpan * kUnroll);
    return launch_after(true, dispatch_kernel<T, BYTES, kUnroll>,
                        grid_for(pad + d.n * slices, num_sms, 64), kRowThreads, 0, stream, d,
                        static_cast<int>(slices), pad);
  } else if (op == 1) {
    if constexpr (BYTES >= 16) {
      if (d.k == 1) return run_combine_ring<T, 1>(d, num_sms, stream);
      if (d.k == 2) return run_combine_ring<T, 2>(d, num_sms, stream);
      return run_combine_ring<T, 4>(d, num_sms, stream);
    } else {
      const int64_t slices = slices_of(d.cols, 32 * kAcross);
      return launch_after(true, combine_kernel<T>, grid_for(d.n * slices, num_sms, 64), kRowThreads, 0,
                          stream, d, static_cast<int>(slices));
    }
  } else {
    if constexpr (BYTES >= 16) {
      if (d.dweight != nullptr) {
        if (d.k <= 2) return run_backward_ring<T, 2>(d, pad, num_sms, stream);
        if (d.k <= 4) return run_backward_ring<T, 4>(d, pad, num_sms, stream);
        return run_backward_ring<T, 8>(d, pad, num_sms, stream);
      }
    }
    // more warps a token where the tokens alone do not fill the device
    int team = 1;
    while (team < 8 && d.n * team < num_sms * 48LL && team * kSpan < d.cols) team *= 2;
    // CTAs an SM: without the weights 8 (4096 tokens of 8 rows of 2048 in fp32: 54 us, 61 with 4; in
    // bf16 28.5 and 28.3), with them 4 (8192 tokens of 2 rows of 4095 in bf16: 90 us, 91.5 with 8)
    const unsigned grid = grid_for(pad + d.n * team, num_sms, d.dweight != nullptr ? 4 : 8);
    constexpr int kAcrossOf2 = BYTES < 16 ? 4 : 1, kAcrossOf4 = BYTES < 16 ? 2 : 1;
    auto launch = [&](auto kern) {
      return launch_after(true, kern, grid, kRowThreads, 0, stream, d, team, pad);
    };
    if constexpr (BYTES < 16) {
      if (d.dweight != nullptr)
        return d.k <= 2 ? launch(combine_backward_kernel<T, BYTES, 2, kAcrossOf2, true>)
                        : launch(combine_backward_kernel<T, BYTES, 4, kAcrossOf4, true>);
    }
    return d.k <= 2 ? launch(combine_backward_kernel<T, BYTES, 2, kAcrossOf2, false>)
                    : launch(combine_backward_kernel<T, BYTES, 4, kAcrossOf4, false>);
  }
}

template <typename T>
cudaError_t typed(const mxg_expert_rows_t& d, int op, int num_sms, cudaStream_t stream) {
  const int bytes = piece_bytes(d, sizeof(T));
  if (bytes == 32) return run<T, 32>(d, op, num_sms, stream);
  if (bytes == 16) return run<T, 16>(d, op, num_sms, stream);
  return run<T, static_cast<int>(sizeof(T))>(d, op, num_sms, stream);
}

}  // namespace

// op: 0 dispatch, 1 combine, 2 its gradients
cudaError_t launch_expert_rows(const mxg_expert_rows_t& d, int op, int num_sms,
                               cudaStream_t stream) {
  if (d.dtype == MXG_F32) return typed<float>(d, op, num_sms, stream);
  if (d.dtype == MXG_BF16) return typed<Bf16>(d, op, num_sms, stream);
  return typed<F16>(d, op, num_sms, stream);
}

}  // namespace mxg
