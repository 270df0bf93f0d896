// rows.cuh -- rows of a matrix worked on by teams of threads: who owns which
// columns, the shared-memory rings the rows come through, packed fp32 pairs,
// and sums over a team.  Used by the norms around a block, both directions.
//
// A team of threads owns a row -- 8 to 32 lanes up to 256 columns, else a CTA
// with 8 or 16 columns a thread -- and walks rows in a grid stride.  What a row
// needs of its inputs is the same few 16-byte pieces for a thread every time,
// so each thread keeps its own ring of them in shared memory, filled by
// asynchronous copies up to three rows ahead: no barrier guards it, and the
// copies in flight do not depend on how far the row's reductions are.
#pragma once

#include <algorithm>
#include <atomic>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

struct RowShape {
  int team;     // threads per row
  int threads;  // per CTA: one team, or several of at most a warp
  int iter;     // chunks of 8 columns per thread
  int split;    // CTAs (a cluster) that share a row
};

// Columns of a row that one CTA of a cluster of `split` holds: a multiple of 8
// (the last one may have fewer).
__host__ __device__ inline int64_t cols_per_cta(int64_t cols, int split) {
  return split == 1 ? cols : (cols + 8 * split - 1) / (8 * split) * 8;
}

constexpr int kMaxRowCols = 16384;  // the widest row that a call accepts
constexpr int kNarrowCols = 256;    // up to which a team is a warp or less

// What a kernel lets row_shape choose from.
struct RowLimits {
  int small_cta;  // CTA size of narrow rows
  int team[2];    // threads a row may take with 8, and with 16, columns a thread
  int fit[2];     // threads an SM holds of either kernel
  int split_at;   // columns above which two CTAs share a row (7168 of an fp32
                  // stream, 2777 rows: 87 us in one CTA, 115 us in two)
};

// 8 or 16 columns a thread, whichever keeps more of an SM's threads on columns;
// where both do alike, 8.  1 <= cols <= kMaxRowCols.
inline RowShape row_shape(int64_t cols, const RowLimits& lim) {
  RowShape r = {32, 32, 1, 1};
  r.split = cols > lim.split_at ? 2 : 1;
  cols = cols_per_cta(cols, r.split);
  if (cols <= kNarrowCols) {
    r.team = 8;
    while (r.team * 8 < cols) r.team *= 2;
    r.threads = lim.small_cta;
    r.iter = 1;
    return r;
  }
  double best = -1.0;
  for (int iter = 1; iter <= 2; ++iter) {
    const int64_t busy = (cols + 8 * iter - 1) / (8 * iter);
    const int team = static_cast<int>((busy + 31) / 32 * 32);
    if (team > lim.team[iter - 1]) continue;
    if (r.split > 1 && iter == 1) continue;  // shared rows: kernels of 16 columns a thread
    const int fit = lim.fit[iter - 1];
    const double used = static_cast<double>(std::max(1, fit / team) * busy) / fit;
    if (used > best + 1e-9) {
      best = used;
      r.iter = iter;
      r.team = r.threads = team;
    }
  }
  return r;
}

// CTAs an SM holds at once.
inline int row_ctas(const RowShape& r, const RowLimits& lim, int most) {
  return std::max(1, std::min(most, lim.fit[r.iter - 1] / r.threads));
}

constexpr int kRowSmem = 220 * 1024;  // of an SM's 227 KB, for the rings of its CTAs

inline bool aligned_rows(const void* p, int64_t ld, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * static_cast<int64_t>(size)) % 16 == 0;
}

// Launches KERN with its ring, in clusters of `split`.  The shared memory that a
// kernel may be launched with belongs to the kernel, for all host threads: it is set
// once per device, to the most that any shape takes.  Set for each launch to what
// that one takes, another thread's launch of a larger shape was refused now and then
// (2761 of 30000 with three threads).
template <auto KERN, typename... Args>
cudaError_t launch_rows(const RowShape& r, int64_t grid, int smem, cudaStream_t stream,
                        const Args&... args) {
  constexpr int kMaxDev = 64;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev)
    return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(r.split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid * r.split));
  cfg.blockDim = dim3(static_cast<unsigned>(r.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = r.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, KERN, args...);
}

// ---------------------------------------------------------------- fp32 pairs
// Two fp32 in one 64-bit register pair; each half is rounded as the scalar
// instruction rounds it.
typedef uint64_t F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float v) { return f2(v, v); }
__device__ __forceinline__ float f2_lo(F2 v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return lo;
}
__device__ __forceinline__ float f2_hi(F2 v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return hi;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(F2 v) { return f2_lo(v) + f2_hi(v); }

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& v, F2 (&f)[4]) {
  float g[8];
  unpack8<T>(v, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(g[2 * i], g[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const F2 (&f)[4]) {
  Raw8<T> v;
  if constexpr (sizeof(T) == 4) {
    v.q = make_uint4(__float_as_uint(f2_lo(f[0])), __float_as_uint(f2_hi(f[0])),
                     __float_as_uint(f2_lo(f[1])), __float_as_uint(f2_hi(f[1])));
    v.r = make_uint4(__float_as_uint(f2_lo(f[2])), __float_as_uint(f2_hi(f[2])),
                     __float_as_uint(f2_lo(f[3])), __float_as_uint(f2_hi(f[3])));
  } else {
    v.q = make_uint4(pack2<T>(f2_lo(f[0]), f2_hi(f[0])), pack2<T>(f2_lo(f[1]), f2_hi(f[1])),
                     pack2<T>(f2_lo(f[2]), f2_hi(f[2])), pack2<T>(f2_lo(f[3]), f2_hi(f[3])));
  }
  return v;
}
__device__ __forceinline__ void zero4(F2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = 0;
}

// ---------------------------------------------------------------- a thread's columns
// VEC: 8 neighbouring columns a chunk, moved as 16-byte accesses; else columns
// `team` apart, one element at a time (any alignment, any width).  That costs:
// 8192 x 4099 takes 463 us backward and 152 us forward, a quarter or less of what
// memory gives.  4-byte asynchronous copies (457 us), all of a row's loads before
// the first store (444 and 163 us) and loads without branches (517 and 220 us)
// did not change that.
template <typename T, bool VEC>
struct RowIo {
  // column of (chunk it, slot e) of lane `lane` in a team of `team`
  static __device__ __forceinline__ int col(int it, int e, int lane, int team) {
    return VEC ? (it * team + lane) * 8 + e : (it * 8 + e) * team + lane;
  }
  // columns at or past `cols` are 0
  static __device__ __forceinline__ Raw8<T> load(const T* row, int cols, int it, int lane,
                                                 int team) {
    Raw8<T> v{};
    if constexpr (VEC) {
      const int c = col(it, 0, lane, team);
      if (c < cols) v = load8<T>(row + c);
    } else {
      T t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col(it, e, lane, team);
        t[e] = T{};
        if (c < cols) t[e] = row[c];
      }
      uint32_t w[sizeof(T) * 2];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(t[e]);
        v.r = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = t[2 * e].bits | (static_cast<uint32_t>(t[2 * e + 1].bits) << 16);
      }
      v.q = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
  static __device__ __forceinline__ void store(T* row, int cols, int it, int lane, int team,
                                               const F2 (&f)[4]) {
    if constexpr (VEC) {
      const int c = col(it, 0, lane, team);
      if (c < cols) {
        const Raw8<T> v = pack8<T>(f);
        if constexpr (sizeof(T) == 4) {
          // whole 32-byte sectors, where the row allows it
          if ((reinterpret_cast<uintptr_t>(row) & 31u) == 0) {
            const uint32_t w[8] = {v.q.x, v.q.y, v.q.z, v.q.w, v.r.x, v.r.y, v.r.z, v.r.w};
            st_global_32B(row + c, w);
            return;
          }
          reinterpret_cast<uint4*>(row + c)[1] = v.r;
        }
        reinterpret_cast<uint4*>(row + c)[0] = v.q;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = col(it, e, lane, team);
        if (c < cols) row[c] = from_f32<T>(e & 1 ? f2_hi(f[e >> 1]) : f2_lo(f[e >> 1]));
      }
    }
  }
};

// ---------------------------------------------------------------- the ring
// Slot, then chunk, then input, then 16-byte half, then thread.  Its addresses
// are 32-bit shared-memory ones: as generic pointers they cost two instructions
// at each of the dozen places that form one for a row.
template <typename T>
constexpr int kHalves = static_cast<int>(sizeof(T)) / 2;

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// One chunk of an input into the ring, `src` being the thread's first column of
// it: copied asynchronously where rows come in vectors, through registers where
// they do not.  `in`: the chunk lies in the row (VEC).
template <typename T, bool VEC>
__device__ __forceinline__ void ring_fill(uint32_t at, const T* src, bool in, int cols, int it,
                                          int lane, int team, int nt) {
  if constexpr (VEC) {
    if (in)
#pragma unroll
      for (int h = 0; h < kHalves<T>; ++h)
        cp_async_16_l2(at + h * nt * 16, reinterpret_cast<const uint8_t*>(src) + 16 * h);
  } else {
    const Raw8<T> v =
        RowIo<T, VEC>::load(src - RowIo<T, VEC>::col(it, 0, lane, team), cols, it, lane, team);
    st_shared_v4(at, v.q.x, v.q.y, v.q.z, v.q.w);
    if constexpr (sizeof(T) == 4) st_shared_v4(at + nt * 16, v.r.x, v.r.y, v.r.z, v.r.w);
  }
}
// A chunk back out of it.
template <typename T>
__device__ __forceinline__ void ring_read(uint32_t at, int nt, F2 (&f)[4]) {
  Raw8<T> v;
  v.q = lds16(at);
  if constexpr (sizeof(T) == 4) v.r = lds16(at + nt * 16);
  unpack8<T>(v, f);
}
// Zeros in this thread's pieces of `bytes` bytes of the ring.
__device__ __forceinline__ void ring_clear(uint32_t mine, int bytes, int nt) {
  for (int o = 0; o < bytes; o += nt * 16) st_shared_v4(mine + o, 0, 0, 0, 0);
}

// All but the newest `n` groups of this thread's copies have landed.
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n >= 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A thread's columns of a weight (ones where there is none).  REG: kept in
// registers as they lie in memory -- read again for each row, they come from L2,
// since the ring leaves L1 little room.  The forward pass on rows of over 8192
// columns has no registers to spare and does that.
template <typename T, bool VEC, int ITER, bool REG = true>
struct Weight {
  Raw8<T> raw[REG ? ITER : 1];
  const T* at;
  int cols, lane, team;
  // `w` is read from the CTA's first column, `off`, on
  __device__ __forceinline__ Weight(const void* w, int64_t off, int cols, int lane, int team)
      : at(w != nullptr ? static_cast<const T*>(w) + off : nullptr),
        cols(cols),
        lane(lane),
        team(team) {
    if constexpr (REG) {
      F2 one[4] = {f2(1.0f), f2(1.0f), f2(1.0f), f2(1.0f)};
#pragma unroll
      for (int it = 0; it < ITER; ++it)
        raw[it] = w != nullptr ? RowIo<T, VEC>::load(at, cols, it, lane, team) : pack8<T>(one);
    }
  }
  // f *= weight
  __device__ __forceinline__ void apply(int it, F2 (&f)[4]) const {
    F2 w[4];
    if constexpr (REG) {
      unpack8<T>(raw[it], w);
    } else {
      if (at == nullptr) return;
      unpack8<T>(RowIo<T, VEC>::load(at, cols, it, lane, team), w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w[i]);
  }
};

// ---------------------------------------------------------------- sums
// Sums over the team, in a fixed order, of one value or of four.  For teams of
// more than a warp (the whole CTA) `buf` holds 32 floats a value, and is written
// again only after another such sum on another buffer, or a barrier, has
// passed.
__device__ __forceinline__ float lanes_sum(float v, int span) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < span) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// A CTA's barrier, or the cluster's where two CTAs share a row.
template <int SPLIT>
__device__ __forceinline__ void team_sync() {
  if constexpr (SPLIT == 1)
    __syncthreads();
  else
    cluster_sync();
}
// A warp's sum into place `at` of the buffer of every CTA that shares the row.
template <int SPLIT>
__device__ __forceinline__ void team_post(float* buf, int at, float v) {
  buf[at] = v;
  if constexpr (SPLIT == 2)
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                     mapa_shared(smem_u32(buf + at), cluster_ctarank() ^ 1u)),
                 "f"(v)
                 : "memory");
}

__device__ __forceinline__ float team_sum(float v, float* buf, int team) {
  if (team < 32) return lanes_sum(v, team);
  v = lanes_sum(v, 32);
  if (team == 32) return v;
  const int warps = team >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[w] = v;
  __syncthreads();
  v = lane < warps ? buf[lane] : 0.0f;
  if (warps <= 8) {
    v = lanes_sum(v, 8);
    return __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return lanes_sum(v, 32);
}

// Four at once, for CTAs of at most 16 warps (SPLIT 2: rank r's warps take places
// 16 r and on).  Within a warp the lanes halve the values between them as they
// halve the span, so that four sums cost 6 shuffles and not 20.
template <int SPLIT>
__device__ __forceinline__ void team_sum4(float (&v)[4], float* buf, int team) {
  if (SPLIT == 1 && team < 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lanes_sum(v[i], team);
    return;
  }
  const int lane = threadIdx.x & 31;
  const bool h16 = (lane & 16) != 0, h8 = (lane & 8) != 0;
  // lanes with bit 4 take values 2 and 3, the others 0 and 1; bit 3 then
  // chooses within the pair
  float a = h16 ? v[2] : v[0], b = h16 ? v[3] : v[1];
  a += __shfl_xor_sync(0xFFFFFFFFu, h16 ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xFFFFFFFFu, h16 ? v[1] : v[3], 16);
  float s = h8 ? b : a;
  s += __shfl_xor_sync(0xFFFFFFFFu, h8 ? a : b, 8);
  s = lanes_sum(s, 8);
  if (SPLIT > 1 || team > 32) {
    const int warps = team >> 5, w = threadIdx.x >> 5, j = lane & 7;
    float* mine = buf + (lane >> 3) * 32;
    if (j == 0) team_post<SPLIT>(mine, SPLIT == 1 ? w : 16 * cluster_ctarank() + w, s);
    team_sync<SPLIT>();
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; k += 8)
      if (j + k < warps) {
        s += mine[j + k];
        if (SPLIT > 1) s += mine[16 + j + k];
      }
    s = lanes_sum(s, 8);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, 8 * i);
}

}  // namespace mxg
