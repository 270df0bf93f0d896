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

#include "elem.cuh"
#include "mxg_host.h"

namespace mxg {

struct RowShape {
  int team;     // threads per row
  int threads;  // per CTA: one team, or several of at most a warp
  int iter;     // chunks of 8 columns per thread
};

// `wide`: columns above which a thread takes 16 of them.
inline RowShape row_shape(int64_t cols, int small_cta, int64_t wide) {
  RowShape r;
  if (cols <= 256) {
    r.team = 8;
    while (r.team * 8 < cols) r.team *= 2;
    r.threads = small_cta;
    r.iter = 1;
  } else {
    r.iter = cols > wide ? 2 : 1;
    r.team = static_cast<int>((cols + 8 * r.iter - 1) / (8 * r.iter) + 31) / 32 * 32;
    r.threads = r.team;
  }
  return r;
}

constexpr int kRowSmem = 220 * 1024;  // of an SM's 227 KB, for the rings of its CTAs

inline bool aligned_rows(const void* p, int64_t ld, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * static_cast<int64_t>(size)) % 16 == 0;
}

// Launches `kern` with its ring; more than 48 KB of shared memory in all has to be
// asked for.
template <typename Kern, typename... Args>
cudaError_t launch_rows(Kern kern, int64_t grid, int threads, int smem, cudaStream_t stream,
                        Args... args) {
  if (smem > 40 * 1024) {  // 48 KB with the static part
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<static_cast<unsigned>(grid), threads, smem, stream>>>(args...);
  return cudaGetLastError();
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
// `team` apart, one element at a time (any alignment, any width).
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
// since the ring leaves L1 little room.  Rows of over 8192 columns have no
// registers to spare and do that.
template <typename T, bool VEC, int ITER, bool REG>
struct Weight {
  Raw8<T> raw[REG ? ITER : 1];
  const T* at;
  int cols, lane, team;
  __device__ __forceinline__ Weight(const void* w, int cols, int lane, int team)
      : at(static_cast<const T*>(w)), cols(cols), lane(lane), team(team) {
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

// Four at once.  Within a warp the lanes halve the values between them as they
// halve the span, so that four sums cost 6 shuffles and not 20.
__device__ __forceinline__ void team_sum4(float (&v)[4], float* buf, int team) {
  if (team < 32) {
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
  if (team > 32) {
    const int warps = team >> 5, w = threadIdx.x >> 5, j = lane & 7;
    float* mine = buf + (lane >> 3) * 32;
    if (j == 0) mine[w] = s;
    __syncthreads();
    s = j < warps ? mine[j] : 0.0f;
#pragma unroll
    for (int k = 8; k < 32; k += 8)
      if (j + k < warps) s += mine[j + k];
    s = lanes_sum(s, 8);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, 8 * i);
}

}  // namespace mxg
