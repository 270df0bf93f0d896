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

// Above 2048 columns 16 a thread: a row's reductions cost a warp some 60
// instructions whatever its width, and at 8 columns a thread (512 threads on
// 4096 columns) they were a third of all that was issued.
inline RowShape row_shape(int64_t cols, int small_cta) {
  RowShape r;
  if (cols <= 256) {
    r.team = 8;
    while (r.team * 8 < cols) r.team *= 2;
    r.threads = small_cta;
    r.iter = 1;
  } else {
    r.iter = cols > 2048 ? 2 : 1;
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
        reinterpret_cast<uint4*>(row + c)[0] = v.q;
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(row + c)[1] = v.r;
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
// Slot, then chunk, then input, then 16-byte half, then thread.
template <typename T>
constexpr int kHalves = static_cast<int>(sizeof(T)) / 2;

// One chunk of an input into the ring: asynchronously where rows come in
// vectors, through registers where they do not.  Columns past `cols` are left
// out (VEC) or zero.
template <typename T, bool VEC>
__device__ __forceinline__ void ring_fill(uint8_t* at, const T* row, int cols, int it, int lane,
                                          int team, int nt) {
  if constexpr (VEC) {
    const int c = RowIo<T, VEC>::col(it, 0, lane, team);
    if (c < cols)
#pragma unroll
      for (int h = 0; h < kHalves<T>; ++h)
        cp_async_16_l2(smem_u32(at + h * nt * 16),
                       reinterpret_cast<const uint8_t*>(row + c) + 16 * h);
  } else {
    const Raw8<T> v = RowIo<T, VEC>::load(row, cols, it, lane, team);
    *reinterpret_cast<uint4*>(at) = v.q;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(at + nt * 16) = v.r;
  }
}
// A chunk back out of it; 0 for a thread whose columns are past `cols`.
template <typename T, bool VEC>
__device__ __forceinline__ void ring_read(const uint8_t* at, int cols, int it, int lane, int team,
                                          int nt, F2 (&f)[4]) {
  Raw8<T> v{};
  if (RowIo<T, VEC>::col(it, 0, lane, team) < cols) {
    v.q = *reinterpret_cast<const uint4*>(at);
    if constexpr (sizeof(T) == 4) v.r = *reinterpret_cast<const uint4*>(at + nt * 16);
  }
  unpack8<T>(v, f);
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

// A thread's columns of a weight, kept in registers as they lie in memory: read
// again for each row, they come from L2, since the ring leaves L1 little room.
template <typename T, bool VEC, int ITER>
struct Weight {
  Raw8<T> raw[ITER];
  bool present;
  __device__ __forceinline__ Weight(const void* w, int cols, int lane, int team)
      : present(w != nullptr) {
#pragma unroll
    for (int it = 0; it < ITER; ++it)
      raw[it] = RowIo<T, VEC>::load(static_cast<const T*>(w), present ? cols : 0, it, lane, team);
  }
  // f *= weight
  __device__ __forceinline__ void apply(int it, F2 (&f)[4]) const {
    if (!present) return;
    F2 w[4];
    unpack8<T>(raw[it], w);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w[i]);
  }
};

// ---------------------------------------------------------------- sums
// Sums of NV values over the team, in a fixed order.  For teams of more than a
// warp (the whole CTA) `buf` holds 32 * NV floats, and is written again only
// after another team_sum on another buffer, or a barrier, has passed.
template <int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float* buf, int team) {
  if (team >= 32) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
    if (team == 32) return;
    const int warps = team >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) buf[i * 32 + w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = lane < warps ? buf[i * 32 + lane] : 0.0f;
    // 8 warps: three steps in lanes 0-7, read from lane 0
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (d < warps)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, v[i], 0);
  } else {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (d < team)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  }
}

}  // namespace mxg
