// gated_act.cu -- the activation between an expert's two products, with its inputs kept
// in 8 bits for the backward pass:
//   h = act(gate) up,  act(x) = x sigmoid(z(x));  z = x, or 2 sqrt(2 / pi) (x + 0.044715 x^3)
//   kept: E4M3 with one E8M0 scale for each 32 columns of a row (mx_exponent's rule)
//   dgate = dh up act'(gate),  dup = dh act(gate),  act' = s + x s (1 - s) z'
//
// A thread owns 16 columns -- 32 bytes of a 16-bit tensor, 16 of the kept values -- and the
// thread beside it the other half of the 32 that share a scale, so a block's largest
// magnitude is one shuffle away.  Rows that do not start on 16 bytes, or whose columns are no
// multiple of 8, have a lane for each column and a warp for each block.  Each input is read once
// and each output written once: memory is the bound.
//
// Forward, 16384 x 14336 in bf16 with the checkpoint: 289 us, 6.55 TB/s of the 6.78 that a copy
// reaches (14328 columns, rows on 16 bytes: 301 us; 14335, a lane a column: 683 us).  Backward,
// 32768 x 1408 in fp16 with h again: 70.5 us, 6.6 TB/s; 5 us more without the next half's loads
// ahead.
#include <algorithm>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

constexpr int kActThreads = 256;

// 16 neighbouring values of a 16-bit type as packed pairs, by accesses of ALIGN = 32 or 16 bytes;
// of the latter only the first where n is 8.
template <typename T, int ALIGN>
__device__ __forceinline__ void load16(const T* p, int n, uint32_t (&w)[8]) {
  // (volatile: in order with the stores)
  if constexpr (ALIGN == 32) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
    w[4] = w[5] = w[6] = w[7] = 0;
    if (n > 8)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p + 8));
  }
}
template <typename T, int ALIGN>
__device__ __forceinline__ void store16(T* p, int n, const float (&f)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
  if constexpr (ALIGN == 32) {
    st_global_32B(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (n > 8) reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
template <typename T>
__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) unpack2<T>(w[i], f[2 * i], f[2 * i + 1]);
}

// Four E4M3 bytes -> fp32, exact.
__device__ __forceinline__ void e4m3x4_values(uint32_t b, float* f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(b));
  f[0] = f16lo(lo);
  f[1] = f16hi(lo);
  f[2] = f16lo(hi);
  f[3] = f16hi(hi);
}

// The value of a scale byte: 2^(b - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : (b == 255u ? 0x7FC00000u : b << 23);
  return __uint_as_float(bits);
}

// sigmoid(z(x)), and z'(x).
template <int ACT>
__device__ __forceinline__ float act_z(float x) {
  if constexpr (ACT == MXG_ACT_SILU) return x;
  const float u = 1.59576912f * x;
  return fmaf(0.0713548163f * x * x, x, u);
}
template <int ACT>
__device__ __forceinline__ float act_dz(float x) {
  if constexpr (ACT == MXG_ACT_SILU) return 1.0f;
  // (bounded: it meets a slope of 0 there)
  return fmaf(0.214064449f, fminf(x * x, 1e30f), 1.59576912f);
}

// Rows that take part: the sum of the group sizes, at most `rows`.
__device__ __forceinline__ int64_t act_rows(const mxg_gated_act_t& d) {
  if (d.group_ws == nullptr) return d.rows;
  int64_t sum = 0;
  for (int g = lane_id(); g < d.G; g += 32) {
    const int64_t s = d.group_ws[g];
    sum += s < 0 ? 0 : (s < d.rows ? s : d.rows);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum < d.rows ? sum : d.rows;
}

// A thread's walk through the halves of blocks, `halves` (even) a row, a grid apart.
struct HalfWalk {
  int64_t row;
  int half;
  int64_t row_step;
  int half_step, halves;
  __device__ __forceinline__ HalfWalk(int halves) : halves(halves) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kActThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kActThreads;
    row = at / halves;
    half = static_cast<int>(at - row * halves);
    row_step = step / halves;
    half_step = static_cast<int>(step - row_step * halves);
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    half += half_step;
    if (half >= halves) {
      half -= halves;
      ++row;
    }
  }
};

// 16 of a block's values to E4M3 bytes and the block's scale byte, with the lane beside
// this one; all lanes of the warp take part.
template <int ALIGN>
__device__ __forceinline__ void keep16(const float (&v)[16], bool on, int n, uint8_t* q,
                                       uint8_t* sf, bool first) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = v[i];
  if (isinf(top)) {  // an infinity is kept as NaN
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (isinf(f[i])) f[i] = __uint_as_float(0x7FC00000u);
      top = fmaxf(top, fabsf(f[i]));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  const int e = mx_exponent(top);
  const float scale = pow2_neg(e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = cvt_e4m3x2(f[4 * i] * scale, f[4 * i + 1] * scale) |
           (cvt_e4m3x2(f[4 * i + 2] * scale, f[4 * i + 3] * scale) << 16);
  if (!on) return;
  if constexpr (ALIGN == 32) {
    if (n > 0) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {  // (kept rows on 8 bytes)
    if (n > 0) reinterpret_cast<uint2*>(q)[0] = make_uint2(w[0], w[1]);
    if (n > 8) reinterpret_cast<uint2*>(q)[1] = make_uint2(w[2], w[3]);
  }
  if (first) *sf = static_cast<uint8_t>(e + 127);
}

template <typename T, int ACT, bool GATED, int ALIGN>
__global__ void __launch_bounds__(kActThreads)
    gated_act_kernel(const mxg_gated_act_t d, int blocks) {
  const int cols = static_cast<int>(d.cols);
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t live = act_rows(d);
  const bool keep = d.q != nullptr;
  HalfWalk at(2 * blocks);
  const int64_t sf_row = (GATED ? 2 : 1) * static_cast<int64_t>(blocks);
  // (a row ends with a warp's pair of lanes, so both of a pair go on or both stop)
  while (__any_sync(0xFFFFFFFFu, at.row < live)) {
    const bool on = at.row < live;
    const int c = at.half * 16;
    const int n = on ? min(cols - c, 16) : 0;  // 0 or less: the half is empty
    uint32_t gw[8] = {}, uw[8] = {};
    if (n > 0) {
      load16<T, ALIGN>(static_cast<const T*>(d.gate) + at.row * d.ldg + c, n, gw);
      if (GATED) load16<T, ALIGN>(static_cast<const T*>(d.up) + at.row * d.ldu + c, n, uw);
    }
    float g[16], u[16], h[16];
    unpack16<T>(gw, g);
    if (GATED) unpack16<T>(uw, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      h[i] = g[i] * rcp_approx(1.0f + exp_approx(-act_z<ACT>(g[i])));
      if (GATED) h[i] *= u[i];
    }
    if (n > 0) store16<T, ALIGN>(static_cast<T*>(d.h) + at.row * d.ldh + c, n, h);
    if (keep) {
      uint8_t* q = d.q + at.row * d.ldq + c;
      uint8_t* sf = d.sf + at.row * sf_row + (at.half >> 1);
      const bool first = (at.half & 1) == 0;
      keep16<ALIGN>(g, on, n, q, sf, first);
      if (GATED) keep16<ALIGN>(u, on, n, q + cols, sf + blocks, first);
    }
    at.next();
  }
}

// 16 kept bytes as words, and the values that they stand for.
template <int ALIGN>
__device__ __forceinline__ void load_kept(const uint8_t* q, int n, uint32_t (&w)[4]) {
  if constexpr (ALIGN == 32) {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(q));
  } else {
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(q));
    w[2] = w[3] = 0;
    if (n > 8) asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[2]), "=r"(w[3]) : "l"(q + 8));
  }
}

// What a thread reads for 16 columns.
template <typename T, bool GATED, int ALIGN>
struct KeptHalf {
  uint32_t dh[8], g[4], u[4];
  uint32_t sf_g, sf_u;
  __device__ __forceinline__ void load(const mxg_gated_act_t& d, const HalfWalk& at, int64_t live,
                                       int blocks) {
    const int c = at.half * 16, cols = static_cast<int>(d.cols);
    const int n = min(cols - c, 16);
    if (at.row >= live || n <= 0) return;
    const uint8_t* q = d.q + at.row * d.ldq + c;
    const uint8_t* sf =
        d.sf + at.row * ((GATED ? 2 : 1) * static_cast<int64_t>(blocks)) + (at.half >> 1);
    load_kept<ALIGN>(q, n, g);
    sf_g = sf[0];
    if (GATED) {
      load_kept<ALIGN>(q + cols, n, u);
      sf_u = sf[blocks];
    }
    load16<T, ALIGN>(static_cast<const T*>(d.dh) + at.row * d.lddh + c, n, dh);
  }
};

template <typename T, int ACT, bool GATED, int ALIGN>
__global__ void __launch_bounds__(kActThreads, 3)
    gated_act_backward_kernel(const mxg_gated_act_t d, int blocks) {
  const int cols = static_cast<int>(d.cols);
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t live = act_rows(d);
  HalfWalk at(2 * blocks), then = at;
  KeptHalf<T, GATED, ALIGN> in;
  in.load(d, at, live, blocks);
  for (; at.row < live; at = then) {
    // the next ones are asked for before these are worked on
    then.next();
    KeptHalf<T, GATED, ALIGN> in2;
    in2.load(d, then, live, blocks);
    const int c = at.half * 16;
    const int n = min(cols - c, 16);
    if (n > 0) {
      T* dgate = static_cast<T*>(d.dgate) + at.row * d.lddg + c;
      T* dup = GATED ? static_cast<T*>(d.dup) + at.row * d.lddu + c : nullptr;
      T* h = d.h != nullptr ? static_cast<T*>(d.h) + at.row * d.ldh + c : nullptr;
      const float scale_g = e8m0_value(in.sf_g), scale_u = GATED ? e8m0_value(in.sf_u) : 0.0f;
      float dg[16], du[16], again[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float g[4], u[4], dh[4];
        e4m3x4_values(in.g[i], g);
        if (GATED) e4m3x4_values(in.u[i], u);
        unpack2<T>(in.dh[2 * i], dh[0], dh[1]);
        unpack2<T>(in.dh[2 * i + 1], dh[2], dh[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = g[j] * scale_g;
          const float s = rcp_approx(1.0f + exp_approx(-act_z<ACT>(x)));
          const float a = x * s;
          const float slope = fmaf(a * (1.0f - s), act_dz<ACT>(x), s);
          if (GATED) {
            const float y = u[j] * scale_u;
            dg[4 * i + j] = dh[j] * y * slope;
            du[4 * i + j] = dh[j] * a;
            again[4 * i + j] = y * a;
          } else {
            dg[4 * i + j] = dh[j] * slope;
            again[4 * i + j] = a;
          }
        }
      }
      store16<T, ALIGN>(dgate, n, dg);
      if (GATED) store16<T, ALIGN>(dup, n, du);
      if (h != nullptr) store16<T, ALIGN>(h, n, again);
    }
    in = in2;
  }
}

// ---------------------------------------------------------------- rows of any alignment
// A warp's item: kAcross blocks of a row side by side, a lane a column of each.
constexpr int kAcross = 4;

struct BlockWalk {
  int64_t row, row_step;
  int group, group_step, groups;
  __device__ __forceinline__ BlockWalk(int blocks) : groups((blocks + kAcross - 1) / kAcross) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kActThreads / 32);
    row = at / groups;
    group = static_cast<int>(at - row * groups);
    row_step = step / groups;
    group_step = static_cast<int>(step - row_step * groups);
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    group += group_step;
    if (group >= groups) {
      group -= groups;
      ++row;
    }
  }
};

// A column's value to its E4M3 byte, and the block's scale byte; by a whole warp.
__device__ __forceinline__ uint32_t keep_column(float v, uint32_t& byte) {
  // magnitudes are in the order of their bits
  uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v)));
  if (top >= 0x7F800000u) {  // infinities are kept as NaN, and neither is among the magnitudes
    const bool fine = fabsf(v) < INFINITY;
    top = __reduce_max_sync(0xFFFFFFFFu, fine ? __float_as_uint(fabsf(v)) : 0u);
    if (!fine) v = __uint_as_float(0x7FC00000u);
  }
  const int e = mx_exponent(__uint_as_float(top));
  byte = cvt_e4m3x2(v * pow2_neg(e), 0.0f);
  return static_cast<uint32_t>(e + 127);
}

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kActThreads)
    gated_act_columns_kernel(const mxg_gated_act_t d, int blocks) {
  const int cols = static_cast<int>(d.cols), lane = threadIdx.x & 31;
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t live = act_rows(d), sf_row = (GATED ? 2 : 1) * static_cast<int64_t>(blocks);
  for (BlockWalk at(blocks); at.row < live; at.next()) {
    const T* gate = static_cast<const T*>(d.gate) + at.row * d.ldg;
    const T* up = GATED ? static_cast<const T*>(d.up) + at.row * d.ldu : nullptr;
    T* h = static_cast<T*>(d.h) + at.row * d.ldh;
    const int b0 = at.group * kAcross;
    float g[kAcross], u[kAcross];
#pragma unroll
    for (int i = 0; i < kAcross; ++i) {
      const int c = (b0 + i) * 32 + lane;
      g[i] = c < cols ? to_f32(gate[c]) : 0.0f;
      u[i] = GATED && c < cols ? to_f32(up[c]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kAcross; ++i) {
      const int c = (b0 + i) * 32 + lane;
      float v = g[i] * rcp_approx(1.0f + exp_approx(-act_z<ACT>(g[i])));
      if (GATED) v *= u[i];
      if (c < cols) h[c] = from_f32<T>(v);
    }
    if (d.q == nullptr) continue;
    uint8_t* q = d.q + at.row * d.ldq;
    uint8_t* sf = d.sf + at.row * sf_row;
    uint32_t mine_g = 0, mine_u = 0;  // lane i keeps the scale of block i
#pragma unroll
    for (int i = 0; i < kAcross; ++i) {
      const int c = (b0 + i) * 32 + lane;
      uint32_t byte;
      const uint32_t scale = keep_column(g[i], byte);
      if (c < cols) q[c] = static_cast<uint8_t>(byte);
      if (lane == i) mine_g = scale;
      if (GATED) {
        const uint32_t scale_u = keep_column(u[i], byte);
        if (c < cols) q[cols + c] = static_cast<uint8_t>(byte);
        if (lane == i) mine_u = scale_u;
      }
    }
    if (lane < kAcross && b0 + lane < blocks) {
      sf[b0 + lane] = static_cast<uint8_t>(mine_g);
      if (GATED) sf[blocks + b0 + lane] = static_cast<uint8_t>(mine_u);
    }
  }
}

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kActThreads)
    gated_act_backward_columns_kernel(const mxg_gated_act_t d, int blocks) {
  const int cols = static_cast<int>(d.cols), lane = threadIdx.x & 31;
  grid_wait_for_previous();
  grid_launch_dependents();
  const int64_t live = act_rows(d), sf_row = (GATED ? 2 : 1) * static_cast<int64_t>(blocks);
  for (BlockWalk at(blocks); at.row < live; at.next()) {
    const T* dh = static_cast<const T*>(d.dh) + at.row * d.lddh;
    T* dgate = static_cast<T*>(d.dgate) + at.row * d.lddg;
    T* dup = GATED ? static_cast<T*>(d.dup) + at.row * d.lddu : nullptr;
    T* h = d.h != nullptr ? static_cast<T*>(d.h) + at.row * d.ldh : nullptr;
    const uint8_t* q = d.q + at.row * d.ldq;
    const uint8_t* sf = d.sf + at.row * sf_row;
    const int b0 = at.group * kAcross;
    uint32_t qg[kAcross], qu[kAcross], sg[kAcross], su[kAcross];
    float y[kAcross];
#pragma unroll
    for (int i = 0; i < kAcross; ++i) {
      const int b = b0 + i, c = b * 32 + lane;
      const bool in = c < cols;
      qg[i] = in ? q[c] : 0u;
      qu[i] = GATED && in ? q[cols + c] : 0u;
      sg[i] = in ? sf[b] : 0u;
      su[i] = GATED && in ? sf[blocks + b] : 0u;
      y[i] = in ? to_f32(dh[c]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kAcross; ++i) {
      const int c = (b0 + i) * 32 + lane;
      float f[4];
      e4m3x4_values(qg[i] | (qu[i] << 8), f);
      const float x = f[0] * e8m0_value(sg[i]), u = f[1] * e8m0_value(su[i]);
      const float s = rcp_approx(1.0f + exp_approx(-act_z<ACT>(x))), a = x * s;
      const float slope = fmaf(a * (1.0f - s), act_dz<ACT>(x), s);
      if (c < cols) {
        dgate[c] = from_f32<T>(GATED ? y[i] * u * slope : y[i] * slope);
        if (GATED) dup[c] = from_f32<T>(y[i] * a);
        if (h != nullptr) h[c] = from_f32<T>(GATED ? u * a : a);
      }
    }
  }
}

namespace {

// The widest accesses that every row allows: 32 or 16 bytes (of the kept values half as many), or
// 2, an element's.
int act_align(const mxg_gated_act_t& d) {
  const uintptr_t kept = reinterpret_cast<uintptr_t>(d.q) |
                         (d.q != nullptr ? static_cast<uintptr_t>(d.ldq | d.cols) : 0);
  uintptr_t all = 2 * kept | static_cast<uintptr_t>(2 * d.cols);
  auto add = [&](const void* p, int64_t ld) {
    if (p != nullptr) all |= reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(2 * ld);
  };
  add(d.gate, d.ldg);
  add(d.up, d.ldu);
  add(d.h, d.ldh);
  add(d.dh, d.lddh);
  add(d.dgate, d.lddg);
  add(d.dup, d.lddu);
  return (all & 31u) == 0 ? 32 : ((all & 15u) == 0 ? 16 : 2);
}

template <typename T, int ACT, bool GATED>
cudaError_t run(const mxg_gated_act_t& d, bool backward, int num_sms, cudaStream_t stream) {
  const int blocks = static_cast<int>((d.cols + 31) / 32), align = act_align(d);
  const int64_t threads = align == 2 ? d.rows * ((blocks + kAcross - 1) / kAcross) * 32
                                     : d.rows * 2 * blocks;
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>((threads + kActThreads - 1) / kActThreads, num_sms * 16LL));
  auto launch = [&](auto kern) {
    return launch_after(true, kern, grid, kActThreads, 0, stream, d, blocks);
  };
  if (backward)
    return align == 32   ? launch(gated_act_backward_kernel<T, ACT, GATED, 32>)
           : align == 16 ? launch(gated_act_backward_kernel<T, ACT, GATED, 16>)
                         : launch(gated_act_backward_columns_kernel<T, ACT, GATED>);
  return align == 32   ? launch(gated_act_kernel<T, ACT, GATED, 32>)
         : align == 16 ? launch(gated_act_kernel<T, ACT, GATED, 16>)
                       : launch(gated_act_columns_kernel<T, ACT, GATED>);
}

template <typename T>
cudaError_t typed(const mxg_gated_act_t& d, bool backward, int num_sms, cudaStream_t stream) {
  if (d.act == MXG_ACT_SILU)
    return d.gated ? run<T, MXG_ACT_SILU, true>(d, backward, num_sms, stream)
                   : run<T, MXG_ACT_SILU, false>(d, backward, num_sms, stream);
  return d.gated ? run<T, MXG_ACT_GELU_TANH, true>(d, backward, num_sms, stream)
                 : run<T, MXG_ACT_GELU_TANH, false>(d, backward, num_sms, stream);
}

}  // namespace

cudaError_t launch_gated_act(const mxg_gated_act_t& d, bool backward, int num_sms,
                             cudaStream_t stream) {
  return d.dtype == MXG_BF16 ? typed<Bf16>(d, backward, num_sms, stream)
                             : typed<F16>(d, backward, num_sms, stream);
}

}  // namespace mxg
