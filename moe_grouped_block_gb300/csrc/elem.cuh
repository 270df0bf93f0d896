// elem.cuh -- element types of the 16-bit operators: conversions between
// bf16 / fp16 / fp32 storage and fp32 registers, one element or 8 at a time.
#pragma once

#include "device16.cuh"

namespace mxg {

struct Bf16 {
  uint16_t bits;
};
struct F16 {
  uint16_t bits;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Bf16 v) {
  return __uint_as_float(static_cast<uint32_t>(v.bits) << 16);
}
__device__ __forceinline__ float to_f32(F16 v) {
  float r;
  asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(v.bits));
  return r;
}

// 1 / v to one unit in the last place, e^v to 2 + 1.2 |v| of them; a result below fp32's normal
// numbers is 0 (with them the exponential takes five instructions and not two).
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float exp_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.44269504f));
  return r;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) {
  Bf16 r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r.bits) : "f"(v));
  return r;
}
template <>
__device__ __forceinline__ F16 from_f32<F16>(float v) {
  F16 r;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r.bits) : "f"(v));
  return r;
}

// Two fp32 -> packed fp16x2 (round to nearest even); `lo` in the low half.
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16lo(uint32_t w) {
  return to_f32(F16{static_cast<uint16_t>(w & 0xFFFFu)});
}
__device__ __forceinline__ float f16hi(uint32_t w) {
  return to_f32(F16{static_cast<uint16_t>(w >> 16)});
}

template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi);
template <>
__device__ __forceinline__ void unpack2<Bf16>(uint32_t w, float& lo, float& hi) {
  lo = bf16lo(w);
  hi = bf16hi(w);
}
template <>
__device__ __forceinline__ void unpack2<F16>(uint32_t w, float& lo, float& hi) {
  lo = f16lo(w);
  hi = f16hi(w);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<Bf16>(float lo, float hi) {
  return cvt_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<F16>(float lo, float hi) {
  return cvt_f16x2(lo, hi);
}

// 8 consecutive elements as they lie in memory (16 or 32 bytes).
template <typename T>
struct Raw8 {
  uint4 q;
};
template <>
struct Raw8<float> {
  uint4 q, r;
};

// Vector forms: the address is 16-byte aligned.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> v;
  v.q = *reinterpret_cast<const uint4*>(p);
  if constexpr (sizeof(T) == 4) v.r = reinterpret_cast<const uint4*>(p)[1];
  return v;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& v, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    f[0] = __uint_as_float(v.q.x);
    f[1] = __uint_as_float(v.q.y);
    f[2] = __uint_as_float(v.q.z);
    f[3] = __uint_as_float(v.q.w);
    f[4] = __uint_as_float(v.r.x);
    f[5] = __uint_as_float(v.r.y);
    f[6] = __uint_as_float(v.r.z);
    f[7] = __uint_as_float(v.r.w);
  } else {
    unpack2<T>(v.q.x, f[0], f[1]);
    unpack2<T>(v.q.y, f[2], f[3]);
    unpack2<T>(v.q.z, f[4], f[5]);
    unpack2<T>(v.q.w, f[6], f[7]);
  }
}
}  // namespace mxg
