// grad_clip.cu -- the norm of a list of gradients and their clipping:
//   norm = sqrt(sum over tensors and elements of g^2)
//   dst  = g * min(1, max_norm / (norm + 1e-6))
//
// The list travels in the kernels' parameters (no copy to the device), cut
// into chunks of 32 KB that the CTAs take in turn: one kernel leaves
// a partial sum per CTA, the next one adds those -- each CTA the same ones in
// the same order -- and scales.  Both are bound by memory; the second walks the
// chunks backwards, so that it finds in L2 what the first read last.
//
// 1.41 G bf16 elements in 24 tensors: 1.28 ms, 6.6 TB/s for the three passes over
// 2.8 GB (a copy reaches 6.78); nothing stays in an L2 of 126 MB but the last 4 %
// read.  48 tensors of 1 to 262147 elements: 10.3 us, the two kernels' latency.
//
// Squares are summed in fp32 over 8 elements, over a thread's share of a chunk
// (8 or fewer such sums) and over a warp, and in fp64 from there on.  A sum of 8
// outside [2^-96, 2^120] -- where fp32 squares have overflowed, or may have lost
// something -- is made again from values scaled by a power of two, and kept
// apart.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

constexpr int kThreads = 512;
constexpr int kChunkBytes = 32768;            // of a source: 16384 or 8192 elements
constexpr int kVecs = kChunkBytes / 16 / kThreads;  // 16-byte pieces a thread has in flight
constexpr int kMaxBlocks = 1024;              // partial sums (fp64) in the workspace

struct GradEntry {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t first_chunk;  // chunks of the list before this tensor
  uint8_t src_type, dst_type;
  uint8_t head;     // elements before the first 16-byte boundary of src
  uint8_t dst_vec;  // dst + head lies on a 16-byte boundary too
};

template <int CAP>
struct GradList {
  GradEntry e[CAP];
  int32_t n, chunks;
};

template <int CAP>
__device__ __forceinline__ int find_entry(const GradList<CAP>& l, int chunk) {
  int lo = 0, hi = l.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.e[mid].first_chunk <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__host__ __device__ constexpr int chunk_elems(int type) {
  return kChunkBytes / (type == MXG_F32 ? 4 : 2);
}

// A chunk: elements [at, at + n) from the entry's first 16-byte boundary on;
// the first one takes the `head` elements before it too.
struct Chunk {
  int64_t at;
  int n;     // <= chunk_elems
  int head;  // > 0 in the first chunk only
};
__device__ __forceinline__ Chunk chunk_of(const GradEntry& e, int c) {
  Chunk k;
  const int most = chunk_elems(e.src_type);
  k.at = static_cast<int64_t>(c - e.first_chunk) * most;
  const int64_t left = e.numel - e.head - k.at;
  k.n = static_cast<int>(left < most ? left : most);
  k.head = k.at == 0 ? e.head : 0;
  k.at += e.head;
  return k;
}

// 16 bytes of a source as fp32: 8 or 4 elements.
template <typename T>
constexpr int kPer16 = 16 / static_cast<int>(sizeof(T));
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& q, float (&f)[kPer16<T>]) {
  if constexpr (sizeof(T) == 4) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
  } else {
    unpack2<T>(q.x, f[0], f[1]);
    unpack2<T>(q.y, f[2], f[3]);
    unpack2<T>(q.z, f[4], f[5]);
    unpack2<T>(q.w, f[6], f[7]);
  }
}

// ---------------------------------------------------------------- the norm
struct SquareSum {
  float mid = 0.0f, big = 0.0f, tiny = 0.0f;  // big: of x 2^-80, tiny: of x 2^100
  __device__ __forceinline__ void add(float q, const float* f, int n) {
    if (q >= 0x1p-96f && q <= 0x1p120f) {
      mid += q;
    } else if (!(q < 1.0f)) {  // over the range, or NaN
      for (int i = 0; i < n; ++i) {
        const float s = f[i] * 0x1p-80f;
        big = fmaf(s, s, big);
      }
    } else {
      for (int i = 0; i < n; ++i) {
        const float s = f[i] * 0x1p100f;
        tiny = fmaf(s, s, tiny);
      }
    }
  }
  template <int N>
  __device__ __forceinline__ void add_all(const float (&f)[N]) {
    float q = f[0] * f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) q = fmaf(f[i], f[i], q);
    add(q, f, N);
  }
};

template <typename T>
__device__ __forceinline__ void chunk_squares(const GradEntry& e, const Chunk& k, SquareSum& s) {
  constexpr int P = kPer16<T>;
  const T* src = static_cast<const T*>(e.src) + k.at;
  const int tid = threadIdx.x, whole = k.n & ~(P - 1);
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = (i * kThreads + tid) * P;
    v[i] = make_uint4(0, 0, 0, 0);
    if (at < whole) v[i] = *reinterpret_cast<const uint4*>(src + at);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float f[P];
    unpack16<T>(v[i], f);
    s.add_all(f);
  }
  // what 16-byte pieces do not cover: less than one at either end
  const T* rest = tid < k.head ? src - k.head + tid : src + whole + (tid - 32);
  if (tid < k.head || (tid >= 32 && tid - 32 < k.n - whole)) {
    const float f[1] = {to_f32(*rest)};
    s.add_all(f);
  }
}

template <typename T>
struct Tag {
  using type = T;
};
// fn(Tag<T>{}) with T the type of an entry: S itself, or -- void, for lists of
// several types -- whatever `type` says.
template <typename S, typename F>
__device__ __forceinline__ void with_type(int type, F&& fn) {
  if constexpr (!std::is_void<S>::value) {
    fn(Tag<S>{});
  } else {
    if (type == MXG_F32)
      fn(Tag<float>{});
    else if (type == MXG_BF16)
      fn(Tag<Bf16>{});
    else
      fn(Tag<F16>{});
  }
}

template <int CAP, typename S>
__global__ void __launch_bounds__(kThreads, 3)
    grad_squares_kernel(const __grid_constant__ GradList<CAP> list, double* partial, int first) {
  __shared__ double warp_sum[kThreads / 32];
  grid_launch_dependents();
  double sum = 0.0;  // of this warp's chunks, in its lane 0
  for (int c = blockIdx.x; c < list.chunks; c += gridDim.x) {
    const GradEntry& e = list.e[find_entry(list, c)];
    const Chunk k = chunk_of(e, c);
    SquareSum s;
    with_type<S>(e.src_type,
                 [&](auto t) { chunk_squares<typename decltype(t)::type>(e, k, s); });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s.mid += __shfl_xor_sync(0xFFFFFFFFu, s.mid, d);
    sum += static_cast<double>(s.mid);
    if (__any_sync(0xFFFFFFFFu, s.big != 0.0f || s.tiny != 0.0f)) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        s.big += __shfl_xor_sync(0xFFFFFFFFu, s.big, d);
        s.tiny += __shfl_xor_sync(0xFFFFFFFFu, s.tiny, d);
      }
      sum += static_cast<double>(s.big) * 0x1p160 + static_cast<double>(s.tiny) * 0x1p-200;
    }
  }
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += warp_sum[w];
    partial[blockIdx.x] = first ? sum : partial[blockIdx.x] + sum;
  }
}

// sqrt(total) by one warp: every lane gets it.  fp64 is slow here, so the root
// is fp32's with one Newton step (error 2^-46).
__device__ __forceinline__ double norm_of(const double* partial, int n) {
  double v = 0.0;
  for (int i = lane_id(); i < n; i += 32) v += partial[i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (!(v > 0.0) || isinf(v)) return v;  // 0, infinity, NaN
  // v = m 4^k with m in [1, 4)
  const int k = (static_cast<int>(__double2hiint(v) >> 20) - 1023) >> 1;
  const double m = __hiloint2double(__double2hiint(v) - (k << 21), __double2loint(v));
  const float r = sqrtf(static_cast<float>(m));
  const double root = static_cast<double>(r) +
                      static_cast<double>(static_cast<float>(fma(-static_cast<double>(r), r, m)) /
                                          (2.0f * r));
  return __hiloint2double(__double2hiint(root) + (k << 20), __double2loint(root));
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const double* partial, int n, float* norm) {
  const double v = norm_of(partial, n);
  if (lane_id() == 0) *norm = static_cast<float>(v);
}

// ---------------------------------------------------------------- clipping
template <typename T, typename D>
__device__ __forceinline__ void chunk_scale(const GradEntry& e, const Chunk& k, float2 factor) {
  constexpr int P = kPer16<T>;
  const T* src = static_cast<const T*>(e.src) + k.at;
  D* dst = static_cast<D*>(e.dst) + k.at;
  const int tid = threadIdx.x, whole = k.n & ~(P - 1);
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = (i * kThreads + tid) * P;
    if (at < whole) v[i] = *reinterpret_cast<const uint4*>(src + at);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = (i * kThreads + tid) * P;
    if (at >= whole) break;
    float f[P];
    unpack16<T>(v[i], f);
#pragma unroll
    for (int j = 0; j < P; ++j) f[j] = f[j] * factor.x * factor.y;
    if (e.dst_vec) {  // 8 or 4 elements of 4 or 2 bytes: 8 bytes at least
      uint32_t w[P * sizeof(D) / 4];
#pragma unroll
      for (int j = 0; j < static_cast<int>(P * sizeof(D) / 4); ++j) {
        if constexpr (sizeof(D) == 4)
          w[j] = __float_as_uint(f[j]);
        else
          w[j] = pack2<D>(f[2 * j], f[2 * j + 1]);
      }
      if constexpr (P * sizeof(D) == 8) {
        *reinterpret_cast<uint2*>(dst + at) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int j = 0; j < static_cast<int>(P * sizeof(D) / 16); ++j)
          reinterpret_cast<uint4*>(dst + at)[j] =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < P; ++j) dst[at + j] = from_f32<D>(f[j]);
    }
  }
  const int rest = tid < k.head ? tid - k.head : whole + (tid - 32);
  if (tid < k.head || (tid >= 32 && tid - 32 < k.n - whole))
    dst[rest] = from_f32<D>(to_f32(src[rest]) * factor.x * factor.y);
}

// min(1, max_norm / (norm + 1e-6)) as a product x y that is applied factor by factor:
// x = 1, but where the quotient is no normal fp32 number -- a norm may pass fp32's
// range.  There x = 2^-100 or 2^-126 and y makes up for it: g x is exact unless the
// result is below the smallest subnormal, and y keeps its bits down to quotients of
// 2^-252, whose results are fp32 subnormals or 0.
__device__ __forceinline__ float2 clip_factor(float max_norm, double norm) {
  if (isinf(max_norm))  // nothing is clipped, whatever the norm
    return make_float2(1.0f, isnan(norm) ? static_cast<float>(norm) : 1.0f);
  const double to = norm + 1e-6;
  const float f = max_norm / static_cast<float>(to);
  if (f < 0x1p-126f && !isinf(norm)) {
    const double q = static_cast<double>(max_norm) / to;
    return q < 0x1p-226 ? make_float2(0x1p-126f, static_cast<float>(q * 0x1p126))
                        : make_float2(0x1p-100f, static_cast<float>(q * 0x1p100));
  }
  return make_float2(1.0f, f > 1.0f ? 1.0f : f);  // NaN stays NaN
}

template <int CAP, typename S, typename D>
__global__ void __launch_bounds__(kThreads, std::is_void<S>::value ? 1 : 3)
    grad_scale_kernel(const __grid_constant__ GradList<CAP> list, const double* partial,
                      int partials, float max_norm, float* norm) {
  __shared__ float2 shared_factor;
  grid_wait_for_previous();  // the partial sums
  if (threadIdx.x < 32) {
    const double total = norm_of(partial, partials);
    if (threadIdx.x == 0) {
      if (norm != nullptr && blockIdx.x == 0) *norm = static_cast<float>(total);
      shared_factor = clip_factor(max_norm, total);
    }
  }
  __syncthreads();
  const float2 factor = shared_factor;
  for (int c = list.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const GradEntry& e = list.e[find_entry(list, c)];
    const Chunk k = chunk_of(e, c);
    with_type<S>(e.src_type, [&](auto s) {
      with_type<D>(e.dst_type, [&](auto d) {
        chunk_scale<typename decltype(s)::type, typename decltype(d)::type>(e, k, factor);
      });
    });
  }
}

namespace {

constexpr int kSmallList = 64, kLargeList = 512;

// Fills one launch's list from grads[*next ...]; empty tensors are skipped.
template <int CAP>
void fill(GradList<CAP>& l, const mxg_grad_t* grads, int n, int* next) {
  l.n = 0;
  l.chunks = 0;
  while (*next < n && l.n < CAP) {
    const mxg_grad_t& t = grads[*next];
    const int64_t size = t.src_type == MXG_F32 ? 4 : 2;
    const int64_t to_16 = (16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.src) & 15u)) % 16;
    const int64_t head = std::min<int64_t>(t.numel, to_16 / size);
    const int64_t per = chunk_elems(t.src_type);
    const int64_t chunks = std::max<int64_t>(1, (t.numel - head + per - 1) / per);
    if (l.chunks + chunks > INT32_MAX) break;
    ++*next;
    if (t.numel == 0) continue;
    GradEntry& e = l.e[l.n++];
    e.src = t.src;
    e.dst = t.dst;
    e.numel = t.numel;
    e.first_chunk = l.chunks;
    e.src_type = static_cast<uint8_t>(t.src_type);
    e.dst_type = static_cast<uint8_t>(t.dst_type);
    e.head = static_cast<uint8_t>(head);
    const uintptr_t to = reinterpret_cast<uintptr_t>(t.dst) +
                         static_cast<uintptr_t>(head * (t.dst_type == MXG_F32 ? 4 : 2));
    e.dst_vec = (to & 15u) == 0;
    l.chunks += static_cast<int32_t>(chunks);
  }
}

// S, D: the type of every source and of every destination of the list, or void.
template <int CAP, typename S, typename D>
cudaError_t run_list(const mxg_grad_t* grads, int n, bool clip, float max_norm, float* norm,
                     double* partial, int num_sms, cudaStream_t stream, int* launches) {
  GradList<CAP> l;
  const int most = std::min(num_sms * 3, kMaxBlocks);
  int next = 0, partials = 0;
  do {
    fill(l, grads, n, &next);
    // the first launch decides how many partial sums there are; a list that
    // goes on has 512 tensors in it, and takes them all
    const int grid = partials > 0 ? partials
                     : next < n   ? most
                                  : std::max(1, std::min(most, static_cast<int>(l.chunks)));
    grad_squares_kernel<CAP, S><<<grid, kThreads, 0, stream>>>(l, partial, partials == 0);
    ++*launches;
    partials = grid;
  } while (next < n);
  if (!clip) {
    grad_norm_kernel<<<1, 32, 0, stream>>>(partial, partials, norm);
    ++*launches;
    return cudaGetLastError();
  }
  next = 0;
  do {
    const bool whole = next == 0;
    fill(l, grads, n, &next);
    const int grid = std::max(1, std::min(most, static_cast<int>(l.chunks)));
    float* const to = whole ? norm : nullptr;
    // the first of these is set up while the squares are summed
    const cudaError_t e = launch_after(whole, grad_scale_kernel<CAP, S, D>,
                                       static_cast<unsigned>(grid), kThreads, 0, stream, l,
                                       static_cast<const double*>(partial), partials, max_norm, to);
    if (e != cudaSuccess) return e;
    ++*launches;
  } while (next < n);
  return cudaGetLastError();
}

// A list of one source type and one destination type, as nearly all are, gets
// kernels for these: the one for any types holds nine versions of its loop, and
// the registers of the worst.
template <int CAP>
cudaError_t run_types(const mxg_grad_t* grads, int n, bool clip, float max_norm, float* norm,
                      double* partial, int num_sms, cudaStream_t stream, int* launches) {
  bool one = n > 0;
  for (int i = 1; i < n; ++i)
    one = one && grads[i].src_type == grads[0].src_type &&
          (!clip || grads[i].dst_type == grads[0].dst_type);
  auto run = [&](auto s, auto d) {
    return run_list<CAP, typename decltype(s)::type, typename decltype(d)::type>(
        grads, n, clip, max_norm, norm, partial, num_sms, stream, launches);
  };
  if (!one) return run(Tag<void>{}, Tag<void>{});
  const int st = grads[0].src_type, dt = clip ? grads[0].dst_type : MXG_F32;
  auto to = [&](auto s) {
    return dt == MXG_F32 ? run(s, Tag<float>{})
                         : (dt == MXG_BF16 ? run(s, Tag<Bf16>{}) : run(s, Tag<F16>{}));
  };
  return st == MXG_F32 ? to(Tag<float>{}) : (st == MXG_BF16 ? to(Tag<Bf16>{}) : to(Tag<F16>{}));
}

}  // namespace

size_t grad_ws_bytes() { return kMaxBlocks * sizeof(double); }

cudaError_t launch_grad_clip(const mxg_grad_t* grads, int n, bool clip, float max_norm,
                             float* norm, void* ws, int num_sms, cudaStream_t stream,
                             int* launches) {
  double* partial = static_cast<double*>(ws);
  if (n <= kSmallList)
    return run_types<kSmallList>(grads, n, clip, max_norm, norm, partial, num_sms, stream, launches);
  return run_types<kLargeList>(grads, n, clip, max_norm, norm, partial, num_sms, stream, launches);
}

}  // namespace mxg
