// grad_clip.cu -- the norm of a list of gradients and their clipping:
//   norm = sqrt(sum over tensors and elements of g^2)
//   dst  = g * min(1, max_norm / (norm + 1e-6))
//
// The list travels in the kernels' parameters (no copy to the device), cut
// into chunks of kChunk elements that the CTAs take in turn.  Squares are
// summed in fp32 within a chunk (at most 64 an accumulator) and in fp64 from
// there on, always in the same order.  So that fp32 neither overflows nor
// loses what is tiny, 8 elements whose largest magnitude is outside
// [2^-50, 2^50] are scaled by a power of two before they are squared, and
// summed apart.
#include "elem.cuh"
#include "mxg_host.h"

namespace mxg {

constexpr int kChunk = 16384;
constexpr int kGradThreads = 256;
constexpr int kGradMaxBlocks = 1024;  // partial sums (fp64) in the workspace

struct GradEntry {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t first_chunk;  // chunks of the list before this tensor
  uint8_t src_type, dst_type, src_vec, both_vec;
};

template <int CAP>
struct GradList {
  GradEntry e[CAP];
  int32_t n, chunks;
};

struct SquareSum {
  float mid = 0.0f, big = 0.0f, tiny = 0.0f;
  __device__ __forceinline__ void add(const float* f, int n) {
    float m = 0.0f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, fabsf(f[i]));
    if (m <= 0x1p50f && (m >= 0x1p-50f || m == 0.0f)) {
      for (int i = 0; i < n; ++i) mid = fmaf(f[i], f[i], mid);
    } else if (m > 0x1p50f) {
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
    // (fmaxf drops a NaN, but every branch squares all n values)
  }
  __device__ __forceinline__ double value() const {
    return static_cast<double>(mid) + static_cast<double>(big) * 0x1p160 +
           static_cast<double>(tiny) * 0x1p-200;
  }
};

template <int CAP>
__device__ __forceinline__ int find_entry(const GradList<CAP>& l, int chunk) {
  int lo = 0, hi = l.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.e[mid].first_chunk <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// Sum of v over the CTA in a fixed order (every thread gets it).
__device__ __forceinline__ double block_sum_f64(double v, double* buf) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  const int warps = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[w] = v;
  __syncthreads();
  v = lane < warps ? buf[lane] : 0.0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* src, int64_t n, bool vec) {
  SquareSum s;
  int64_t done = 0;
  if (vec) {
    done = n & ~static_cast<int64_t>(7);
    for (int64_t i = threadIdx.x * 8; i < done; i += kGradThreads * 8) {
      float f[8];
      unpack8<T>(load8<T>(src + i), f);
      s.add(f, 8);
    }
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kGradThreads) {
    const float f[1] = {to_f32(src[i])};
    s.add(f, 1);
  }
  return s.value();
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads)
    grad_squares_kernel(const __grid_constant__ GradList<CAP> list, double* partial, int first) {
  __shared__ double buf[32];
  double sum = 0.0;
  for (int c = blockIdx.x; c < list.chunks; c += gridDim.x) {
    const GradEntry& e = list.e[find_entry(list, c)];
    const int64_t at = static_cast<int64_t>(c - e.first_chunk) * kChunk;
    const int64_t n = min(e.numel - at, static_cast<int64_t>(kChunk));
    if (e.src_type == MXG_F32)
      sum += chunk_squares(static_cast<const float*>(e.src) + at, n, e.src_vec);
    else if (e.src_type == MXG_BF16)
      sum += chunk_squares(static_cast<const Bf16*>(e.src) + at, n, e.src_vec);
    else
      sum += chunk_squares(static_cast<const F16*>(e.src) + at, n, e.src_vec);
  }
  sum = block_sum_f64(sum, buf);
  if (threadIdx.x == 0) partial[blockIdx.x] = first ? sum : partial[blockIdx.x] + sum;
}

__device__ __forceinline__ double total_squares(const double* partial, int n, double* buf) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += partial[i];
  return block_sum_f64(v, buf);
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* partial, int n, float* norm) {
  __shared__ double buf[32];
  const double s = total_squares(partial, n, buf);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <typename T, typename D>
__device__ __forceinline__ void chunk_scale(const T* src, D* dst, int64_t n, bool vec,
                                            float factor) {
  int64_t done = 0;
  if (vec) {
    done = n & ~static_cast<int64_t>(7);
    for (int64_t i = threadIdx.x * 8; i < done; i += kGradThreads * 8) {
      float f[8];
      unpack8<T>(load8<T>(src + i), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= factor;
      store8<D>(dst + i, f);
    }
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kGradThreads)
    dst[i] = from_f32<D>(to_f32(src[i]) * factor);
}

template <typename T>
__device__ __forceinline__ void chunk_scale_to(const GradEntry& e, int64_t at, int64_t n,
                                               float factor) {
  const T* src = static_cast<const T*>(e.src) + at;
  if (e.dst_type == MXG_F32)
    chunk_scale(src, static_cast<float*>(e.dst) + at, n, e.both_vec, factor);
  else if (e.dst_type == MXG_BF16)
    chunk_scale(src, static_cast<Bf16*>(e.dst) + at, n, e.both_vec, factor);
  else
    chunk_scale(src, static_cast<F16*>(e.dst) + at, n, e.both_vec, factor);
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads)
    grad_scale_kernel(const __grid_constant__ GradList<CAP> list, const double* partial,
                      int partials, float max_norm, float* norm) {
  __shared__ double buf[32];
  const double total = sqrt(total_squares(partial, partials, buf));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const double f = static_cast<double>(max_norm) / (total + 1e-6);
  const float factor = f > 1.0 ? 1.0f : static_cast<float>(f);  // NaN stays NaN
  for (int c = blockIdx.x; c < list.chunks; c += gridDim.x) {
    const GradEntry& e = list.e[find_entry(list, c)];
    const int64_t at = static_cast<int64_t>(c - e.first_chunk) * kChunk;
    const int64_t n = min(e.numel - at, static_cast<int64_t>(kChunk));
    if (e.src_type == MXG_F32) chunk_scale_to<float>(e, at, n, factor);
    else if (e.src_type == MXG_BF16) chunk_scale_to<Bf16>(e, at, n, factor);
    else chunk_scale_to<F16>(e, at, n, factor);
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
    const int64_t chunks = (t.numel + kChunk - 1) / kChunk;
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
    e.src_vec = (reinterpret_cast<uintptr_t>(t.src) & 15u) == 0;
    e.both_vec = e.src_vec && (reinterpret_cast<uintptr_t>(t.dst) & 15u) == 0;
    l.chunks += static_cast<int32_t>(chunks);
  }
}

template <int CAP>
cudaError_t run_list(const mxg_grad_t* grads, int n, bool clip, float max_norm, float* norm,
                     double* partial, int num_sms, cudaStream_t stream, int* launches) {
  GradList<CAP> l;
  const int grid = num_sms * 4 < kGradMaxBlocks ? num_sms * 4 : kGradMaxBlocks;
  int next = 0, first = 1;
  do {
    fill(l, grads, n, &next);
    grad_squares_kernel<CAP><<<grid, kGradThreads, 0, stream>>>(l, partial, first);
    ++*launches;
    first = 0;
  } while (next < n);
  if (!clip) {
    grad_norm_kernel<<<1, kGradThreads, 0, stream>>>(partial, grid, norm);
    ++*launches;
    return cudaGetLastError();
  }
  next = 0;
  do {
    fill(l, grads, n, &next);
    grad_scale_kernel<CAP><<<grid, kGradThreads, 0, stream>>>(l, partial, grid, max_norm, norm);
    ++*launches;
    norm = nullptr;
  } while (next < n);
  return cudaGetLastError();
}

}  // namespace

size_t grad_ws_bytes() { return kGradMaxBlocks * sizeof(double); }

cudaError_t launch_grad_clip(const mxg_grad_t* grads, int n, bool clip, float max_norm,
                             float* norm, void* ws, int num_sms, cudaStream_t stream,
                             int* launches) {
  double* partial = static_cast<double*>(ws);
  if (n <= kSmallList)
    return run_list<kSmallList>(grads, n, clip, max_norm, norm, partial, num_sms, stream, launches);
  return run_list<kLargeList>(grads, n, clip, max_norm, norm, partial, num_sms, stream, launches);
}

}  // namespace mxg
