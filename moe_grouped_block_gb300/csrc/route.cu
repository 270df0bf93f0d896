// route.cu -- tokens to experts: the k best logits of each token, their weights, the
// tokens of each expert, the balance loss, and the rows that the tokens take among
// the experts' groups; and the gradient of the weights and of the loss.
//
//   s = softmax(l) or sigmoid(l);  p = s / sum(s);  weight = scale * s [/ sum of the chosen s]
//   loss = sum_e slope_e sum_t p_te,  slope_e = balance * E / n * counts_e / sum(counts)
//
// A token is worked on by a team of 1 to 32 lanes that keep its logits in registers, 8 to
// 32 neighbouring columns a lane.  Logits are compared as integers of the same order; an
// expert is taken out by a maximum over the team and a ballot for the lowest lane that
// holds it.
//
// The tokens are cut into chunks, one for each CTA, which leaves its chunk's tokens per
// expert and sums of p in the workspace.  A second kernel adds these up -- each CTA the
// same ones in the same order -- and gives its chunk's tokens their rows: the expert's
// start, the tokens of it in earlier chunks, those of earlier warps, and the rank among
// the warp's lanes.  One chunk alone is finished by the first kernel.  No floating-point
// atomics and no counters kept between calls.
#include <algorithm>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxChunks = 304;
constexpr uint32_t kNoLogit = 0x007FFFFFu;  // the key of -infinity: it and all below are not chosen
constexpr int kBufWords = 4096;

// The workspace: chunk by chunk, tokens per expert, sums of p, tokens that take part.
struct RouteWs {
  int32_t* hist;  // [chunks][experts]
  float* psum;    // [chunks][experts]
  int32_t* live;  // [chunks]
};

// What the second half needs to know.
struct RowPlan {
  const int32_t* expert;
  int32_t* counts;
  float* loss;
  float* slope;
  int32_t* row_of;
  int64_t* group_ws;
  int32_t* status;
  int64_t tokens, per;  // per: tokens a chunk
  int64_t last_dim;
  uint32_t capacity;  // a multiple of align
  int32_t experts, k, align, chunks;
  float balance;
};

struct RouteShared {
  uint32_t buf[kBufWords];  // sums of p by warp, then tokens per expert by warp
  int32_t hist[kMaxExperts];
  float psum[kMaxExperts];
  uint32_t total[kMaxExperts], before[kMaxExperts], start[kMaxExperts];
  uint32_t warp_sum[kRouteWarps];
  float warp_f[kRouteWarps];
  int32_t live;
  uint32_t sum;
};

// Logits as unsigned integers of the same order: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  if (v != v) return 0xFFFFFFFFu;
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// sigmoid(l) e^-m, with m <= 0: shares of a token whose sigmoids all underflow are still
// right (m the largest logit where that is negative).
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
  const float e = __expf(-fabsf(l));
  const float num = l >= 0.0f ? 1.0f : (m < 0.0f ? __expf(l - m) : e);
  return l != l ? l : __fdividef(num, 1.0f + e);
}

template <int LPT>
__device__ __forceinline__ float team_add(float v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  if constexpr (LPT == 32) return __reduce_max_sync(0xFFFFFFFFu, v);
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}

// A lane's columns of a row, as they lie in memory; -infinity past the last expert.
template <typename T, int VPL>
struct LogitRow {
  Raw8<T> raw[VPL / 8];
  __device__ __forceinline__ void load(const T* row, int c0, int experts, bool vec) {
#pragma unroll
    for (int i = 0; i < VPL / 8; ++i) {
      const int c = c0 + 8 * i;
      if (vec && c < experts) {
        raw[i] = load8<T>(row + c);
      } else {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          t[j] = from_f32<T>(-INFINITY);
          if (c + j < experts) t[j] = row[c + j];
        }
        uint32_t w[sizeof(T) * 2];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(t[j]);
          raw[i].r = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = t[2 * j].bits | (static_cast<uint32_t>(t[2 * j + 1].bits) << 16);
        }
        raw[i].q = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[VPL]) const {
#pragma unroll
    for (int i = 0; i < VPL / 8; ++i) {
      float f[8];
      unpack8<T>(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * i + j] = f[j];
    }
  }
};

// ---------------------------------------------------------------- rows
// Everything that needs the whole batch's counts, by the CTA of chunk c.  `hist`, `psum`
// and `live` are the chunks' (this CTA's own where there is one chunk).  The first CTA
// writes counts and group_ws, the last one slope and loss.
__device__ void finish_chunk(const RowPlan& p, RouteShared& sh, const int32_t* hist,
                             const float* psum, const int32_t* live, int c) {
  const int tid = threadIdx.x, E = p.experts;
  const int lane = tid & 31, warp = tid >> 5;
  int wide = 1;  // experts, as a power of two
  while (wide < E) wide *= 2;
  const int parts = max(1, min(min(kRouteThreads / wide, 16), p.chunks));
  uint32_t* part_total = sh.buf;
  uint32_t* part_before = sh.buf + kBufWords / 2;
  // tokens of each expert, in all chunks and in those before this one
  for (int i = tid; i < parts * wide; i += kRouteThreads) {
    const int e = i & (wide - 1), part = i / wide;
    uint32_t total = 0, before = 0;
    if (e < E) {
#pragma unroll 8
      for (int h = part; h < p.chunks; h += parts) {
        const uint32_t v = static_cast<uint32_t>(hist[static_cast<int64_t>(h) * E + e]);
        total += v;
        before += h < c ? v : 0u;
      }
    }
    part_total[i] = total;
    part_before[i] = before;
  }
  __syncthreads();
  // starts of the padded groups: two experts a thread, a scan over the warp and the CTA
  uint32_t size[2], total[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    uint32_t t = 0, b = 0;
    if (e < E) {
      for (int part = 0; part < parts; ++part) {
        t += part_total[part * wide + e];
        b += part_before[part * wide + e];
      }
      sh.total[e] = t;
      sh.before[e] = b;
    }
    total[i] = t;
    const uint32_t a = static_cast<uint32_t>(p.align);
    size[i] = a == 1 ? t : (t + a - 1) / a * a;
  }
  uint32_t incl = size[0] + size[1], sum = total[0] + total[1];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  sum = __reduce_add_sync(0xFFFFFFFFu, sum);
  __syncthreads();  // part_total has been read
  if (lane == 31) {
    sh.warp_sum[warp] = incl;
    sh.buf[warp] = sum;
  }
  __syncthreads();
  uint32_t ahead = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w < warp) ahead += sh.warp_sum[w];
    all += sh.buf[w];
  }
  uint32_t start = ahead + incl - size[0] - size[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    if (e < E) {
      sh.start[e] = start;
      if (c == 0) {
        if (p.counts != nullptr) p.counts[e] = static_cast<int32_t>(total[i]);
        if (p.group_ws != nullptr) {
          const uint32_t from = min(start, p.capacity), to = min(start + size[i], p.capacity);
          p.group_ws[e] = static_cast<int64_t>(to - from);
          p.group_ws[E + 1 + e] = static_cast<int64_t>(to) * p.last_dim;
          if (e == 0) p.group_ws[E] = 0;
          if (start + size[i] > p.capacity) status_set(p.status, MXG_DEV_SUM_OVER_CAPACITY);
        }
      }
    }
    start += size[i];
  }
  __syncthreads();

  if (c == static_cast<int>(gridDim.x) - 1 && (p.loss != nullptr || p.slope != nullptr)) {
    float* part_p = reinterpret_cast<float*>(sh.buf);
    int n = 0;
    for (int h = tid; h < p.chunks; h += kRouteThreads) n += live[h];
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (p.loss != nullptr) {
      for (int i = tid; i < parts * wide; i += kRouteThreads) {
        const int e = i & (wide - 1), part = i / wide;
        float v = 0.0f;
        if (e < E)
#pragma unroll 8
          for (int h = part; h < p.chunks; h += parts) v += psum[static_cast<int64_t>(h) * E + e];
        part_p[i] = v;
      }
    }
    if (lane == 0) sh.warp_sum[warp] = static_cast<uint32_t>(n);
    __syncthreads();
    uint32_t tokens = 0;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) tokens += sh.warp_sum[w];
    // all and tokens are 0 together
    const float unit = all == 0 ? 0.0f
                                : p.balance * static_cast<float>(E) / static_cast<float>(tokens);
    float mine = 0.0f;
    for (int e = tid; e < E; e += kRouteThreads) {
      const float s = all == 0 ? 0.0f
                               : unit * (static_cast<float>(sh.total[e]) / static_cast<float>(all));
      if (p.slope != nullptr) p.slope[e] = s;
      if (p.loss != nullptr) {
        float v = 0.0f;
        for (int part = 0; part < parts; ++part) v += part_p[part * wide + e];
        mine += s * v;
      }
    }
    if (p.loss != nullptr) {
      mine = team_add<32>(mine);
      if (lane == 0) sh.warp_f[warp] = mine;
      __syncthreads();
      if (tid == 0) {
        float v = 0.0f;
        for (int w = 0; w < kRouteWarps; ++w) v += sh.warp_f[w];
        *p.loss = v;
      }
    }
    __syncthreads();
  }
  if (p.row_of == nullptr) return;

  // rows: as many warps as the counts have room for, each a run of the chunk's choices
  const int warps = min(kRouteWarps, kBufWords / wide);
  uint32_t* mine = sh.buf + warp * E;
  const int64_t begin = static_cast<int64_t>(c) * p.per;
  const int64_t end = min(begin + p.per, p.tokens);
  const int32_t items = begin < end ? static_cast<int32_t>((end - begin) * p.k) : 0;
  const int32_t run = ((items + warps - 1) / warps + 31) / 32 * 32;
  const int32_t* expert = p.expert + begin * p.k;
  int32_t* row_of = p.row_of + begin * p.k;
  const int32_t from = min(warp * run, items), to = warp < warps ? min(from + run, items) : from;
  for (int i = tid; i < warps * E; i += kRouteThreads) sh.buf[i] = 0;
  __syncthreads();
  for (int i = from + lane; i < to; i += 32) {
    const int32_t e = expert[i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&mine[e], 1u);
  }
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads) {
    uint32_t at = sh.start[e] + sh.before[e];
    for (int w = 0; w < warps; ++w) {
      const uint32_t n = sh.buf[w * E + e];
      sh.buf[w * E + e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int base = from; base < to; base += 32) {
    const int i = base + lane;
    int32_t e = i < to ? expert[i] : -1;
    if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E)) e = -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const uint32_t rank = __popc(same & ((1u << lane) - 1u));
    uint32_t row = 0;
    if (e >= 0) row = mine[e] + rank;
    __syncwarp();
    if (e >= 0 && rank == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i < to) row_of[i] = e >= 0 && row < p.capacity ? static_cast<int32_t>(row) : -1;
  }
}

__global__ void __launch_bounds__(kRouteThreads)
    route_finish_kernel(const RowPlan p, const RouteWs ws) {
  __shared__ RouteShared sh;
  grid_wait_for_previous();
  finish_chunk(p, sh, ws.hist, ws.psum, ws.live, blockIdx.x);
}

// Tokens per expert of a chunk, for experts chosen elsewhere.
template <bool ONE>
__global__ void __launch_bounds__(kRouteThreads)
    route_count_kernel(const RowPlan p, const RouteWs ws) {
  __shared__ RouteShared sh;
  const int tid = threadIdx.x, c = blockIdx.x, E = p.experts;
  if (!ONE) grid_launch_dependents();
  for (int e = tid; e < E; e += kRouteThreads) sh.hist[e] = 0;
  __syncthreads();
  const int64_t begin = c * p.per, end = min(begin + p.per, p.tokens);
  const int32_t items = begin < end ? static_cast<int32_t>((end - begin) * p.k) : 0;
  for (int i = tid; i < items; i += kRouteThreads) {
    const int32_t e = p.expert[begin * p.k + i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&sh.hist[e], 1);
  }
  __syncthreads();
  if (ONE) {
    finish_chunk(p, sh, sh.hist, nullptr, nullptr, 0);
  } else {
    for (int e = tid; e < E; e += kRouteThreads) ws.hist[static_cast<int64_t>(c) * E + e] = sh.hist[e];
  }
}

// ---------------------------------------------------------------- the choice
template <typename T, int LPT, int VPL, bool ONE>
__global__ void __launch_bounds__(kRouteThreads)
    route_kernel(const mxg_route_t d, const RowPlan p, const RouteWs ws, int vec) {
  __shared__ RouteShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int gl = lane & (LPT - 1), c0 = gl * VPL, E = d.experts, k = d.k;
  constexpr int kTeams = kRouteThreads / LPT;
  if (!ONE) grid_launch_dependents();
  for (int e = tid; e < E; e += kRouteThreads) sh.hist[e] = 0;
  if (tid == 0) sh.live = 0;
  __syncthreads();

  const int64_t begin = c * p.per, end = min(begin + p.per, d.tokens);
  const T* logits = static_cast<const T*>(d.logits);
  const bool softmax = d.score == MXG_SCORE_SOFTMAX;
  const bool shares = d.loss != nullptr, whole = shares || (softmax && !d.normalize);
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int live = 0;
  int64_t t = begin + tid / LPT;
  LogitRow<T, VPL> next;
  bool next_on = false;
  auto fetch = [&](int64_t at) {
    next_on = at < end && (d.mask == nullptr || d.mask[at] != 0);
    if (at < end) next.load(logits + at * d.ld, c0, E, vec != 0);
  };
  fetch(t);
  for (int64_t base = begin; base < end; base += kTeams, t += kTeams) {
    float v[VPL];
    next.values(v);
    const bool on = next_on;
    fetch(t + kTeams);
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = on && c0 + i < E ? logit_key(v[i]) : 0u;
    // the k best: lane j of the team keeps the j-th
    uint32_t my_key = 0, top = 0;
    int my_e = -1;
    for (int j = 0; j < k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
      const uint32_t m = team_max<LPT>(best);
      if (j == 0) top = m;
      int slot = 0;
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == m) slot = i;
      const uint32_t holds = __ballot_sync(0xFFFFFFFFu, best == m) >> (lane & ~(LPT - 1));
      const int who = __ffs(holds) - 1;  // the team's lowest lane of them
      const int e = __shfl_sync(0xFFFFFFFFu, c0 + slot, who, LPT);
      if (gl == who)
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (i == slot) key[i] = 0u;
      if (gl == j && m > kNoLogit) {
        my_e = e;
        my_key = m;
      }
    }
    const bool taken = top > kNoLogit;
    const float best = key_logit(top), mine = key_logit(my_key);
    const float shift = softmax ? best : fminf(best, 0.0f);
    float sum = 0.0f, s[VPL];
    if (whole) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = softmax ? __expf(v[i] - shift) : sigmoid_scaled(v[i], shift);
        sum += s[i];
      }
      sum = team_add<LPT>(sum);
    }
    float w = 0.0f;
    if (my_e >= 0) {
      if (softmax)
        w = __expf(mine - shift);
      else
        w = sigmoid_scaled(mine, d.normalize ? shift : 0.0f);
    }
    const float chosen = d.normalize ? team_add<LPT>(w) : (softmax ? sum : 1.0f);
    if (t < end && gl < k) {
      d.expert[t * k + gl] = my_e;
      d.weight[t * k + gl] = my_e >= 0 ? d.scale * (w / chosen) : 0.0f;
    }
    if (my_e >= 0) atomicAdd(&sh.hist[my_e], 1);
    if (taken) {
      if (gl == 0) ++live;
      if (shares) {
        const float r = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = fmaf(s[i], r, acc[i]);
      }
    }
  }

  // the chunk's sums, in a fixed order: teams of a warp, then warps
  live = __reduce_add_sync(0xFFFFFFFFu, live);
  if (lane == 0 && live != 0) atomicAdd(&sh.live, live);
  if (shares) {
    float* rows = reinterpret_cast<float*>(sh.buf);
    int wide = 1;
    while (wide < E) wide *= 2;
    const int fit = min(kRouteWarps, kBufWords / wide);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    for (int w0 = 0; w0 < kRouteWarps; w0 += fit) {
      if (warp >= w0 && warp < w0 + fit && lane < LPT) {
        float* row = rows + (warp - w0) * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (c0 + i < E) row[c0 + i] = w0 == 0 ? acc[i] : row[c0 + i] + acc[i];
      }
      __syncthreads();
    }
    for (int e = tid; e < E; e += kRouteThreads) {
      float v = 0.0f;
      for (int w = 0; w < fit; ++w) v += rows[w * E + e];
      sh.psum[e] = v;
    }
  }
  __syncthreads();
  if (ONE) {
    finish_chunk(p, sh, sh.hist, sh.psum, &sh.live, 0);
  } else {
    for (int e = tid; e < E; e += kRouteThreads) {
      ws.hist[static_cast<int64_t>(c) * E + e] = sh.hist[e];
      if (shares) ws.psum[static_cast<int64_t>(c) * E + e] = sh.psum[e];
    }
    if (tid == 0) ws.live[c] = sh.live;
  }
}

// ---------------------------------------------------------------- the gradient
// With a the gradient of the shares p (slope * dloss) and b that of the chosen scores
// (scale * dweight), all sums over a token:
//   softmax : dl = p (a - sum a p) + extra;  extra of a chosen expert, normalised: q (b - sum b q)
//             with q = s / sum of the chosen s, else p b, with sum b p joining sum a p
//   sigmoid : dl = p (1 - s) (a - sum a p) + extra;  normalised: q (1 - s) (b - sum b q), else
//             b s (1 - s)
constexpr int kGradThreads = 256;

template <typename T, int LPT, int VPL>
__global__ void __launch_bounds__(kGradThreads)
    route_backward_kernel(const mxg_route_grad_t d, int vec) {
  extern __shared__ float team_rows[];  // a row of LPT * VPL columns a team
  const int tid = threadIdx.x, lane = tid & 31;
  const int gl = lane & (LPT - 1), c0 = gl * VPL, E = d.experts, k = d.k;
  constexpr int kTeams = kGradThreads / LPT;
  float* mine = team_rows + tid / LPT * (LPT * VPL);
  const bool softmax = d.score == MXG_SCORE_SOFTMAX, balance = d.slope != nullptr;
  const bool joined = softmax && !d.normalize;  // the weights' gradient goes through the shares
  float a[VPL];
  const float dloss = balance ? *d.dloss : 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) a[i] = balance && c0 + i < E ? d.slope[c0 + i] * dloss : 0.0f;
  const T* logits = static_cast<const T*>(d.logits);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTeams; base < d.tokens; base += step) {
    const int64_t t = base + tid / LPT;
    const bool in = t < d.tokens;
    const T* row = logits + (in ? t : 0) * d.ld;
    LogitRow<T, VPL> raw;
    float v[VPL];
    raw.load(row, c0, in ? E : 0, vec != 0);
    raw.values(v);
    int e = -1;
    float b = 0.0f, l = -INFINITY;
    if (in && gl < k) e = d.expert[t * k + gl];
    if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E)) e = -1;
    if (e >= 0) {
      l = to_f32(row[e]);
      if (d.dweight != nullptr) b = d.scale * d.dweight[t * k + gl];
    }
    const uint32_t any = __ballot_sync(0xFFFFFFFFu, e >= 0) >> (lane & ~(LPT - 1));
    const bool taken = (LPT == 32 ? any : any & ((1u << (LPT & 31)) - 1u)) != 0;

    float top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float shift = softmax ? top : fminf(top, 0.0f);
    // the shares and their part of the sums
    float p[VPL], rest[VPL], sum = 0.0f, dot = 0.0f;
    if (balance || joined) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = softmax ? __expf(v[i] - shift) : sigmoid_scaled(v[i], shift);
        // 1 - s, without its cancellation
        rest[i] = softmax ? 1.0f : sigmoid_scaled(-v[i], 0.0f);
        sum += p[i];
        dot = fmaf(a[i], p[i], dot);
      }
      sum = team_add<LPT>(sum);
    }
    // the chosen experts'
    float s = 0.0f, extra = 0.0f;
    const float other = softmax ? 1.0f : sigmoid_scaled(-l, 0.0f);
    if (e >= 0) s = softmax ? __expf(l - shift) : sigmoid_scaled(l, d.normalize ? shift : 0.0f);
    if (d.normalize) {
      const float chosen = team_add<LPT>(s);
      const float q = e >= 0 ? s / chosen : 0.0f;
      const float bq = team_add<LPT>(b * q);
      extra = q * other * (b - bq);
    } else if (softmax) {
      extra = b * s / sum;
      dot = fmaf(b, s, dot);
    } else {
      extra = b * s * other;
    }
    float r = 0.0f;
    if (balance || joined) {
      dot = team_add<LPT>(dot);
      r = 1.0f / sum;
      dot *= r;
    }
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      *reinterpret_cast<float4*>(mine + c0 + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    if (e >= 0) atomicAdd(&mine[e], extra);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(mine + c0 + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
    if (balance || joined)
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = fmaf(p[i] * r * rest[i], a[i] - dot, v[i]);
    if (in) {
      T* out = static_cast<T*>(d.dlogits) + t * d.ldd;
#pragma unroll
      for (int i = 0; i < VPL; i += 8) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = taken ? v[i + j] : 0.0f;
        if (vec && c0 + i < E) {
          if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(out + c0 + i)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(out + c0 + i)[1] = make_float4(f[4], f[5], f[6], f[7]);
          } else {
            *reinterpret_cast<uint4*>(out + c0 + i) =
                make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                           pack2<T>(f[6], f[7]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + i + j < E) out[c0 + i + j] = from_f32<T>(f[j]);
        }
      }
    }
    __syncwarp();
  }
}

namespace {

// Lanes a token: 8 columns each, and one for each of the k chosen.
int lanes_per_token(int experts, int k) {
  int lanes = 1;
  while (lanes < 32 && (lanes * 8 < experts || lanes < k)) lanes *= 2;
  return lanes;
}

struct Chunks {
  int n;
  int64_t per;  // tokens each
};

// At least a pass of a CTA's teams a chunk.
Chunks chunks_of(int64_t tokens, int experts, int k) {
  const int64_t pass = kRouteThreads / lanes_per_token(experts, k);
  const int64_t n = std::max<int64_t>(1, std::min<int64_t>(kMaxChunks, (tokens + pass - 1) / pass));
  Chunks c;
  c.per = std::max<int64_t>(1, (tokens + n - 1) / n);
  c.n = static_cast<int>(std::max<int64_t>(1, (tokens + c.per - 1) / c.per));
  return c;
}

RouteWs carve(void* ws, int chunks, int experts) {
  RouteWs w;
  w.hist = static_cast<int32_t*>(ws);
  w.psum = reinterpret_cast<float*>(w.hist + static_cast<int64_t>(chunks) * experts);
  w.live = reinterpret_cast<int32_t*>(w.psum + static_cast<int64_t>(chunks) * experts);
  return w;
}

bool rows_of_16(const void* p, int64_t ld, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * static_cast<int64_t>(size)) % 16 == 0;
}

cudaError_t launch_finish(const RowPlan& p, const RouteWs& ws, cudaStream_t stream, int* launches) {
  ++*launches;
  return launch_after(true, route_finish_kernel,
                      static_cast<unsigned>(p.row_of != nullptr ? p.chunks : 1), kRouteThreads, 0,
                      stream, p, ws);
}

template <typename T, int LPT, int VPL>
cudaError_t run_route(const mxg_route_t& d, const RowPlan& p, const RouteWs& ws, int vec,
                      cudaStream_t stream) {
  if (p.chunks == 1)
    route_kernel<T, LPT, VPL, true><<<1, kRouteThreads, 0, stream>>>(d, p, ws, vec);
  else
    route_kernel<T, LPT, VPL, false>
        <<<static_cast<unsigned>(p.chunks), kRouteThreads, 0, stream>>>(d, p, ws, vec);
  return cudaGetLastError();
}

template <typename T, int LPT, int VPL>
cudaError_t run_backward(const mxg_route_grad_t& d, int vec, int num_sms, cudaStream_t stream) {
  constexpr int kTeams = kGradThreads / LPT;
  const int64_t grid = std::min<int64_t>((d.tokens + kTeams - 1) / kTeams, num_sms * 8LL);
  const size_t smem = static_cast<size_t>(kGradThreads) * VPL * sizeof(float);
  route_backward_kernel<T, LPT, VPL>
      <<<static_cast<unsigned>(grid), kGradThreads, smem, stream>>>(d, vec);
  return cudaGetLastError();
}

// fn<T, LPT, VPL>() for a type, and the lanes and columns a lane that experts and k take.
#define MXG_BY_LANES(T, CALL)                     \
  switch (lanes_per_token(d.experts, d.k)) {      \
    case 1: return CALL(T, 1, 8);                 \
    case 2: return CALL(T, 2, 8);                 \
    case 4: return CALL(T, 4, 8);                 \
    case 8: return CALL(T, 8, 8);                 \
    case 16: return CALL(T, 16, 8);               \
  }                                               \
  if (d.experts <= 256) return CALL(T, 32, 8);    \
  if (d.experts <= 512) return CALL(T, 32, 16);   \
  return CALL(T, 32, 32);

template <typename T>
cudaError_t route_typed(const mxg_route_t& d, const RowPlan& p, const RouteWs& ws,
                        cudaStream_t stream) {
  const int vec = d.experts % 8 == 0 && rows_of_16(d.logits, d.ld, sizeof(T));
#define MXG_CALL(T, L, V) (run_route<T, L, V>(d, p, ws, vec, stream))
  MXG_BY_LANES(T, MXG_CALL)
#undef MXG_CALL
}

template <typename T>
cudaError_t backward_typed(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream) {
  const int vec = d.experts % 8 == 0 && rows_of_16(d.logits, d.ld, sizeof(T)) &&
                  rows_of_16(d.dlogits, d.ldd, sizeof(T));
#define MXG_CALL(T, L, V) (run_backward<T, L, V>(d, vec, num_sms, stream))
  MXG_BY_LANES(T, MXG_CALL)
#undef MXG_CALL
}
#undef MXG_BY_LANES

}  // namespace

size_t route_ws_bytes(int64_t tokens, int experts, int k) {
  const int64_t n = chunks_of(tokens, experts, k).n;
  return static_cast<size_t>((n * (2 * experts + 1) * 4 + 15) / 16 * 16);
}

cudaError_t launch_route(const mxg_route_t& d, void* workspace, int32_t* status,
                         cudaStream_t stream, int* launches) {
  const Chunks c = chunks_of(d.tokens, d.experts, d.k);
  RowPlan p = {};
  p.expert = d.expert;
  p.counts = d.counts;
  p.loss = d.loss;
  p.slope = d.slope;
  p.row_of = d.row_of;
  p.group_ws = d.group_ws;
  p.status = status;
  p.tokens = d.tokens;
  p.per = c.per;
  p.last_dim = d.last_dim;
  p.capacity = static_cast<uint32_t>(d.rows_capacity / d.align * d.align);
  p.experts = d.experts;
  p.k = d.k;
  p.align = d.align;
  p.chunks = c.n;
  p.balance = d.balance;
  const RouteWs ws = carve(workspace, c.n, d.experts);
  const cudaError_t e = d.dtype == MXG_F32    ? route_typed<float>(d, p, ws, stream)
                        : d.dtype == MXG_BF16 ? route_typed<Bf16>(d, p, ws, stream)
                                              : route_typed<F16>(d, p, ws, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  return c.n == 1 ? cudaSuccess : launch_finish(p, ws, stream, launches);
}

cudaError_t launch_route_rows(const int32_t* expert, int64_t tokens, int experts, int k, int align,
                              int64_t capacity, int64_t last_dim, int32_t* counts, int32_t* row_of,
                              int64_t* group_ws, void* workspace, int32_t* status,
                              cudaStream_t stream, int* launches) {
  const Chunks c = chunks_of(tokens, experts, k);
  RowPlan p = {};
  p.expert = expert;
  p.counts = counts;
  p.row_of = row_of;
  p.group_ws = group_ws;
  p.status = status;
  p.tokens = tokens;
  p.per = c.per;
  p.last_dim = last_dim;
  p.capacity = static_cast<uint32_t>(capacity / align * align);
  p.experts = experts;
  p.k = k;
  p.align = align;
  p.chunks = c.n;
  const RouteWs ws = carve(workspace, c.n, experts);
  ++*launches;
  if (c.n == 1) {
    route_count_kernel<true><<<1, kRouteThreads, 0, stream>>>(p, ws);
    return cudaGetLastError();
  }
  route_count_kernel<false><<<static_cast<unsigned>(c.n), kRouteThreads, 0, stream>>>(p, ws);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_finish(p, ws, stream, launches);
}

cudaError_t launch_route_backward(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream) {
  if (d.dtype == MXG_F32) return backward_typed<float>(d, num_sms, stream);
  if (d.dtype == MXG_BF16) return backward_typed<Bf16>(d, num_sms, stream);
  return backward_typed<F16>(d, num_sms, stream);
}

}  // namespace mxg
