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

constexpr int kMaxExperts = 1024;
constexpr int kMaxChunks = 152;
constexpr uint32_t kNoLogit = 0x007FFFFFu;  // the key of -infinity: it and all below are not chosen
constexpr int kOneItems = 4096;  // choices of a batch that one CTA finishes

// Threads of a CTA: of the kernels that work on a whole batch alone, and of the others.  With
// 16 or 32 columns a lane the choice needs the registers of two or four.
constexpr int kOneThreads = 512;
constexpr int kManyThreads = 1024;
constexpr int threads_of(int vpl, bool one) {
  const int most = vpl > 16 ? 256 : (vpl > 8 ? 512 : 1024);
  return one && most > kOneThreads ? kOneThreads : most;
}

// The workspace: chunk by chunk, tokens per expert, sums of p, tokens that take part.  A
// chunk's experts are padded to a multiple of 4, to be read 16 bytes at a time.
struct RouteWs {
  int32_t* hist;  // [chunks][pitch]
  float* psum;    // [chunks][pitch]
  int32_t* live;  // [chunks]
  int32_t pitch;
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

constexpr int kBufWords = 8192;

// BUF: words for sums by part or by warp, and for tokens per expert by warp.
template <int BUF>
struct RouteShared {
  uint4 buf[BUF / 4];
  int32_t hist[kMaxExperts];
  float psum[kMaxExperts];
  uint32_t start[kMaxExperts];
  uint32_t warp_sum[32], warp_total[32];
  float warp_f[32];
  int32_t live;
};

// Logits as unsigned integers of the same order: -0 as 0, NaN above all (an addition
// gives the NaN of positive sign).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// sigmoid(l), and sigmoid(l) e^-m with m < 0: shares of a token whose sigmoids all underflow
// are still right (m the largest logit where that is negative, so l <= m).
__device__ __forceinline__ float sigmoid(float l) {
  const float e = exp_approx(-fabsf(l));
  return (l < 0.0f ? e : 1.0f) * rcp_approx(1.0f + e);
}
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
  return m < 0.0f ? exp_approx(l - m) * rcp_approx(1.0f + exp_approx(l)) : sigmoid(l);
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
// Sums over the chunks of `n` columns, `pitch` apart from one chunk to the next, into
// parts of shared memory: part p, column c at [p * 4 * quads + c].  LOW: beside the sums, those
// of the chunks below `low`, `kBufWords / 2` further on.  The parts are returned.
template <int NT, bool LOW, typename V4, typename V>
__device__ __forceinline__ int sum_chunks(V* to, const V* from, int pitch, int chunks, int low) {
  const int quads = pitch / 4;
  int wide = 1;
  while (wide < quads) wide *= 2;
  const int parts = min(min(NT / wide, 16), chunks);
  const int q = threadIdx.x & (wide - 1), part = threadIdx.x / wide;
  if (q < quads && part < parts) {
    V4 all = {}, under = {};
    const V4* at = reinterpret_cast<const V4*>(from) + q;
    // ten loads at once: all of a part's where there are 16 parts
    for (int h0 = part; h0 < chunks; h0 += 10 * parts) {
      V4 v[10];
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        v[i] = V4{};
        if (h0 + i * parts < chunks) v[i] = at[(h0 + i * parts) * quads];
      }
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        all.x += v[i].x;
        all.y += v[i].y;
        all.z += v[i].z;
        all.w += v[i].w;
        if (LOW && h0 + i * parts < low) {
          under.x += v[i].x;
          under.y += v[i].y;
          under.z += v[i].z;
          under.w += v[i].w;
        }
      }
    }
    V4* out = reinterpret_cast<V4*>(to) + part * quads + q;
    out[0] = all;
    if (LOW) out[kBufWords / 8] = under;
  }
  return parts;
}

// Everything that needs the whole batch's counts, by the CTA of chunk c, of NT threads
// (at least as many as experts, but for ONE).  ONE: this CTA has all tokens, whose counts and
// sums are in `sh`.  The first CTA writes counts and group_ws; the last one, which has no
// tokens where there are several, slope and loss.
template <int NT, bool ONE, int BUF>
__device__ __forceinline__ void finish_chunk(const RowPlan& p, RouteShared<BUF>& sh,
                                             const RouteWs& ws, const int32_t* expert, int c) {
  static_assert(ONE || BUF == kBufWords, "sums of chunks take two halves of a whole buffer");
  constexpr int kPer = (kMaxExperts + NT - 1) / NT;  // experts a thread
  constexpr int kWarps = NT / 32;
  const int tid = threadIdx.x, E = p.experts;
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t* buf = reinterpret_cast<uint32_t*>(sh.buf);
  // this chunk's choices: as many warps as the counts have room for, each a run of them, of which
  // the first kHeld of a lane are asked for now
  constexpr int kHeld = 4;
  const int64_t begin = static_cast<int64_t>(c) * p.per;
  const int64_t end = min(begin + p.per, p.tokens);
  const int32_t items =
      begin < end && p.row_of != nullptr ? static_cast<int32_t>((end - begin) * p.k) : 0;
  const int warps = min(min(kWarps, BUF / E), (items + 31) / 32);
  const int32_t run = warps == 0 ? 0 : ((items + warps - 1) / warps + 31) / 32 * 32;
  const int32_t from = min(warp * run, items), to = warp < warps ? min(from + run, items) : from;
  auto choice = [&](int i) {
    const int32_t e = i < to ? expert[i] : -1;
    return static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;
  };
  int32_t held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = choice(from + 32 * i + lane);
  // tokens of each expert, in all chunks and in those before this one
  int parts = 1;
  if (!ONE) {
    parts = sum_chunks<NT, true, uint4>(buf, reinterpret_cast<const uint32_t*>(ws.hist), ws.pitch,
                                        p.chunks, c);
    __syncthreads();
  }
  // starts of the padded groups: a scan over a thread's experts, the warp and the CTA
  uint32_t size[kPer], total[kPer], before[kPer], incl = 0, sum = 0;
  const uint32_t a = static_cast<uint32_t>(p.align);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * tid + i;
    total[i] = before[i] = 0;
    if (e < E) {
      if (ONE) {
        total[i] = static_cast<uint32_t>(sh.hist[e]);
      } else {
#pragma unroll
        for (int part = 0; part < 16; ++part) {
          if (part >= parts) break;
          total[i] += buf[part * ws.pitch + e];
          before[i] += buf[kBufWords / 2 + part * ws.pitch + e];
        }
      }
    }
    size[i] = a == 1 ? total[i] : (total[i] + a - 1) / a * a;
    incl += size[i];
    sum += total[i];
  }
  const uint32_t mine_size = incl;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  sum = __reduce_add_sync(0xFFFFFFFFu, sum);
  if (lane == 31) {
    sh.warp_sum[warp] = incl;
    sh.warp_total[warp] = sum;
  }
  __syncthreads();
  const uint32_t w_size = lane < kWarps ? sh.warp_sum[lane] : 0u;
  const uint32_t ahead = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w_size : 0u);
  const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.warp_total[lane] : 0u);
  uint32_t start = ahead + incl - mine_size;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * tid + i;
    if (e < E) {
      sh.start[e] = start + before[i];  // of this chunk's tokens
      if (!ONE) sh.hist[e] = static_cast<int32_t>(total[i]);
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
    int tokens = 0, p_parts = 1;
    if (ONE) {
      tokens = sh.live;
    } else {
      for (int h = lane; h < p.chunks; h += 32) tokens += ws.live[h];
      tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
      if (p.loss != nullptr)
        p_parts = sum_chunks<NT, false, float4>(part_p, ws.psum, ws.pitch, p.chunks, 0);
      __syncthreads();
    }
    // all and tokens are 0 together
    const float unit =
        all == 0 ? 0.0f : p.balance * static_cast<float>(E) / static_cast<float>(tokens);
    float mine = 0.0f;
    for (int e = tid; e < E; e += NT) {
      const float s =
          all == 0 ? 0.0f : unit * (static_cast<float>(sh.hist[e]) / static_cast<float>(all));
      if (p.slope != nullptr) p.slope[e] = s;
      if (p.loss != nullptr) {
        float v = 0.0f;
        if (ONE) {
          v = sh.psum[e];
        } else {
          for (int part = 0; part < p_parts; ++part) v += part_p[part * ws.pitch + e];
        }
        mine += s * v;
      }
    }
    if (p.loss != nullptr) {
      mine = team_add<32>(mine);
      if (lane == 0) sh.warp_f[warp] = mine;
      __syncthreads();
      if (warp == 0) {
        const float v = team_add<32>(lane < kWarps ? sh.warp_f[lane] : 0.0f);
        if (lane == 0) *p.loss = v;
      }
    }
  }

  if (items == 0) return;
  // A choice's place among its expert's: those of earlier lanes, of earlier rounds of the
  // warp (both now), then of earlier warps, chunks and experts.
  uint32_t* mine = buf + warp * E;
  int32_t* row_of = p.row_of + begin * p.k;
  if (warp < warps)
    for (int i = lane; i < E; i += 32) mine[i] = 0;
  __syncwarp();
  auto place = [&](int32_t e) {
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const uint32_t rank = __popc(same & ((1u << lane) - 1u));
    uint32_t at = rank;
    if (e >= 0) at += mine[e];
    __syncwarp();
    if (e >= 0 && rank == 0) mine[e] += __popc(same);
    __syncwarp();
    return at;
  };
  uint32_t at[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    at[i] = 0;
    if (from + 32 * i < to) at[i] = place(held[i]);
  }
  for (int base = from + 32 * kHeld; base < to; base += 32) place(choice(base + lane));
  __syncthreads();
  for (int e = tid; e < E; e += NT) {
    uint32_t first = sh.start[e];
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const uint32_t n = buf[w * E + e];
      buf[w * E + e] = first;
      first += n;
    }
  }
  __syncthreads();
  auto write = [&](int i, int32_t e, uint32_t row) {
    if (i < to) row_of[i] = e >= 0 && row < p.capacity ? static_cast<int32_t>(row) : -1;
  };
  const bool more = to - from > 32 * kHeld;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (from + 32 * i < to)
      write(from + 32 * i + lane, held[i], held[i] >= 0 ? mine[held[i]] + at[i] : 0u);
  if (!more) return;
  // the others' places are found again, after those of the held ones
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kHeld; ++i) place(held[i]);
  for (int base = from + 32 * kHeld; base < to; base += 32) {
    const int32_t e = choice(base + lane);
    write(base + lane, e, place(e));
  }
}

__global__ void __launch_bounds__(kManyThreads)
    route_finish_kernel(const RowPlan p, const RouteWs ws) {
  __shared__ RouteShared<kBufWords> sh;
  grid_wait_for_previous();
  const int c = static_cast<int>(blockIdx.x);
  finish_chunk<kManyThreads, false>(p, sh, ws, p.expert + c * p.per * p.k, c);
}

// Tokens per expert of a chunk, for experts chosen elsewhere.
template <int NT, bool ONE>
__global__ void __launch_bounds__(NT) route_count_kernel(const RowPlan p, const RouteWs ws) {
  __shared__ RouteShared<ONE ? kBufWords / 2 : kBufWords> sh;
  const int tid = threadIdx.x, c = blockIdx.x, E = p.experts;
  if (!ONE) grid_launch_dependents();
  for (int e = tid; e < E; e += NT) sh.hist[e] = 0;
  __syncthreads();
  const int64_t begin = c * p.per, end = min(begin + p.per, p.tokens);
  const int32_t items = begin < end ? static_cast<int32_t>((end - begin) * p.k) : 0;
  const int32_t* expert = p.expert + begin * p.k;
  for (int i = tid; i < items; i += NT) {
    const int32_t e = expert[i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&sh.hist[e], 1);
  }
  __syncthreads();
  if (ONE) {
    finish_chunk<NT, true>(p, sh, ws, expert, 0);
  } else {
    for (int e = tid; e < ws.pitch; e += NT)
      ws.hist[static_cast<int64_t>(c) * ws.pitch + e] = e < E ? sh.hist[e] : 0;
  }
}

// ---------------------------------------------------------------- the choice
// A team's k best keys: lane j keeps the j-th, with its column.
struct Chosen {
  uint32_t key;  // 0 where there is none
  int expert;    // -1 there
};

// One after the other: the maximum over the team, and the lowest lane that holds it.  The keys
// are used up.
template <int LPT, int VPL>
__device__ __forceinline__ Chosen choose_in_turn(uint32_t (&key)[VPL], int k, int gl) {
  const int lane = threadIdx.x & 31, c0 = gl * VPL;
  Chosen r = {0u, -1};
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    const uint32_t m = team_max<LPT>(best);
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
      r.expert = e;
      r.key = m;
    }
  }
  return r;
}

// By counting, among the few keys that can be of the best.  The lanes form `groups` groups, at
// least k of them, so none below the least of the groups' maxima is chosen (above 8, where that
// leaves too many, none below the k-th largest of the lanes' maxima).  The others -- for 8 of
// 64 some 15, for 8 of 256 some 17 -- are laid out in shared memory in the order of their
// columns, and the lanes count those above each.  Where there are more than kMost, one after
// the other after all.  `slots` has room for the warp's teams.
constexpr int kMost = 31;  // (a stride that keeps the teams' slots on different banks)

template <int LPT, int VPL>
__device__ __forceinline__ Chosen choose_by_rank(uint32_t (&key)[VPL], int k, int gl, int groups,
                                                 uint2* slots) {
  constexpr int kRounds = (kMost + LPT - 1) / LPT;
  const int lane = threadIdx.x & 31;
  uint32_t bound = key[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) bound = max(bound, key[i]);
  if (LPT == 32 && k > 8) {
    uint32_t best = bound;
    bound = __reduce_max_sync(0xFFFFFFFFu, best);
    for (int j = 1; j < k; ++j) {
      if (best == bound) best = 0u;  // all alike at once: the bound is only lower for it
      bound = __reduce_max_sync(0xFFFFFFFFu, best);
    }
  } else {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) {
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, bound, d);
      bound = d >= groups ? max(bound, other) : min(bound, other);
    }
  }
  bound = max(bound, kNoLogit + 1u);
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) n += key[i] >= bound ? 1 : 0;
  int at = n;
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, at, d, LPT);
    if (gl >= d) at += v;
  }
  const int all = __shfl_sync(0xFFFFFFFFu, at, LPT - 1, LPT);
  const int most = __reduce_max_sync(0xFFFFFFFFu, all);
  if (most > kMost) return choose_in_turn<LPT, VPL>(key, k, gl);
  uint2* team = slots + lane / LPT * kMost;
  uint2* to = team + (at - n);
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (key[i] >= bound) *to++ = make_uint2(key[i], static_cast<uint32_t>(gl * VPL + i));
  __syncwarp();
  uint2 mine[kRounds];
  int above[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    mine[r] = make_uint2(0xFFFFFFFFu, 0u);
    if (r * LPT + gl < all) mine[r] = team[r * LPT + gl];
    above[r] = 0;
  }
#pragma unroll 4
  for (int j = 0; j < most; ++j) {
    const uint32_t other = j < all ? team[j].x : 0u;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) above[r] += other > mine[r].x ? 1 : 0;
  }
  // without equal keys the counts are 0, 1, 2, ...
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) sum += above[r];
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (__any_sync(0xFFFFFFFFu, 2 * sum != all * (all - 1))) {
    for (int j = 0; j < all; ++j)
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        above[r] += team[j].x == mine[r].x && j < r * LPT + gl ? 1 : 0;
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (r * LPT + gl < all && above[r] < k) team[above[r]] = mine[r];
  __syncwarp();
  Chosen c = {0u, -1};
  if (gl < min(all, k)) {
    const uint2 v = team[gl];
    c.key = v.x;
    c.expert = static_cast<int>(v.y);
  }
  __syncwarp();  // the slots are written again for the next token
  return c;
}

template <typename T, int LPT, int VPL, int NT, bool ONE>
__global__ void __launch_bounds__(NT)
    route_kernel(const mxg_route_t d, const RowPlan p, const RouteWs ws, int vec) {
  constexpr int kTeams = NT / LPT, kWarps = NT / 32;
  constexpr int kBuf = ONE ? kBufWords / 2 : kBufWords;
  __shared__ RouteShared<kBuf> sh;
  __shared__ int32_t choices[ONE ? kOneItems : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int gl = lane & (LPT - 1), c0 = gl * VPL, E = d.experts, k = d.k;
  if (!ONE) grid_launch_dependents();
  for (int e = tid; e < E; e += NT) sh.hist[e] = 0;
  if (tid == 0) sh.live = 0;
  __syncthreads();

  const int64_t begin = c * p.per;
  const int count = static_cast<int>(max(min(begin + p.per, d.tokens) - begin, int64_t{0}));
  const T* row = static_cast<const T*>(d.logits) + (begin + tid / LPT) * d.ld;
  const uint8_t* mask = d.mask != nullptr ? d.mask + begin : nullptr;
  int32_t* const expert = d.expert + begin * k;
  float* const weight = d.weight + begin * k;
  const bool softmax = d.score == MXG_SCORE_SOFTMAX;
  const bool shares = d.loss != nullptr, whole = shares || (softmax && !d.normalize);
  int groups = 1;
  while (groups < k) groups *= 2;
  // a few are found sooner in turn; and groups without columns have no maximum
  const bool by_rank = LPT >= 8 && k > 3 && (LPT == 32 || k <= 8) && groups * VPL <= E;
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int live = 0;
  int t = tid / LPT;  // in the chunk
  LogitRow<T, VPL> next;
  bool next_on = false;
  auto fetch = [&](int at) {
    next_on = at < count && (mask == nullptr || mask[at] != 0);
    if (at < count) next.load(row, c0, E, vec != 0);
    row += kTeams * d.ld;
  };
  fetch(t);
  for (int base = 0; base < count; base += kTeams, t += kTeams) {
    float v[VPL];
    next.values(v);
    const bool on = next_on;
    fetch(t + kTeams);
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = on ? logit_key(v[i]) : 0u;
    Chosen best;
    if (LPT >= 8 && by_rank)
      best = choose_by_rank<LPT, VPL>(key, k, gl, groups, reinterpret_cast<uint2*>(sh.buf) +
                                                              warp * (kMost * 32 / LPT));
    else
      best = choose_in_turn<LPT, VPL>(key, k, gl);
    const float mine = key_logit(best.key);
    const float top = __shfl_sync(0xFFFFFFFFu, mine, 0, LPT);
    const bool taken = __shfl_sync(0xFFFFFFFFu, best.expert, 0, LPT) >= 0;
    const float shift = softmax ? top : fminf(top, 0.0f);
    float sum = 0.0f, s[VPL];
    if (whole) {
      if (softmax) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = exp_approx(v[i] - shift);
      } else if (shift < 0.0f) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = sigmoid_scaled(v[i], shift);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = sigmoid(v[i]);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += s[i];
      sum = team_add<LPT>(sum);
    }
    float w = 0.0f;
    if (best.expert >= 0)
      w = softmax ? exp_approx(mine - shift) : sigmoid_scaled(mine, d.normalize ? shift : 0.0f);
    const float chosen = d.normalize ? team_add<LPT>(w) : (softmax ? sum : 1.0f);
    if (t < count && gl < k) {
      expert[t * k + gl] = best.expert;
      weight[t * k + gl] = best.expert >= 0 ? d.scale * (w / chosen) : 0.0f;
      if (ONE) choices[t * k + gl] = best.expert;
    }
    if (best.expert >= 0) atomicAdd(&sh.hist[best.expert], 1);
    if (taken) {
      if (gl == 0) ++live;
      if (shares) {
        const float r = rcp_approx(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = fmaf(s[i], r, acc[i]);
      }
    }
  }

  // the chunk's sums, in a fixed order: teams of a warp, then warps
  live = __reduce_add_sync(0xFFFFFFFFu, live);
  if (lane == 0 && live != 0) atomicAdd(&sh.live, live);
  __syncthreads();  // the warps' slots give way to the sums
  if (shares) {
    float* rows = reinterpret_cast<float*>(sh.buf);
    const int fit = min(kWarps, kBuf / E);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    for (int w0 = 0; w0 < kWarps; w0 += fit) {
      if (warp >= w0 && warp < w0 + fit && lane < LPT) {
        float* row = rows + (warp - w0) * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (c0 + i < E) row[c0 + i] = w0 == 0 ? acc[i] : row[c0 + i] + acc[i];
      }
      __syncthreads();
    }
    for (int e = tid; e < E; e += NT) {
      float v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < fit; ++w) v += rows[w * E + e];
      if (ONE)
        sh.psum[e] = v;
      else
        ws.psum[static_cast<int64_t>(c) * ws.pitch + e] = v;
    }
  }
  if (ONE) {
    __syncthreads();
    finish_chunk<NT, true>(p, sh, ws, choices, 0);
  } else {
    for (int e = tid; e < ws.pitch; e += NT)
      ws.hist[static_cast<int64_t>(c) * ws.pitch + e] = e < E ? sh.hist[e] : 0;
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
        p[i] = softmax ? exp_approx(v[i] - shift) : sigmoid_scaled(v[i], shift);
        // 1 - s, without its cancellation
        rest[i] = softmax ? 1.0f : sigmoid(-v[i]);
        sum += p[i];
        dot = fmaf(a[i], p[i], dot);
      }
      sum = team_add<LPT>(sum);
    }
    // the chosen experts'
    float s = 0.0f, extra = 0.0f;
    const float other = softmax ? 1.0f : sigmoid(-l);
    if (e >= 0) s = softmax ? exp_approx(l - shift) : sigmoid_scaled(l, d.normalize ? shift : 0.0f);
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

// Columns a lane.
int columns_per_lane(int experts) { return experts > 512 ? 32 : (experts > 256 ? 16 : 8); }

struct Chunks {
  int n;
  int64_t per;  // tokens each
};

// One CTA up to four passes of its teams (a second kernel costs more than three of them),
// else a pass at least a CTA.
Chunks chunks_of(int64_t tokens, int experts, int k) {
  const int lanes = lanes_per_token(experts, k), vpl = columns_per_lane(experts);
  if (tokens <= 4 * (threads_of(vpl, true) / lanes) && tokens * k <= kOneItems)
    return {1, std::max<int64_t>(1, tokens)};
  const int64_t pass = threads_of(vpl, false) / lanes;
  const int64_t n = std::min<int64_t>(kMaxChunks, (tokens + pass - 1) / pass);
  Chunks c;
  c.per = (tokens + n - 1) / n;
  c.n = static_cast<int>(std::max<int64_t>(2, (tokens + c.per - 1) / c.per));
  return c;
}

int pitch_of(int experts) { return (experts + 3) / 4 * 4; }

RouteWs carve(void* ws, int chunks, int experts) {
  RouteWs w;
  w.pitch = pitch_of(experts);
  w.hist = static_cast<int32_t*>(ws);
  w.psum = reinterpret_cast<float*>(w.hist + static_cast<int64_t>(chunks) * w.pitch);
  w.live = reinterpret_cast<int32_t*>(w.psum + static_cast<int64_t>(chunks) * w.pitch);
  return w;
}

bool rows_of_16(const void* p, int64_t ld, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * static_cast<int64_t>(size)) % 16 == 0;
}

cudaError_t launch_finish(const RowPlan& p, const RouteWs& ws, cudaStream_t stream, int* launches) {
  ++*launches;
  return launch_after(true, route_finish_kernel,
                      static_cast<unsigned>(p.row_of != nullptr ? p.chunks + 1 : 1), kManyThreads,
                      0, stream, p, ws);
}

template <typename T, int LPT, int VPL>
cudaError_t run_route(const mxg_route_t& d, const RowPlan& p, const RouteWs& ws, int vec,
                      cudaStream_t stream) {
  constexpr int kThreads = threads_of(VPL, false), kOne = threads_of(VPL, true);
  if (p.chunks == 1)
    route_kernel<T, LPT, VPL, kOne, true><<<1, kOne, 0, stream>>>(d, p, ws, vec);
  else
    route_kernel<T, LPT, VPL, kThreads, false>
        <<<static_cast<unsigned>(p.chunks), kThreads, 0, stream>>>(d, p, ws, vec);
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
  if (columns_per_lane(d.experts) == 8) return CALL(T, 32, 8);   \
  if (columns_per_lane(d.experts) == 16) return CALL(T, 32, 16); \
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
  return n == 1 ? 16 : static_cast<size_t>((n * (2 * pitch_of(experts) + 1) * 4 + 15) / 16 * 16);
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
    route_count_kernel<kOneThreads, true><<<1, kOneThreads, 0, stream>>>(p, ws);
    return cudaGetLastError();
  }
  route_count_kernel<kManyThreads, false>
      <<<static_cast<unsigned>(c.n), kManyThreads, 0, stream>>>(p, ws);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_finish(p, ws, stream, launches);
}

cudaError_t launch_route_backward(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream) {
  if (d.dtype == MXG_F32) return backward_typed<float>(d, num_sms, stream);
  if (d.dtype == MXG_BF16) return backward_typed<Bf16>(d, num_sms, stream);
  return backward_typed<F16>(d, num_sms, stream);
}

}  // namespace mxg
