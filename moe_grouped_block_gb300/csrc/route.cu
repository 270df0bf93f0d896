// route.cu -- tokens to experts: the k best logits of each token, their weights, the
// tokens of each expert, the balance loss, and the rows that the tokens take among
// the experts' groups; and the gradient of the weights and of the loss.
//
//   s = softmax(l) or sigmoid(l);  p = s / sum(s);  weight = scale * s [/ sum of the chosen s]
//   loss = sum_e slope_e sum_t p_te,  slope_e = balance * E / n * counts_e / sum(counts)
//
// A token is worked on by a team of 1 to 32 lanes that keep its logits in registers, 8 to
// 32 columns a lane in runs of 8: few lanes with many columns for large batches, where
// instructions are the bound and those between lanes cost most, and 8 columns a lane for
// small ones.
//
// The tokens are cut into chunks, one for each CTA, which leaves its chunk's tokens per
// expert and sums of p in the workspace.  A second kernel adds these up -- each CTA the
// same ones in the same order -- and gives its chunk's tokens their rows: the expert's
// start, the tokens of it in earlier chunks, those of earlier warps, and the rank among
// the warp's tokens.  One chunk alone is finished by the first kernel.  No floating-point
// atomics and no counters kept between calls.
//
// Instructions and the latency of dependent steps are the bound, not memory: 65536 tokens
// to 8 of 256 experts (fp32, sigmoids, with the loss and the rows) take 39.5 us, 1.9 TB/s: 30 in the
// first kernel (alone), 281 instructions a token, and the rest in the second.  4 of those are a second
// wave: with 152 chunks its 153 CTAs, of an SM's whole register file each, do not fit 152 SMs at once,
// and the last one starts when another has ended (35.1 us with 151 chunks).  16384 tokens to 8 of 64:
// 11.3 us, 128 chunks, half of it the second kernel and the step between the two.  8 tokens to 2 of 8:
// 5.9 us, one CTA.  The gradient of the first: 29 us, 4.8 TB/s of the 6.78 that a copy reaches.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "host16.h"

namespace mxg {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChunks = 152;  // a CTA an SM (of the first kernel; the second has one more)
constexpr uint32_t kNoLogit = 0x007FFFFFu;  // the key of -infinity: it and all below are not chosen
constexpr int kOneItems = 4096;  // choices of a batch that one CTA finishes

// Threads of a CTA: of the kernels that work on a whole batch alone, and of the others.  With
// 16 or 32 columns a lane the choice needs the registers of two or four.
constexpr int kOneThreads = 512;
constexpr int kManyThreads = 1024;
constexpr int threads_of(int lpt, int vpl, bool one) {
  return lpt == 32 && vpl == 32 ? 256 : (one || vpl > 8 || lpt == 1 ? 512 : 1024);
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
  // how the second half is cut, found on the host: a division takes a kernel 150 cycles
  int32_t warps, rounds, each;  // a chunk's tokens over warps and rounds, 32 at most each
  int32_t inverse;              // 65536 / k, rounded up
  int32_t pitch;                // of a warp's words: odd, a column of them lies on different banks
  int32_t share_bits, each_share;  // neighbouring lanes that take an expert's words, words of each
  int32_t quad_bits, parts;        // threads that read a chunk's experts, chunks read at once
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

// A key that orders a token's logits, and among equal ones the lower column first: of 16-bit
// types, whose order fits into 16 bits, the rest of the word is the column.  kUnique: no two of
// a token are equal.
template <typename T>
constexpr bool kUnique = sizeof(T) == 2;
template <typename T>
__device__ __forceinline__ uint32_t order_key(T v, int column) {
  if constexpr (sizeof(T) == 4) {
    return logit_key(v);
  } else {
    constexpr uint32_t kInf = std::is_same<T, Bf16>::value ? 0x7F80u : 0x7C00u;
    uint32_t u = v.bits;
    if ((u & 0x7FFFu) > kInf) u = 0x7FFFu;  // NaN, of either sign
    if (u == 0x8000u) u = 0u;
    u ^= u & 0x8000u ? 0xFFFFu : 0x8000u;
    return (u << 16) | (0xFFFFu - static_cast<uint32_t>(column));
  }
}

// sigmoid(l), and sigmoid(l) e^-m with m < 0: shares of a token whose sigmoids all underflow
// are still right (m the largest logit where that is negative, so l <= m).
__device__ __forceinline__ float sigmoid(float l) { return rcp_approx(1.0f + exp_approx(-l)); }
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
  return m < 0.0f ? exp_approx(l - m) * rcp_approx(1.0f + exp_approx(l)) : sigmoid(l);
}
// The same and 1 - sigmoid(l), without the subtraction's cancellation.
__device__ __forceinline__ float sigmoid_scaled(float l, float m, float& rest) {
  if (m < 0.0f) {
    rest = rcp_approx(1.0f + exp_approx(l));
    return exp_approx(l - m) * rest;
  }
  const float e = exp_approx(-l), r = rcp_approx(1.0f + e);
  rest = fminf(e * r, 1.0f);  // (infinity times 0 becomes 1)
  return r;
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

// A lane's columns of a row: runs of 8, LPT of them from one to the next.
template <int LPT>
__device__ __forceinline__ int column(int i, int gl) {
  return ((i >> 3) * LPT + gl) * 8 + (i & 7);
}

// As they lie in memory; -infinity past the last expert.
template <typename T, int LPT, int VPL>
struct LogitRow {
  Raw8<T> raw[VPL / 8];
  __device__ __forceinline__ void load(const T* row, int gl, int experts, bool vec) {
#pragma unroll
    for (int i = 0; i < VPL / 8; ++i) {
      const int c = column<LPT>(8 * i, gl);
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
  // asks for the lines of a row that is loaded later
  static __device__ __forceinline__ void ahead(const T* row, int gl, int experts) {
#pragma unroll
    for (int i = 0; i < VPL / 8; ++i) {
      const int c = column<LPT>(8 * i, gl);
      if (c < experts) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + c));
    }
  }
};

// ---------------------------------------------------------------- rows
// Sums over the chunks, `pitch` columns each, into parts of shared memory: part p, column c at
// [p * pitch + c].  LOW: beside the sums, those
// of the chunks below `low`, `kBufWords / 2` further on.
template <bool LOW, typename V4, typename V>
__device__ __forceinline__ void sum_chunks(V* to, const V* from, int pitch, int chunks, int low,
                                           int quad_bits, int parts) {
  const int quads = pitch >> 2;
  const int q = threadIdx.x & ((1 << quad_bits) - 1), part = threadIdx.x >> quad_bits;
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
}

// Everything that needs the whole batch's counts, by the CTA of chunk c, of NT threads
// (at least as many as experts, but for ONE).  ONE: this CTA has all tokens, whose counts and
// sums are in `sh`.  Else the CTA behind the last chunk's, which has no tokens, writes counts,
// group_ws, slope and loss.
template <int NT, bool ONE, int BUF>
__device__ __forceinline__ void finish_chunk(const RowPlan& p, RouteShared<BUF>& sh,
                                             const RouteWs& ws, const int32_t* expert, int c) {
  static_assert(ONE || BUF == kBufWords, "sums of chunks take two halves of a whole buffer");
  constexpr int kPer = (kMaxExperts + NT - 1) / NT;  // experts a thread
  constexpr int kWarps = NT / 32;
  const int tid = threadIdx.x, E = p.experts;
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t* buf = reinterpret_cast<uint32_t*>(sh.buf);
  // this chunk's choices, 32 tokens at most a warp and round (as many warps as the counts
  // have room for); the first kHeld of a lane are asked for now
  constexpr int kHeld = 4;
  const int64_t begin = static_cast<int64_t>(c) * p.per;
  const int tokens_here =
      p.row_of == nullptr ? 0 : static_cast<int>(max(min(begin + p.per, p.tokens) - begin, int64_t{0}));
  const int warps = p.warps, each = p.each, pitch = p.pitch, inverse = p.inverse;
  const int rounds = tokens_here == 0 ? 0 : p.rounds;
  int from = 0, items = 0;  // of this warp and round
  auto take = [&](int round) {
    const int first = warp < warps ? min((round * warps + warp) * each, tokens_here) : 0;
    from = first * p.k;
    items = warp < warps ? (min(first + each, tokens_here) - first) * p.k : 0;
  };
  auto choice = [&](int i) {
    const int32_t e = i < items ? expert[from + i] : -1;
    return static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;
  };
  int32_t held[kHeld];
  auto hold = [&] {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = choice(32 * i + lane);
  };
  take(0);
  hold();
  // tokens of each expert, in all chunks and in those before this one
  const int parts = p.parts;
  const bool losses = (ONE || c == p.chunks) && (p.loss != nullptr || p.slope != nullptr);
  if (!ONE) {
    const uint32_t* hist = reinterpret_cast<const uint32_t*>(ws.hist);
    if (c == p.chunks) {  // no tokens: the sums of p in the place of those before them
      sum_chunks<false, uint4>(buf, hist, ws.pitch, p.chunks, 0, p.quad_bits, p.parts);
      if (losses && p.loss != nullptr)
        sum_chunks<false, float4>(reinterpret_cast<float*>(buf) + kBufWords / 2, ws.psum, ws.pitch,
                                  p.chunks, 0, p.quad_bits, p.parts);
    } else {
      sum_chunks<true, uint4>(buf, hist, ws.pitch, p.chunks, c, p.quad_bits, p.parts);
    }
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
      if (ONE || c == p.chunks) {
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

  if (losses) {
    const float* part_p = reinterpret_cast<const float*>(buf) + kBufWords / 2;
    int tokens = 0;
    if (ONE) {
      tokens = sh.live;
    } else {
      for (int h = lane; h < p.chunks; h += 32) tokens += ws.live[h];
      tokens = __reduce_add_sync(0xFFFFFFFFu, tokens);
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
          for (int part = 0; part < parts; ++part) v += part_p[part * ws.pitch + e];
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

  // A choice's place among its expert's: those of earlier tokens of the warp, then of earlier
  // warps, chunks and experts.  The warp's tokens of an expert are bits of a word (a token
  // names an expert once), so their order does not depend on that of the atomics.
  uint32_t* mine = buf + warp * pitch;
  int32_t* row_of = p.row_of + begin * p.k;
  const int shares = 1 << p.share_bits;
  for (int round = 0; round < rounds; ++round) {
    if (round > 0) {
      __syncthreads();  // the words of the round before have been read
      take(round);
      hold();
    }
    if (warp < warps)
      for (int i = lane; i < E; i += 32) mine[i] = 0;
    __syncwarp();
    auto bit = [&](int i) { return 1u << ((i * inverse) >> 16); };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (held[i] >= 0) atomicOr(&mine[held[i]], bit(32 * i + lane));
    for (int i = 32 * kHeld + lane; i < items; i += 32) {
      const int32_t e = choice(i);
      if (e >= 0) atomicOr(&mine[e], bit(i));
    }
    __syncwarp();
    uint32_t at[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      at[i] = held[i] < 0 ? 0u : __popc(mine[held[i]] & (bit(32 * i + lane) - 1u));
    // (more than a lane holds: their places wait in row_of)
    for (int i = 32 * kHeld + lane; i < items; i += 32) {
      const int32_t e = choice(i);
      row_of[from + i] = e < 0 ? 0 : __popc(mine[e] & (bit(i) - 1u));
    }
    __syncthreads();
    // an expert's tokens in the warps before: neighbouring lanes take a part of the warps each
    for (int i = tid; (i & ~31) < E << p.share_bits; i += NT) {
      const int e = i >> p.share_bits, share = i & (shares - 1);
      const int w0 = share * p.each_share, w1 = min(w0 + p.each_share, warps);
      uint32_t n = 0;
      if (e < E)
#pragma unroll 4
        for (int w = w0; w < w1; ++w) n += __popc(buf[w * pitch + e]);
      uint32_t upto = n;
      for (int d = 1; d < shares; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (share >= d) upto += v;
      }
      uint32_t first = e < E ? sh.start[e] + upto - n : 0u;
      __syncwarp();  // an expert's lanes have all read its start
      if (e < E) {
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
          n = __popc(buf[w * pitch + e]);
          buf[w * pitch + e] = first;
          first += n;
        }
        if (share == shares - 1) sh.start[e] = first;
      }
    }
    __syncthreads();
    auto write = [&](int i, int32_t e, uint32_t place) {
      const uint32_t row = e >= 0 ? mine[e] + place : p.capacity;
      row_of[from + i] = row < p.capacity ? static_cast<int32_t>(row) : -1;
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (32 * i + lane < items) write(32 * i + lane, held[i], at[i]);
    for (int i = 32 * kHeld + lane; i < items; i += 32)
      write(i, choice(i), static_cast<uint32_t>(row_of[from + i]));
  }
}

__global__ void __launch_bounds__(kManyThreads)
    route_finish_kernel(const RowPlan p, const RouteWs ws, int first) {
  __shared__ RouteShared<kBufWords> sh;
  grid_wait_for_previous();
  grid_launch_dependents();
  const int c = first + static_cast<int>(blockIdx.x);
  finish_chunk<kManyThreads, false>(p, sh, ws, p.expert + c * p.per * p.k, c);
}

// Tokens per expert of a chunk, for experts chosen elsewhere.
template <int NT, bool ONE>
__global__ void __launch_bounds__(NT) route_count_kernel(const RowPlan p, const RouteWs ws) {
  __shared__ RouteShared<ONE ? kBufWords / 2 : kBufWords> sh;
  const int tid = threadIdx.x, c = blockIdx.x, E = p.experts;
  grid_wait_for_previous();
  grid_launch_dependents();
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
// A team's k best logits in falling order: lane j of the team keeps the j-th, the one LPT after it,
// and so on, KPL of them.
template <int KPL>
struct Chosen {
  float logit[KPL];  // -infinity where there is none
  int expert[KPL];   // -1 there
};

// One after the other: the maximum over the team, and the lowest column that holds it.
template <int LPT, int VPL, int KPL>
__device__ __forceinline__ Chosen<KPL> choose_in_turn(const float (&v)[VPL], bool on, int k,
                                                      int gl) {
  const int lane = threadIdx.x & 31;
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = on ? logit_key(v[i]) : 0u;
  Chosen<KPL> r;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    r.logit[i] = -INFINITY;
    r.expert[i] = -1;
  }
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    const uint32_t m = team_max<LPT>(best);
    int slot = 0;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == m) slot = i;
    int e = column<LPT>(slot, gl);
    bool here = best == m;
    if constexpr (VPL == 8) {  // the lanes are in the order of their columns
      const uint32_t holds = __ballot_sync(0xFFFFFFFFu, here) >> (lane & ~(LPT - 1));
      const int who = __ffs(holds) - 1;
      e = __shfl_sync(0xFFFFFFFFu, e, who, LPT);
      here = gl == who;
    } else {
      const uint32_t mine = here ? static_cast<uint32_t>(e) : 0xFFFFFFFFu;
      e = static_cast<int>(~team_max<LPT>(~mine));
      here = static_cast<uint32_t>(e) == mine;
    }
    if (here)
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == slot) key[i] = 0u;
    if (gl == (j & (LPT - 1)) && m > kNoLogit) {
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (i == j / LPT) {
          r.expert[i] = e;
          r.logit[i] = key_logit(m);
        }
    }
  }
  return r;
}

// By counting, among the few logits that can be of the best: the team's columns form 16 parts
// (32, one a lane, where it is a whole warp), and nothing below the k-th largest of their maxima
// is chosen.  The others -- for 8 of 64 some 10, for 8 of 256 some 11 -- are laid out in shared
// memory, and the lanes count those above each.  Where there are more than kMost, one after
// the other after all.  (The least maximum of 8 parts takes fewer steps to find, but leaves more
// than kMost so often -- at 256 columns for 13 % of the tokens -- that all took longer.)
// `slots` has room for the warp's teams.
constexpr int kMost = 31;  // (a stride that keeps the teams' slots on different banks)

template <typename T, int LPT, int VPL, int KPL>
__device__ __forceinline__ Chosen<KPL> choose_by_rank(const float (&v)[VPL], const T* row, bool on,
                                                      int k, int gl, uint2* slots) {
  constexpr int kParts = LPT < 16 ? 16 / LPT : 1;    // of a lane
  constexpr int kRun = kParts <= VPL / 8 ? 8 : 4;    // columns in a row of a part
  const int lane = threadIdx.x & 31;
  float part[kParts];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int at = i / kRun % kParts;
    part[at] = i < kRun * kParts && i % kRun == 0 ? v[i] : fmaxf(part[at], v[i]);
  }
  float bound = INFINITY;
  if constexpr (LPT == 32) {
    uint32_t best = logit_key(part[0]), m = __reduce_max_sync(0xFFFFFFFFu, best);
    for (int j = 1; j < k; ++j) {
      if (best == m) best = 0u;  // all alike at once: the bound is only lower for it
      m = __reduce_max_sync(0xFFFFFFFFu, best);
    }
    bound = key_logit(m);
  } else {
    int above[kParts] = {};
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int o = 0; o < LPT; ++o) {
        const float other = __shfl_sync(0xFFFFFFFFu, part[i], o, LPT);
#pragma unroll
        for (int j = 0; j < kParts; ++j) above[j] += other > part[j] ? 1 : 0;
      }
#pragma unroll
    for (int j = 0; j < kParts; ++j)
      if (above[j] < k) bound = fminf(bound, part[j]);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1)
      bound = fminf(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, o));
  }
  bound = fmaxf(bound, -3.40282347e38f);  // -infinity is not chosen; NaN is not below anything
  uint32_t among = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) among |= !(v[i] < bound) ? 1u << i : 0u;
  if (!on) among = 0;
  const int n = __popc(among);
  int at = n;
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, at, d, LPT);
    if (gl >= d) at += x;
  }
  const int all = __shfl_sync(0xFFFFFFFFu, at, LPT - 1, LPT);
  const int most = __reduce_max_sync(0xFFFFFFFFu, all);
  if (most > kMost) return choose_in_turn<LPT, VPL, KPL>(v, on, k, gl);
  uint2* team = slots + lane / LPT * kMost;
  for (uint2* to = team + (at - n); among != 0; among &= among - 1u) {
    const int i = __ffs(static_cast<int>(among)) - 1;
    const int e = ((i >> 3) * LPT + gl) * 8 + (i & 7);
    // (read again: a register cannot be picked by a number)
    *to++ = make_uint2(order_key<T>(row[e], e), static_cast<uint32_t>(e));
  }
  // no key in the slots behind, up to those of the team that has most
  for (int i = all + gl; i < most; i += LPT) team[i].x = 0u;
  __syncwarp();
  // two a lane at once, as often as it takes: mostly once for 8 lanes, twice for 4
  constexpr int kPairs = (kMost + 2 * LPT - 1) / (2 * LPT);
  uint2 mine[2 * kPairs];
  int above[2 * kPairs];
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kPairs; ++r) {
    const int i0 = 2 * r * LPT + gl, i1 = i0 + LPT;
    above[2 * r] = above[2 * r + 1] = k;  // of a slot that is empty
    if (2 * r * LPT < most) {
      const uint2 a = i0 < all ? team[i0] : make_uint2(0xFFFFFFFFu, 0u);
      const uint2 b = i1 < all ? team[i1] : make_uint2(0xFFFFFFFFu, 0u);
      int x = 0, y = 0;
#pragma unroll 4
      for (int j = 0; j < most; ++j) {
        const uint32_t other = team[j].x;
        x += other > a.x ? 1 : 0;
        y += other > b.x ? 1 : 0;
      }
      sum += x + y;
      mine[2 * r] = a;
      mine[2 * r + 1] = b;
      if (i0 < all) above[2 * r] = x;
      if (i1 < all) above[2 * r + 1] = y;
    }
  }
  // without equal keys the counts are 0, 1, 2, ...; else the lower column comes first
  if constexpr (!kUnique<T>) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (__any_sync(0xFFFFFFFFu, 2 * sum != all * (all - 1))) {
      for (int j = 0; j < all; ++j) {
        const uint2 other = team[j];
#pragma unroll
        for (int r = 0; r < 2 * kPairs; ++r)
          if (r * LPT + gl < all && other.x == mine[r].x && other.y < mine[r].y) ++above[r];
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 2 * kPairs; ++r)
    if (above[r] < k) team[above[r]] = mine[r];
  __syncwarp();
  Chosen<KPL> c;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    uint2 x = make_uint2(0u, 0xFFFFFFFFu);
    if (i * LPT + gl < min(all, k)) x = team[i * LPT + gl];
    c.expert[i] = static_cast<int>(x.y);
    c.logit[i] = c.expert[i] >= 0 ? to_f32(row[c.expert[i]]) : -INFINITY;
  }
  __syncwarp();  // the slots are written again for the next token
  return c;
}

// KPL * LPT >= k; KPL > 1 in the kernels of few lanes a token.  With 32 columns a lane the 128
// registers of 512 threads are just too few: 4 lanes a token put 28 to 136 bytes a thread on the stack,
// 8 and 16 lanes 12 to 88 (16-bit logits alone).
template <typename T, int LPT, int VPL, int KPL, int NT, bool ONE>
__global__ void __launch_bounds__(NT)
    route_kernel(const mxg_route_t d, const RowPlan p, const RouteWs ws, int vec) {
  constexpr int kTeams = NT / LPT, kWarps = NT / 32;
  constexpr int kBuf = ONE ? kBufWords / 2 : kBufWords;
  // room for the teams' slots; many CTAs take 8 columns by 16 lanes for more than 8 of the experts alone
  constexpr bool kRank = (LPT >= 8 && (ONE || LPT != 16 || VPL != 8)) || (LPT == 4 && KPL > 1);
  constexpr bool kAhead = VPL <= 16;  // registers for the next row
  static_assert(!kRank || kWarps * kMost * (32 / LPT) * 2 <= kBuf, "slots of every team");
  __shared__ RouteShared<kBuf> sh;
  __shared__ int32_t choices[ONE ? kOneItems : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int gl = lane & (LPT - 1), E = d.experts, k = d.k;
  for (int e = tid; e < E; e += NT) sh.hist[e] = 0;
  if (tid == 0) sh.live = 0;
  __syncthreads();
  grid_wait_for_previous();
  grid_launch_dependents();

  const int64_t begin = c * p.per;
  const int count = static_cast<int>(max(min(begin + p.per, d.tokens) - begin, int64_t{0}));
  const T* const logits = static_cast<const T*>(d.logits) + begin * d.ld;
  const T* row = logits + tid / LPT * d.ld;
  const uint8_t* mask = d.mask != nullptr ? d.mask + begin : nullptr;
  int32_t* const expert = d.expert + begin * k;
  float* const weight = d.weight + begin * k;
  const bool softmax = d.score == MXG_SCORE_SOFTMAX;
  const bool shares = d.loss != nullptr, whole = shares || (softmax && !d.normalize);
  // a few are found sooner in turn, and of more than 8 the bound by 16 parts leaves too many
  const bool by_rank = kRank && k > 3 && (LPT == 32 || k <= 8);
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int live = 0;
  int t = tid / LPT;  // in the chunk
  LogitRow<T, LPT, VPL> next;
  bool next_on = false;
  auto fetch = [&](int at) {
    next_on = at < count && (mask == nullptr || mask[at] != 0);
    if (at < count) next.load(row, gl, E, vec != 0);
    row += kTeams * d.ld;
  };
  if (kAhead) fetch(t);
  for (int base = 0; base < count; base += kTeams, t += kTeams) {
    if (!kAhead) {
      fetch(t);
      if (t + kTeams < count) next.ahead(row, gl, E);
    }
    float v[VPL];
    next.values(v);
    const bool on = next_on;
    if (kAhead) fetch(t + kTeams);
    Chosen<KPL> best;
    if (kRank && by_rank)
      best = choose_by_rank<T, LPT, VPL, KPL>(
          v, logits + t * d.ld, on, k, gl, reinterpret_cast<uint2*>(sh.buf) + warp * (kMost * (32 / LPT)));
    else
      best = choose_in_turn<LPT, VPL, KPL>(v, on, k, gl);
    const float top = __shfl_sync(0xFFFFFFFFu, best.logit[0], 0, LPT);
    const bool taken = __shfl_sync(0xFFFFFFFFu, best.expert[0], 0, LPT) >= 0;
    const float shift = softmax ? top : fminf(top, 0.0f);
    float w[KPL], chosen = 0.0f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const float l = best.logit[i];
      w[i] = best.expert[i] < 0 ? 0.0f
             : softmax          ? exp_approx(l - shift)
                                : sigmoid_scaled(l, d.normalize ? shift : 0.0f);
      chosen += w[i];
    }
    if (d.normalize) chosen = team_add<LPT>(chosen);
    float sum = 0.0f;
    if (whole) {
      if (softmax) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = exp_approx(v[i] - shift);
      } else if (shift < 0.0f) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = sigmoid_scaled(v[i], shift);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = sigmoid(v[i]);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += v[i];
      sum = team_add<LPT>(sum);
    }
    if (!d.normalize) chosen = softmax ? sum : 1.0f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = i * LPT + gl, e = best.expert[i];
      if (t < count && j < k) {
        expert[t * k + j] = e;
        weight[t * k + j] = e >= 0 ? d.scale * (w[i] / chosen) : 0.0f;
        if (ONE) choices[t * k + j] = e;
      }
      if (e >= 0) atomicAdd(&sh.hist[e], 1);
    }
    if (taken) {
      if (gl == 0) ++live;
      if (shares) {
        const float r = rcp_approx(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = fmaf(v[i], r, acc[i]);
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
        float* to = rows + (warp - w0) * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = column<LPT>(i, gl);
          if (e < E) to[e] = w0 == 0 ? acc[i] : to[e] + acc[i];
        }
      }
      __syncthreads();
    }
    for (int e = tid; e < E; e += NT) {
      float x = 0.0f;
#pragma unroll 4
      for (int w = 0; w < fit; ++w) x += rows[w * E + e];
      if (ONE)
        sh.psum[e] = x;
      else
        ws.psum[static_cast<int64_t>(c) * ws.pitch + e] = x;
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
// The extras reach the lanes that own their columns through a row of shared memory a team.
constexpr int kGradThreads = 256;

// A row of n columns in shared memory: the first halves of its runs of 8, then the second ones, so
// that neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ int halves_at(int c, int n) {
  return (c >> 3) * 4 + (c & 3) + ((c & 4) != 0 ? n / 2 : 0);
}

// CTAs an SM: four, which 64 registers a thread allow.  Lanes of 8 or 4 choices put 44 to 164 bytes of
// theirs on the stack for it (32 experts or fewer); with two CTAs and 12 bytes there at most, 65536
// tokens took 3.0 and not 3.6 us (2 of 8, bf16), 4.3 and not 5.5 (4 of 16), but 8.4 and not 7.7 (8 of 32).
template <typename T, int LPT, int VPL, int KPL>
__global__ void __launch_bounds__(kGradThreads, VPL <= 16 ? 4 : 1)
    route_backward_kernel(const mxg_route_grad_t d, int vec) {
  constexpr int kTeams = kGradThreads / LPT, kCols = LPT * VPL;
  __shared__ float4 team_rows[kTeams][kCols / 4];
  __shared__ float4 slopes[kCols / 4];
  const int tid = threadIdx.x, gl = tid & (LPT - 1), E = d.experts, k = d.k;
  float4* const mine = team_rows[tid / LPT];
  const bool softmax = d.score == MXG_SCORE_SOFTMAX, balance = d.slope != nullptr;
  // the weights' gradient goes through the shares; whether any of it does
  const bool joined = softmax && !d.normalize, shares = balance || joined;
  grid_wait_for_previous();
  grid_launch_dependents();
  const float dloss = balance ? *d.dloss : 0.0f;
  for (int e = tid; e < kCols; e += kGradThreads)
    reinterpret_cast<float*>(slopes)[halves_at(e, kCols)] = balance && e < E ? d.slope[e] * dloss : 0.0f;
  __syncthreads();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + tid / LPT;
  // the chosen experts and their weights' gradients are asked for a token ahead
  int e[KPL];
  float b[KPL];
  auto choices = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int j = i * LPT + gl;
      e[i] = at < d.tokens && j < k ? d.expert[at * k + j] : -1;
      b[i] = at < d.tokens && j < k && d.dweight != nullptr ? d.dweight[at * k + j] : 0.0f;
    }
  };
  choices(t);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTeams; base < d.tokens;
       base += step, t += step) {
    const bool in = t < d.tokens;
    const T* row = static_cast<const T*>(d.logits) + (in ? t : 0) * d.ld;
    LogitRow<T, LPT, VPL> raw;
    raw.load(row, gl, in ? E : 0, vec != 0);
    if (t + step < d.tokens) raw.ahead(row + step * d.ld, gl, E);
    int at[KPL], have = 0;
    float l[KPL], db[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      at[i] = static_cast<uint32_t>(e[i]) < static_cast<uint32_t>(E) ? e[i] : -1;
      l[i] = at[i] >= 0 ? to_f32(row[at[i]]) : -INFINITY;
      db[i] = at[i] >= 0 ? d.scale * b[i] : 0.0f;
      have |= at[i] >= 0 ? 1 : 0;
    }
    choices(t + step);
    float v[VPL];
    raw.values(v);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) have |= __shfl_xor_sync(0xFFFFFFFFu, have, o);

    float top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float shift = softmax ? top : fminf(top, 0.0f);
    // the shares (times 1 - s for sigmoids, once they are summed up) and their part of the sums
    float sum = 0.0f, dot = 0.0f;
    if (shares) {
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        const float4 a4 = slopes[halves_at(column<LPT>(i, gl), kCols) / 4];
        const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float rest = 1.0f;
          const float p = softmax ? exp_approx(v[i + j] - shift)
                                  : sigmoid_scaled(v[i + j], shift, rest);
          sum += p;
          dot = fmaf(a[j], p, dot);
          v[i + j] = softmax ? p : p * rest;
        }
      }
      sum = team_add<LPT>(sum);
    }
    // the chosen experts'
    float s[KPL], rest[KPL], chosen = 0.0f, bq = 0.0f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      rest[i] = 1.0f;
      s[i] = 0.0f;
      if (at[i] >= 0)
        s[i] = softmax ? exp_approx(l[i] - shift)
                       : sigmoid_scaled(l[i], d.normalize ? shift : 0.0f, rest[i]);
      chosen += s[i];
      bq = fmaf(db[i], s[i], bq);
    }
    if (d.normalize) {
      chosen = team_add<LPT>(chosen);
      bq = team_add<LPT>(bq) / chosen;
    } else {
      if (joined) dot += bq;
      chosen = joined ? sum : 1.0f;
      bq = 0.0f;
    }
    float r = 0.0f;
    if (shares) {
      r = rcp_approx(sum);
      dot = -team_add<LPT>(dot) * r * r;
    }
#pragma unroll
    for (int i = 0; i < VPL; i += 4)
      mine[halves_at(column<LPT>(i, gl), kCols) / 4] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (at[i] >= 0)
        atomicAdd(reinterpret_cast<float*>(mine) + halves_at(at[i], kCols),
                  s[i] / chosen * rest[i] * (db[i] - bq));
    __syncwarp();
    T* out = static_cast<T*>(d.dlogits) + (in ? t : 0) * d.ldd;
#pragma unroll
    for (int i = 0; i < VPL; i += 8) {
      const int c = column<LPT>(i, gl);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const int q = halves_at(c + j, kCols) / 4;
        const float4 x = mine[q], a = slopes[q];
        f[j] = x.x;
        f[j + 1] = x.y;
        f[j + 2] = x.z;
        f[j + 3] = x.w;
        if (shares) {  // p / sum (a - dot / sum) + extra
          f[j] = fmaf(v[i + j], fmaf(a.x, r, dot), f[j]);
          f[j + 1] = fmaf(v[i + j + 1], fmaf(a.y, r, dot), f[j + 1]);
          f[j + 2] = fmaf(v[i + j + 2], fmaf(a.z, r, dot), f[j + 2]);
          f[j + 3] = fmaf(v[i + j + 3], fmaf(a.w, r, dot), f[j + 3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = have ? f[j] : 0.0f;
      if (!in) continue;
      if (vec && c < E) {
        if constexpr (sizeof(T) == 4) {
          reinterpret_cast<float4*>(out + c)[0] = make_float4(f[0], f[1], f[2], f[3]);
          reinterpret_cast<float4*>(out + c)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          *reinterpret_cast<uint4*>(out + c) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]),
                                                          pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < E) out[c + j] = from_f32<T>(f[j]);
      }
    }
    __syncwarp();
  }
}

namespace {

// How a token is laid out over lanes: few lanes (kpl > 0 choices each) with many columns, where
// k is at most 8 and there are at most 512 experts; else 8 columns a lane (up to 32 lanes), and a
// lane for each of the k.
struct Shape {
  int lpt, vpl, kpl;
};
Shape few_lanes(int experts) {
  if (experts <= 8) return {1, 8, 8};
  if (experts <= 16) return {1, 16, 8};
  if (experts <= 32) return {2, 16, 4};
  if (experts <= 64) return {4, 16, 2};
  if (experts <= 128) return {4, 32, 2};
  if (experts <= 256) return {8, 32, 1};
  return {16, 32, 1};
}
Shape many_lanes(int experts, int k) {
  int lanes = 1;
  while (lanes < 32 && (lanes * 8 < experts || lanes < k)) lanes *= 2;
  return {lanes, experts > 512 ? 32 : (experts > 256 ? 16 : 8), 1};
}
bool few_serve(int experts, int k) { return k <= 8 && experts <= 512; }

struct Chunks {
  int n;
  int64_t per;  // tokens each
  int room;     // no fewer than a smaller batch has: tokens rounded up a chunk can leave n below that
};

Chunks cut(int64_t tokens, int64_t pass) {
  const int64_t n = std::min<int64_t>(kMaxChunks, (tokens + pass - 1) / pass);
  Chunks c;
  c.per = (tokens + n - 1) / n;
  c.n = static_cast<int>(std::max<int64_t>(2, (tokens + c.per - 1) / c.per));
  c.room = static_cast<int>(std::max<int64_t>(2, n));
  return c;
}

// One CTA up to two passes of its teams, else a pass at least a CTA: 256 tokens of 64 experts, four
// passes, took 13.6 us in one CTA and 10.6 in four.
Chunks chunks_of(int64_t tokens, int experts, int k) {
  const Shape one = many_lanes(experts, k);
  if (tokens <= 2 * (threads_of(one.lpt, one.vpl, true) / one.lpt) && tokens * k <= kOneItems)
    return {1, std::max<int64_t>(1, tokens), 1};
  const Shape s = few_serve(experts, k) ? few_lanes(experts) : one;
  return cut(tokens, threads_of(s.lpt, s.vpl, false) / s.lpt);
}

// For choices made elsewhere, each counted as a token with one.
Chunks chunks_of_choices(int64_t choices) {
  if (choices <= 4 * kOneThreads) return {1, std::max<int64_t>(1, choices), 1};
  return cut(choices, kManyThreads);
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

// How finish_chunk cuts its work, in a CTA of `threads`.
void cut_finish(RowPlan* p, int threads) {
  const int words = p->chunks == 1 ? kBufWords / 2 : kBufWords;
  p->pitch = p->experts | 1;
  p->warps = std::min(threads / 32, words / p->pitch);
  p->rounds = static_cast<int>(std::max<int64_t>(1, (p->per + 32 * p->warps - 1) / (32 * p->warps)));
  p->each = static_cast<int>((p->per + p->rounds * p->warps - 1) / (p->rounds * p->warps));
  p->inverse = (65536 + p->k - 1) / p->k;
  int wide = 1, quads = 1;
  while (wide < p->experts) wide *= 2;
  p->share_bits = 0;
  while (p->share_bits < 5 && (wide << (p->share_bits + 1)) <= threads) ++p->share_bits;
  p->each_share = (p->warps + (1 << p->share_bits) - 1) >> p->share_bits;
  p->quad_bits = 0;
  while (quads < (p->experts + 3) / 4) {
    quads *= 2;
    ++p->quad_bits;
  }
  p->parts = std::max(1, std::min({threads / quads, 16, p->chunks}));
}

cudaError_t launch_finish(const RowPlan& p, const RouteWs& ws, cudaStream_t stream, int* launches) {
  ++*launches;
  return launch_after(true, route_finish_kernel,
                      static_cast<unsigned>(p.row_of != nullptr ? p.chunks + 1 : 1), kManyThreads,
                      0, stream, p, ws, p.row_of != nullptr ? 0 : p.chunks);
}

template <typename T, int LPT, int VPL, int KPL, bool ONE>
cudaError_t run_route(const mxg_route_t& d, const RowPlan& p, const RouteWs& ws, int vec,
                      cudaStream_t stream) {
  constexpr int kThreads = threads_of(LPT, VPL, ONE);
  return launch_after(true, route_kernel<T, LPT, VPL, KPL, kThreads, ONE>,
                      static_cast<unsigned>(p.chunks), kThreads, 0, stream, d, p, ws, vec);
}

template <typename T>
cudaError_t route_typed(const mxg_route_t& d, const RowPlan& p, const RouteWs& ws,
                        cudaStream_t stream) {
  const int vec = d.experts % 8 == 0 && rows_of_16(d.logits, d.ld, sizeof(T));
  if (p.chunks > 1 && few_serve(d.experts, d.k)) {
    const Shape s = few_lanes(d.experts);
    if (s.vpl == 8) return run_route<T, 1, 8, 8, false>(d, p, ws, vec, stream);
    if (s.lpt == 1) return run_route<T, 1, 16, 8, false>(d, p, ws, vec, stream);
    if (s.lpt == 2) return run_route<T, 2, 16, 4, false>(d, p, ws, vec, stream);
    if (d.experts <= 64) return run_route<T, 4, 16, 2, false>(d, p, ws, vec, stream);
    if (s.lpt == 4) return run_route<T, 4, 32, 2, false>(d, p, ws, vec, stream);
    if (s.lpt == 8) return run_route<T, 8, 32, 1, false>(d, p, ws, vec, stream);
    return run_route<T, 16, 32, 1, false>(d, p, ws, vec, stream);
  }
  const Shape s = many_lanes(d.experts, d.k);
  if (p.chunks > 1) {  // (more than 8 of the experts, or more than 512 of them: 16 lanes at least)
    if (s.lpt == 16) return run_route<T, 16, 8, 1, false>(d, p, ws, vec, stream);
    if (s.vpl == 8) return run_route<T, 32, 8, 1, false>(d, p, ws, vec, stream);
    if (s.vpl == 16) return run_route<T, 32, 16, 1, false>(d, p, ws, vec, stream);
    return run_route<T, 32, 32, 1, false>(d, p, ws, vec, stream);
  }
  if (s.lpt == 1) return run_route<T, 1, 8, 1, true>(d, p, ws, vec, stream);
  if (s.lpt == 2) return run_route<T, 2, 8, 1, true>(d, p, ws, vec, stream);
  if (s.lpt == 4) return run_route<T, 4, 8, 1, true>(d, p, ws, vec, stream);
  if (s.lpt == 8) return run_route<T, 8, 8, 1, true>(d, p, ws, vec, stream);
  if (s.lpt == 16) return run_route<T, 16, 8, 1, true>(d, p, ws, vec, stream);
  if (s.vpl == 8) return run_route<T, 32, 8, 1, true>(d, p, ws, vec, stream);
  if (s.vpl == 16) return run_route<T, 32, 16, 1, true>(d, p, ws, vec, stream);
  return run_route<T, 32, 32, 1, true>(d, p, ws, vec, stream);
}

template <typename T, int LPT, int VPL, int KPL>
cudaError_t run_backward(const mxg_route_grad_t& d, int vec, int num_sms, cudaStream_t stream) {
  constexpr int kTeams = kGradThreads / LPT;
  // as many CTAs as the device holds: 29.4 us for 65536 x 256 in fp32, 31.1 with two waves of them
  const int64_t grid = std::min<int64_t>((d.tokens + kTeams - 1) / kTeams, num_sms * 4LL);
  return launch_after(true, route_backward_kernel<T, LPT, VPL, KPL>, static_cast<unsigned>(grid),
                      kGradThreads, 0, stream, d, vec);
}

template <typename T>
cudaError_t backward_typed(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream) {
  const int vec = d.experts % 8 == 0 && rows_of_16(d.logits, d.ld, sizeof(T)) &&
                  rows_of_16(d.dlogits, d.ldd, sizeof(T));
  if (d.k <= 8 && d.experts <= 256) {
    // (16 columns a lane: more warps an SM than with 32, 29.3 against 32.3 us for 65536 x 256 in fp32)
    if (d.experts <= 8) return run_backward<T, 1, 8, 8>(d, vec, num_sms, stream);
    if (d.experts <= 16) return run_backward<T, 1, 16, 8>(d, vec, num_sms, stream);
    if (d.experts <= 32) return run_backward<T, 2, 16, 4>(d, vec, num_sms, stream);
    if (d.experts <= 64) return run_backward<T, 4, 16, 2>(d, vec, num_sms, stream);
    if (d.experts <= 128) return run_backward<T, 8, 16, 1>(d, vec, num_sms, stream);
    return run_backward<T, 16, 16, 1>(d, vec, num_sms, stream);
  }
  const Shape s = many_lanes(d.experts, d.k);
  if (s.lpt == 16) return run_backward<T, 16, 8, 1>(d, vec, num_sms, stream);
  if (s.vpl == 8) return run_backward<T, 32, 8, 1>(d, vec, num_sms, stream);
  if (s.vpl == 16) return run_backward<T, 32, 16, 1>(d, vec, num_sms, stream);
  return run_backward<T, 32, 32, 1>(d, vec, num_sms, stream);
}

}  // namespace

// Grows with the tokens, so that what is made for the largest batch serves them all.
size_t route_ws_bytes(int64_t tokens, int experts, int k) {
  const int64_t n = std::max(chunks_of(tokens, experts, k).room, chunks_of_choices(tokens * k).room);
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
  const Shape one = many_lanes(d.experts, d.k);
  cut_finish(&p, c.n == 1 ? threads_of(one.lpt, one.vpl, true) : kManyThreads);
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
  // an expert may be named twice for a token here: each choice is a token with one
  const Chunks c = chunks_of_choices(tokens * k);
  RowPlan p = {};
  p.expert = expert;
  p.counts = counts;
  p.row_of = row_of;
  p.group_ws = group_ws;
  p.status = status;
  p.tokens = tokens * k;
  p.per = c.per;
  p.last_dim = last_dim;
  p.capacity = static_cast<uint32_t>(capacity / align * align);
  p.experts = experts;
  p.k = 1;
  p.align = align;
  p.chunks = c.n;
  cut_finish(&p, c.n == 1 ? kOneThreads : kManyThreads);
  const RouteWs ws = carve(workspace, c.n, experts);
  ++*launches;
  if (c.n == 1)
    return launch_after(true, route_count_kernel<kOneThreads, true>, 1, kOneThreads, 0, stream, p, ws);
  const cudaError_t e = launch_after(true, route_count_kernel<kManyThreads, false>,
                                     static_cast<unsigned>(c.n), kManyThreads, 0, stream, p, ws);
  return e != cudaSuccess ? e : launch_finish(p, ws, stream, launches);
}

cudaError_t launch_route_backward(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream) {
  if (d.dtype == MXG_F32) return backward_typed<float>(d, num_sms, stream);
  if (d.dtype == MXG_BF16) return backward_typed<Bf16>(d, num_sms, stream);
  return backward_typed<F16>(d, num_sms, stream);
}

}  // namespace mxg
