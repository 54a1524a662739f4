// Balance loss of a router over sequences of tokens, with the experts'
// counts, and its gradient, for gfx950.
//
// Of a token t, share[t][i] = s_i / sum_j s_j with s the softmax or the
// sigmoid of its logits; masked experts (-inf, NaN) have none, and a token
// with nothing else is not counted.  Over the n counted tokens of a sequence
//   count[i] = entries of idx that name i,
//   slope[i] = scale E / (k n^2) count[i],   loss = sum_i slope[i] sum_t share[t][i]
// (E / (k n) count is the load of an expert relative to an even one, the mean
// of the shares its probability).  slope is also the loss's derivative by every
// share, so that the gradient needs nothing else:
//   c = dloss slope,  m = sum_i c_i share_i
//   softmax: dl_j = share_j (c_j - m),  sigmoid: dl_j = share_j (1 - s_j) (c_j - m)
// A sigmoid's share is formed from exp(l - m'), m' = min(max l, 0), in place
// of s, so that scores that underflow keep their ratios.
//
// The tokens are cut into chunks, and the chunks by the sequences that they
// meet into pieces: the piece of chunk c and sequence s has the number c + s,
// which no other piece has, since along the tokens every step raises c or s.  Each
// piece has one partial sum, and a sequence's are added in their order: no
// result depends on the order in which workgroups run.
//
// The bytes are few (16384 x 256 f32: 17 MB, 3.4 us at a device copy's rate); what
// counts is latency: two dependent launches (9 and 5 us of 14 to 15), the loads of
// bounds, then of tokens, and the fetching of code that each workgroup runs
// through once or twice.  With the loops unrolled and both scores in one kernel the first
// took 12 us; with the largest logit of every token 14.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"
#include "tiles.h"

namespace fp8fg {

namespace {

// Threads of a workgroup that sums tokens: with 16 experts to a lane the registers of
// 1024 do not hold two tokens.
template <int NE>
constexpr int kPartThreads = NE < 16 ? 1024 : 512;
constexpr int kMostWaves = 16;
constexpr int kMaxE = kRouteMaxExperts;

// ------------------------------------------------------------- one token
// LPT lanes hold a token's experts, NE each: 4 consecutive ones at a time
// (VEC), or every LPT-th.
template <int LPT, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return VEC ? 4 * (lane + LPT * (i >> 2)) + (i & 3) : lane + LPT * i;
}

template <int LT, int LPT, int NE, bool VEC>
__device__ __forceinline__ void load_token(const void* __restrict__ p, int64_t at, int lane, int E, float (&y)[NE]) {
  // (without branches: past the last expert it reads that one again, which is masked)
#pragma unroll
  for (int i = 0; i < NE; i += VEC ? 4 : 1) {
    const int e = expert_of<LPT, VEC>(lane, i), last = VEC ? E - 4 : E - 1;
    const int64_t x = at + (e < last ? e : last);
    if constexpr (VEC && LT == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + x);
      y[i] = bf16_lo(w.x);
      y[i + 1] = bf16_hi(w.x);
      y[i + 2] = bf16_lo(w.y);
      y[i + 3] = bf16_hi(w.y);
    } else if constexpr (VEC) {
      const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + x);
      y[i] = w.x;
      y[i + 1] = w.y;
      y[i + 2] = w.z;
      y[i + 3] = w.w;
    } else {
      y[i] = LT == 0 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[x] << 16)
                     : reinterpret_cast<const float*>(p)[x];
    }
  }
}
// -inf past the last expert.
template <int LPT, int NE, bool VEC>
__device__ __forceinline__ void mask_token(int lane, int E, float (&y)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) y[i] = expert_of<LPT, VEC>(lane, i) < E ? y[i] : -INFINITY;
}

template <int LT, int LPT, int NE, bool VEC>
__device__ __forceinline__ void store_token(void* __restrict__ p, int64_t at, int lane, int E, const float (&y)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += VEC ? 4 : 1) {
    const int e = expert_of<LPT, VEC>(lane, i);
    if (e >= E) continue;
    if constexpr (VEC) {
      if constexpr (LT == 0)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at + e) =
            make_uint2(pack2_bf16(y[i], y[i + 1]), pack2_bf16(y[i + 2], y[i + 3]));
      else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at + e) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else if constexpr (LT == 0) {
      reinterpret_cast<uint16_t*>(p)[at + e] = (uint16_t)pack2_bf16(y[i], 0.0f);
    } else {
      reinterpret_cast<float*>(p)[at + e] = y[i];
    }
  }
}

// Sum and maximum over a token's lanes.
template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
  v = row16_sum(v);
  if constexpr (LPT >= 32) v = pair_sum<16>(v);
  if constexpr (LPT >= 64) v = pair_sum<32>(v);
  return v;
}
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  v = row16_max(v);
  if constexpr (LPT >= 32) v = pair_max<16>(v);
  if constexpr (LPT >= 64) v = pair_max<32>(v);
  return v;
}

// exp(x) = 2^t exp(x - t ln 2), t = RN(x RN32(log2 e)): within an ulp of the
// hardware's 2^t and |x| 2^-28 of RN32(ln 2), of which a softmax's shares have the
// differences' alone.  x at least -120; infinite or NaN above 2^128.
__device__ __forceinline__ float exp_from(float x) {
  const float t = x * 1.44269502f;
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, __builtin_fmaf(t, -0.693147181f, x), p);
}
// 0 below 2^-126 and for a NaN.
__device__ __forceinline__ float exp_of(float x) { return exp_from(fmaxf(x, -120.0f)); }

// RN-close 1 / x of a normal x.
__device__ __forceinline__ float reciprocal(float x) {
  const float y = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, y, 1.0f), y, y);
}

// Scores of a token below its largest logit (softmax), or of one whose
// sigmoids may all underflow (their common factor exp(min(top, 0)) taken out),
// and their sum over the token; masked and NaN logits give 0.
template <int LPT, int NE, int SCORE, bool REST>
__device__ __forceinline__ float scores_below_top(const float (&l)[NE], float (&y)[NE], float (&r)[NE]) {
  float top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    y[i] = l[i] == l[i] ? l[i] : -INFINITY;
    top = fmaxf(top, y[i]);
  }
  top = token_max<LPT>(top);
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float v = y[i];
    if (SCORE == 0) {
      y[i] = exp_below(v, top);
    } else {
      const float t = exp_of(-fabsf(v)), inv = __builtin_amdgcn_rcpf(1.0f + t);
      if (REST) r[i] = v >= 0.0f ? t * inv : inv;
      y[i] = (top < 0.0f ? exp_below(v, top) : v >= 0.0f ? 1.0f : t) * inv;
    }
    total += y[i];
  }
  return token_sum<LPT>(total);
}

// Scores of a token's logits, up to a common factor, in y, of a sigmoid also 1 -
// s in r (REST); returns 1 / their sum, 0 where all experts are masked (live
// false).
//
// They are formed directly first: exp(l) and 1 / (1 + exp(-l)) are within fp32's
// range unless the logits are far out, what underflows is below 2^-126 of
// a sum that is not small, and without a difference to round a score's error
// does not grow with its logit.  The sum tells: with one below 1 (softmax) or 1/2
// (sigmoid), above 2^100 or NaN in the wave the scores are formed again
// below the largest logit (16384 x 256, softmax: around 0 11 us, around -8, where all
// waves do, 14).  That maximum and its checks cost half of the instructions.  (A NaN
// logit comes out as a masked one; one whose exponential overflows makes the sum
// infinite or NaN.)
template <int LPT, int NE, int SCORE, bool REST>
__device__ __forceinline__ float token_scores(const float (&l)[NE], float (&y)[NE], float (&r)[NE], bool& live) {
  float total = 0.0f;
  live = true;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (SCORE == 0) {
      y[i] = exp_of(l[i]);
    } else if (REST) {
      const float t = exp_of(-fabsf(l[i])), inv = __builtin_amdgcn_rcpf(1.0f + t);
      r[i] = l[i] >= 0.0f ? t * inv : inv;
      y[i] = l[i] >= 0.0f ? inv : t * inv;
    } else {
      // (from -87 on down, and for a NaN, 2^-125.5)
      y[i] = __builtin_amdgcn_rcpf(1.0f + exp_from(-fmaxf(l[i], -87.0f)));
    }
    total += y[i];
  }
  total = token_sum<LPT>(total);
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(!(total >= (SCORE == 0 ? 1.0f : 0.5f) && total <= 0x1p100f)) != 0, 0)) {
    total = scores_below_top<LPT, NE, SCORE, REST>(l, y, r);
    live = total > 0.0f;
    return live ? reciprocal(total) : 0.0f;
  }
  return reciprocal(total);
}

// ---------------------------------------------------------- sequences
// Offset i, held within the rows (the caller's offsets are not checked).
__device__ __forceinline__ int64_t bound(const int32_t* __restrict__ off, int64_t i, int64_t rows) {
  if (!off) return i ? rows : 0;
  const int64_t v = off[i];
  return v < 0 ? 0 : v < rows ? v : rows;
}

// The first sequence that ends behind token t, or seqs: 64 ends at a time, by a
// whole wave with the same t.  (In 32 bits: with int64_t bounds the compiler
// selected the lower one by a stale condition code.)
__device__ __forceinline__ int64_t find_seq(const int32_t* __restrict__ off, int64_t seqs, int64_t rows, int64_t t) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, hi = (uint32_t)seqs;
  while (lo < hi) {
    const uint32_t step = (hi - lo + 63) >> 6, i = lo + (lane + 1) * step - 1;
    const uint64_t past = __builtin_amdgcn_ballot_w64(i >= hi || bound(off, (int64_t)i + 1, rows) > t);
    if (past == 0) return hi;
    const uint32_t f = (uint32_t)__builtin_ctzll(past), end = lo + (f + 1) * step - 1;
    lo += f * step;
    hi = end < hi ? end : hi;
  }
  return lo;
}

// 64 consecutive bounds in a wave's lanes, lane i the start of sequence base + i;
// with fewer than 64 sequences one load serves a whole chunk.
struct Bounds {
  int64_t base;
  int32_t at;  // (rows fit an int32)
};
__device__ __forceinline__ Bounds load_bounds(const int32_t* __restrict__ off, int64_t seqs, int64_t rows, int64_t t) {
  const int lane = threadIdx.x & 63;
  const int64_t base = seqs < 64 ? 0 : find_seq(off, seqs, rows, t);
  const int64_t i = base + lane;
  return {base, (int32_t)bound(off, i < seqs ? i : seqs, rows)};
}
struct Seq {
  int64_t s, first, end;
};
// The first sequence of the window that ends behind t; s = seqs where there is
// none.  t at least the base sequence's predecessor's end.
__device__ __forceinline__ Seq seq_of(const Bounds& w, int64_t seqs, int64_t t) {
  const int lane = threadIdx.x & 63;
  const uint64_t past = __builtin_amdgcn_ballot_w64(lane > 0 && w.base + lane <= seqs && (int64_t)w.at > t);
  if (past == 0) return {seqs, 0, 0};
  const int f = __builtin_ctzll(past);
  return {w.base + f - 1, __builtin_amdgcn_readlane(w.at, f - 1), __builtin_amdgcn_readlane(w.at, f)};
}

// ------------------------------------------------------- partial sums
struct BalanceLds {
  float sum[kMostWaves][kMaxE];
  int hist[kMaxE];
  int live[kMostWaves];
};

// What a workgroup loads of the tokens from `a` on before it knows how far its
// piece reaches: one token of each lane group and one entry of idx.
template <int NE>
struct Ahead {
  float y[NE];
  int entry;
};
__device__ __forceinline__ int load_entry(const BalanceArgs& p, const FastDiv& by_k, int64_t a, uint32_t i, int64_t end) {
  const uint32_t t = fast_div(i, by_k), j = i - t * by_k.d;
  return a + t < end ? p.idx[(a + t) * p.ld_idx + j] : -1;
}
template <int LT, int LPT, int NE, bool VEC>
__device__ __forceinline__ void load_ahead(const BalanceArgs& p, const FastDiv& by_k, int64_t a, int64_t end, Ahead<NE>& h) {
  const int64_t t = a + threadIdx.x / LPT;
  load_token<LT, LPT, NE, VEC>(p.logits, (t < end ? t : end - 1) * p.ldl, threadIdx.x & (LPT - 1), p.experts, h.y);
  h.entry = load_entry(p, by_k, a, threadIdx.x, end);
}

// Sums of the tokens [a, b), b > a, by the whole workgroup, h loaded from a on:
// on return thread e's column of `sum` is added by column_sum, hist and
// live are whole.  The loops are kept rolled: a workgroup runs through this
// code once or twice, and what it costs then is the fetching of it.
template <int LT, int LPT, int NE, bool VEC, int SCORE>
__device__ __forceinline__ void sum_tokens(const BalanceArgs& p, const FastDiv& by_k, int64_t a, int64_t b, Ahead<NE>& h,
                                           BalanceLds& m) {
  constexpr int kThreads = kPartThreads<NE>, kStep = kThreads / LPT;
  const int lane = threadIdx.x & (LPT - 1), wave = threadIdx.x >> 6;
  float acc[NE] = {}, next[NE];
  int live = 0;
  const int64_t t0 = a + threadIdx.x / LPT;
  load_token<LT, LPT, NE, VEC>(p.logits, (t0 + kStep < b ? t0 + kStep : b - 1) * p.ldl, lane, p.experts, next);
  for (int e = threadIdx.x; e < p.experts; e += kThreads) m.hist[e] = 0;
#pragma unroll 1
  for (int64_t t = t0; t < b; t += kStep) {
    float after[NE], y[NE], none[NE];
    load_token<LT, LPT, NE, VEC>(p.logits, (t + 2 * kStep < b ? t + 2 * kStep : b - 1) * p.ldl, lane, p.experts, after);
    mask_token<LPT, NE, VEC>(lane, p.experts, h.y);
    bool counts;
    const float inv = token_scores<LPT, NE, SCORE, false>(h.y, y, none, counts);
    live += counts;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      acc[i] = __builtin_fmaf(y[i], inv, acc[i]);
      h.y[i] = next[i];
      next[i] = after[i];
    }
  }
  // the wave's tokens, then the waves'
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if constexpr (LPT == 16) acc[i] = pair_sum<16>(acc[i]);
    if constexpr (LPT <= 32) acc[i] = pair_sum<32>(acc[i]);
    const int e = expert_of<LPT, VEC>(lane, i);
    if ((threadIdx.x & 63) < LPT && e < p.experts) m.sum[wave][e] = acc[i];
  }
  if constexpr (LPT == 16) live += __shfl_xor(live, 16);
  if constexpr (LPT <= 32) live += __shfl_xor(live, 32);
  if ((threadIdx.x & 63) == 0) m.live[wave] = live;
  __syncthreads();
  const uint32_t n = (uint32_t)((b - a) * p.k);
  int entry = h.entry;
#pragma unroll 1
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    if ((uint32_t)entry < (uint32_t)p.experts) atomicAdd(&m.hist[entry], 1);
    entry = load_entry(p, by_k, a, i + kThreads, b);
  }
  __syncthreads();
}

template <int WAVES>
__device__ __forceinline__ float column_sum(const BalanceLds& m, int e) {
  float s = 0.0f;
#pragma unroll 4
  for (int w = 0; w < WAVES; ++w) s += m.sum[w][e];
  return s;
}
template <int WAVES>
__device__ __forceinline__ int live_sum(const BalanceLds& m) {
  int s = 0;
#pragma unroll 4
  for (int w = 0; w < WAVES; ++w) s += m.live[w];
  return s;
}

// Slope of a count and its part of the loss.
__device__ __forceinline__ double finish(const BalanceArgs& p, int64_t s, int e, int count, int64_t n, double share) {
  const double per = n > 0 ? (double)p.scale * p.experts / ((double)p.k * (double)n * (double)n) : 0.0;
  const double slope = per * count;
  p.counts[s * p.experts + e] = count;
  p.slope[s * p.experts + e] = (float)slope;
  return slope * share;
}

// Sum over the workgroup, in a fixed order; thread 0 has it.
__device__ __forceinline__ double block_sum64(double v, double* part) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += part[w];
  __syncthreads();
  return s;
}

// Few rows: a workgroup takes a whole sequence.
template <int LT, int LPT, int NE, bool VEC, int SCORE>
__global__ __launch_bounds__(kPartThreads<NE>) void balance_one_kernel(BalanceArgs p, FastDiv by_k) {
  __shared__ BalanceLds m;
  __shared__ double part[kMostWaves];
  for (int64_t s = blockIdx.x; s < p.seqs; s += gridDim.x) {
    const int64_t a = bound(p.offsets, s, p.rows), b = bound(p.offsets, s + 1, p.rows);
    constexpr int kThreads = kPartThreads<NE>;
    if (a < b) {
      Ahead<NE> h;
      load_ahead<LT, LPT, NE, VEC>(p, by_k, a, b, h);
      sum_tokens<LT, LPT, NE, VEC, SCORE>(p, by_k, a, b, h, m);
    }
    const int n = a < b ? live_sum<kThreads / 64>(m) : 0;
    double v = 0.0;
    for (int e = threadIdx.x; e < p.experts; e += kThreads)
      v += finish(p, s, e, a < b ? m.hist[e] : 0, n, a < b ? column_sum<kThreads / 64>(m, e) : 0.0f);
    v = block_sum64(v, part);
    if (threadIdx.x == 0) p.loss[s] = (float)v;
  }
}

struct BalancePieces {
  int64_t chunk, chunks;  // tokens of a chunk, chunks
  FastDiv by_chunk;
  float* sum;             // [chunks + seqs][experts]
  int32_t* count;         // the same
  int32_t* live;          // [chunks + seqs]
};

template <int LT, int LPT, int NE, bool VEC, int SCORE>
__global__ __launch_bounds__(kPartThreads<NE>) void balance_part_kernel(BalanceArgs p, FastDiv by_k, BalancePieces q) {
  __shared__ BalanceLds m;
  const int64_t c = blockIdx.x;
  const int64_t lo = c * q.chunk, hi = lo + q.chunk < p.rows ? lo + q.chunk : p.rows;
  int64_t at = lo;
  Bounds w;
  bool known = false;
  while (at < hi) {
    // (loads return in order: the bounds first; nearly every piece starts where the last one
    // ended, so that its tokens need not wait for them)
    if (!known) w = load_bounds(p.offsets, p.seqs, p.rows, at);
    Ahead<NE> h;
    load_ahead<LT, LPT, NE, VEC>(p, by_k, at, hi, h);
    const Seq f = seq_of(w, p.seqs, at);
    if (f.s >= p.seqs) {
      if (!known || w.base + 64 > p.seqs) break;
      known = false;
      continue;
    }
    known = true;
    if (f.first > at) {
      at = f.first;
      continue;
    }
    const int64_t b = f.end < hi ? f.end : hi, piece = c + f.s;
    sum_tokens<LT, LPT, NE, VEC, SCORE>(p, by_k, at, b, h, m);
    at = b;
    for (int e = threadIdx.x; e < p.experts; e += kPartThreads<NE>) {
      q.sum[piece * p.experts + e] = column_sum<kPartThreads<NE> / 64>(m, e);
      q.count[piece * p.experts + e] = m.hist[e];
    }
    if (threadIdx.x == 0) q.live[piece] = live_sum<kPartThreads<NE> / 64>(m);
    __syncthreads();  // (the next piece writes m again)
  }
}

// The pieces of a sequence, added: thread (part, e) takes W experts of every
// PARTS-th piece.
constexpr int kJoinThreads = 1024;

template <int W>
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(BalanceArgs p, BalancePieces q) {
  __shared__ double sums[kJoinThreads * W];
  __shared__ int counts[kJoinThreads * W];
  __shared__ double part[kJoinThreads / 64];
  __shared__ int lives[kJoinThreads / 64];
  const uint32_t E = p.experts, groups = E / W;
  const uint32_t shift = groups > 1 ? 32 - __builtin_clz(groups - 1) : 0, cols = 1u << shift;  // columns of threads
  // (the parts are added one after the other: not more of them than 32)
  const uint32_t parts = (kJoinThreads >> shift) < 32 ? kJoinThreads >> shift : 32;
  const uint32_t g = threadIdx.x & (cols - 1), mine = threadIdx.x >> shift;
  for (int64_t s = blockIdx.x; s < p.seqs; s += gridDim.x) {
    const uint32_t a = (uint32_t)bound(p.offsets, s, p.rows), b = (uint32_t)bound(p.offsets, s + 1, p.rows);
    // the sequence's pieces, from the one in a's chunk on
    const int64_t first = s + fast_div(a, q.by_chunk);
    const uint32_t pieces = b > a ? fast_div(b - 1, q.by_chunk) - fast_div(a, q.by_chunk) + 1 : 0;
    const float* sum = q.sum + first * E;
    const int32_t* count = q.count + first * E;
    double t[W] = {};
    int c[W] = {}, live = 0;
    if (g < groups && mine < parts) {
#pragma unroll 2
      for (uint32_t i = mine; i < pieces; i += parts) {
        const int64_t at = (int64_t)i * E + g * W;
        if constexpr (W == 4) {
          const float4 f = *reinterpret_cast<const float4*>(sum + at);
          const int4 n = *reinterpret_cast<const int4*>(count + at);
          t[0] += f.x; t[1] += f.y; t[2] += f.z; t[3] += f.w;
          c[0] += n.x; c[1] += n.y; c[2] += n.z; c[3] += n.w;
        } else {
          t[0] += sum[at];
          c[0] += count[at];
        }
      }
    }
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < pieces; i += kJoinThreads) live += q.live[first + i];
#pragma unroll
    for (int x = 0; x < W; ++x) {
      sums[((mine * W + x) << shift) + g] = t[x];
      counts[((mine * W + x) << shift) + g] = c[x];
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) live += __shfl_xor(live, k);
    if ((threadIdx.x & 63) == 0) lives[threadIdx.x >> 6] = live;
    __syncthreads();
    int64_t n = 0;
#pragma unroll 4
    for (int w = 0; w < kJoinThreads / 64; ++w) n += lives[w];
    double v = 0.0;
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < cols * W; i += kJoinThreads) {
      const uint32_t gi = i & (cols - 1), x = i >> shift;
      if (gi >= groups) continue;
      double total = 0.0;
      int all = 0;
#pragma unroll 4
      for (uint32_t r = 0; r < parts; ++r) {
        total += sums[((r * W + x) << shift) + gi];
        all += counts[((r * W + x) << shift) + gi];
      }
      v += finish(p, s, gi * W + x, all, n, total);
    }
    v = block_sum64(v, part);
    if (threadIdx.x == 0) p.loss[s] = (float)v;
  }
}

// ----------------------------------------------------------- gradient
constexpr int kGradThreads = 256;

// A wave takes `run` consecutive tokens (per lane group every kPer-th of
// them); the next token's logits and base are loaded while this one is formed.
// 16384 x 256 f32 with base: 12.1 us (50 MB, 4.2 TB/s; 16 waves per CU: with 32
// and two tokens to each 13 to 14, with 8 as many).
template <int LT, int LPT, int NE, bool VEC, int SCORE>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(BalanceGradArgs p, int64_t run) {
  constexpr int kPer = 64 / LPT;
  const int lane = threadIdx.x & (LPT - 1), E = p.experts;
  const int64_t wave = (int64_t)blockIdx.x * (kGradThreads / 64) + (threadIdx.x >> 6);
  const int64_t lo = wave * run, hi = lo + run < p.rows ? lo + run : p.rows;
  if (lo >= hi) return;
  int64_t held = -1;
  float c[NE], y[NE], base[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) c[i] = base[i] = 0.0f;
  const Bounds bounds = load_bounds(p.offsets, p.seqs, p.rows, lo);  // (loads return in order)
  int64_t t = lo + ((threadIdx.x & 63) / LPT);
  load_token<LT, LPT, NE, VEC>(p.logits, (t < hi ? t : hi - 1) * p.ldl, lane, E, y);
  if (p.base) load_token<LT, LPT, NE, VEC>(p.base, (t < hi ? t : hi - 1) * p.ldb, lane, E, base);
  const Seq f = seq_of(bounds, p.seqs, lo);
  int64_t s = f.s, first = f.first, end = f.end;
#pragma unroll 1
  for (; t < hi; t += kPer) {
    float ny[NE], nb[NE];
    const int64_t n = t + kPer < hi ? t + kPer : t;
    load_token<LT, LPT, NE, VEC>(p.logits, n * p.ldl, lane, E, ny);
    if (p.base) load_token<LT, LPT, NE, VEC>(p.base, n * p.ldb, lane, E, nb);
    if (s < p.seqs && end <= t) {
      // the first sequence behind s that ends past t
      int64_t l = s + 1, h = p.seqs;
#pragma unroll 1
      while (l < h) {
        const int64_t mid = l + ((h - l) >> 1);
        if (bound(p.offsets, mid + 1, p.rows) > t) h = mid; else l = mid + 1;
      }
      s = l;
      if (s < p.seqs) {
        first = bound(p.offsets, s, p.rows);
        end = bound(p.offsets, s + 1, p.rows);
      }
    }
    const int64_t now = s < p.seqs && first <= t ? s : p.seqs;
    if (now != held) {
      held = now;
      const float d = now < p.seqs ? p.dloss ? p.dloss[now] : 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = expert_of<LPT, VEC>(lane, i);
        c[i] = now < p.seqs && e < E ? d * p.slope[now * E + e] : 0.0f;
      }
    }
    mask_token<LPT, NE, VEC>(lane, E, y);
    float r[NE], o[NE], share[NE];
    bool live;
    const float inv = token_scores<LPT, NE, SCORE, true>(y, share, r, live);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = __builtin_fmaf(c[i], share[i], m);
    m = token_sum<LPT>(m) * inv;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      o[i] = share[i] * inv * (c[i] - m);
      if (SCORE != 0) o[i] *= r[i];
      if (p.base) o[i] += base[i];
    }
    store_token<LT, LPT, NE, VEC>(p.dl, t * p.lddl, lane, E, o);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      y[i] = ny[i];
      base[i] = nb[i];
    }
  }
}

// Whether a workgroup takes a whole sequence, in one launch: while the longest that
// the rows allow is 12 passes of the workgroup's lane groups (rows of 256
// experts: 192 in 9.7 us a call, in two launches 10.1 to 11.7; 256 in 11.8, 10.2;
// of 64 experts 700 in 8.5, 10.2 to 11.9).
bool one_launch(int64_t rows, int64_t experts) {
  const int64_t per_pass = experts <= 64 ? 1024 / 16 : experts <= 128 ? 1024 / 32 : experts <= 512 ? 1024 / 64 : 512 / 64;
  return rows <= 12 * per_pass;
}
constexpr int64_t kMostChunks = 256;
constexpr int64_t kMaxChunk = 4096;
constexpr int64_t kMaxBlocks = 1 << 20;

int64_t chunk_tokens(int64_t rows) {
  int64_t c = (rows + kMostChunks - 1) / kMostChunks;
  c = (c + 7) / 8 * 8;
  return c < 32 ? 32 : c < kMaxChunk ? c : kMaxChunk;
}

template <int LT, int LPT, int NE, bool VEC, int SCORE>
hipError_t balance_as(const BalanceArgs& a, hipStream_t st) {
  const FastDiv by_k = make_fast_div((uint32_t)a.k);
  const unsigned seqs = (unsigned)(a.seqs < kMaxBlocks ? a.seqs : kMaxBlocks);
  if (one_launch(a.rows, a.experts)) {
    hipLaunchKernelGGL((balance_one_kernel<LT, LPT, NE, VEC, SCORE>), dim3(seqs), dim3(kPartThreads<NE>), 0, st, a, by_k);
    return hipGetLastError();
  }
  BalancePieces q;
  q.chunk = chunk_tokens(a.rows);
  q.chunks = (a.rows + q.chunk - 1) / q.chunk;
  q.by_chunk = make_fast_div((uint32_t)q.chunk);
  const int64_t pieces = q.chunks + a.seqs;
  q.sum = reinterpret_cast<float*>(a.workspace);
  q.count = reinterpret_cast<int32_t*>(q.sum + pieces * a.experts);
  q.live = q.count + pieces * a.experts;
  // (at most 2^19 chunks: 2^31 rows, 4096 to each)
  hipLaunchKernelGGL((balance_part_kernel<LT, LPT, NE, VEC, SCORE>), dim3((unsigned)q.chunks), dim3(kPartThreads<NE>), 0, st, a, by_k, q);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.experts % 4 == 0)
    hipLaunchKernelGGL((balance_join_kernel<4>), dim3(seqs), dim3(kJoinThreads), 0, st, a, q);
  else
    hipLaunchKernelGGL((balance_join_kernel<1>), dim3(seqs), dim3(kJoinThreads), 0, st, a, q);
  return hipGetLastError();
}

template <int LT, int LPT, int NE, bool VEC, int SCORE>
hipError_t grad_as(const BalanceGradArgs& a, hipStream_t st) {
  constexpr int kPer = 64 / LPT;
  const int64_t waves = (int64_t)device_cu_count() * 16;
  int64_t run = (a.rows + waves - 1) / waves;
  run = (run + kPer - 1) / kPer * kPer;
  const int64_t per = run * (kGradThreads / 64);
  hipLaunchKernelGGL((balance_grad_kernel<LT, LPT, NE, VEC, SCORE>), dim3((unsigned)((a.rows + per - 1) / per)), dim3(kGradThreads),
                     0, st, a, run);
  return hipGetLastError();
}

// f.template go<LT, LPT, NE, VEC, SCORE>() by the number of experts.
template <int LT, bool VEC, int SCORE, typename F>
hipError_t by_experts(int E, F f) {
  if (E <= 64) return f.template go<LT, 16, 4, VEC, SCORE>();
  if (E <= 128) return f.template go<LT, 32, 4, VEC, SCORE>();
  if (E <= 256) return f.template go<LT, 64, 4, VEC, SCORE>();
  if (E <= 512) return f.template go<LT, 64, 8, VEC, SCORE>();
  return f.template go<LT, 64, 16, VEC, SCORE>();
}
template <int SCORE, typename F>
hipError_t by_type(int l_type, bool vec, int E, F f) {
  if (l_type == 0) return vec ? by_experts<0, true, SCORE>(E, f) : by_experts<0, false, SCORE>(E, f);
  return vec ? by_experts<1, true, SCORE>(E, f) : by_experts<1, false, SCORE>(E, f);
}
template <typename F>
hipError_t choose(int l_type, bool vec, int E, int score, F f) {
  return score == 0 ? by_type<0>(l_type, vec, E, f) : by_type<1>(l_type, vec, E, f);
}

struct GoBalance {
  const BalanceArgs& a;
  hipStream_t st;
  template <int LT, int LPT, int NE, bool VEC, int SCORE>
  hipError_t go() const { return balance_as<LT, LPT, NE, VEC, SCORE>(a, st); }
};
struct GoGrad {
  const BalanceGradArgs& a;
  hipStream_t st;
  template <int LT, int LPT, int NE, bool VEC, int SCORE>
  hipError_t go() const { return grad_as<LT, LPT, NE, VEC, SCORE>(a, st); }
};

// Whether rows of 4 elements at a time are aligned.
bool fours(const void* p, int64_t ld, int l_type) {
  return reinterpret_cast<uintptr_t>(p) % (l_type == 0 ? 8 : 16) == 0 && ld % 4 == 0;
}

}  // namespace

int64_t balance_workspace(int64_t rows, int64_t experts, int64_t seqs) {
  if (one_launch(rows, experts)) return 16;
  const int64_t chunk = chunk_tokens(rows), pieces = (rows + chunk - 1) / chunk + seqs;
  return pieces * (2 * experts + 1) * (int64_t)sizeof(float);
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
  return choose(a.l_type, a.experts % 4 == 0 && fours(a.logits, a.ldl, a.l_type), a.experts, a.score, GoBalance{a, st});
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t st) {
  const bool vec = a.experts % 4 == 0 && fours(a.logits, a.ldl, a.l_type) && fours(a.base, a.ldb, a.l_type) &&
                   fours(a.dl, a.lddl, a.l_type);
  return choose(a.l_type, vec, a.experts, a.score, GoGrad{a, st});
}

}  // namespace fp8fg
