// Routing of tokens to experts and its gradient, for gfx950.
//
// Per token with logits l over E experts (a logit of -inf, or a NaN, is a
// masked expert):
//   score   s = RN32(1 / (1 + exp(-l)))   or   RN32(softmax(l));  masked: 0
//   choice  c = s + bias in fp32;  masked: never chosen
//   groups  the experts are `groups` equal runs; a group's value is the sum
//           of its `group_top` best choices; the experts of all but the
//           `top_groups` best groups are out
//   top-k   by c, the lower index on equal values (groups likewise)
//   weight  w = scale * s, or scale * s / (sum of the chosen s); the latter for
//           softmax is scale * softmax over the chosen logits alone and is
//           formed from them: where the bias keeps the largest logits out,
//           the chosen scores may have underflowed, their shares have not
// Slots that find no expert get index -1 and weight 0.
//
// The choice is discrete, so the scores' last bits matter: they are formed
// in fp64 to about 2^-36 and rounded once, which gives the correctly rounded
// fp32 value for all but one in some thousand logits; the others are one step off,
// and choices that lie so close to another are rarer still.  A token's results
// depend neither on the other tokens nor on their number.  (gfx950 issues fp64
// FMAs at the fp32 rate.)
//
// Gradient of w with respect to l, from the logits and the indexes alone:
//   v_j = scale * dw_j;  renormalised: v_j <- (v_j - sum_i v_i s_i / S) / S
//   sigmoid: dl_j = v_j s_j (1 - s_j) for the chosen, 0 elsewhere
//   softmax: dl_e = s_e (v_e - sum_i v_i s_i); renormalised, the weights are
//            the softmax over the chosen logits alone and the rest get 0.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"

namespace fp8fg {

namespace {

constexpr int kRouteWaves = 4;

// exp(x) for -200 <= x <= 0, relative error below 2^-36: exp(x) = 2^n exp(r),
// |r| <= ln(2)/2, with the Taylor polynomial of degree 9 (remainder
// r^10/10! < 2^-37).  The coefficients come in scalar registers (as literals
// each would be moved into vector registers before its FMA).
struct ExpCoef {
  double c[7];  // 1/9! .. 1/3!
};

__device__ __forceinline__ ExpCoef exp_coef() {
  ExpCoef k = {{1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0}};
#pragma unroll
  for (int i = 0; i < 7; ++i) asm("" : "+s"(k.c[i]));
  return k;
}

__device__ __forceinline__ double exp_acc(double x, const ExpCoef& k) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -0.6931471805599453, x);
  double p = __builtin_fma(k.c[0], r, k.c[1]);
#pragma unroll
  for (int i = 2; i < 7; ++i) p = __builtin_fma(p, r, k.c[i]);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// What lies this far below the largest has score 0 in fp32 (exp(-200) is
// 2^-288), without an infinity's special cases.
constexpr float kExpFloor = -200.0f;

// RN32(1 / (1 + exp(-l))), from e = exp(-|l|) <= 1 without overflow: the
// reciprocal of 1 + e is fp32's with one Newton step in fp64 (error squared:
// 2^-44).
__device__ __forceinline__ float sigmoid_acc(float l, const ExpCoef& k) {
  const double e = exp_acc((double)fmaxf(-fabsf(l), kExpFloor), k);
  const double d = 1.0 + e;
  double y = (double)__builtin_amdgcn_rcpf((float)d);
  y = __builtin_fma(y, __builtin_fma(-d, y, 1.0), y);
  return (float)(l >= 0.0f ? y : y * e);
}

// exp(l - top) to be summed and divided by the sum; masked logits end at the
// floor (where everything is masked, at 1: no score of theirs is used).
__device__ __forceinline__ double softmax_term(float l, float top, const ExpCoef& k) {
  const double d = l == top ? 0.0 : (double)l - (double)top;
  return exp_acc(__builtin_fmax(d, (double)kExpFloor), k);
}

// A term as it enters the sum: rounded to a multiple of 2^-42, so that the
// sum of up to 1024 of them is exact in any order and the scores do not depend
// on how many lanes hold a token (which goes by the number of tokens).  The
// sum, at least 1, is off by 2^-33 at most and usually by far less.
__device__ __forceinline__ double on_grid(double term) {
  constexpr double kShift = 1536.0;  // (1.5 * 2^10: units of 2^-42 in its last place)
  return (term + kShift) - kShift;
}

// exp(l - top), a lane's part of the softmax over the chosen logits with the
// largest at `top`; 0 for a lane without one.  Within 2 units of fp32 at every
// distance: 2^t by the hardware's 2^f, f = t - rint(t), with t formed in fp64.
// (No choice hangs on it, so it needs no more bits than that.)
__device__ __forceinline__ float chosen_term(float l, bool chosen, float top) {
  const double d = l == top ? 0.0 : (double)l - (double)top;
  const double t = __builtin_fmax(d * 1.4426950408889634, (double)kExpFloor);  // (2^-200: 0 in fp32)
  const double n = __builtin_rint(t);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(t - n)), (int)n);
  return chosen ? e : 0.0f;
}

// fp32 -> unsigned whose order is the floats' (no NaN reaches it); -0 counts
// as +0.  Every key of a number is above 0, the key of "not a candidate".
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t o = __shfl_xor(v, m);
    v = o > v ? o : v;
  }
  return v;
}

// A logit as it lies in memory, and its value (NaN: masked).
template <int LT>
struct RawLogitOf {
  using type = float;
};
template <>
struct RawLogitOf<0> {
  using type = uint16_t;
};
template <int LT>
using RawLogit = typename RawLogitOf<LT>::type;

__device__ __forceinline__ float logit_value(float v) { return v == v ? v : -INFINITY; }
__device__ __forceinline__ float logit_value(uint16_t v) { return logit_value(bf16_lo(v)); }

template <int LT>
__device__ __forceinline__ float load_logit(const void* __restrict__ l, int64_t off) {
  return logit_value(reinterpret_cast<const RawLogit<LT>*>(l)[off]);
}

// ------------------------------------------------- lanes of one token
// Reductions over the LANES (32 or 64) that hold a token; every
// one of them gets the result.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);  // (every lane has a source)
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_u32<CTRL>((uint32_t)(u >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)u));
}

template <int LANES>
__device__ __forceinline__ float lanes_max_f32(float v) {
  v = pair_max<16>(row16_max(v));
  return LANES == 64 ? pair_max<32>(v) : v;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum_f32(float v) {
  v = pair_sum<16>(row16_sum(v));
  return LANES == 64 ? pair_sum<32>(v) : v;
}

template <int STEP>
__device__ __forceinline__ double pair_sum_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const LanePair lo = lane_pair<STEP>((uint32_t)u), hi = lane_pair<STEP>((uint32_t)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi.a << 32 | lo.a) + __builtin_bit_cast(double, (uint64_t)hi.b << 32 | lo.b);
}

template <int LANES>
__device__ __forceinline__ double lanes_sum_f64(double v) {
  v += dpp_f64<kDppQuadXor1>(v);
  v += dpp_f64<kDppQuadXor2>(v);
  v += dpp_f64<kDppRowHalfMirror>(v);
  v += dpp_f64<kDppRowMirror>(v);
  v = pair_sum_f64<16>(v);
  return LANES == 64 ? pair_sum_f64<32>(v) : v;
}

// (`same`: log2 of the consecutive lanes that hold equal values already.)
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int same = 0) {
  if (same < 1) v = max(v, dpp_u32<kDppQuadXor1>(v));
  if (same < 2) v = max(v, dpp_u32<kDppQuadXor2>(v));
  v = max(v, dpp_u32<kDppRowHalfMirror>(v));
  v = max(v, dpp_u32<kDppRowMirror>(v));
  LanePair p = lane_pair<16>(v);
  v = max(p.a, p.b);
  if constexpr (LANES == 64) {
    p = lane_pair<32>(v);
    v = max(p.a, p.b);
  }
  return v;
}

// The first `n` lanes from the lowest set one on, of every token's part of a
// lane mask (scalar arithmetic; n at most LANES / 2).
template <int LANES>
__device__ __forceinline__ uint64_t first_lanes(uint64_t m, int n) {
  if constexpr (LANES == 64) return m ? ((1ull << n) - 1) << __builtin_ctzll(m) : 0;
  const uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32), span = (1u << n) - 1;
  return (uint64_t)((hi & (0u - hi)) * span) << 32 | (lo & (0u - lo)) * span;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A candidate as one number: its key, then 1023 - place, so that the larger
// candidate, the lower place on equal keys, is the larger number.  As the
// bits of a double between 2 and 4 it is compared and selected by one
// v_max_f64 / v_min_f64, which this chip issues at the full rate.
__device__ __forceinline__ double pack(uint32_t key, int place) {
  const uint64_t u = (uint64_t)key << 10 | (uint32_t)(1023 - place);
  return __builtin_bit_cast(double, u | 0x4000000000000000ull);
}
constexpr double kNoPack = 2.0;  // below every candidate; its key is 0
__device__ __forceinline__ int pack_place(double v) {
  return 1023 - (int)((uint32_t)__builtin_bit_cast(uint64_t, v) & 1023u);
}
__device__ __forceinline__ uint32_t pack_key(double v) {
  return (uint32_t)(__builtin_bit_cast(uint64_t, v) >> 10);
}

// The two largest of two disjoint sets' two largest (a >= b).
__device__ __forceinline__ void merge_top2(double& a, double& b, double oa, double ob) {
  b = __builtin_fmax(__builtin_fmin(a, oa), __builtin_fmax(b, ob));
  a = __builtin_fmax(a, oa);
}

__device__ __forceinline__ void order2(double& a, double& b) {
  const double x = __builtin_fmax(a, b);
  b = __builtin_fmin(a, b);
  a = x;
}

// How the experts lie in a token's lanes: each group has `lanes` consecutive
// lanes (a power of two), each of which has `slots` consecutive experts of
// the group.  The lower expert is in the lower lane, then the lower slot:
// place = lane * NS + slot orders candidates as their indexes do.
struct RouteLayout {
  int groups;  // 1 where groups play no part
  int size;    // experts per group
  int lanes;   // log2
  int slots;
  int vec;     // every lane's experts are NS whole ones, aligned: 16-byte loads
};

// The NS values from e0 on of a row of E (past its end the last ones: loads
// without branches, all in flight).
template <typename T, int NS>
__device__ __forceinline__ void load_slots(const T* __restrict__ row, int e0, int E, int vec, T (&v)[NS]) {
  if (vec && NS * sizeof(T) >= 16) {
    struct alignas(16) Run {
      T v[NS];
    };
    const Run r = *reinterpret_cast<const Run*>(row + min(e0, E - NS));
#pragma unroll
    for (int s = 0; s < NS; ++s) v[s] = r.v[s];
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) v[s] = row[min(e0 + s, E - 1)];
  }
}

// LANES lanes per token, NS >= slots experts per lane in registers, as NS / 4
// descending lists of 4: an expert that is taken only moves up the list that
// it heads.  A step of the selection is a maximum over the lists' heads and
// the lanes (32-bit keys, by DPP and row swaps), a ballot, and scalar
// arithmetic for the lowest lane that has it.
//
// Bound by instruction issue: 790 vector instructions a wave, some 200 of them
// the scores; the vector units issue in 86% of the busy cycles (counters).
// 16384 x 256, 8 of 256 in 4 of 8 groups, f32: 13.3 us with two tokens to a wave
// (the logits' bytes at a device copy's rate: 3.5), softmax 14.4; 25.7 with one,
// 22 with four (16 experts to a lane: too few waves to hide the loads).
// 5 x 256: 3.8 us.
template <int LT, int LANES, int NS, int SCORE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p, RouteLayout q) {
  constexpr int kTokens = 64 / LANES;  // of a wave
  constexpr int NL = NS / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LANES;
  const int E = p.experts;
  const int group = sub >> q.lanes;
  const int in_group = (sub - (group << q.lanes)) * q.slots;
  const int e0 = group * q.size + in_group;
  const int n = group < q.groups ? min(q.slots, q.size - in_group) : 0;  // this lane's experts (<= 0: none)
  const ExpCoef coef = exp_coef();
  __shared__ float scores[kRouteWaves][64 * NS];  // softmax: the logits
  __shared__ int picks[kRouteWaves][64];
  float* mine = scores[wave] + (lane / LANES) * LANES * NS;
  float bias[NS];
  if (p.bias) load_slots<float, NS>(p.bias, e0, E, q.vec, bias);

  for (int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * kTokens; t0 < p.rows;
       t0 += (int64_t)gridDim.x * kRouteWaves * kTokens) {
    // (lanes without experts or token read the last one's)
    const int64_t t = t0 + lane / LANES;
    const int64_t row = min(t, p.rows - 1) * p.ldl;
    RawLogit<LT> in[NS];
    load_slots<RawLogit<LT>, NS>(reinterpret_cast<const RawLogit<LT>*>(p.logits) + row, e0, E, q.vec, in);
    float l[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) l[s] = s < n ? logit_value(in[s]) : -INFINITY;

    float top = -INFINITY;
    double inv = 0.0;
    double c[NL][4];  // softmax: the terms, until the scores replace them
    if constexpr (SCORE == 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        mine[sub * NS + s] = l[s];
        top = fmaxf(top, l[s]);
      }
      top = lanes_max_f32<LANES>(top);
      double sum = 0.0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        c[s / 4][s % 4] = softmax_term(l[s], top, coef);
        sum += s < n ? on_grid(c[s / 4][s % 4]) : 0.0;
      }
      inv = 1.0 / lanes_sum_f64<LANES>(sum);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float sc = SCORE == 0 ? (float)(c[s / 4][s % 4] * inv) : sigmoid_acc(l[s], coef);
      const float v = p.bias ? sc + bias[s] : sc;
      const bool live = l[s] > -INFINITY && v > -INFINITY;  // (a NaN compares false)
      if constexpr (SCORE == 1) mine[sub * NS + s] = sc;
      c[s / 4][s % 4] = live ? pack(order_key(v), sub * NS + s) : kNoPack;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {  // a sorting network for 4
      order2(c[i][0], c[i][1]);
      order2(c[i][2], c[i][3]);
      order2(c[i][0], c[i][2]);
      order2(c[i][1], c[i][3]);
      order2(c[i][1], c[i][2]);
    }

    if (q.groups > 1) {
      double a = c[0][0], b = c[0][1];
#pragma unroll
      for (int i = 1; i < NL; ++i) merge_top2(a, b, c[i][0], c[i][1]);
      if (q.lanes > 0) merge_top2(a, b, dpp_f64<kDppQuadXor1>(a), dpp_f64<kDppQuadXor1>(b));
      if (q.lanes > 1) merge_top2(a, b, dpp_f64<kDppQuadXor2>(a), dpp_f64<kDppQuadXor2>(b));
      if (q.lanes > 2) merge_top2(a, b, dpp_f64<kDppRowHalfMirror>(a), dpp_f64<kDppRowHalfMirror>(b));
      if (q.lanes > 3) merge_top2(a, b, dpp_f64<kDppRowMirror>(a), dpp_f64<kDppRowMirror>(b));
      if constexpr (LANES == 64) {
        if (q.lanes > 4) merge_top2(a, b, __shfl_xor(a, 16), __shfl_xor(b, 16));
      }
      // (0: no candidate; where nothing else is left, such groups are kept)
      uint32_t g = p.group_top > 1 && b != kNoPack ? order_key(key_value(pack_key(a)) + key_value(pack_key(b))) : pack_key(a);
      uint64_t keep = 0;
      for (int r = 0; r < p.top_groups; ++r) {
        const uint32_t best = lanes_max<LANES>(g, q.lanes);
        const uint64_t won = first_lanes<LANES>(__builtin_amdgcn_ballot_w64(g == best), 1 << q.lanes);
        keep |= won;
        g = __builtin_amdgcn_inverse_ballot_w64(won) ? 0u : g;
      }
      if (!__builtin_amdgcn_inverse_ballot_w64(keep)) {
#pragma unroll
        for (int i = 0; i < NL; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = kNoPack;
        asm volatile("" : "+v"(c[0][0]));
      }
    }

    picks[wave][lane] = -1;
    wave_fence();
    for (int j = 0; j < p.k; ++j) {
      uint32_t head = pack_key(c[0][0]);
#pragma unroll
      for (int i = 1; i < NL; ++i) head = max(head, pack_key(c[i][0]));
      const uint32_t best = lanes_max<LANES>(head);
      // the lowest lane that has it, and there the first list (lower places)
      bool mine_now = __builtin_amdgcn_inverse_ballot_w64(first_lanes<LANES>(__builtin_amdgcn_ballot_w64(head == best), 1));
      mine_now = mine_now && best != 0;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        if (mine_now && pack_key(c[i][0]) == best) {
          picks[wave][(lane & ~(LANES - 1)) + j] = pack_place(c[i][0]);
          c[i][0] = c[i][1];
          c[i][1] = c[i][2];
          c[i][2] = c[i][3];
          c[i][3] = kNoPack;
          mine_now = false;
          asm volatile("" : "+v"(c[i][0]));  // moves under the lanes' mask, no selects
        }
      }
    }
    wave_fence();
    int at = sub < p.k ? picks[wave][lane] : -1;  // lane j of the token: the place of its j-th expert
    float s = 0.0f;
    if (at >= 0) {
      s = mine[at];
      const int from = at / NS;
      at = (from >> q.lanes) * q.size + (from & ((1 << q.lanes) - 1)) * q.slots + at % NS;
    }
    if constexpr (SCORE == 0) {  // from the chosen logits; unnormalised, the score once more
      if (p.renorm)
        s = chosen_term(s, at >= 0, lanes_max_f32<LANES>(at >= 0 ? s : -INFINITY));
      else
        s = at >= 0 ? (float)(softmax_term(s, top, coef) * inv) : 0.0f;
    }
    const float sum = lanes_sum_f32<LANES>(s);
    if (t < p.rows && sub < p.k) {
      p.idx[t * p.ld_idx + sub] = at;
      p.w[t * p.ldw + sub] = p.renorm ? (sum > 0.0f ? s / sum * p.scale : 0.0f) : s * p.scale;
    }
    wave_fence();  // the scores' places are free for the next tokens
  }
}

// Any number of groups: one wave per token, lane i holds the experts i,
// i + 64, ..; group values are formed from LDS.  For what route_kernel's
// layout does not fit (more than 64 groups, or over 16 experts to a lane).
template <int LT, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_any_kernel(RouteArgs p) {
  __shared__ float cbuf[kRouteWaves][64 * NE];
  __shared__ float sbuf[kRouteWaves][64 * NE];
  const ExpCoef coef = exp_coef();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.experts;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < p.rows; t += (int64_t)gridDim.x * kRouteWaves) {
    float s[NE], c[NE];
    float l[NE], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < E ? load_logit<LT>(p.logits, t * p.ldl + e) : -INFINITY;
      top = fmaxf(top, l[i]);
    }
    if (p.score == 0) {
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
      double ex[NE], sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        ex[i] = softmax_term(l[i], top, coef);
        sum += lane + 64 * i < E ? on_grid(ex[i]) : 0.0;
      }
      const double inv = 1.0 / lanes_sum_f64<64>(sum);
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = (float)(ex[i] * inv);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = sigmoid_acc(l[i], coef);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      c[i] = s[i];
      if (p.bias && e < E) c[i] += p.bias[e];
      if (!(l[i] > -INFINITY) || !(c[i] == c[i])) c[i] = -INFINITY;
      cbuf[wave][e] = c[i];
      sbuf[wave][e] = p.score == 0 && p.renorm ? l[i] : s[i];  // what the weights are formed from
    }
    wave_fence();

    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = c[i] > -INFINITY ? order_key(c[i]) : 0u;
    if (p.top_groups < p.groups) {
      const int size = E / p.groups;
      // group values, lane g holding the groups g, g + 64, ..
      uint64_t gk[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int g = lane + 64 * i;
        gk[i] = 0;
        if (g >= p.groups) continue;
        float a = -INFINITY, b = -INFINITY;
        for (int e = g * size; e < (g + 1) * size; ++e) {
          const float v = cbuf[wave][e];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
        if (a == -INFINITY) continue;
        const float v = p.group_top > 1 && b > -INFINITY ? a + b : a;
        gk[i] = (uint64_t)order_key(v) << 32 | (uint32_t)~g;
      }
      bool keep[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) keep[i] = false;
      for (int r = 0; r < p.top_groups; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) best = gk[i] > best ? gk[i] : best;
        best = wave_max64(best);
        if (best == 0) break;
        const int g = (int)~(uint32_t)best;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          if (lane + 64 * i == g) gk[i] = 0;
          keep[i] = keep[i] || (lane + 64 * i) / size == g;
        }
      }
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (!keep[i]) key[i] = 0u;
    }

    float sum = 0.0f, mine = 0.0f;
    int at = -1;
    for (int j = 0; j < p.k; ++j) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const uint64_t v = key[i] ? (uint64_t)key[i] << 32 | (uint32_t)~(lane + 64 * i) : 0;
        best = v > best ? v : best;
      }
      best = wave_max64(best);
      if (best == 0) break;
      const int e = (int)~(uint32_t)best;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i == e) key[i] = 0;
      const float v = sbuf[wave][e];
      sum += v;
      if (lane == j) {
        at = e;
        mine = v;
      }
    }
    if (p.score == 0 && p.renorm) {
      mine = chosen_term(mine, at >= 0, lanes_max_f32<64>(at >= 0 ? mine : -INFINITY));
      sum = lanes_sum_f32<64>(mine);
    }
    if (lane < p.k) {
      p.idx[t * p.ld_idx + lane] = at;
      p.w[t * p.ldw + lane] = p.renorm ? (sum > 0.0f ? mine / sum * p.scale : 0.0f) : mine * p.scale;
    }
    wave_fence();  // the buffers are free for the next token
  }
}

// exp(x) for x <= 0 by the hardware's 2^t, t = x log2(e) with the product's
// rounding error and the constant's made good to first order: within 2 ulp
// down to 2^-126, 0 below.
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -120.0f);
  const float t = x * 1.44269502f;                                    // RN32(log2 e)
  const float e = __builtin_fmaf(x, 1.44269502f, -t) + x * 1.92596299e-8f;  // log2 e - RN32(log2 e)
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, e * 0.693147181f, p);
}

// exp(l - top), 0 for a masked logit, 1 at the top (also where both are
// +inf).
__device__ __forceinline__ float exp_below(float l, float top) {
  const float e = exp_neg(l == top ? 0.0f : l - top);
  return l == -INFINITY ? 0.0f : e;
}

// One wave per token: lane j < k has the j-th chosen expert, and lane i the
// logits (where the gradient is dense) and gradients i, i + 64, ..  Only the
// dense form reads a whole row.  Bound by instruction issue (341 vector
// instructions a token; 89% of the busy cycles): 8191 x 160 bf16, dense: 6.0 us
// (its bytes at a device copy's rate: 1.1; a smallest kernel 3.8).
template <int LT, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_grad_kernel(RouteGradArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.experts;
  const bool dense = p.score == 0 && !p.renorm;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < p.rows; t += (int64_t)gridDim.x * kRouteWaves) {
    RawLogit<LT> in[NE];
    float y[NE];
    if (dense) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        in[i] = reinterpret_cast<const RawLogit<LT>*>(p.logits)[t * p.ldl + min(lane + 64 * i, E - 1)];
    }
    float l = -INFINITY, v = 0.0f, top = -INFINITY, total = 0.0f, dot = 0.0f;
    int e = -1;
    if (lane < p.k) {
      e = p.idx[t * p.ld_idx + lane];
      if ((uint32_t)e < (uint32_t)E) {
        l = load_logit<LT>(p.logits, t * p.ldl + e);
        v = p.scale * p.dw[t * p.lddw + lane];
      } else {
        e = -1;
      }
    }
    if (p.score == 0) {
      top = l;
      if (dense) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          y[i] = lane + 64 * i < E ? logit_value(in[i]) : -INFINITY;
          top = fmaxf(top, y[i]);
        }
      }
      top = lanes_max_f32<64>(top);
      float s = exp_below(l, top);
      total = s;
      if (dense) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          y[i] = exp_below(y[i], top);
          total += y[i];
        }
      }
      total = wave_sum(total);
      s = total > 0.0f ? s / total : 0.0f;
      dot = wave_sum(v * s);
      if (!dense) v = s * (v - dot);
    } else {
      const float e1 = expf(-fabsf(l));  // (a masked logit: 0; denormals count, shares are quotients)
      const float s = (l >= 0.0f ? 1.0f : e1) / (1.0f + e1);
      float share = s;  // s_j / S when renormalised
      if (p.renorm) {
        total = wave_sum(s);
        share = total > 0.0f ? s / total : 0.0f;
        v -= wave_sum(v * share);
      }
      v = v * share * ((l >= 0.0f ? e1 : 1.0f) / (1.0f + e1));  // 1 - s without cancellation
    }
    float d[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) d[i] = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] = lane + 64 * i == ej ? vj : d[i];
    }
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int x = lane + 64 * i;
      if (x >= E) continue;
      if (dense) d[i] = y[i] * inv * (d[i] - dot);
      if constexpr (LT == 0)
        reinterpret_cast<uint16_t*>(p.dl)[t * p.lddl + x] = (uint16_t)pack2_bf16(d[i], 0.0f);
      else
        reinterpret_cast<float*>(p.dl)[t * p.lddl + x] = d[i];
    }
  }
}

constexpr int64_t kMaxRouteBlocks = 1 << 20;

unsigned route_blocks(int64_t rows, int tokens_per_wave) {
  const int64_t per = (int64_t)kRouteWaves * tokens_per_wave;
  const int64_t n = (rows + per - 1) / per;
  return (unsigned)(n < kMaxRouteBlocks ? n : kMaxRouteBlocks);
}

// The layout over `lanes` lanes; slots = 0 where there is none.
RouteLayout route_layout(const RouteArgs& a, int lanes) {
  RouteLayout q{a.top_groups < a.groups ? a.groups : 1, 0, 0, 0, 0};
  q.size = a.experts / q.groups;
  if (q.groups > lanes) return q;
  while ((q.groups << (q.lanes + 1)) <= lanes) ++q.lanes;
  q.slots = (q.size + (1 << q.lanes) - 1) >> q.lanes;
  return q;
}

template <int LT, int LANES, int NS>
hipError_t route_as(const RouteArgs& a, const RouteLayout& q, hipStream_t st) {
  RouteLayout l = q;
  constexpr int kPer16 = LT == 0 ? 8 : 4;
  l.vec = NS % kPer16 == 0 && q.slots == NS && q.size % NS == 0 && a.ldl % kPer16 == 0 &&
          reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  const dim3 grid(route_blocks(a.rows, 64 / LANES)), block(64 * kRouteWaves);
  if (a.score == 0)
    hipLaunchKernelGGL((route_kernel<LT, LANES, NS, 0>), grid, block, 0, st, a, l);
  else
    hipLaunchKernelGGL((route_kernel<LT, LANES, NS, 1>), grid, block, 0, st, a, l);
  return hipGetLastError();
}

// From this many tokens on, two to a wave: fewer instructions per token, but
// a longer chain of them (8 of 256 experts, 2048 tokens: 5.1 us, one to a wave
// 4.8; 4096: 6.0 and 6.5; 8192: 8.4 and 9.8).
constexpr int64_t kRouteManyRows = 2560;

template <int LT>
hipError_t route_t(const RouteArgs& a, hipStream_t st) {
  if (a.rows >= kRouteManyRows && a.k <= 32) {
    const RouteLayout q = route_layout(a, 32);
    if (q.slots > 0 && q.slots <= 8) return route_as<LT, 32, 8>(a, q, st);
  }
  const RouteLayout q = route_layout(a, 64);
  if (q.slots > 0 && q.slots <= 4) return route_as<LT, 64, 4>(a, q, st);
  if (q.slots > 0 && q.slots <= 8) return route_as<LT, 64, 8>(a, q, st);
  if (q.slots > 0 && q.slots <= 16) return route_as<LT, 64, 16>(a, q, st);
  hipLaunchKernelGGL((route_any_kernel<LT, kRouteMaxExperts / 64>), dim3(route_blocks(a.rows, 1)),
                     dim3(64 * kRouteWaves), 0, st, a);
  return hipGetLastError();
}

template <int LT>
hipError_t route_grad_t(const RouteGradArgs& a, hipStream_t st) {
  const dim3 grid(route_blocks(a.rows, 1)), block(64 * kRouteWaves);
  if (a.experts <= 256)
    hipLaunchKernelGGL((route_grad_kernel<LT, 4>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((route_grad_kernel<LT, kRouteMaxExperts / 64>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  return a.l_type == 0 ? route_t<0>(a, st) : route_t<1>(a, st);
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t st) {
  return a.l_type == 0 ? route_grad_t<0>(a, st) : route_grad_t<1>(a, st);
}

}  // namespace fp8fg
