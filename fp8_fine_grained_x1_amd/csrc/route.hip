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
//   weight  w = scale * s, or scale * s / (sum of the chosen s)
// Slots that find no expert get index -1 and weight 0.
//
// The choice is discrete, so the scores' last bits matter: they are formed
// in fp64 to about 2^-40 and rounded once, which gives the correctly rounded
// fp32 value for all but a few of a million logits.  (gfx950 issues fp64
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

// exp(x) for x <= 709, relative error below 2^-41: exp(x) = 2^n exp(r),
// |r| <= ln(2)/2, with the Taylor polynomial of degree 11 (remainder
// r^12/12! < 2^-47 of the sum).
__device__ __forceinline__ double exp_acc(double x) {
  if (x < -745.0) return 0.0;
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -0.6931471805599453, x);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
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

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <int LT>
__device__ __forceinline__ float load_logit(const void* __restrict__ l, int64_t off) {
  float v;
  if constexpr (LT == 0)
    v = bf16_lo(reinterpret_cast<const uint16_t*>(l)[off]);
  else
    v = reinterpret_cast<const float*>(l)[off];
  return v == v ? v : -INFINITY;
}

// One wave per token; lane i holds the experts i, i + 64, ..
template <int LT, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
  __shared__ float cbuf[kRouteWaves][64 * NE];
  __shared__ float sbuf[kRouteWaves][64 * NE];
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
        ex[i] = l[i] == -INFINITY ? 0.0 : l[i] == top ? 1.0 : exp_acc((double)l[i] - (double)top);
        sum += ex[i];
      }
      sum = wave_sum64(sum);
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = sum > 0.0 ? (float)(ex[i] / sum) : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = l[i] < -700.0f ? 0.0f : (float)(1.0 / (1.0 + exp_acc(-(double)l[i])));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      c[i] = s[i];
      if (p.bias && e < E) c[i] += p.bias[e];
      if (!(l[i] > -INFINITY) || !(c[i] == c[i])) c[i] = -INFINITY;
      cbuf[wave][e] = c[i];
      sbuf[wave][e] = s[i];
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
    if (lane < p.k) {
      p.idx[t * p.ld_idx + lane] = at;
      p.w[t * p.ldw + lane] = p.renorm ? (sum > 0.0f ? mine / sum * p.scale : 0.0f) : mine * p.scale;
    }
    wave_fence();  // the buffers are free for the next token
  }
}

// exp(l - top), 0 for a masked logit, 1 at the top (also where both are
// +inf).
__device__ __forceinline__ float exp_below(float l, float top) {
  return l == -INFINITY ? 0.0f : l == top ? 1.0f : expf(l - top);
}

// One wave per token.  Lane j < k holds the j-th chosen expert.
template <int LT>
__global__ __launch_bounds__(64 * kRouteWaves) void route_grad_kernel(RouteGradArgs p) {
  __shared__ float vbuf[kRouteWaves][kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.experts;
  const bool dense = p.score == 0 && !p.renorm;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < p.rows; t += (int64_t)gridDim.x * kRouteWaves) {
    float top = -INFINITY, total = 0.0f, s = 0.0f, v = 0.0f, dot = 0.0f;
    int e = -1;
    for (int x = lane; x < E; x += 64) vbuf[wave][x] = 0.0f;
    float l = -INFINITY;
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
      if (dense)
        for (int x = lane; x < E; x += 64) top = fmaxf(top, load_logit<LT>(p.logits, t * p.ldl + x));
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
      s = exp_below(l, top);
      total = s;
      if (dense) {
        total = 0.0f;
        for (int x = lane; x < E; x += 64) total += exp_below(load_logit<LT>(p.logits, t * p.ldl + x), top);
      }
      total = wave_sum(total);
      s = total > 0.0f ? s / total : 0.0f;
      dot = wave_sum(v * s);
      if (!dense) v = s * (v - dot);
    } else {
      s = l == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(-l));
      float share = s;  // s_j / S when renormalised
      if (p.renorm) {
        total = wave_sum(s);
        share = total > 0.0f ? s / total : 0.0f;
        v -= wave_sum(v * share);
      }
      v = v * share * (1.0f - s);
    }
    wave_fence();
    if (e >= 0) vbuf[wave][e] = v;
    wave_fence();
    for (int x = lane; x < E; x += 64) {
      float d = vbuf[wave][x];
      if (dense) {
        const float y = exp_below(load_logit<LT>(p.logits, t * p.ldl + x), top);
        d = total > 0.0f ? y / total * (d - dot) : 0.0f;
      }
      if constexpr (LT == 0)
        reinterpret_cast<uint16_t*>(p.dl)[t * p.lddl + x] = (uint16_t)pack2_bf16(d, 0.0f);
      else
        reinterpret_cast<float*>(p.dl)[t * p.lddl + x] = d;
    }
    wave_fence();
  }
}

constexpr int64_t kMaxRouteBlocks = 1 << 20;

int64_t token_blocks(int64_t rows) {
  const int64_t n = (rows + kRouteWaves - 1) / kRouteWaves;
  return n < kMaxRouteBlocks ? n : kMaxRouteBlocks;
}

template <int LT>
hipError_t route_t(const RouteArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)token_blocks(a.rows)), block(64 * kRouteWaves);
  if (a.experts <= 64)
    hipLaunchKernelGGL((route_kernel<LT, 1>), grid, block, 0, st, a);
  else if (a.experts <= 128)
    hipLaunchKernelGGL((route_kernel<LT, 2>), grid, block, 0, st, a);
  else if (a.experts <= 256)
    hipLaunchKernelGGL((route_kernel<LT, 4>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((route_kernel<LT, 16>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  return a.l_type == 0 ? route_t<0>(a, st) : route_t<1>(a, st);
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)token_blocks(a.rows)), block(64 * kRouteWaves);
  if (a.l_type == 0)
    hipLaunchKernelGGL(route_grad_kernel<0>, grid, block, 0, st, a);
  else
    hipLaunchKernelGGL(route_grad_kernel<1>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace fp8fg
