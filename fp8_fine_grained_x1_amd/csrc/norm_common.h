// Helpers shared by the kernels that hold a row in one workgroup's registers
// (norm.hip, block_norm.hip).
#pragma once

#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace fp8fg {

namespace {

constexpr int kMaxWaves = 16;

// Sum over the workgroup's waves (at most 16); every thread gets the result,
// the waves' sums added by a row of 16 lanes.  `part` may be written again
// after the next call's barrier: callers alternate between two of them.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  const int i = threadIdx.x & 15;
  return row16_sum(i < waves ? part[i] : 0.0f);
}

// gamma's elements N v .. N v + N - 1, undecoded.
template <int N>
struct RawGamma {
  uint4 a, b;
};

template <int N>
__device__ __forceinline__ RawGamma<N> load_gamma(const void* __restrict__ g, int g_type, int v) {
  RawGamma<N> r = {};
  if (g_type == 0) {
    if constexpr (N == 8) {
      r.a = reinterpret_cast<const uint4*>(g)[v];
    } else {
      const uint2 h = reinterpret_cast<const uint2*>(g)[v];
      r.a.x = h.x;
      r.a.y = h.y;
    }
  } else {
    r.a = reinterpret_cast<const uint4*>(g)[N / 4 * v];
    if constexpr (N == 8) r.b = reinterpret_cast<const uint4*>(g)[2 * v + 1];
  }
  return r;
}

template <int N>
__device__ __forceinline__ void decode_gamma(const RawGamma<N>& r, int g_type, float (&v)[N]) {
  if (g_type == 0) {
    v[0] = bf16_lo(r.a.x); v[1] = bf16_hi(r.a.x);
    v[2] = bf16_lo(r.a.y); v[3] = bf16_hi(r.a.y);
    if constexpr (N == 8) {
      v[4] = bf16_lo(r.a.z); v[5] = bf16_hi(r.a.z);
      v[6] = bf16_lo(r.a.w); v[7] = bf16_hi(r.a.w);
    }
  } else {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    if constexpr (N == 8) {
      v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
      v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
    }
  }
}

// Means of squares (with eps) from here to the largest fp32 number come from
// fp32 sums: below it squares that fp32 rounds to subnormal numbers (each off
// by 2^-150 at most, 2^15 of them) could count, above it the sum overflows
// (elements of 2e17 in 7168 columns).
constexpr float kLeastMean = 0x1p-100f;

// rstd of a row beyond that range, whose squares are summed in fp64 (2^-298
// to 2^256 hold those of every number): rare, and never with ordinary eps
// and values.  A row of zeros with eps 0 gets 0: its y is 0 and no gradient
// passes.  Every thread of the workgroup takes part.
template <int XT, int NV>
__device__ __forceinline__ float wide_range_rstd(const Raw8<XT> (&raw)[NV], int nvec, int64_t cols, float eps, double* part) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((int)(threadIdx.x + i * blockDim.x) >= nvec) continue;
    float f[8];
    decode8<XT>(raw[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)f[e] * (double)f[e];
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) sum += part[w];
  __syncthreads();  // (the next such row writes them again)
  const double m = sum / (double)cols + (double)eps;
  const double r = m == 0.0 ? 0.0 : 1.0 / sqrt(m);
  return (float)(r > (double)FLT_MAX ? (double)FLT_MAX : r);
}

template <int XT, int N>
struct Unit {  // N elements, undecoded
  uint4 w[N / kPer16<XT>];
};

// Unit v of the row that starts `row` elements in.
template <int XT, bool NT, int N>
__device__ __forceinline__ Unit<XT, N> load_unit(const void* __restrict__ p, int64_t row, uint32_t v) {
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + row * (XT == 0 ? 2 : 4));
  Unit<XT, N> u;
#pragma unroll
  for (int i = 0; i < N / kPer16<XT>; ++i) u.w[i] = NT ? ld_nt16(q + v * (N / kPer16<XT>) + i) : q[v * (N / kPer16<XT>) + i];
  return u;
}
template <int XT, int N>
__device__ __forceinline__ void store_unit(void* __restrict__ p, int64_t row, uint32_t v, const float (&x)[N]) {
  constexpr int M = kPer16<XT>;
  uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<char*>(p) + row * (XT == 0 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < N / M; ++i) {
    float f[M];
#pragma unroll
    for (int e = 0; e < M; ++e) f[e] = x[i * M + e];
    q[v * (N / M) + i] = encode16<XT>(f);
  }
}
template <int XT, int N>
__device__ __forceinline__ void decode_unit(const Unit<XT, N>& u, float (&v)[N]) {
  constexpr int M = kPer16<XT>;
#pragma unroll
  for (int i = 0; i < N / M; ++i) {
    float f[M];
    decode16<XT>(u.w[i], f);
#pragma unroll
    for (int e = 0; e < M; ++e) v[i * M + e] = f[e];
  }
}

constexpr int64_t kMaxRowBlocks = 1 << 20;

// Elements (8 `per` thread) and threads of a workgroup for a row: at most 512
// threads, whose register budget holds a row of up to 16384 elements, and
// 1024 beyond.  The columns alone decide, and with them the order of a row's
// additions: its results do not depend on the other rows.
struct RowShape {
  int per, threads;
};
inline RowShape row_shape(int64_t cols) {
  const int64_t groups = cols / 8;
  const int per = groups <= 512 ? 1 : groups <= 1024 ? 2 : 4;
  const int64_t t = (groups + per - 1) / per;
  return {per, (int)((t + 63) / 64 * 64)};
}

}  // namespace

}  // namespace fp8fg
