// Root-mean-square norm with the residual's addition and an E4M3 output with
// 1x128 scales, and its gradient, for gfx950.
//
// Forward, per row:  h = RN(x + r) in x's type,  rstd = 1 / sqrt(mean(h^2) + eps)
//   (0 for a row of zeros with eps 0, at most the largest fp32 number),
//   y = (h * rstd) * gamma in fp32;  per 1x128 tile the quantizers' scale
//   s = max(amax |y| / 448, 2^-126) (or its power of two) and
//   q = E4M3(RN32(y / s)).  y is rounded once into each output: q comes from
//   the fp32 value, not from the stored y.  The norm is taken of the rounded
//   h, so that the gradient, which reads h, differentiates what was computed.
// Backward:  xh = h * rstd,  a = dy * gamma,
//   dx = rstd * (a - xh * mean(a * xh)) + dh,  dgamma = sum over rows dy * xh.
//   (The quantizer is passed straight through; dh is the gradient that
//   reaches h along the residual stream.)
//
// Both are bound by HBM: a row's elements are read once and stay in
// registers, undecoded, between the statistics and the outputs.  Of the
// outputs y, or h where there is no y, and dx are stored ordinarily and may
// stay in the caches for what reads them next, the others pass them by;
// measured on 8192 x 7168 bf16 with every output: 90 us (5.9 TB/s), all
// ordinary 99.5, all non-temporal 95.  (q, too, passes them by: ordinary stores
// of it cost the norm itself 7.8 us instead of 7.3 on 1111 x 5120 f32 and 97
// instead of 90 here, though a dispatch right after it gains more than that
// while its rows fit the caches.)  The gradient takes 85 us, 7 of them dgamma's
// strips (5.5 TB/s); dx non-temporal 90, dy read ordinarily 93.  A large device
// copy moves 5.1 TB/s on this card.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"

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

// One row per workgroup iteration; thread t holds the 8-element vectors
// t, t + blockDim, ..: 16 consecutive lanes hold one 1x128 tile.  (For f32, 16
// bytes a lane and tiles of 32 lanes form every scale in twice the lanes and
// take more registers: 1111 x 5120 11.4 us instead of 8.6.)
//
// STREAM: x and r pass the caches by.  On inputs that fit the caches, where
// their producer left them, that costs (bf16 of 7168 columns with r, 117 MB of
// inputs: 51.3 us; 44.6 with ordinary reads), on larger ones it gains (143 MB:
// 60.3; 66.3).  The ordinary form also loads gamma before the reduction, which
// shortens its chain (2048 rows: 24.2 -> 23.1 us, one row 4.2 -> 3.8); the
// streams want those registers (8192 rows: 98 us instead of 93), as do the
// widest rows.
template <int XT, int NV, bool STREAM, bool WITH_Y>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs p) {
  constexpr bool AHEAD = !STREAM && NV <= 2;
  __shared__ float part[2][kMaxWaves];
  __shared__ double wide[kMaxWaves];
  const int nvec = (int)(p.cols >> 3);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    Raw8<XT> raw[NV];
    RawGamma<8> gamma[NV];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      raw[i] = load_raw8<XT, STREAM>(p.x, row * p.ldx + v * 8);
      if (AHEAD) gamma[i] = load_gamma<8>(p.gamma, p.g_type, v);
      if (p.r) {
        float a[8], b[8];
        decode8<XT>(raw[i], a);
        decode8<XT>(load_raw8<XT, STREAM>(p.r, row * p.ldr + v * 8), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
        raw[i] = encode8<XT>(a);
      }
      if (p.h) store_raw8<XT, WITH_Y && STREAM>(p.h, row * p.ldh + v * 8, raw[i]);
      float f[8];
      decode8<XT>(raw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
    }
    ss = block_sum(ss, part[flip]);
    const float mean = ss / (float)p.cols + p.eps;
    float rstd = 1.0f / sqrtf(mean);
    if (__builtin_expect(!(mean >= kLeastMean && mean <= FLT_MAX), 0))
      rstd = wide_range_rstd<XT, NV>(raw, nvec, p.cols, p.eps, wide);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    if (!p.q && !WITH_Y) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float f[8], g[8];
      decode8<XT>(raw[i], f);
      decode_gamma<8>(AHEAD ? gamma[i] : load_gamma<8>(p.gamma, p.g_type, v), p.g_type, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[e];
      if constexpr (WITH_Y) store_raw8<XT, false>(p.y, row * p.ldy + v * 8, encode8<XT>(f));
      if (p.q) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
        m = row16_max(m);
        TileScale sc;
        if (p.rule == 0) {
          sc = scale_amax(m);
          quotient8<0>(f, sc);
        } else {
          sc = scale_pow2(m);
          quotient8<1>(f, sc);
        }
        uint2 out;
        out.x = pack4_e4m3(f[0], f[1], f[2], f[3]);
        out.y = pack4_e4m3(f[4], f[5], f[6], f[7]);
        st_nt8(p.q + row * p.ldq + v * 8, out);
        if ((threadIdx.x & 15) == 0) p.s[row * p.s_rs + (int64_t)(v >> 4) * p.s_ts] = sc.s;
      }
    }
  }
}

// A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ..; its
// threads keep their columns' part of dgamma in registers and write it once.
// The next row is loaded before the reduction of this one where the registers
// hold both (PREFETCH); the widest rows (1024 threads) leave gamma and dh in
// memory until their use, too.  A lane holds units of 16 bytes, so that a
// wave's accesses are contiguous (f32 4096 x 7168 with dh: 94 us; 32 bytes a
// lane, in two accesses, 101); the widest rows units of 8 elements, of which
// f32 then has half as many to guard (1024 x 20480: 90 us with 8 registers
// spilled; in 16-byte units 124 with 54).  A row's address is formed once for
// the wave, in scalar registers (per lane and unit 77 spilled, 140 us).
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

template <int XT, int NV, int N>
struct GradRow {
  Unit<XT, N> d[NV], h[NV], b[NV];
  float rstd;
};

template <int XT, int NV, int N, bool NT, bool WITH_B>
__device__ __forceinline__ void load_grad_row(const NormGradArgs& p, int64_t row, int nvec, GradRow<XT, NV, N>& r) {
  r.rstd = p.rstd[row];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    r.d[i] = load_unit<XT, NT, N>(p.dy, row * p.lddy, v);
    r.h[i] = load_unit<XT, NT, N>(p.h, row * p.ldh, v);
    if (WITH_B && p.dh) r.b[i] = load_unit<XT, NT, N>(p.dh, row * p.lddh, v);
  }
}

template <int XT, int NV, int THREADS, bool PREFETCH, bool NT>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(NormGradArgs p) {
  constexpr int N = THREADS <= 512 ? kPer16<XT> : 8;
  constexpr bool kKeepGamma = THREADS <= 512;
  __shared__ float part[2][kMaxWaves];
  const int nvec = (int)(p.cols / N);
  const float inv_cols = 1.0f / (float)p.cols;
  float g[NV][N], acc[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < N; ++e) g[i][e] = acc[i][e] = 0.0f;
    if (kKeepGamma && v < nvec) decode_gamma<N>(load_gamma<N>(p.gamma, p.g_type, v), p.g_type, g[i]);
  }
  int flip = 0;
  GradRow<XT, NV, N> r;
  int64_t row = blockIdx.x;
  if (PREFETCH && row < p.rows) load_grad_row<XT, NV, N, NT, PREFETCH>(p, row, nvec, r);
  for (; row < p.rows; row += gridDim.x, flip ^= 1) {
    if (!PREFETCH) load_grad_row<XT, NV, N, NT, PREFETCH>(p, row, nvec, r);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float d[N], h[N];
      decode_unit<XT, N>(r.d[i], d);
      decode_unit<XT, N>(r.h[i], h);
      if (!kKeepGamma) decode_gamma<N>(load_gamma<N>(p.gamma, p.g_type, v), p.g_type, g[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float dx = d[e] * (h[e] * r.rstd);
        c = __builtin_fmaf(dx, g[i][e], c);
        acc[i][e] += dx;
      }
    }
    GradRow<XT, NV, N> next;
    if (PREFETCH && row + gridDim.x < p.rows) load_grad_row<XT, NV, N, NT, PREFETCH>(p, row + gridDim.x, nvec, next);
    c = block_sum(c, part[flip]) * inv_cols;
    // xh = h * rstd once more (rstd * c could leave fp32's range, xh does
    // not).  Formed from a copy that the compiler takes for another value: kept
    // from the loop above instead, f32 rows of 12288 take 64 us, not 54.
    float rstd = r.rstd;
    asm("" : "+v"(rstd));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float d[N], h[N], o[N];
      decode_unit<XT, N>(r.d[i], d);
      decode_unit<XT, N>(r.h[i], h);
      if (!kKeepGamma) decode_gamma<N>(load_gamma<N>(p.gamma, p.g_type, v), p.g_type, g[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = rstd * __builtin_fmaf(-(h[e] * rstd), c, d[e] * g[i][e]);
      if (p.dh) {
        float b[N];
        decode_unit<XT, N>(PREFETCH ? r.b[i] : load_unit<XT, NT, N>(p.dh, row * p.lddh, v), b);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += b[e];
      }
      store_unit<XT, N>(p.dx, row * p.lddx, v, o);
    }
    if (PREFETCH) r = next;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float* out = p.partial + blockIdx.x * p.cols + v * N;
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<float4*>(out + e) = make_float4(acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]);
  }
}

// dgamma[c] = sum over the strips' partial sums: 4 lanes hold 16 columns,
// 128 thread rows take every 128th strip, then the rows are added, 16 of a
// wave and the 8 waves.  Narrow columns make many workgroups.
constexpr int kSumThreads = 512;

__global__ __launch_bounds__(kSumThreads) void norm_grad_sum_kernel(const float* __restrict__ partial, int strips,
                                                                    int64_t cols, float* __restrict__ dgamma) {
  __shared__ float part[kSumThreads / 64][16];
  const int c = threadIdx.x & 3, s0 = threadIdx.x >> 2;
  const int64_t col = (int64_t)blockIdx.x * 16 + c * 4;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < cols) {
#pragma unroll 8
    for (int s = s0; s < strips; s += kSumThreads / 4) {
      const float4 v = *reinterpret_cast<const float4*>(partial + s * cols + col);
      t[0] += v.x;
      t[1] += v.y;
      t[2] += v.z;
      t[3] += v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int m = 4; m < 64; m <<= 1) t[e] += __shfl_xor(t[e], m);
    if ((threadIdx.x & 63) < 4) part[threadIdx.x >> 6][c * 4 + e] = t[e];
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const int64_t at = (int64_t)blockIdx.x * 16 + threadIdx.x;
    float s = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kSumThreads / 64; ++w) s += part[w][threadIdx.x];
    if (at < cols) dgamma[at] = s;
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
RowShape row_shape(int64_t cols) {
  const int64_t groups = cols / 8;
  const int per = groups <= 512 ? 1 : groups <= 1024 ? 2 : 4;
  const int64_t t = (groups + per - 1) / per;
  return {per, (int)((t + 63) / 64 * 64)};
}

template <int XT, bool STREAM, bool WITH_Y>
hipError_t norm_as(const NormArgs& a, hipStream_t st) {
  const RowShape sh = row_shape(a.cols);
  const dim3 grid((unsigned)(a.rows < kMaxRowBlocks ? a.rows : kMaxRowBlocks)), block(sh.threads);
  if (sh.per == 1)
    hipLaunchKernelGGL((norm_kernel<XT, 1, STREAM, WITH_Y>), grid, block, 0, st, a);
  else if (sh.per == 2)
    hipLaunchKernelGGL((norm_kernel<XT, 2, STREAM, WITH_Y>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_kernel<XT, 4, STREAM, WITH_Y>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int XT>
hipError_t norm_t(const NormArgs& a, hipStream_t st) {
  const int64_t bytes = a.rows * a.cols * (XT == 0 ? 2 : 4) * (a.r ? 2 : 1);
  if (bytes > kStreamBytes) return a.y ? norm_as<XT, true, true>(a, st) : norm_as<XT, true, false>(a, st);
  return a.y ? norm_as<XT, false, true>(a, st) : norm_as<XT, false, false>(a, st);
}

template <int XT, bool NT>
hipError_t norm_grad_as(const NormGradArgs& a, hipStream_t st) {
  constexpr int U = 8 / kPer16<XT>;  // units of 8 elements
  const RowShape sh = row_shape(a.cols);
  const dim3 grid((unsigned)norm_grad_strips(a.rows, a.cols)), block(sh.threads);
  if (sh.per == 1)
    hipLaunchKernelGGL((norm_grad_kernel<XT, U, 512, true, NT>), grid, block, 0, st, a);
  else if (sh.per == 2)
    hipLaunchKernelGGL((norm_grad_kernel<XT, 2 * U, 512, true, NT>), grid, block, 0, st, a);
  else if (sh.threads <= 512)
    hipLaunchKernelGGL((norm_grad_kernel<XT, 4 * U, 512, false, NT>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_grad_kernel<XT, 4, 1024, false, NT>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int XT>
hipError_t norm_grad_t(const NormGradArgs& a, hipStream_t st) {
  const int64_t bytes = a.rows * a.cols * (XT == 0 ? 2 : 4) * (a.dh ? 3 : 2);
  return bytes > kStreamBytes ? norm_grad_as<XT, true>(a, st) : norm_grad_as<XT, false>(a, st);
}

}  // namespace

// Up to 64 rows each their own strip, then four rows to a strip (a strip's
// partial sums are written and read again: 512 rows of 7168 bf16 take 13.2 us
// in 128 strips, 19.6 in 512, 14.9 in 256), two strips per CU at most and four
// where rows are short (16384 x 1024: 27 us in 1024 strips, 30 in 512, 29 in
// 2048; 8192 x 7168 in 768 strips 89 us, in 512 85).
int64_t norm_grad_strips(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 1024 ? 1024 : 512;
  const int64_t n = rows < 64 ? rows : rows < 256 ? 64 : (rows + 3) / 4;
  return n < most ? n : most;
}

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  return a.x_type == 0 ? norm_t<0>(a, st) : norm_t<1>(a, st);
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  if (a.rows > 0) {
    const hipError_t e = a.x_type == 0 ? norm_grad_t<0>(a, st) : norm_grad_t<1>(a, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_grad_sum_kernel, dim3((unsigned)((a.cols + 15) / 16)), dim3(kSumThreads), 0, st, a.partial,
                     (int)norm_grad_strips(a.rows, a.cols), a.cols, a.dgamma);
  return hipGetLastError();
}

}  // namespace fp8fg
