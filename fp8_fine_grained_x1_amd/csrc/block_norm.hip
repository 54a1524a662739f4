// Root-mean-square norms after and before a block, with the block's gate, the
// scaled residual addition and an E4M3 output, and their gradient, for gfx950.
//
// Forward, per row, z the block's output and r the residual stream:
//   zh = z rstd_post,  t = zh gamma_post gate block_scale
//   h = RN(residual_scale r + t) in z's type, each product in fp32
//   y = (h rstd) gamma;  q, s as the norm's (norm.hip)
// rstd = 1 / sqrt(mean of squares + eps) of z and of the rounded h.
// Backward, dy the gradient of y, dh what reaches h along the stream:
//   xh = h rstd,  a = dy gamma,  dH = rstd (a - xh mean(a xh)) + dh
//   dr = residual_scale dH
//   b = block_scale dH gate,  dz = rstd_post (b gamma_post - zh mean(b gamma_post zh))
//   dgamma = sum over rows dy xh,  dgamma_post = sum over rows b zh
//   dgate = block_scale dH zh gamma_post: of a gate per column summed over
//   the rows, which is gamma_post's sum without the gate: one sum
//   D = sum dH zh gives both.
// A row stays in the workgroup's registers, undecoded, from its one reading to
// its outputs.
//
// Both are bound by HBM, and by two sums over the row, one after the other, that
// the outputs wait for: while they run nothing of that row moves, so the next
// one is loaded ahead.  Measured on 8192 x 7168 bf16 with a gate per column: 97 us
// forward with every output (530 MB, 5.5 TB/s), gradient with dh 143 us (705 MB,
// 4.9 TB/s), 7 of it the sums over strips.  A large device copy moves 5.1 TB/s
// on this card.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"
#include "norm_common.h"
#include "tiles.h"

namespace fp8fg {

namespace {

enum { kGateNone = 0, kGateCols = 1, kGateRows = 2 };

template <int XT, int NV>
__device__ __forceinline__ float rstd_of(const Raw8<XT> (&raw)[NV], float ss, float inv_cols, int nvec, int64_t cols, float eps,
                                         double* wide) {
  const float mean = __builtin_fmaf(ss, inv_cols, eps);
  if (__builtin_expect(!(mean >= kLeastMean && mean <= FLT_MAX), 0)) return wide_range_rstd<XT, NV>(raw, nvec, cols, eps, wide);
  // the hardware's root (1 ulp) and one Newton step, y + y (1 - mean y^2) / 2: within an ulp, in 5
  // instructions; a root and a quotient take 50, which every wave of the row
  // runs twice between two barriers
  const float y = __builtin_amdgcn_rsqf(mean), my = mean * y;
  return __builtin_fmaf(__builtin_fmaf(-my, y, 1.0f) * 0.5f, y, y);
}

// Thread t holds the 8-element vectors t, t + blockDim, .. of its rows
// blockIdx.x, blockIdx.x + gridDim.x, ..: 16 consecutive lanes hold one 1x128
// tile.  With one vector to a thread (up to 8192 columns: AHEAD) the gammas
// stay in registers and the next row is loaded while this one is worked on
// (8192 x 7168 bf16: 97 us, loaded behind the first sum's squares 99.5, where narrow
// rows gain, 8192 x 2048: 33.0, this 33.7; two vectors to a thread and two workgroups
// per CU, without loading ahead, 121; with it 122).  The gammas are decoded where
// the first row needs them, not before its first sum (10 us more).  Large calls
// read and store past the caches (STREAM: 3 us less than without), others ordinarily,
// for the readers of h and y: 2048 rows take 29.8 us, with stores past the
// caches 24.1, but with three readers after it 52.9 and 57.5.
template <int XT, int NV, int GATE>
struct BlockIn {
  Raw8<XT> z[NV], r[NV], g[GATE == kGateRows ? NV : 1];
};
template <int XT, int NV, int GATE, bool STREAM>
__device__ __forceinline__ void load_block_in(const BlockNormArgs& p, int64_t row, int nvec, BlockIn<XT, NV, GATE>& in) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    in.z[i] = load_raw8<XT, STREAM>(p.z, row * p.ldz + v * 8);
    in.r[i] = load_raw8<XT, STREAM>(p.r, row * p.ldr + v * 8);
    if (GATE == kGateRows) in.g[i] = load_raw8<XT, STREAM>(p.gate, row * p.ldg + v * 8);
  }
}

template <int XT, int NV, int GATE, bool STREAM>
__global__ __launch_bounds__(1024) void block_norm_kernel(BlockNormArgs p) {
  constexpr bool AHEAD = NV == 1;
  __shared__ float part[2][kMaxWaves];
  __shared__ double wide[kMaxWaves];
  const int nvec = (int)(p.cols >> 3);
  const float inv_cols = 1.0f / (float)p.cols;
  float gm[8], gp[8], gc[8];  // gamma, gamma_post, a gate per column
  RawGamma<8> raw_gm, raw_gp, raw_gate;
  auto load_gammas = [&](int v) {
    raw_gp = load_gamma<8>(p.gamma_post, p.g_type, v);
    if (GATE == kGateCols) raw_gate = load_gamma<8>(p.gate, p.g_type, v);
    raw_gm = load_gamma<8>(p.gamma, p.g_type, v);
  };
  auto decode_gammas = [&]() {
    decode_gamma<8>(raw_gp, p.g_type, gp);
    if (GATE == kGateCols) decode_gamma<8>(raw_gate, p.g_type, gc);
    decode_gamma<8>(raw_gm, p.g_type, gm);
  };
  BlockIn<XT, NV, GATE> in;
  int64_t row = blockIdx.x;
  if (AHEAD) {
    load_block_in<XT, NV, GATE, STREAM>(p, row, nvec, in);
    if ((int)threadIdx.x < nvec) load_gammas(threadIdx.x);
  }
  for (; row < p.rows; row += gridDim.x) {
    if (!AHEAD) load_block_in<XT, NV, GATE, STREAM>(p, row, nvec, in);
    BlockIn<XT, NV, GATE> next;
    if (AHEAD && row + gridDim.x < p.rows) load_block_in<XT, NV, GATE, STREAM>(p, row + gridDim.x, nvec, next);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float f[8];
      decode8<XT>(in.z[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
    }
    ss = block_sum(ss, part[0]);
    const float post = rstd_of<XT, NV>(in.z, ss, inv_cols, nvec, p.cols, p.eps, wide);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float f[8], x[8];
      if (!AHEAD) load_gammas(v);
      if (!AHEAD || row == blockIdx.x) decode_gammas();
      decode8<XT>(in.z[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * post * gp[e];
      if constexpr (GATE != kGateNone) {
        if (GATE == kGateRows) decode8<XT>(in.g[i], gc);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= gc[e];
      }
      decode8<XT>(in.r[i], x);
      // Each product rounded by itself, as in the formula taken step by step:
      // h then rounds to z's type as that does but for 100 of 58.7 million values
      // (8192 x 7168 bf16).  With the scales and gates multiplied before
      // the rows and a fused sum 370 differ (3 us less), and where one is a tile's
      // largest, its scale follows by a step of z's type.
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = p.residual_scale * x[e] + p.block_scale * f[e];
      in.r[i] = encode8<XT>(x);
      store_raw8<XT, STREAM>(p.h, row * p.ldh + v * 8, in.r[i]);
      decode8<XT>(in.r[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
    }
    ss = block_sum(ss, part[1]);
    const float rstd = rstd_of<XT, NV>(in.r, ss, inv_cols, nvec, p.cols, p.eps, wide);
    if (threadIdx.x == 0) {
      if (p.rstd_post) p.rstd_post[row] = post;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec || (!p.q && !p.y)) continue;
      float f[8];
      if (!AHEAD) {
        load_gammas(v);
        decode_gammas();
      }
      decode8<XT>(in.r[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * gm[e];
      if (p.y) store_raw8<XT, STREAM>(p.y, row * p.ldy + v * 8, encode8<XT>(f));
      if (p.q) {
        uint32_t out[2];
        const float m = row16_max(amax_of(f));
        const float sc = p.rule == 0 ? quantize<0, 8>(f, m, out) : quantize<1, 8>(f, m, out);
        st_nt8(p.q + row * p.ldq + v * 8, make_uint2(out[0], out[1]));
        if ((threadIdx.x & 15) == 0) p.s[row * p.s_rs + (int64_t)(v >> 4) * p.s_ts] = sc;
      }
    }
    if (AHEAD) in = next;
  }
}

// A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ..; its
// threads keep their columns' part of the two sums over rows in registers
// (D = sum dH zh, with a gate of rows sum dH zh gate; and sum dy xh) and
// write them once.  8 elements to a thread, up to 1024 threads: the next row is
// loaded while this one is worked on (PREFETCH, rows of up to 8192 columns)
// at 94 registers, and one strip per CU suffices (8192 x 7168 bf16: 143 us, loaded
// before the first sum's terms 156, behind that sum 149; 16
// elements to a thread, 512 strips and nothing ahead: 197).
template <int XT, int NV, int GATE>
struct BlockRow {
  Unit<XT, kPer16<XT>> d[NV], h[NV], z[NV], b[NV], g[GATE == kGateRows ? NV : 1];
  float rstd, post;
};

template <int XT, int NV, int GATE, bool NT>
__device__ __forceinline__ void load_block_row(const BlockNormGradArgs& p, int64_t row, int nvec, BlockRow<XT, NV, GATE>& r) {
  constexpr int N = kPer16<XT>;
  r.rstd = p.rstd[row];
  r.post = p.rstd_post[row];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    r.d[i] = load_unit<XT, NT, N>(p.dy, row * p.lddy, v);
    r.h[i] = load_unit<XT, NT, N>(p.h, row * p.ldh, v);
    r.z[i] = load_unit<XT, NT, N>(p.z, row * p.ldz, v);
    if (p.dh) r.b[i] = load_unit<XT, NT, N>(p.dh, row * p.lddh, v);
    if (GATE == kGateRows) r.g[i] = load_unit<XT, NT, N>(p.gate, row * p.ldg, v);
  }
}

template <int XT, int NV, int GATE, bool NT, bool PREFETCH>
__global__ __launch_bounds__(1024) void block_norm_grad_kernel(BlockNormGradArgs p) {
  constexpr int N = kPer16<XT>;
  __shared__ float part[2][kMaxWaves];
  const int nvec = (int)(p.cols / N);
  const float inv_cols = 1.0f / (float)p.cols;
  // gamma, and what dH is multiplied by on its way to z (without a gate of
  // rows): kept, or for the widest rows loaded at each use
  constexpr int KEPT = PREFETCH ? NV : 1;
  float gm[KEPT][N], gp[KEPT][N], acc[2][NV][N];
  auto load_gm = [&](int i, int v) {
    decode_gamma<N>(load_gamma<N>(p.gamma, p.g_type, v), p.g_type, gm[i]);
  };
  auto load_gp = [&](int i, int v) {
    decode_gamma<N>(load_gamma<N>(p.gamma_post, p.g_type, v), p.g_type, gp[i]);
    float g[N];
    if (GATE == kGateCols) decode_gamma<N>(load_gamma<N>(p.gate, p.g_type, v), p.g_type, g);
#pragma unroll
    for (int e = 0; e < N; ++e) gp[i][e] *= GATE == kGateCols ? p.block_scale * g[e] : p.block_scale;
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[0][i][e] = acc[1][i][e] = 0.0f;
    if (!PREFETCH || v >= nvec) continue;
    load_gm(i, v);
    load_gp(i, v);
  }
  BlockRow<XT, NV, GATE> r;
  int64_t row = blockIdx.x;
  if (PREFETCH && row < p.rows) load_block_row<XT, NV, GATE, NT>(p, row, nvec, r);
  for (; row < p.rows; row += gridDim.x) {
    if (!PREFETCH) load_block_row<XT, NV, GATE, NT>(p, row, nvec, r);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float dy[N], x[N];
      decode_unit<XT, N>(r.d[i], dy);
      decode_unit<XT, N>(r.h[i], x);
      if (!PREFETCH) load_gm(0, v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float dx = dy[e] * (x[e] * r.rstd);
        c = __builtin_fmaf(dx, gm[i % KEPT][e], c);
        acc[1][i][e] += dx;
      }
    }
    BlockRow<XT, NV, GATE> next;
    if (PREFETCH && row + gridDim.x < p.rows) load_block_row<XT, NV, GATE, NT>(p, row + gridDim.x, nvec, next);
    c = block_sum(c, part[0]) * inv_cols;
    // dH, then w = block_scale dH gate gamma_post and its mean with zh
    float w[NV][N], m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float x[N], zv[N], o[N];
      decode_unit<XT, N>(r.d[i], o);
      decode_unit<XT, N>(r.h[i], x);
      decode_unit<XT, N>(r.z[i], zv);
      if (!PREFETCH) {
        load_gm(0, v);
        load_gp(0, v);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = r.rstd * __builtin_fmaf(-(x[e] * r.rstd), c, o[e] * gm[i % KEPT][e]);
      if (p.dh) {
        decode_unit<XT, N>(r.b[i], x);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] += x[e];
      }
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = p.residual_scale * o[e];
      store_unit<XT, N>(p.dr, row * p.lddr, v, x);
#pragma unroll
      for (int e = 0; e < N; ++e) zv[e] *= r.post;
      if constexpr (GATE == kGateRows) {
        float gv[N];
        decode_unit<XT, N>(r.g[i], gv);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          x[e] = o[e] * zv[e] * gp[i % KEPT][e];
          o[e] *= gv[e];
        }
        store_unit<XT, N>(p.dgate, row * p.lddg, v, x);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        acc[0][i][e] = __builtin_fmaf(o[e], zv[e], acc[0][i][e]);
        w[i][e] = o[e] * gp[i % KEPT][e];
        m = __builtin_fmaf(w[i][e], zv[e], m);
      }
    }
    m = block_sum(m, part[1]) * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float zv[N], o[N];
      decode_unit<XT, N>(r.z[i], zv);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = r.post * __builtin_fmaf(-(zv[e] * r.post), m, w[i][e]);
      store_unit<XT, N>(p.dz, row * p.lddz, v, o);
    }
    if (PREFETCH) r = next;
  }
  const int64_t strips = gridDim.x;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float* out = p.partial + (a * strips + blockIdx.x) * p.cols + v * N;
#pragma unroll
      for (int e = 0; e < N; e += 4)
        *reinterpret_cast<float4*>(out + e) =
            make_float4(acc[a][i][e], acc[a][i][e + 1], acc[a][i][e + 2], acc[a][i][e + 3]);
    }
}

// Element c of a vector of g_type.
__device__ __forceinline__ float gamma_at(const void* g, int g_type, int64_t c) {
  return g_type == 0 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(g)[c] << 16)
                     : reinterpret_cast<const float*>(g)[c];
}

// The strips' sums, added as norm_grad_sum_kernel adds them: blockIdx.y 0
// gives dgamma_post and a column gate's gradient, 1 dgamma.
constexpr int kSumThreads = 512;

template <int GATE>
__global__ __launch_bounds__(kSumThreads) void block_norm_sum_kernel(BlockNormGradArgs p, int strips) {
  __shared__ float part[kSumThreads / 64][16];
  const float* partial = p.partial + (int64_t)blockIdx.y * strips * p.cols;
  const int c = threadIdx.x & 3, s0 = threadIdx.x >> 2;
  const int64_t col = (int64_t)blockIdx.x * 16 + c * 4;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < p.cols) {
#pragma unroll 8
    for (int s = s0; s < strips; s += kSumThreads / 4) {
      const float4 v = *reinterpret_cast<const float4*>(partial + s * p.cols + col);
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
    if (at < p.cols) {
      if (blockIdx.y == 1) {
        p.dgamma[at] = s;
      } else {
        s *= p.block_scale;
        p.dgamma_post[at] = GATE == kGateCols ? s * gamma_at(p.gate, p.g_type, at) : s;
        if (GATE == kGateCols && p.dgate) reinterpret_cast<float*>(p.dgate)[at] = s * gamma_at(p.gamma_post, p.g_type, at);
      }
    }
  }
}

// Threads of a workgroup for rows of up to 8192 columns, 8 to each, and up to 16384,
// 16 to each: a function of the columns alone, and with it the order of a row's
// additions.
int block_threads(int64_t cols) {
  const int64_t groups = cols / 8, t = groups <= 1024 ? groups : (groups + 1) / 2;
  return (int)((t + 63) / 64 * 64);
}

template <int XT, int GATE, bool STREAM>
hipError_t norm_as(const BlockNormArgs& a, hipStream_t st) {
  const int threads = block_threads(a.cols);
  // Workgroups that take row after row (AHEAD): one to a CU of rows past 4096 columns, 8
  // waves down to 1152, then 14 (bf16: 8192 x 4096 57.3 us, with two workgroups 63;
  // 8192 x 2048 31.8, with 16 waves 33; 8192 x 1024 15.7, with 8 waves 16.8).
  const int waves = threads / 64, per_cu = waves > 8 ? 1 : waves > 2 ? 8 / waves : 14 / waves;
  const int64_t fit = (int64_t)device_cu_count() * per_cu;
  if (a.cols <= 8192)
    hipLaunchKernelGGL((block_norm_kernel<XT, 1, GATE, STREAM>), dim3((unsigned)(a.rows < fit ? a.rows : fit)), dim3(threads), 0,
                       st, a);
  else
    hipLaunchKernelGGL((block_norm_kernel<XT, 2, GATE, STREAM>), dim3((unsigned)(a.rows < kMaxRowBlocks ? a.rows : kMaxRowBlocks)),
                       dim3(threads), 0, st, a);
  return hipGetLastError();
}

template <int XT, int GATE>
hipError_t norm_t(const BlockNormArgs& a, hipStream_t st) {
  const bool big = past_caches(a.rows, GATE == kGateRows ? 3 : 2, a.cols, XT == 0 ? 2 : 4);
  return big ? norm_as<XT, GATE, true>(a, st) : norm_as<XT, GATE, false>(a, st);
}

template <int XT, int GATE, bool NT>
hipError_t grad_as(const BlockNormGradArgs& a, hipStream_t st) {
  constexpr int U = 8 / kPer16<XT>;  // units of 8 elements
  const dim3 grid((unsigned)block_norm_strips(a.rows, a.cols)), block(block_threads(a.cols));
  if (a.cols <= 8192)
    hipLaunchKernelGGL((block_norm_grad_kernel<XT, U, GATE, NT, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((block_norm_grad_kernel<XT, 2 * U, GATE, NT, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int XT, int GATE>
hipError_t grad_t(const BlockNormGradArgs& a, hipStream_t st) {
  const bool big = past_caches(a.rows, 3 + (a.dh != nullptr) + (GATE == kGateRows), a.cols, XT == 0 ? 2 : 4);
  return big ? grad_as<XT, GATE, true>(a, st) : grad_as<XT, GATE, false>(a, st);
}

// f.template go<XT, GATE>() by the type and the gate.
template <typename F>
hipError_t choose(int x_type, const void* gate, int64_t ldg, F f) {
  if (x_type == 0)
    return !gate ? f.template go<0, kGateNone>() : ldg == 0 ? f.template go<0, kGateCols>() : f.template go<0, kGateRows>();
  return !gate ? f.template go<1, kGateNone>() : ldg == 0 ? f.template go<1, kGateCols>() : f.template go<1, kGateRows>();
}
struct GoNorm {
  const BlockNormArgs& a;
  hipStream_t st;
  template <int XT, int GATE>
  hipError_t go() const { return norm_t<XT, GATE>(a, st); }
};
struct GoGrad {
  const BlockNormGradArgs& a;
  hipStream_t st;
  template <int XT, int GATE>
  hipError_t go() const { return grad_t<XT, GATE>(a, st); }
};

}  // namespace

// Row strips of the gradient, one workgroup each: one per CU where a row takes
// more than 512 threads, two down to 128 and four below (6000 rows of 2048 bf16: 39.8
// us in 512 strips, 42.3 in 1024; of 4096: 66 in 512, 69 in 256; 8000 x 512: 18 in 1024, 23
// in 512).  A strip has at least two rows, since its sums are written and read
// again (200 rows of 7168: 15.4 us, in strips of one row 19, of four 17), and all
// the same number of them but the last (856 rows of 5376 f32: 33 us in 214 strips,
// 35 in 256).
int64_t block_norm_strips(int64_t rows, int64_t cols) {
  const int64_t most = cols > 4096 ? 256 : cols > 1024 ? 512 : 1024;
  if (rows <= 64) return rows;
  const int64_t per = (rows + most - 1) / most;
  return (rows + (per < 2 ? 2 : per) - 1) / (per < 2 ? 2 : per);
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t st) {
  return choose(a.x_type, a.gate, a.ldg, GoNorm{a, st});
}

hipError_t launch_block_norm_grad(const BlockNormGradArgs& a, hipStream_t st) {
  if (a.rows > 0) {
    const hipError_t e = choose(a.x_type, a.gate, a.ldg, GoGrad{a, st});
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)((a.cols + 15) / 16), 2);
  const int strips = (int)block_norm_strips(a.rows, a.cols);
  if (a.gate && a.ldg == 0)
    hipLaunchKernelGGL((block_norm_sum_kernel<kGateCols>), grid, dim3(kSumThreads), 0, st, a, strips);
  else
    hipLaunchKernelGGL((block_norm_sum_kernel<kGateNone>), grid, dim3(kSumThreads), 0, st, a, strips);
  return hipGetLastError();
}

}  // namespace fp8fg
