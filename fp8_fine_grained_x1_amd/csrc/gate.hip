// Silu gate between the two products of an expert, with 8-bit outputs and
// 8-bit activation checkpoints, and its gradient from a checkpoint, for
// gfx950.
//
// u = [g | l] holds the gate and the linear half of a row, `inner` columns
// each.  With sg = 1 / (1 + exp(-g)), all in fp32:
//   forward     a = (g sg) l;  (q, s) = 1x128 tiles of a, (uq, us) = 1x128
//               tiles of u, by the quantizers' rules
//   backward    g, l = RN32(dec(uq) us);  dg = (da l) sg (1 + g (1 - sg)),
//               dl = da (g sg), a = (g sg) l;  1x128 tiles of [dg | dl] and,
//               in the other form, the transposed 128x1 tiles of [dg | dl] and
//               of a.  (Both quantizers are passed straight through.)
// Every output is rounded once, from the fp32 value.  With t = exp(-|g|),
// sg and 1 - sg are 1 / (1 + t) and t / (1 + t), in the order of g's sign:
// neither cancels, and both go to 0 as they should.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"
#include "tiles.h"

namespace fp8fg {

namespace {

constexpr int kGThreads = 256;
constexpr int kGroups = kGThreads / 16;
constexpr int kUnroll = 2;
constexpr int kGateBlocksPerCu = 28;

// sigmoid(g) and 1 - sigmoid(g)
struct Sigmoid {
  float s, r;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float g) {
  const float t = exp_neg(-fabsf(g));
  const float i = __builtin_amdgcn_rcpf(1.0f + t);
  const float ti = t * i;
  return {g >= 0.0f ? i : ti, g >= 0.0f ? ti : i};
}

struct GateParts {
  float dg, dl, a;
};
__device__ __forceinline__ GateParts gate_parts(float da, float g, float l) {
  const Sigmoid s = sigmoid_of(g);
  const float silu = g * s.s;
  return {da * l * s.s * __builtin_fmaf(g, s.r, 1.0f), da * silu, silu * l};
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// A 1x128 tile held by 16 lanes, 8 elements each: its bytes and its scale.
template <int RULE>
__device__ __forceinline__ void quantize_tile(float (&v)[8], uint8_t* __restrict__ q, float* __restrict__ s) {
  const float m = row16_max(amax8(v));
  const TileScale sc = RULE == 0 ? scale_amax(m) : scale_pow2(m);
  quotient8<RULE>(v, sc);
  uint2 out;
  out.x = pack4_e4m3(v[0], v[1], v[2], v[3]);
  out.y = pack4_e4m3(v[4], v[5], v[6], v[7]);
  st_nt8(q, out);
  if ((threadIdx.x & 15) == 0) *s = sc.s;
}

// Rows in use: all of them, or the first *used.
__device__ __forceinline__ uint32_t rows_used(int64_t rows, const int32_t* used) {
  if (!used) return (uint32_t)rows;
  const int64_t n = *used;
  return (uint32_t)(n < 0 ? 0 : n < rows ? n : rows);
}

struct GateGrid {
  FastDiv tpr, band;  // tiles of a row's half, of a band of 16 rows
};

// 16 lanes own a tile of both halves; two tiles per iteration, so that the
// loads of both are in flight before either is processed.
template <int XT, int RULE, int ORDER, bool KEEP, bool NT>
__global__ __launch_bounds__(kGThreads) void gate_kernel(GateArgs p, GateGrid gr) {
  const int c = (threadIdx.x & 15) * 8;
  const uint32_t group = blockIdx.x * kGroups + (threadIdx.x >> 4);
  const uint32_t ngroups = gridDim.x * kGroups;
  const uint32_t rows = rows_used(p.rows, p.used);
  const uint32_t ntiles = rows * gr.tpr.d;
  for (uint32_t t0 = group; t0 < ntiles; t0 += kUnroll * ngroups) {
    Raw8<XT> g[kUnroll], l[kUnroll];
    uint32_t r[kUnroll], tc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t t = t0 + u * ngroups;
      if (t >= ntiles) continue;
      tile_rc<ORDER>(t, gr.tpr, gr.band, rows, r[u], tc[u]);
      const int64_t at = (int64_t)r[u] * p.ldu + tc[u] * 128 + c;
      g[u] = load_raw8<XT, NT>(p.u, at);
      l[u] = load_raw8<XT, NT>(p.u, at + p.inner);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t t = t0 + u * ngroups;
      if (t >= ntiles) continue;
      float a[8], b[8], v[8];
      decode8<XT>(g[u], a);
      decode8<XT>(l[u], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a[i] * sigmoid_of(a[i]).s * b[i];
      const int64_t row = r[u], col = tc[u] * 128 + c;
      quantize_tile<RULE>(v, p.q + row * p.ldq + col, p.s + row * p.s_rs + tc[u] * p.s_ts);
      if constexpr (KEEP) {
        uint8_t* k = p.uq + row * p.lduq + col;
        float* ks = p.us + row * p.us_rs + tc[u] * p.us_ts;
        quantize_tile<RULE>(a, k, ks);
        quantize_tile<RULE>(b, k + p.inner, ks + (p.inner >> 7) * p.us_ts);
      }
    }
  }
}

// 8 values of a checkpoint: RN32(dec(q) s).
__device__ __forceinline__ void decode_kept(uint2 w, float s, float (&v)[8]) {
  float a[4], b[4];
  unpack4_e4m3(w.x, a);
  unpack4_e4m3(w.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i] * s;
    v[4 + i] = b[i] * s;
  }
}

template <int XT, int RULE, int ORDER, bool WIDE, bool NT>
__global__ __launch_bounds__(kGThreads) void gate_grad_kernel(GateGradArgs p, GateGrid gr) {
  const int c = (threadIdx.x & 15) * 8;
  const uint32_t group = blockIdx.x * kGroups + (threadIdx.x >> 4);
  const uint32_t ngroups = gridDim.x * kGroups;
  const uint32_t rows = rows_used(p.rows, p.used);
  const uint32_t ntiles = rows * gr.tpr.d;
  const int64_t half = p.inner >> 7;
  for (uint32_t t0 = group; t0 < ntiles; t0 += kUnroll * ngroups) {
    Raw8<XT> d[kUnroll];
    uint2 g[kUnroll], l[kUnroll];
    float gs[kUnroll], ls[kUnroll];
    uint32_t r[kUnroll], tc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t t = t0 + u * ngroups;
      if (t >= ntiles) continue;
      tile_rc<ORDER>(t, gr.tpr, gr.band, rows, r[u], tc[u]);
      const int64_t row = r[u], col = tc[u] * 128 + c;
      d[u] = load_raw8<XT, NT>(p.da, row * p.ldda + col);
      const uint8_t* k = p.uq + row * p.lduq + col;
      const float* ks = p.us + row * p.us_rs + tc[u] * p.us_ts;
      g[u] = ld_nt8(k);
      l[u] = ld_nt8(k + p.inner);
      gs[u] = *ks;
      ls[u] = ks[half * p.us_ts];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t t = t0 + u * ngroups;
      if (t >= ntiles) continue;
      float x[8], gv[8], lv[8], dg[8], dl[8], a[8];
      decode8<XT>(d[u], x);
      decode_kept(g[u], gs[u], gv);
      decode_kept(l[u], ls[u], lv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const GateParts o = gate_parts(x[i], gv[i], lv[i]);
        dg[i] = o.dg;
        dl[i] = o.dl;
        a[i] = o.a;
      }
      const int64_t row = r[u], col = tc[u] * 128 + c;
      if constexpr (WIDE) {
        if (p.du) {
          store_raw8<XT, false>(p.du, row * p.lddu + col, encode8<XT>(dg));
          store_raw8<XT, false>(p.du, row * p.lddu + p.inner + col, encode8<XT>(dl));
        }
        if (p.a) store_raw8<XT, false>(p.a, row * p.lda + col, encode8<XT>(a));
        if (!p.q) continue;
      }
      uint8_t* q = p.q + row * p.ldq + col;
      float* s = p.s + row * p.s_rs + tc[u] * p.s_ts;
      quantize_tile<RULE>(dg, q, s);
      quantize_tile<RULE>(dl, q + p.inner, s + half * p.s_ts);
    }
  }
}

// One 128 x 128 block of da per workgroup, with both halves of the
// checkpoint: thread (rg, cg) holds rows 8 rg .. + 7 of columns 8 cg .. + 7,
// undecoded.  The first pass forms the rows' values (1x128 tiles: their
// maxima within 16 lanes, their bytes stored at once) and the columns' maxima
// (through LDS); the second forms the values again, in column order, and
// stages the transposed bytes in LDS.
template <int XT, int RULE>
__global__ __launch_bounds__(kGThreads) void gate_grad_tile_kernel(GateGradTileArgs p) {
  __shared__ __align__(16) uint8_t tbuf[3 * 128 * kTPitch];
  __shared__ TileScale col_sc[3][128];
  __shared__ float row_s[2][128];
  float(*part)[16][128] = reinterpret_cast<float(*)[16][128]>(tbuf);  // 24 of its 54 KB, before the bytes

  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  const int64_t tr = blockIdx.y, tc = blockIdx.x, half = p.inner >> 7;

  RawRow<XT> d[8];
  RawRow<2> g[8], l[8];
  float gs[8], ls[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + rg * 8 + i, col = c0 + cg * 8;
    d[i] = load_raw<XT>(p.da, row * p.ldda + col);
    g[i] = load_raw<2>(p.uq, row * p.lduq + col);
    l[i] = load_raw<2>(p.uq, row * p.lduq + p.inner + col);
    gs[i] = p.us[row * p.us_rs + tc * p.us_ts];
    ls[i] = p.us[row * p.us_rs + (half + tc) * p.us_ts];
  }
  auto pair = [&](int i, auto col, GateParts& x, GateParts& y) {
    constexpr int J = decltype(col)::value;
    float d0, d1, g0, g1, l0, l1;
    raw_pair<J>(d[i], d0, d1);
    raw_pair<J>(g[i], g0, g1);
    raw_pair<J>(l[i], l0, l1);
    x = gate_parts(d0, g0 * gs[i], l0 * ls[i]);
    y = gate_parts(d1, g1 * gs[i], l1 * ls[i]);
  };

  float mc[3][8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float dg[8], dl[8];
    for_pairs([&](auto col) {
      constexpr int J = decltype(col)::value;
      GateParts x, y;
      pair(i, col, x, y);
      dg[J] = x.dg;
      dg[J + 1] = y.dg;
      dl[J] = x.dl;
      dl[J + 1] = y.dl;
      mc[0][J] = fmaxf(mc[0][J], fabsf(x.dg));
      mc[0][J + 1] = fmaxf(mc[0][J + 1], fabsf(y.dg));
      mc[1][J] = fmaxf(mc[1][J], fabsf(x.dl));
      mc[1][J + 1] = fmaxf(mc[1][J + 1], fabsf(y.dl));
      mc[2][J] = fmaxf(mc[2][J], fabsf(x.a));
      mc[2][J + 1] = fmaxf(mc[2][J + 1], fabsf(y.a));
    });
    uint8_t* q = p.q + (r0 + rg * 8 + i) * p.ldq + c0 + cg * 8;
    quantize_tile<RULE>(dg, q, &row_s[0][rg * 8 + i]);
    quantize_tile<RULE>(dl, q + p.inner, &row_s[1][rg * 8 + i]);
  }
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int j = 0; j < 8; ++j) part[o][rg][cg * 8 + j] = mc[o][j];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    refresh(d[i]);
    refresh(g[i]);
    refresh(l[i]);
  }
  __syncthreads();
  // the rows' scales, and the columns'
  p.s[(r0 + (tid & 127)) * p.s_rs + (tc + (tid >> 7) * half) * p.s_ts] = row_s[tid >> 7][tid & 127];
  for (int k = tid; k < 3 * 128; k += kGThreads) {
    const int o = k >> 7, c = k & 127;
    float m = part[o][0][c];
#pragma unroll
    for (int r = 1; r < 16; ++r) m = fmaxf(m, part[o][r][c]);
    const TileScale sc = RULE == 0 ? scale_amax(m) : scale_pow2(m);
    col_sc[o][c] = sc;
    if (o < 2)
      p.st[(o * p.inner + c0 + c) * p.st_rs + tr * p.st_ts] = sc.s;
    else
      p.as[(c0 + c) * p.as_rs + tr * p.as_ts] = sc.s;
  }
  __syncthreads();
  for_pairs([&](auto col) {
    constexpr int J = decltype(col)::value;
    float v[3][2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      GateParts x, y;
      pair(i, col, x, y);
      v[0][0][i] = x.dg;
      v[0][1][i] = y.dg;
      v[1][0][i] = x.dl;
      v[1][1][i] = y.dl;
      v[2][0][i] = x.a;
      v[2][1][i] = y.a;
    }
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = cg * 8 + J + h;
        quotient8<RULE>(v[o][h], col_sc[o][c]);
        const float(&w)[8] = v[o][h];
        uint2 out;
        out.x = pack4_e4m3(w[0], w[1], w[2], w[3]);
        out.y = pack4_e4m3(w[4], w[5], w[6], w[7]);
        const int chunk = (rg >> 1) ^ ((c >> 4) & 7);
        *reinterpret_cast<uint2*>(tbuf + (o * 128 + c) * kTPitch + chunk * 16 + (rg & 1) * 8) = out;
      }
  });
  __syncthreads();
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    uint8_t* out = o < 2 ? p.qt + (o * p.inner + c0) * p.ldqt : p.aq + c0 * p.ldaq;
    const int64_t ld = o < 2 ? p.ldqt : p.ldaq;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int k = it * kGThreads + tid;
      const int c = k >> 3, chunk = k & 7;
      const uint4 w = *reinterpret_cast<const uint4*>(tbuf + (o * 128 + c) * kTPitch + ((chunk ^ ((c >> 4) & 7)) << 4));
      st_nt16(out + c * ld + r0 + chunk * 16, w);
    }
  }
}

// Workgroups for `rows` (all of them: how many are in use is known on the
// device alone) and the tiles' division constants.
unsigned gate_grid(int64_t rows, int64_t inner, GateGrid& gr) {
  const int64_t tpr = inner / 128, ntiles = rows * tpr, per = kGroups * kUnroll;
  const int64_t want = (ntiles + per - 1) / per, cap = (int64_t)device_cu_count() * kGateBlocksPerCu;
  gr.tpr = make_fast_div((uint32_t)tpr);
  gr.band = make_fast_div((uint32_t)(16 * tpr));
  return (unsigned)(want < cap ? want : cap);
}
// Bands of 16 rows where the scales of consecutive rows are adjacent (see
// the 1x128 quantizer).
bool by_bands(int64_t s_rs) { return s_rs == 1; }

template <int XT, int RULE, int ORDER, bool NT>
hipError_t gate_as(const GateArgs& a, hipStream_t st) {
  GateGrid gr;
  const unsigned blocks = gate_grid(a.rows, a.inner, gr);
  if (a.uq)
    hipLaunchKernelGGL((gate_kernel<XT, RULE, ORDER, true, NT>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  else
    hipLaunchKernelGGL((gate_kernel<XT, RULE, ORDER, false, NT>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  return hipGetLastError();
}
template <int XT, int RULE, int ORDER, bool NT>
hipError_t grad_as(const GateGradArgs& a, hipStream_t st) {
  GateGrid gr;
  const unsigned blocks = gate_grid(a.rows, a.inner, gr);
  if (a.du || a.a)
    hipLaunchKernelGGL((gate_grad_kernel<XT, RULE, ORDER, true, NT>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  else
    hipLaunchKernelGGL((gate_grad_kernel<XT, RULE, ORDER, false, NT>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  return hipGetLastError();
}

template <int XT, int RULE>
hipError_t gate_t(const GateArgs& a, hipStream_t st) {
  const bool nt = past_caches(a.rows, 2, a.inner, XT == 0 ? 2 : 4);
  if (by_bands(a.s_rs)) return nt ? gate_as<XT, RULE, 1, true>(a, st) : gate_as<XT, RULE, 1, false>(a, st);
  return nt ? gate_as<XT, RULE, 0, true>(a, st) : gate_as<XT, RULE, 0, false>(a, st);
}
template <int XT, int RULE>
hipError_t grad_t(const GateGradArgs& a, hipStream_t st) {
  const bool nt = past_caches(a.rows, 1, a.inner, XT == 0 ? 2 : 4);
  if (by_bands(a.q ? a.s_rs : 0)) return nt ? grad_as<XT, RULE, 1, true>(a, st) : grad_as<XT, RULE, 1, false>(a, st);
  return nt ? grad_as<XT, RULE, 0, true>(a, st) : grad_as<XT, RULE, 0, false>(a, st);
}
template <int XT, int RULE>
hipError_t grad_tile_t(const GateGradTileArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.inner / 128), (unsigned)(a.rows / 128));
  hipLaunchKernelGGL((gate_grad_tile_kernel<XT, RULE>), grid, dim3(kGThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t st) {
  if (a.u_type == 0) return a.rule == 0 ? gate_t<0, 0>(a, st) : gate_t<0, 1>(a, st);
  return a.rule == 0 ? gate_t<1, 0>(a, st) : gate_t<1, 1>(a, st);
}

hipError_t launch_gate_grad(const GateGradArgs& a, hipStream_t st) {
  if (a.type == 0) return a.rule == 0 ? grad_t<0, 0>(a, st) : grad_t<0, 1>(a, st);
  return a.rule == 0 ? grad_t<1, 0>(a, st) : grad_t<1, 1>(a, st);
}

hipError_t launch_gate_grad_tile(const GateGradTileArgs& a, hipStream_t st) {
  if (a.type == 0) return a.rule == 0 ? grad_tile_t<0, 0>(a, st) : grad_tile_t<0, 1>(a, st);
  return a.rule == 0 ? grad_tile_t<1, 0>(a, st) : grad_tile_t<1, 1>(a, st);
}

}  // namespace fp8fg
