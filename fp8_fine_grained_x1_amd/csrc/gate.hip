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
// Every output is rounded once, from the fp32 value.
//
// An element costs 36 vector instructions in either direction, which keep the
// vector units busy in 85% of the forward's cycles, which HBM bounds, and 94% of
// the gradient's, which they bound.  Measured on 16384 x 4096 bf16: forward with
// checkpoint 80 us (476 MB, 6.0 TB/s), gradient 74 to 78 us over boxes (411 MB,
// 5.4); with the 128x1 operands, 8192 x 4096, 67 to 72 us (309 MB, 4.5).  A large
// device copy moves 5.1 TB/s on this card.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "launch.h"
#include "tiles.h"

namespace fp8fg {

namespace {

constexpr int kGThreads = 256;

// sigmoid(g) = 1 / (1 + exp(-g)) and g sigmoid(g): gates are held to [-87, 87] in the
// exponent, and from below in the product.  Below -87 the sigmoid stays at 2^-125.5
// instead of falling on to 0, above 87 it is 1 in fp32.  r = 1 - s without
// cancellation.  A NaN stays one: the limits are IEEE 754's minimum and maximum (an
// instruction each; med3 and max would give -87).
//
// The correction step of the quotient is by 1 - y - p y, so that the sum's own rounding
// is made good too: dg, dl and a are then closer to 64 bits than a composition of
// fp32 operations (root mean square 0.75 to 0.87 roundings, the composition 0.85 to
// 1.6; without the step up to 0.97, and the gradient of 16384 x 4096 takes 74 us).
// RN32(ln 2) is off by 2^-28.5, which makes up to 4 roundings of the exponential of
// the farthest gates; a second constant there costs 3 us more.
struct Sigmoid {
  float s, r, silu;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float g) {
  const float low = __builtin_elementwise_maximum(g, -87.0f);
  const float x = __builtin_elementwise_minimum(low, 87.0f);
  const float t = x * -1.44269502f;                        // RN(-x RN32(log2 e))
  const float e = __builtin_fmaf(t, -0.693147181f, -x);    // -x - t ln 2
  const float q = __builtin_amdgcn_exp2f(t);
  const float p = __builtin_fmaf(q, e, q);                 // 2^t exp(e) to first order
  const float y = __builtin_amdgcn_rcpf(1.0f + p);
  const float s = __builtin_fmaf(__builtin_fmaf(-p, y, 1.0f - y), y, y);
  return {s, p * s, low * s};
}

struct GateParts {
  float dg, dl, a;
};
__device__ __forceinline__ GateParts gate_parts(float da, float g, float l) {
  const Sigmoid s = sigmoid_of(g);
  return {da * l * __builtin_fmaf(s.silu, s.r, s.s), da * s.silu, s.silu * l};
}

// 8 lanes own a tile of 128 columns, 16 each, in two runs of 8 that start GAP
// apart: 8 (16 columns in a row: 16-byte accesses of E4M3 bytes) or 64 (runs
// of neighbouring lanes adjoin: contiguous 16-byte accesses of bf16).  Where
// most bytes are E4M3 the first gains (gradient of 16384 x 4096: 77.6 us, 79.5),
// where most are written in bf16 the second (with du and a, 5003 x 2048: 27.9
// us, 28.9); the forward pass takes the first (80.7, 85.8).
template <int GAP>
__device__ __forceinline__ uint32_t lane_column() { return (threadIdx.x & 7) * (GAP == 8 ? 16 : 8); }

__device__ __forceinline__ float row8_max(float v) {
  v = fmaxf(v, dpp_mov<kDppQuadXor1>(v));
  v = fmaxf(v, dpp_mov<kDppQuadXor2>(v));
  return fmaxf(v, dpp_mov<kDppRowHalfMirror>(v));
}
// PAST: stored past the caches.
template <int RULE, int GAP, bool PAST>
__device__ __forceinline__ void quantize_tile(float (&v)[16], uint8_t* __restrict__ q, float* __restrict__ s) {
  uint32_t w[4];
  const float sc = quantize<RULE, 16>(v, row8_max(amax_of(v)), w);
  if constexpr (GAP == 8) {
    const uint4 x = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (PAST) st_nt16(q, x); else *reinterpret_cast<uint4*>(q) = x;
  } else {
    const uint2 x = make_uint2(w[0], w[1]), y = make_uint2(w[2], w[3]);
    if constexpr (PAST) {
      st_nt8(q, x);
      st_nt8(q + GAP, y);
    } else {
      *reinterpret_cast<uint2*>(q) = x;
      *reinterpret_cast<uint2*>(q + GAP) = y;
    }
  }
  if ((threadIdx.x & 7) == 0) *s = sc;
}

template <int XT>
struct Raw16 {
  Raw8<XT> a, b;
};
// (Ordinary loads: past the caches 16384 x 4096 takes 82 us instead of 80.5
// forward, 4096 x 4096, whose producer leaves it in them, 24.6 instead of 22.9.)
template <int XT, int GAP>
__device__ __forceinline__ Raw16<XT> load_raw16(const void* __restrict__ p, int64_t off) {
  return {load_raw8<XT, false>(p, off), load_raw8<XT, false>(p, off + GAP)};
}
template <int XT>
__device__ __forceinline__ void decode_raw16(const Raw16<XT>& r, float (&v)[16]) {
  decode8<XT>(r.a, v);
  decode8<XT>(r.b, v + 8);
}
template <int XT, int GAP>
__device__ __forceinline__ void store_raw16(void* __restrict__ p, int64_t off, const float (&v)[16]) {
  store_raw8<XT, false>(p, off, encode8<XT>(v));
  store_raw8<XT, false>(p, off + GAP, encode8<XT>(v + 8));
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
constexpr int kGroups = kGThreads / 8;

template <int XT, int RULE, int ORDER, bool KEEP, bool PAST>
__global__ __launch_bounds__(kGThreads) void gate_kernel(GateArgs p, GateGrid gr) {
  constexpr int GAP = 8;
  const uint32_t c = lane_column<GAP>();
  const uint32_t rows = rows_used(p.rows, p.used), ntiles = rows * gr.tpr.d;
  for (uint32_t t = blockIdx.x * kGroups + (threadIdx.x >> 3); t < ntiles; t += gridDim.x * kGroups) {
    uint32_t r, tc;
    tile_rc<ORDER>(t, gr.tpr, gr.band, rows, r, tc);
    const int64_t row = r, col = tc * 128 + c;
    const Raw16<XT> g = load_raw16<XT, GAP>(p.u, row * p.ldu + col);
    const Raw16<XT> l = load_raw16<XT, GAP>(p.u, row * p.ldu + p.inner + col);
    float a[16], b[16], v[16];
    decode_raw16<XT>(g, a);
    decode_raw16<XT>(l, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = sigmoid_of(a[i]).silu * b[i];
    quantize_tile<RULE, GAP, PAST>(v, p.q + row * p.ldq + col, p.s + row * p.s_rs + tc * p.s_ts);
    if constexpr (KEEP) {
      uint8_t* k = p.uq + row * p.lduq + col;
      float* ks = p.us + row * p.us_rs + tc * p.us_ts;
      quantize_tile<RULE, GAP, true>(a, k, ks);
      quantize_tile<RULE, GAP, true>(b, k + p.inner, ks + (p.inner >> 7) * p.us_ts);
    }
  }
}

template <int GAP>
__device__ __forceinline__ uint4 load_kept(const uint8_t* __restrict__ k) {
  if constexpr (GAP == 8) {
    return ld_nt16(k);
  } else {
    const uint2 a = ld_nt8(k), b = ld_nt8(k + GAP);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
}

// 8 values of a checkpoint: RN32(dec(q) s).
__device__ __forceinline__ void decode_kept(uint2 w, float s, float* v) {
  float a[4], b[4];
  unpack4_e4m3(w.x, a);
  unpack4_e4m3(w.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i] * s;
    v[4 + i] = b[i] * s;
  }
}

template <int XT, int RULE, int ORDER, bool WIDE, bool PAST>
__global__ __launch_bounds__(kGThreads) void gate_grad_kernel(GateGradArgs p, GateGrid gr) {
  constexpr int GAP = WIDE ? 64 : 8;
  const uint32_t c = lane_column<GAP>();
  const uint32_t rows = rows_used(p.rows, p.used), ntiles = rows * gr.tpr.d;
  const int64_t half = p.inner >> 7;
  for (uint32_t t = blockIdx.x * kGroups + (threadIdx.x >> 3); t < ntiles; t += gridDim.x * kGroups) {
    uint32_t r, tc;
    tile_rc<ORDER>(t, gr.tpr, gr.band, rows, r, tc);
    const int64_t row = r, col = tc * 128 + c;
    const Raw16<XT> d = load_raw16<XT, GAP>(p.da, row * p.ldda + col);
    const uint8_t* k = p.uq + row * p.lduq + col;
    const float* ks = p.us + row * p.us_rs + tc * p.us_ts;
    const uint4 gq = load_kept<GAP>(k), lq = load_kept<GAP>(k + p.inner);
    const float gs = *ks, ls = ks[half * p.us_ts];
    float dg[16], dl[16], a[16];
    {
      float x[16], g[16], l[16];
      decode_raw16<XT>(d, x);
      decode_kept(make_uint2(gq.x, gq.y), gs, g);
      decode_kept(make_uint2(gq.z, gq.w), gs, g + 8);
      decode_kept(make_uint2(lq.x, lq.y), ls, l);
      decode_kept(make_uint2(lq.z, lq.w), ls, l + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const GateParts o = gate_parts(x[i], g[i], l[i]);
        dg[i] = o.dg;
        dl[i] = o.dl;
        a[i] = o.a;
      }
    }
    if constexpr (WIDE) {
      if (p.du) {
        store_raw16<XT, GAP>(p.du, row * p.lddu + col, dg);
        store_raw16<XT, GAP>(p.du, row * p.lddu + p.inner + col, dl);
      }
      if (p.a) store_raw16<XT, GAP>(p.a, row * p.lda + col, a);
      if (!p.q) continue;
    }
    uint8_t* q = p.q + row * p.ldq + col;
    float* s = p.s + row * p.s_rs + tc * p.s_ts;
    quantize_tile<RULE, GAP, PAST>(dg, q, s);
    quantize_tile<RULE, GAP, PAST>(dl, q + p.inner, s + half * p.s_ts);
  }
}

// One 128 x 128 block of da per workgroup, with both halves of the
// checkpoint: thread (rg, cg) holds rows 4 rg .. + 3 of columns 8 cg .. + 7, and
// dg, dl and a of them in fp32 from their forming to their last use.  Rows'
// tiles lie in 16 lanes and leave at once; columns' maxima go through LDS, and
// the transposed bytes are staged there, so that a wave stores whole 128-byte
// rows.
//
// 96 values to a thread: 512 threads at 124 registers, two workgroups to a CU.
// (256 threads that formed every value once per tiling, at 256 registers: 160
// us on 8192 x 4096, this 67 on that box.)  What bounds it is the run of load, maxima, bytes
// and stores in only two workgroups per CU: without the sigmoids and quotients
// 96% of the time remains, without the transposed stores 84%.  LDS is active in 16% of
// the cycles, two fifths of them bank conflicts.  Loading the next block ahead
// spills 97 registers (156 us).
constexpr int kTileThreads = 512;

template <int XT, int RULE>
__global__ __launch_bounds__(kTileThreads, 4) void gate_grad_tile_kernel(GateGradTileArgs p) {
  __shared__ __align__(16) uint8_t tbuf[3 * 128 * kTPitch];
  __shared__ __align__(16) float col_s[3][128], col_y[3][128];
  __shared__ float row_s[2][128];
  __shared__ int odd;  // a column's scale is not a plain one, or its maximum is infinite
  float(*part)[32][128] = reinterpret_cast<float(*)[32][128]>(tbuf);  // 48 of its 54 KB, before the bytes

  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
  const int64_t tr = blockIdx.y, tc = blockIdx.x, half = p.inner >> 7;
  if (tid == 0) odd = 0;

  float v[3][4][8];
  {
    RawRow<XT> d[4];
    RawRow<2> g[4], l[4];
    float gs[4], ls[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = r0 + rg * 4 + i, col = c0 + cg * 8;
      d[i] = load_raw<XT>(p.da, row * p.ldda + col);
      g[i] = load_raw<2>(p.uq, row * p.lduq + col);
      l[i] = load_raw<2>(p.uq, row * p.lduq + p.inner + col);
      gs[i] = p.us[row * p.us_rs + tc * p.us_ts];
      ls[i] = p.us[row * p.us_rs + (half + tc) * p.us_ts];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for_pairs([&](auto col) {
        constexpr int J = decltype(col)::value;
        float d0, d1, g0, g1, l0, l1;
        raw_pair<J>(d[i], d0, d1);
        raw_pair<J>(g[i], g0, g1);
        raw_pair<J>(l[i], l0, l1);
        const GateParts x = gate_parts(d0, g0 * gs[i], l0 * ls[i]), y = gate_parts(d1, g1 * gs[i], l1 * ls[i]);
        v[0][i][J] = x.dg;
        v[0][i][J + 1] = y.dg;
        v[1][i][J] = x.dl;
        v[1][i][J + 1] = y.dl;
        v[2][i][J] = x.a;
        v[2][i][J + 1] = y.a;
      });
  }
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      m[j] = fmaxf(fmaxf(fabsf(v[o][0][j]), fabsf(v[o][1][j])), fmaxf(fabsf(v[o][2][j]), fabsf(v[o][3][j])));
    float* at = &part[o][rg][cg * 8];
    *reinterpret_cast<float4*>(at) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<float4*>(at + 4) = make_float4(m[4], m[5], m[6], m[7]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      float x[8];
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = v[o][i][j];
      const float sc = quantize<RULE, 8>(x, row16_max(amax_of(x)), w);
      st_nt8(p.q + (r0 + rg * 4 + i) * p.ldq + o * p.inner + c0 + cg * 8, make_uint2(w[0], w[1]));
      if (cg == 0) row_s[o][rg * 4 + i] = sc;
    }
  __syncthreads();
  if (tid < 3 * 128) {
    const int o = tid >> 7, c = tid & 127;
    float m = part[o][0][c];
#pragma unroll
    for (int r = 1; r < 32; ++r) m = fmaxf(m, part[o][r][c]);
    const TileScale sc = RULE == 0 ? scale_amax(m) : scale_pow2(m);
    col_s[o][c] = sc.s;
    col_y[o][c] = sc.y;
    if (RULE == 0 ? !plain_amax(m) : !(m <= FLT_MAX)) odd = 1;
    if (o < 2)
      p.st[(o * p.inner + c0 + c) * p.st_rs + tr * p.st_ts] = sc.s;
    else
      p.as[(c0 + c) * p.as_rs + tr * p.as_ts] = sc.s;
  }
  if (tid < 2 * 128) p.s[(r0 + (tid & 127)) * p.s_rs + (tc + (tid >> 7) * half) * p.s_ts] = row_s[tid >> 7][tid & 127];
  __syncthreads();
  const bool slow = odd != 0;
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    float s[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 a = *reinterpret_cast<const float4*>(&col_s[o][cg * 8 + j]);
      const float4 b = *reinterpret_cast<const float4*>(&col_y[o][cg * 8 + j]);
      s[j] = a.x; s[j + 1] = a.y; s[j + 2] = a.z; s[j + 3] = a.w;
      y[j] = b.x; y[j + 1] = b.y; y[j + 2] = b.z; y[j + 3] = b.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = cg * 8 + j;
      float x[4] = {v[o][0][j], v[o][1][j], v[o][2][j], v[o][3][j]};
      uint32_t w;
      if (RULE == 1 && !slow) {
        w = pack4_unclamped(x[0] * y[j], x[1] * y[j], x[2] * y[j], x[3] * y[j]);
      } else if (RULE == 1) {
        // (the scale of an infinite maximum is finite: its quotients saturate)
        w = pack4_saturated(x[0] * y[j], x[1] * y[j], x[2] * y[j], x[3] * y[j]);
      } else if (!slow) {
        w = pack4_unclamped(div_by_scale(x[0], s[j], y[j]), div_by_scale(x[1], s[j], y[j]), div_by_scale(x[2], s[j], y[j]),
                            div_by_scale(x[3], s[j], y[j]));
      } else {
        const float pre = s[j] < kTinyScale ? kTinyLift : 1.0f;
        quotients<RULE, 4>(x, TileScale{s[j], s[j] * pre, y[j], pre});
        w = pack4_saturated(x[0], x[1], x[2], x[3]);
      }
      const int chunk = (rg >> 2) ^ ((c >> 4) & 7);
      *reinterpret_cast<uint32_t*>(tbuf + (o * 128 + c) * kTPitch + chunk * 16 + (rg & 3) * 4) = w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 6; ++it) {
    const int k = it * kTileThreads + tid, o = it >> 1;
    const int c = (k >> 3) & 127, chunk = k & 7;
    uint8_t* out = o < 2 ? p.qt + (o * p.inner + c0 + c) * p.ldqt : p.aq + (c0 + c) * p.ldaq;
    const uint4 w = *reinterpret_cast<const uint4*>(tbuf + (o * 128 + c) * kTPitch + ((chunk ^ ((c >> 4) & 7)) << 4));
    st_nt16(out + r0 + chunk * 16, w);
  }
}

// (One tile for each 8 lanes: by their registers 6 to 8 waves fit a SIMD forward, 6 or 7 in
// the gradient, 4 or 5 with du and a.)
constexpr int64_t kMaxGateBlocks = 1 << 20;

// Workgroups for `rows` (all of them: how many are in use is known on the
// device alone) and the tiles' division constants.
unsigned gate_grid(int64_t rows, int64_t inner, GateGrid& gr) {
  const int64_t tpr = inner / 128, blocks = (rows * tpr + kGroups - 1) / kGroups;
  gr.tpr = make_fast_div((uint32_t)tpr);
  gr.band = make_fast_div((uint32_t)(16 * tpr));
  return (unsigned)(blocks < kMaxGateBlocks ? blocks : kMaxGateBlocks);
}
// Bands of 16 rows where the scales of consecutive rows are adjacent (see
// the 1x128 quantizer).
bool by_bands(int64_t s_rs) { return s_rs == 1; }

template <int XT, int RULE, int ORDER, bool PAST>
hipError_t gate_as(const GateArgs& a, hipStream_t st) {
  GateGrid gr;
  const unsigned blocks = gate_grid(a.rows, a.inner, gr);
  if (a.uq)
    hipLaunchKernelGGL((gate_kernel<XT, RULE, ORDER, true, PAST>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  else
    hipLaunchKernelGGL((gate_kernel<XT, RULE, ORDER, false, PAST>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  return hipGetLastError();
}
template <int XT, int RULE, int ORDER, bool PAST>
hipError_t grad_as(const GateGradArgs& a, hipStream_t st) {
  GateGrid gr;
  const unsigned blocks = gate_grid(a.rows, a.inner, gr);
  if (a.du || a.a)
    hipLaunchKernelGGL((gate_grad_kernel<XT, RULE, ORDER, true, true>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  else
    hipLaunchKernelGGL((gate_grad_kernel<XT, RULE, ORDER, false, PAST>), dim3(blocks), dim3(kGThreads), 0, st, a, gr);
  return hipGetLastError();
}

// The next product's operand is stored ordinarily while the inputs fit the
// caches, and past them beyond.  Forward, gradient and a reader after each, inner
// 4096: 4096 rows 57 us, past the caches 62; 8192 rows 111, 121; 16384 rows 248,
// 232.  The checkpoint, which is read much later, always passes them by, and so
// does the operand beside du and a, which stay in them (5003 x 2048: 26.9 us, 28.4
// with all three ordinary).
template <int XT, int RULE>
hipError_t gate_t(const GateArgs& a, hipStream_t st) {
  const bool past = past_caches(a.rows, 2, a.inner, XT == 0 ? 2 : 4);
  if (by_bands(a.s_rs)) return past ? gate_as<XT, RULE, 1, true>(a, st) : gate_as<XT, RULE, 1, false>(a, st);
  return past ? gate_as<XT, RULE, 0, true>(a, st) : gate_as<XT, RULE, 0, false>(a, st);
}
template <int XT, int RULE>
hipError_t grad_t(const GateGradArgs& a, hipStream_t st) {
  const bool past = past_caches(a.rows, 1, a.inner, XT == 0 ? 4 : 6);
  if (by_bands(a.q ? a.s_rs : 0)) return past ? grad_as<XT, RULE, 1, true>(a, st) : grad_as<XT, RULE, 1, false>(a, st);
  return past ? grad_as<XT, RULE, 0, true>(a, st) : grad_as<XT, RULE, 0, false>(a, st);
}
template <int XT, int RULE>
hipError_t grad_tile_t(const GateGradTileArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.inner / 128), (unsigned)(a.rows / 128));
  hipLaunchKernelGGL((gate_grad_tile_kernel<XT, RULE>), grid, dim3(kTileThreads), 0, st, a);
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
