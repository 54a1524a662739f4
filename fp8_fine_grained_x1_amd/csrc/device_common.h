// Device helpers shared by the quantizer and GEMM kernels (gfx950 only).
//
// FP8 here is OCP E4M3 (bias 7, largest finite 448), which gfx950's
// conversion and matrix instructions use natively.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8fg {

constexpr float kE4M3Max = 448.0f;
constexpr float kFltMinNormal = 1.17549435082228750797e-38f;  // 2^-126

// bf16 halves of a 32-bit word -> fp32 (exact).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// DPP row controls (a DPP row is 16 lanes).
constexpr int kDppQuadXor1 = 0xB1;      // quad_perm [1,0,3,2]
constexpr int kDppQuadXor2 = 0x4E;      // quad_perm [2,3,0,1]
constexpr int kDppRowHalfMirror = 0x141;
constexpr int kDppRowMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Max over the 16 lanes of a DPP row; every lane of the row gets the result.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_mov<kDppQuadXor1>(v));
  v = fmaxf(v, dpp_mov<kDppQuadXor2>(v));
  v = fmaxf(v, dpp_mov<kDppRowHalfMirror>(v));
  v = fmaxf(v, dpp_mov<kDppRowMirror>(v));
  return v;
}

// A tile's scale s (the stored dequantization multiplier) and what the
// quotient x / s is formed from: x * pre divided by d = s * pre, with
// y = RN(1/d).  pre is 1 unless s < 2^-64, where it is 2^64: with tiny
// scales the residual of the FMA correction below falls into FP32's
// denormal range and loses bits (the quotient of x ~ 1.4e-38 by
// s ~ 2e-36 came out one ulp low), while the same quotient of the operands
// scaled by 2^64 -- exactly, both being powers of two apart from s -- has a
// normal residual whenever x / s is large enough to matter for E4M3
// (>= 2^-11).
struct TileScale {
  float s;
  float d;
  float y;
  float pre;
};

constexpr float kTinyScale = 5.42101086242752217004e-20f;  // 2^-64
constexpr float kTinyLift = 18446744073709551616.0f;        // 2^64

// s = max(RN(amax / 448), 2^-126); the divisions are the compiler's
// correctly rounded fp32 division (no fast-math is used).
__device__ __forceinline__ TileScale scale_amax(float amax) {
  const float s = fmaxf(amax / kE4M3Max, kFltMinNormal);
  const float pre = s < kTinyScale ? kTinyLift : 1.0f;
  const float d = s * pre;
  return {s, d, 1.0f / d, pre};
}

// s = max(2^k, 2^-126) with k the least integer such that 448 * 2^k >= amax.
// With amax = 1.f * 2^e: amax / 448 = (1.f / 1.75) * 2^(e - 8), so
// k = e - 8 when 1.f <= 1.75 (mantissa field <= 0x600000) and e - 7 otherwise.
// Zero and subnormal amax fall below the floor.  x / s = x * 2^-k is exact
// (or below the E4M3 range), so y = 2^-k is all the quotient needs.
__device__ __forceinline__ TileScale scale_pow2(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int k = (int)((u >> 23) & 0xFFu) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = k < -126 ? -126 : k;
  const float s = __uint_as_float((uint32_t)(k + 127) << 23);
  return {s, s, __uint_as_float((uint32_t)(127 - k) << 23), 1.0f};
}

// Correctly rounded x / d from y = RN(1/d) (Markstein's FMA-based quotient
// correction; P. Markstein, IBM J. Res. Dev. 34(1), 1990), valid while the
// residual does not underflow (see TileScale).  The residual is formed as
// d*q0 - x so that x = -0 keeps its sign.
__device__ __forceinline__ float div_by_scale(float x, float d, float y) {
  const float q0 = x * y;
  const float r = __builtin_fmaf(d, q0, -x);
  return __builtin_fmaf(-r, y, q0);
}

// x / s under either rule (RULE 0: amax, 1: power of two).
template <int RULE>
__device__ __forceinline__ float quotient(float x, const TileScale& t) {
  if constexpr (RULE == 0) {
    return div_by_scale(x * t.pre, t.d, t.y);
  } else {
    return x * t.y;
  }
}

// x / s for N values with one scale per lane.  Under the amax rule the
// pre-scaling multiply is skipped when no active lane of the wave has a tiny
// scale (a wave-uniform branch; there it is a multiply by 1).
template <int RULE, int N>
__device__ __forceinline__ void quotients(float (&v)[N], const TileScale& t) {
  if constexpr (RULE == 0) {
    if (__builtin_amdgcn_ballot_w64(t.pre != 1.0f) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = div_by_scale(v[i], t.d, t.y);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = div_by_scale(v[i] * t.pre, t.d, t.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] * t.y;
  }
}
template <int RULE>
__device__ __forceinline__ void quotient8(float (&v)[8], const TileScale& t) {
  quotients<RULE, 8>(v, t);
}

// Four fp32 values -> four E4M3 bytes (first value in the lowest byte),
// round-to-nearest-even; values are clamped to +-448 first (saturation).
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  a = __builtin_amdgcn_fmed3f(a, -kE4M3Max, kE4M3Max);
  b = __builtin_amdgcn_fmed3f(b, -kE4M3Max, kE4M3Max);
  c = __builtin_amdgcn_fmed3f(c, -kE4M3Max, kE4M3Max);
  d = __builtin_amdgcn_fmed3f(d, -kE4M3Max, kE4M3Max);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Four E4M3 bytes of a word -> fp32 (exact).
__device__ __forceinline__ void unpack4_e4m3(uint32_t w, float out[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  out[0] = lo[0];
  out[1] = lo[1];
  out[2] = hi[0];
  out[3] = hi[1];
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Non-temporal 16- and 8-byte accesses, for data that streams through once.
__device__ __forceinline__ uint4 ld_nt16(const void* p) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint2 ld_nt8(const void* p) {
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
  return make_uint2(v[0], v[1]);
}
__device__ __forceinline__ void st_nt8(void* p, uint2 v) {
  const u32x2 w = {v.x, v.y};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(p));
}
__device__ __forceinline__ void st_nt16(void* p, uint4 v) {
  const u32x4 w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
}

// 8 consecutive elements as fp32 (XT 0: bf16, 1: f32), non-temporal.
template <int XT>
__device__ __forceinline__ void load8(const void* __restrict__ x, int64_t off, float v[8]) {
  if constexpr (XT == 0) {
    const uint4 w = ld_nt16(reinterpret_cast<const uint16_t*>(x) + off);
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
    v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
  } else {
    const float* p = reinterpret_cast<const float*>(x) + off;
    const uint4 a = ld_nt16(p), b = ld_nt16(p + 4);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values -> bf16 pair (round-to-nearest-even), first in the low half.
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// 8 consecutive elements in their own encoding (XT 0: bf16, 1: f32): kept
// undecoded where they wait in registers for a second use.
template <int XT>
struct Raw8;
template <>
struct Raw8<0> {
  uint4 w;
};
template <>
struct Raw8<1> {
  uint4 a, b;
};

template <int XT>
__device__ __forceinline__ void decode8(const Raw8<XT>& r, float v[8]) {
  if constexpr (XT == 0) {
    v[0] = bf16_lo(r.w.x); v[1] = bf16_hi(r.w.x);
    v[2] = bf16_lo(r.w.y); v[3] = bf16_hi(r.w.y);
    v[4] = bf16_lo(r.w.z); v[5] = bf16_hi(r.w.z);
    v[6] = bf16_lo(r.w.w); v[7] = bf16_hi(r.w.w);
  } else {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
  }
}

// fp32 values rounded to the element type (bf16: nearest-even; f32: as is).
template <int XT>
__device__ __forceinline__ Raw8<XT> encode8(const float v[8]) {
  Raw8<XT> r;
  if constexpr (XT == 0) {
    r.w = make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
  } else {
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  }
  return r;
}

// Ordinary (cached) and non-temporal forms; p + off is 16-byte aligned.
template <int XT, bool NT>
__device__ __forceinline__ Raw8<XT> load_raw8(const void* __restrict__ p, int64_t off) {
  Raw8<XT> r;
  if constexpr (XT == 0) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + off;
    r.w = NT ? ld_nt16(q) : *reinterpret_cast<const uint4*>(q);
  } else {
    const float* q = reinterpret_cast<const float*>(p) + off;
    r.a = NT ? ld_nt16(q) : *reinterpret_cast<const uint4*>(q);
    r.b = NT ? ld_nt16(q + 4) : *reinterpret_cast<const uint4*>(q + 4);
  }
  return r;
}

template <int XT, bool NT>
__device__ __forceinline__ void store_raw8(void* __restrict__ p, int64_t off, const Raw8<XT>& r) {
  if constexpr (XT == 0) {
    uint16_t* q = reinterpret_cast<uint16_t*>(p) + off;
    if constexpr (NT) st_nt16(q, r.w); else *reinterpret_cast<uint4*>(q) = r.w;
  } else {
    float* q = reinterpret_cast<float*>(p) + off;
    if constexpr (NT) {
      st_nt16(q, r.a);
      st_nt16(q + 4, r.b);
    } else {
      *reinterpret_cast<uint4*>(q) = r.a;
      *reinterpret_cast<uint4*>(q + 4) = r.b;
    }
  }
}

// Orders the wave's LDS accesses before and after it (a wave runs its LDS
// instructions in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// 16 bytes of elements (XT 0: 8 bf16, 1: 4 f32): what one lane reads or writes
// with one instruction, so that a wave's accesses are contiguous.
template <int XT>
constexpr int kPer16 = XT == 0 ? 8 : 4;

template <int XT, bool NT>
__device__ __forceinline__ uint4 load16(const void* __restrict__ p, int64_t off) {
  const char* q = reinterpret_cast<const char*>(p) + off * (XT == 0 ? 2 : 4);
  return NT ? ld_nt16(q) : *reinterpret_cast<const uint4*>(q);
}
template <int XT, bool NT>
__device__ __forceinline__ void store16(void* __restrict__ p, int64_t off, uint4 w) {
  char* q = reinterpret_cast<char*>(p) + off * (XT == 0 ? 2 : 4);
  if constexpr (NT)
    st_nt16(q, w);
  else
    *reinterpret_cast<uint4*>(q) = w;
}
template <int XT>
__device__ __forceinline__ void decode16(uint4 w, float (&v)[kPer16<XT>]) {
  if constexpr (XT == 0) {
    decode8<0>(Raw8<0>{w}, v);
  } else {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
}
template <int XT>
__device__ __forceinline__ uint4 encode16(const float (&v)[kPer16<XT>]) {
  if constexpr (XT == 0)
    return encode8<0>(v).w;
  else
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// A value and its counterpart 16 or 32 lanes away, in either order (the swap
// of a register with itself leaves the lower half's in one result and the
// upper half's in the other).
struct LanePair {
  uint32_t a, b;
};
template <int STEP>
__device__ __forceinline__ LanePair lane_pair(uint32_t v) {
  static_assert(STEP == 16 || STEP == 32, "rows or halves");
  if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return {r[0], r[1]};
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return {r[0], r[1]};
  }
}
template <int STEP>
__device__ __forceinline__ float pair_sum(float v) {
  const LanePair p = lane_pair<STEP>(__float_as_uint(v));
  return __uint_as_float(p.a) + __uint_as_float(p.b);
}
template <int STEP>
__device__ __forceinline__ float pair_max(float v) {
  const LanePair p = lane_pair<STEP>(__float_as_uint(v));
  return fmaxf(__uint_as_float(p.a), __uint_as_float(p.b));
}

// Sum over the 16 lanes of a DPP row, over 32 or over all 64 lanes of a
// wave; every lane gets the result.  The order of additions is fixed.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_mov<kDppQuadXor1>(v);
  v += dpp_mov<kDppQuadXor2>(v);
  v += dpp_mov<kDppRowHalfMirror>(v);
  v += dpp_mov<kDppRowMirror>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return pair_sum<32>(pair_sum<16>(row16_sum(v))); }

}  // namespace fp8fg
