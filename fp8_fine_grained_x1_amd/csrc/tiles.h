// Helpers shared by the kernels that work tile by tile: the quantizers
// (quant.hip), the silu gate (gate.hip) and, for the quantization of a tile,
// the norms around a block (block_norm.hip).
#pragma once

#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "device_common.h"

namespace fp8fg {

namespace {

constexpr int kTPitch = 144;  // LDS row pitch (bytes) of the transposing store

// n / d for 32-bit n by multiply-high and shift (Granlund & Montgomery,
// "Division by invariant integers using multiplication", PLDI 1994):
// with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (umulhi(n, m) + n) >> l for every n < 2^32 (the sum is formed in
// 64 bits).
struct FastDiv {
  uint32_t d, m, l;
};

__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  const uint64_t t = (uint64_t)__umulhi(n, f.m) + n;
  return (uint32_t)(t >> f.l);
}

inline FastDiv make_fast_div(uint32_t d) {
  uint32_t l = 0;
  while (l < 32 && (1ull << l) < d) ++l;
  const uint64_t m = ((1ull << 32) * ((1ull << l) - d)) / d + 1;
  return FastDiv{d, (uint32_t)m, l};
}

// Tile t's row and tile column.  ORDER 0 numbers the tiles row-major, ORDER 1
// in bands of 16 rows, tile column by tile column (the last band may have
// fewer rows).
template <int ORDER>
__device__ __forceinline__ void tile_rc(uint32_t t, const FastDiv& tpr, const FastDiv& band,
                                        uint32_t rows, uint32_t& r, uint32_t& tc) {
  if constexpr (ORDER == 0) {
    r = fast_div(t, tpr);
    tc = t - r * tpr.d;
  } else {
    const uint32_t b = fast_div(t, band);
    const uint32_t u = t - b * band.d;
    const uint32_t h = rows - 16u * b;  // rows in this band (16 except in the last)
    if (h >= 16u) {
      tc = u >> 4;
      r = 16u * b + (u & 15u);
    } else {
      tc = u / h;
      r = 16u * b + (u - tc * h);
    }
  }
}

// 8 consecutive elements in their input encoding.
template <int XT>
struct RawRow;
template <>
struct RawRow<0> {  // 8 bf16
  uint4 w;
};
template <>
struct RawRow<1> {  // 8 f32
  uint4 a, b;
};
template <>
struct RawRow<2> {  // 8 E4M3 bytes
  uint2 w;
};

template <int XT>
__device__ __forceinline__ RawRow<XT> load_raw(const void* __restrict__ x, int64_t off) {
  RawRow<XT> r;
  if constexpr (XT == 0) {
    r.w = ld_nt16(reinterpret_cast<const uint16_t*>(x) + off);
  } else if constexpr (XT == 1) {
    const float* p = reinterpret_cast<const float*>(x) + off;
    r.a = ld_nt16(p);
    r.b = ld_nt16(p + 4);
  } else {
    r.w = ld_nt8(reinterpret_cast<const uint8_t*>(x) + off);
  }
  return r;
}

// Elements J and J + 1 (J even) of a raw row, exactly as fp32.
template <int J, int XT>
__device__ __forceinline__ void raw_pair(const RawRow<XT>& r, float& a, float& b) {
  static_assert(J % 2 == 0 && J < 8, "pairs start at even columns");
  if constexpr (XT == 0) {
    const uint32_t w = J == 0 ? r.w.x : J == 2 ? r.w.y : J == 4 ? r.w.z : r.w.w;
    a = bf16_lo(w);
    b = bf16_hi(w);
  } else if constexpr (XT == 1) {
    const uint4& h = J < 4 ? r.a : r.b;
    a = __uint_as_float((J & 3) == 0 ? h.x : h.z);
    b = __uint_as_float((J & 3) == 0 ? h.y : h.w);
  } else {
    const auto f = __builtin_amdgcn_cvt_pk_f32_fp8((int)(J < 4 ? r.w.x : r.w.y), (J & 2) != 0);
    a = f[0];
    b = f[1];
  }
}

// Hides a raw row's registers from the optimizer (no instruction is
// emitted): the values decoded before this point cannot be reused after it,
// so the second pass decodes again instead of keeping 64 floats live.
template <int XT>
__device__ __forceinline__ void refresh(RawRow<XT>& r) {
  if constexpr (XT == 0) {
    asm volatile("" : "+v"(r.w.x), "+v"(r.w.y), "+v"(r.w.z), "+v"(r.w.w));
  } else if constexpr (XT == 1) {
    asm volatile("" : "+v"(r.a.x), "+v"(r.a.y), "+v"(r.a.z), "+v"(r.a.w));
    asm volatile("" : "+v"(r.b.x), "+v"(r.b.y), "+v"(r.b.z), "+v"(r.b.w));
  } else {
    asm volatile("" : "+v"(r.w.x), "+v"(r.w.y));
  }
}

template <int J>
struct ColTag {
  static constexpr int value = J;
};
template <typename F, int... P>
__device__ __forceinline__ void for_pairs_impl(F&& f, std::integer_sequence<int, P...>) {
  (f(ColTag<2 * P>{}), ...);
}
// f(ColTag<0>{}), f(ColTag<2>{}), .. f(ColTag<6>{}): the first column of
// each pair as a compile-time constant.
template <typename F>
__device__ __forceinline__ void for_pairs(F&& f) {
  for_pairs_impl(f, std::make_integer_sequence<int, 4>{});
}

template <int N>
__device__ __forceinline__ float amax_of(const float (&v)[N]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// Four E4M3 bytes of quotients by a scale of finite values: none exceeds
// 448 (1 + 2^-24), which rounds to 448 by itself.
__device__ __forceinline__ uint32_t pack4_unclamped(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Four E4M3 bytes of any quotients: beyond 448 they saturate, a NaN stays one
// (as it does above, so that a row's bytes do not depend on which form its
// wave takes).
__device__ __forceinline__ uint32_t pack4_saturated(float a, float b, float c, float d) {
  const auto held = [](float x) { return __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, -kE4M3Max), kE4M3Max); };
  return pack4_unclamped(held(a), held(b), held(c), held(d));
}

// Whether scale_amax and its quotients need none of their steps for tiny
// scales, infinities and NaN.
constexpr float kLeastPlain = 0x1p-55f;
__device__ __forceinline__ bool plain_amax(float m) { return m >= kLeastPlain && m <= 3.40282347e38f; }

// RN(m / 448) and RN(1 / s) of such an m, as scale_amax has them, in 8
// instructions instead of 26.  Both are correction steps in fused
// multiply-adds (Markstein, as in div_by_scale): from RN(1 / 448) for every m,
// and from the hardware's reciprocal for every s -- which a step of one
// correction does not give for any reciprocal within an ulp, but does for
// this one: tests/test_gpu_tile_scale_sweep.py has the scales and quotients of all
// 2^23 significands of m.
__device__ __forceinline__ TileScale plain_scale(float m) {
  const float inv448 = 1.0f / 448.0f;
  const float q = m * inv448;
  const float s = __builtin_fmaf(__builtin_fmaf(-448.0f, q, m), inv448, q);
  const float y = __builtin_amdgcn_rcpf(s);
  return {s, s, __builtin_fmaf(__builtin_fmaf(-s, y, 1.0f), y, y), 1.0f};
}

// N values (a multiple of 4) to E4M3 with the tile's maximum m; `out` gets
// N / 4 words.  Returns the scale.
template <int RULE, int N>
__device__ __forceinline__ float quantize(float (&v)[N], float m, uint32_t (&out)[N / 4]) {
  if (RULE == 0 && __builtin_amdgcn_ballot_w64(!plain_amax(m)) == 0) {
    const TileScale sc = plain_scale(m);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      out[i] = pack4_unclamped(div_by_scale(v[4 * i], sc.d, sc.y), div_by_scale(v[4 * i + 1], sc.d, sc.y),
                               div_by_scale(v[4 * i + 2], sc.d, sc.y), div_by_scale(v[4 * i + 3], sc.d, sc.y));
    return sc.s;
  }
  const TileScale sc = RULE == 0 ? scale_amax(m) : scale_pow2(m);
  quotients<RULE, N>(v, sc);
  // (under the power-of-two rule 448 of the scale are at least a finite maximum)
  if (RULE == 1 && __builtin_amdgcn_ballot_w64(!(m <= FLT_MAX)) == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) out[i] = pack4_unclamped(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    return sc.s;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) out[i] = pack4_saturated(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  return sc.s;
}

}  // namespace

}  // namespace fp8fg
