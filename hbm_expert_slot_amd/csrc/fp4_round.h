// Rounding to 4 bits: the group scale and the codes nearest to the exact quotients.
#pragma once

#include "fp4_device.h"

namespace sc {
namespace fp4 {

// E4M3 byte nearest to t >= 0 (exact quotient up to fp64 rounding, which cannot
// reach a border: borders have 5 bits, the divisor 26, the dividend 24).
__device__ __forceinline__ uint32_t e4m3_of(double t) {
  if (!(t < 448.0)) return 0x7E;
  int e = (int)((__double2hiint(t) >> 20) & 0x7FF) - 1023;
  e = e < -6 ? -6 : e;
  const double up = __hiloint2double((uint32_t)(1023 + 3 - e) << 20, 0);
  const int n = (int)__builtin_rint(t * up);
  return (uint32_t)(((e + 7) << 3) + n - 8);
}

// E2M1 code of a / d, exactly: d * border is exact in fp64.
__device__ __forceinline__ uint32_t e2m1_exact(float a, double d) {
  const double v = a;
  uint32_t c = 0;
  c += v > 0.25 * d;
  c += v >= 0.75 * d;
  c += v > 1.25 * d;
  c += v >= 1.75 * d;
  c += v > 2.5 * d;
  c += v >= 3.5 * d;
  c += v > 5.0 * d;
  return c;
}

// Scale byte and codes (eight to a word) of 16 elements: an NVFP4 group, or half of
// an MXFP4 group, whose other half the neighbouring lane has (they trade maxima).
//
// NVFP4: a quotient in fp32 is off by less than 2^-21 (three roundings and the
// reciprocal's), so where the roundings of (1 -+ 2^-20) times it agree they are the
// exact quotient's; the others are settled in fp64.  MXFP4: the conversion divides by
// a power of two, exactly.
//
// SHORT: the elements are bf16 or fp16 numbers (at most 11 bits).  Where gs is a power
// of two, borders often are quotients then, but no quotient is closer to one without
// being it than 2^-11 (elements and border times divisor have at most 11 and 7 bits),
// so the fp32 quotient rounded to 13 bits is on a border exactly when it should be.
__device__ __forceinline__ float to_13_bits(float q) {
  return __uint_as_float((__float_as_uint(q) + 0x400u) & 0xFFFFF800u);
}
template <int FMT, bool SHORT = false>
__device__ __forceinline__ void round16(const float (&v)[16], float gs, uint32_t& sbyte, u32x2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  if constexpr (FMT == kMx) top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));
  const bool finite = top < 0x7F800000u;
  const bool snap = SHORT && FMT == kNv && (__float_as_uint(gs) & 0x7FFFFFu) == 0;
  float df;   // value of code 1.0, to fp32
  if constexpr (FMT == kNv) {
    const float t = __uint_as_float(top) * (1.0f / (6.0f * gs)), tl = snap ? to_13_bits(t) : t * (1.0f - 0x1p-20f);
    const float th = snap ? tl : t * (1.0f + 0x1p-20f);
    const int two = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(tl, 448.0f), fminf(th, 448.0f), 0, false);
    sbyte = two & 0xFF;
    if (sbyte != (uint32_t)(two >> 8 & 0xFF) || !(gs >= 0x1p-90f && gs <= 0x1p90f))
      sbyte = e4m3_of((double)__uint_as_float(top) / (6.0 * (double)gs));
    if (!finite) sbyte = 0x7F;
    df = __builtin_amdgcn_cvt_pk_f32_fp8((int)sbyte, false)[0] * gs;
  } else {
    // floor(log2) from the exponent field; a denormal max lies below every scale
    const int e = max((int)(top >> 23) - 2, 0);
    sbyte = finite ? (uint32_t)e : 0xFFu;
    df = e == 0 ? 0x1p-127f : __uint_as_float((uint32_t)e << 23);
  }
  uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
  const bool fast = df >= 0x1p-100f && df <= 0x1p100f;
  if (finite && df > 0.0f) {
    if (fast) {
      const float r = __builtin_amdgcn_rcpf(df), rl = r * (1.0f - 0x1p-20f), rh = r * (1.0f + 0x1p-20f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* p = v + 8 * h;
        if constexpr (FMT == kMx) {
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[0], p[1], df, 0);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[2], p[3], df, 1);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[4], p[5], df, 2);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[6], p[7], df, 3);
          hi[h] = lo[h];
        } else if (snap) {
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], to_13_bits(p[0] * r), to_13_bits(p[1] * r), 1.0f, 0);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], to_13_bits(p[2] * r), to_13_bits(p[3] * r), 1.0f, 1);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], to_13_bits(p[4] * r), to_13_bits(p[5] * r), 1.0f, 2);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], to_13_bits(p[6] * r), to_13_bits(p[7] * r), 1.0f, 3);
          hi[h] = lo[h];
        } else {
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[0] * rl, p[1] * rl, 1.0f, 0);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[2] * rl, p[3] * rl, 1.0f, 1);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[4] * rl, p[5] * rl, 1.0f, 2);
          lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], p[6] * rl, p[7] * rl, 1.0f, 3);
          hi[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi[h], p[0] * rh, p[1] * rh, 1.0f, 0);
          hi[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi[h], p[2] * rh, p[3] * rh, 1.0f, 1);
          hi[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi[h], p[4] * rh, p[5] * rh, 1.0f, 2);
          hi[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi[h], p[6] * rh, p[7] * rh, 1.0f, 3);
        }
      }
    }
    if (!fast || lo[0] != hi[0] || lo[1] != hi[1]) {
      // exact: a scale of 4 bits times 24
      const double d = FMT == kNv ? (double)__builtin_amdgcn_cvt_pk_f32_fp8((int)sbyte, false)[0] * (double)gs : (double)df;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __float_as_uint(v[8 * h + e]);
          w |= (e2m1_exact(__uint_as_float(b & 0x7FFFFFFFu), d) | b >> 31 << 3) << (4 * e);
        }
        lo[h] = w;
      }
    }
  }
  codes = u32x2{lo[0], lo[1]};
}

}  // namespace fp4
}  // namespace sc
