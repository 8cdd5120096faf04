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
template <int FMT>
__device__ __forceinline__ void round16(const float (&v)[16], float gs, uint32_t& sbyte, u32x2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  if constexpr (FMT == kMx) top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));
  const bool finite = top < 0x7F800000u;
  double d;   // value of code 1.0: exact
  if constexpr (FMT == kNv) {
    sbyte = finite ? e4m3_of((double)__uint_as_float(top) / (6.0 * (double)gs)) : 0x7Fu;
    const float s = __builtin_amdgcn_cvt_pk_f32_fp8((int)sbyte, false)[0];
    d = (double)s * (double)gs;
  } else {
    // floor(log2) from the exponent field; a denormal max lies below every scale
    const int e = (int)(top >> 23) - 127 - 2;
    const int eb = e < -127 ? -127 : e;
    sbyte = finite ? (uint32_t)(eb + 127) : 0xFFu;
    d = __hiloint2double((uint32_t)(1023 + eb) << 20, 0);
  }
  uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
  const float df = (float)d;
  const bool fast = df >= 0x1p-100f && df <= 0x1p100f;
  if (finite && d > 0.0) {
    if (fast) {
      // the quotient in fp32 is off by less than 2^-22: where the codes of
      // (1 -+ 2^-20) times it agree, they are the exact quotient's
      const float r = 1.0f / df, rl = r * (1.0f - 0x1p-20f), rh = r * (1.0f + 0x1p-20f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* p = v + 8 * h;
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
    if (!fast || lo[0] != hi[0] || lo[1] != hi[1]) {
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
