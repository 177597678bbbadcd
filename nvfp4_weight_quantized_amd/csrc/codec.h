// NVFP4 and E2M1 / E4M3 rounding shared by the quantizers (device code).
#pragma once

#include "common.h"

namespace moe {
namespace {

// Round t in [0, 448] to the nearest E4M3FN value (ties to even); returns the value and its byte.
__device__ __forceinline__ float e4m3_rne(float t, uint32_t* code) {
  if (!(t > 0.f)) {
    *code = 0;
    return 0.f;
  }
  int ex = ilogbf(t);                  // t in [2^ex, 2^(ex+1))
  const int qexp = max(ex, -6) - 3;    // grid spacing 2^qexp
  const float r = rintf(ldexpf(t, -qexp));
  const float v = ldexpf(r, qexp);     // exact
  if (v < 0x1p-6f) {                   // subnormal: m * 2^-9
    *code = (uint32_t)r;
  } else {
    const int ev = ilogbf(v);
    const uint32_t m = (uint32_t)(ldexpf(v, 3 - ev)) - 8u;   // v = (8 + m) * 2^(ev-3)
    *code = ((uint32_t)(ev + 7) << 3) | m;
  }
  return v;
}

// E2M1 code of q (nearest value, ties to even mantissa, saturating at 6); *mag receives the
// magnitude of the value it stands for.
__device__ __forceinline__ uint32_t e2m1_rne(float q, float* mag_out = nullptr) {
  const float mag = fabsf(q);
  const float step_inv = mag < 2.f ? 2.f : (mag < 4.f ? 1.f : 0.5f);
  const float v = fminf(rintf(mag * step_inv) / step_inv, 6.f);
  if (mag_out) *mag_out = v;
  uint32_t c;
  if (v <= 2.f) c = (uint32_t)(v * 2.f);        // 0, .5, 1, 1.5, 2 -> 0..4
  else if (v == 3.f) c = 5u;
  else if (v == 4.f) c = 6u;
  else c = 7u;
  return c | (q < 0.f ? 8u : 0u);
}

// One 16-element group with dequant global scale d: the packed codes (elements 0..7 in `lo`,
// low nibble first), the E4M3 byte of the block scale and (optionally) the values e2m1 * scale the
// codes stand for without the global scale -- at most 6 significant bits, so exact in fp32 and in
// any 16-bit float.
__device__ __forceinline__ void quantize_group16(const float (&v)[16], float d, uint32_t* lo, uint32_t* hi,
                                                 uint32_t* scode, float (*vals)[16] = nullptr) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
  float t = __fdiv_rn(amax, __fmul_rn(6.0f, d));
  t = fminf(t, 448.0f);
  const float s = e4m3_rne(t, scode);
  const float sd = __fmul_rn(s, d);
  *lo = 0;
  *hi = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float qv = (sd > 0.f) ? __fdiv_rn(v[i], sd) : 0.f;
    float mag;
    const uint32_t c = e2m1_rne(qv, &mag);
    if (i < 8) *lo |= c << (4 * i);
    else *hi |= c << (4 * (i - 8));
    if (vals) (*vals)[i] = (c & 8u) ? -(mag * s) : mag * s;
  }
}

// quantize_group16 with the hardware conversions, bit for bit, for 2^-64 <= d <= 2^64 (every
// intermediate below that decides a code is then a normal number).  v_cvt_pk_fp8_f32 and
// v_cvt_scalef32_pk_fp4_f32 round to nearest, ties to even.  The quotients v / (s*d) are correctly rounded:
// with y the correctly rounded reciprocal, two steps q += y * (v - q * sd), the residual exact in the
// fused multiply-add, leave the nearest value (Markstein's theorem: the first step brings q within one
// unit in the last place, the second rounds it correctly).  Values are first limited to 6*s*d, which
// keeps infinities out and turns a NaN into the largest code, as the general routine does; adding +0
// turns -0 into +0, whose code has no sign.
__device__ __forceinline__ void quantize_group16_fast(const float (&v)[16], float d, uint32_t* lo, uint32_t* hi,
                                                      uint32_t* scode) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
  const float t = fminf(__fdiv_rn(amax, __fmul_rn(6.0f, d)), 448.0f);
  const uint32_t sc = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, t, 0, false) & 0xFFu;
  const float s = __builtin_amdgcn_cvt_f32_fp8((int)sc, 0);
  const float sd = __fmul_rn(s, d);
  *scode = sc;
  *lo = *hi = 0;
  if (sd > 0.f) {
    const float y = __fdiv_rn(1.0f, sd), top = 6.0f * sd;
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = fmaxf(fminf(v[i], top), -top);
      float z = x * y;
      z = __fmaf_rn(__fmaf_rn(-z, sd, x), y, z);
      z = __fmaf_rn(__fmaf_rn(-z, sd, x), y, z);
      q[i] = z + 0.0f;
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], q[8 * k], q[8 * k + 1], 1.0f, 0);
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], q[8 * k + 2], q[8 * k + 3], 1.0f, 1);
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], q[8 * k + 4], q[8 * k + 5], 1.0f, 2);
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], q[8 * k + 6], q[8 * k + 7], 1.0f, 3);
    }
    *lo = w[0];
    *hi = w[1];
  }
}

}  // namespace
}  // namespace moe
