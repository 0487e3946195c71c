// The quantizer's arithmetic, one explicitly rounded step at a time (the bit-exact contract of
// include/kvq.h), shared by the prefill quantizers and the multi-token append.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

struct GroupParams {
  float scale;   // fp32 value of the fp16 scale
  float zero;    // fp32 value of the fp16 zero
  __half2 sz;    // (scale, zero) as stored
};

__device__ __forceinline__ GroupParams group_params_b(float mn, float mx, int bits) {
  const float levels = static_cast<float>((1 << bits) - 1);
  const float s32 = __fdiv_rn(__fsub_rn(mx, mn), levels);
  __half s16 = __float2half_rn(s32);
  if (__half2float(s16) == 0.0f) s16 = __ushort_as_half(0);          // canonical +0
  const __half z16 = __float2half_rn(__fadd_rn(mn, 0.0f));            // exact, -0 -> +0
  GroupParams g;
  g.scale = __half2float(s16);
  g.zero = __half2float(z16);
  g.sz = __halves2half2(s16, z16);
  return g;
}

__device__ __forceinline__ uint32_t quant_code_b(float x, const GroupParams& g, int bits) {
  if (g.scale == 0.0f) return 0u;
  const float levels = static_cast<float>((1 << bits) - 1);
  float c = rintf(__fdiv_rn(__fsub_rn(x, g.zero), g.scale));          // half-to-even
  c = fminf(fmaxf(c, 0.0f), levels);
  return static_cast<uint32_t>(c);
}

// The code of one element from the group's zero z and the reciprocal r = fl32(1/s) of its
// scale, equal to the quantizer's clamp(rint(fl32(fl32(x - z) / s)), 0, 2^b - 1) wherever
// `near` stays false:
//   with d = fl32(x - z) >= 0, the exact quotient Q = d/s is below 512 (s is the fp16 rounding
//   of (max - min)/(2^b - 1) with b <= 8, or a subnormal at most 1.5x smaller; s = 0 gives
//   r = 0 and code 0).  P = d * r = Q (1 + e), |e| <= 2^-24, so |P - Q| < 2^-15, and the IEEE
//   quotient F = fl32(Q) is within half an ulp, 2^-16, of Q.  y = fma(d, r, 1.5 * 2^23) rounds
//   the exact P to the nearest integer c (ties to even: spacing 1 at that magnitude, and the
//   constant is even), c = y - 1.5 * 2^23 exactly, and t = fma(d, r, -c) is P - c up to 2^-25.
//   If |t| <= 1/2 - 2^-13 then |F - c| < 1/2 - 2^-14, so rint(F) = c; otherwise `near` is set
//   and the caller takes the IEEE division.  No float-to-integer conversion is needed: the
//   integer c is the low bits of y.
constexpr float kNearHalf = 0.5f - 1.0f / 8192.0f;
constexpr float kRoundMagic = 12582912.0f;         // 1.5 * 2^23
constexpr uint32_t kRoundMagicBits = 0x4B400000u;

__device__ __forceinline__ uint32_t code_fast_l(float x, float z, float r, uint32_t levels, bool& near) {
  const float d = __fsub_rn(x, z);
  const float y = __fmaf_rn(d, r, kRoundMagic);
  const float c = __fsub_rn(y, kRoundMagic);
  near |= fabsf(__fmaf_rn(d, r, -c)) > kNearHalf;
  return min(__float_as_uint(y) - kRoundMagicBits, levels);
}

// The quantizer's code with the IEEE division (the rare elements code_fast leaves undecided).
__device__ __forceinline__ uint32_t code_exact_l(float x, float z, float s, uint32_t levels) {
  if (s == 0.0f) return 0u;
  float c = rintf(__fdiv_rn(__fsub_rn(x, z), s));
  c = fminf(fmaxf(c, 0.0f), static_cast<float>(levels));
  return static_cast<uint32_t>(c);
}

}  // namespace kvq
