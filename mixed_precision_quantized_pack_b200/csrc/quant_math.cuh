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

}  // namespace kvq
