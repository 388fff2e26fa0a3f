// Power-of-two block scales of an e4m3 KV cache: one byte b for the K, one
// for the V of each block of tokens and KV head, standing for 2^(b - 127).
#pragma once

#include <cuda_fp16.h>

#include "qsa_device.cuh"

namespace qsa {

// Exponents are held within +-40: e4m3 then covers 2^-49 .. 448 * 2^40, far
// beyond any key or value, and the quotient of two blocks' scales stays
// inside fp32 beside a softmax weight.
constexpr int kScaleExpMax = 40;

__host__ __device__ __forceinline__ int scale_exp(int byte) {
  const int e = byte - 127;
  return e < -kScaleExpMax ? -kScaleExpMax : e > kScaleExpMax ? kScaleExpMax : e;
}

// 2^e for |e| <= 126
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// |x|, or 0 for an infinity or a NaN
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// The smallest e within the limits with a <= 448 * 2^e = 1.75 * 2^(e + 8),
// from a's exponent and mantissa (a >= 0 and finite).
__device__ __forceinline__ int scale_exp_for(float a) {
  const int bits = __float_as_int(a);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return e < -kScaleExpMax ? -kScaleExpMax : e > kScaleExpMax ? kScaleExpMax : e;
}

// Four e4m3 codes times s (a power of two <= 1), rounded to e4m3.
__device__ __forceinline__ uint32_t rescale4(float s, uint32_t w) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return static_cast<uint32_t>(f32x2_to_e4m3x2(a.x * s, a.y * s)) |
         (static_cast<uint32_t>(f32x2_to_e4m3x2(b.x * s, b.y * s)) << 16);
}
__device__ __forceinline__ uint4 rescale16(float s, uint4 v) {
  return make_uint4(rescale4(s, v.x), rescale4(s, v.y), rescale4(s, v.z), rescale4(s, v.w));
}

}  // namespace qsa
