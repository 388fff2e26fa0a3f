// What the kernels of row_gqa.cu and window_tile.cu share: which rows a call
// owns, and the gated output of a row.
#pragma once

#include "qsa_device.cuh"
#include "qsa_kernels.h"

namespace qsa {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x by the PTX approximate base-2 exponential, subnormal results flushed.
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether a window call's row belongs to the request it names.
__device__ __forceinline__ bool row_live(const RowGqaParams& P, int row, int req) {
  return req >= 0 && req < P.reqs && row >= P.qsl[req] && row < P.qsl[req + 1];
}

// 1 / (1 + 2^(-x log2 e)) by the PTX approximate reciprocal (1 ulp): 0 for a
// gate far below 0, where the exponential is an infinity.
__device__ __forceinline__ float sigmoid_of(uint32_t bf16_bits) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + ex2_ftz(__uint_as_float(bf16_bits << 16) * -kLog2e)));
  return y;
}

// The gate of 8 dims (bf16x8), or zeros when there is none.
__device__ __forceinline__ uint4 load_gate(const RowGqaParams& P, long long at) {
  return P.gate != nullptr ? *reinterpret_cast<const uint4*>(P.gate + at) : make_uint4(0u, 0u, 0u, 0u);
}

// out[8 dims] = bf16(bf16(x) * sigmoid(gate)), or bf16(x) without a gate (the
// rounding before the gate is the sparse GQA stage's).
__device__ __forceinline__ void store_gated8(const RowGqaParams& P, long long at, const float (&x)[8], uint4 g) {
  const uint32_t gv[4] = {g.x, g.y, g.z, g.w};
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = bf16_round(x[2 * e]), b = bf16_round(x[2 * e + 1]);
    if (P.gate != nullptr) {
      a *= sigmoid_of(gv[e] & 0xFFFFu);
      b *= sigmoid_of(gv[e] >> 16);
    }
    o[e] = pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4*>(P.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace qsa
