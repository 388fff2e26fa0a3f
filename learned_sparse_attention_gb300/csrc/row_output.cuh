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

// A window call's position of a row, -1 before the start.  (Room above it for
// the bounds of its key tile; no table reaches there.)
__device__ __forceinline__ int window_position(const RowGqaParams& P, int row) {
  return max(-1, min(P.logical[row], kMaxKeys));
}

// n / page for n >= 0: the multiplication by ceil(2^32 / page) is at most one
// too large.
__device__ __forceinline__ int page_of(const RowGqaParams& P, int n) {
  const unsigned b = __umulhi(static_cast<unsigned>(n), P.page_magic);
  return static_cast<int>(b * P.page > static_cast<unsigned>(n) ? b - 1u : b);
}

// 1 / (1 + 2^(-x log2 e)) by the PTX approximate reciprocal (1 ulp): 0 for a
// gate far below 0, where the exponential is an infinity.
__device__ __forceinline__ float sigmoid_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + ex2_ftz(x * -kLog2e)));
  return y;
}

// The gate of 8 dims (bf16x8), or zeros when there is none.
__device__ __forceinline__ uint4 load_gate(const RowGqaParams& P, long long at) {
  return P.gate != nullptr ? *reinterpret_cast<const uint4*>(P.gate + at) : make_uint4(0u, 0u, 0u, 0u);
}

// out[8 dims] = bf16(x * sigmoid(gate)) of bf16 values x, or x without a gate.
__device__ __forceinline__ void store_gated(const RowGqaParams& P, long long at, uint4 x, uint4 g) {
  if (P.gate != nullptr) {
    uint32_t xv[4] = {x.x, x.y, x.z, x.w};
    const uint32_t gv[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      xv[e] = pack_bf16x2(bf16_lo(xv[e]) * sigmoid_of(bf16_lo(gv[e])), bf16_hi(xv[e]) * sigmoid_of(bf16_hi(gv[e])));
    x = make_uint4(xv[0], xv[1], xv[2], xv[3]);
  }
  *reinterpret_cast<uint4*>(P.out + at) = x;
}
// The same of fp32 values, rounded to bf16 first (the sparse GQA stage's
// rounding before its gate).
__device__ __forceinline__ void store_gated8(const RowGqaParams& P, long long at, const float (&x)[8], uint4 g) {
  store_gated(P, at, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                pack_bf16x2(x[6], x[7])), g);
}

}  // namespace qsa
