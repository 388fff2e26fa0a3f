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

// What a row of a biased call sees: tokens lo .. hi (lo > hi: none) from
// position p.
struct Span {
  int p, lo, hi;
  __host__ __device__ __forceinline__ bool sees() const { return lo <= hi; }
};
__host__ __device__ __forceinline__ Span span_at(int p, int window, int doc, int prefix) {
  if (p < 0) return {-1, 0, -1};
  // (clamped from both sides: prefixes may have any value, and what follows adds
  // up to a tile's keys to the last token)
  return {p, max(max(doc, 0), p - window + 1), max(p, min(max(prefix, 1), kMaxKeys) - 1)};
}
__device__ __forceinline__ Span biased_span(const RowGqaParams& P, int row) {
  return span_at(window_position(P, row), P.window, P.doc_start != nullptr ? P.doc_start[row] : 0,
                 P.prefix_end != nullptr ? P.prefix_end[row] : 0);
}

// 1 / x by the PTX approximate reciprocal (1 ulp); 0 for an infinity.
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A capped score's exponent, c2 tanh(s / cap) with c2 = cap log2 e, from
// u = s 2 log2(e) / cap: c2 (1 - 2 / (1 + 2^u)).  The exponential (2^-22 of
// itself, y (1 - y) <= 1/4 of which reaches y = 1 / (1 + 2^u)), the sum, the
// reciprocal and its rounding move y by at most 2^-23.4 + 2^-24 y + 2^-23 y, so
// the score by less than 2^-20 cap.
__device__ __forceinline__ float capped_exponent(float u, float c2) {
  return fmaf(rcp_ftz(1.0f + ex2_ftz(u)), -2.0f * c2, c2);
}

// The tiles have more use for the polynomial of odd powers that is closest to
// tanh up to kMidX: its coefficients of x^3, x^5, .., x^13 (fitted to the least
// error, with fp32 sums 2^-21.4).
constexpr float kMidX = 1.2f;
__host__ __device__ __forceinline__ constexpr float tanh_term(int k) {
  return k == 0   ? -0.33330211f
         : k == 1 ? 0.132966816f
         : k == 2 ? -0.0523968898f
         : k == 3 ? 0.01851172f
         : k == 4 ? -0.00481772097f
                  : 0.000632195501f;
}

// n / page for n >= 0: the multiplication by ceil(2^32 / page) is at most one
// too large.
__device__ __forceinline__ int page_of(const RowGqaParams& P, int n) {
  const unsigned b = __umulhi(static_cast<unsigned>(n), P.page_magic);
  return static_cast<int>(b * P.page > static_cast<unsigned>(n) ? b - 1u : b);
}

// x * sigmoid(g) of bf16 pairs, rounded once; the sigmoid is 1 / (1 + 2^(-g log2
// e)) by the PTX approximate reciprocal (1 ulp): 0 for a gate far below 0, where
// the exponential is an infinity.
__device__ __forceinline__ uint32_t gated_pair(uint32_t x, uint32_t g) {
  float a, b;
  f32x2_unpack(f32x2_mul(f32x2_pack(bf16_lo(g), bf16_hi(g)), f32x2_pack(-kLog2e, -kLog2e)), a, b);
  f32x2_unpack(f32x2_add(f32x2_pack(ex2_ftz(a), ex2_ftz(b)), f32x2_pack(1.0f, 1.0f)), a, b);
  f32x2_unpack(f32x2_mul(f32x2_pack(bf16_lo(x), bf16_hi(x)), f32x2_pack(rcp_ftz(a), rcp_ftz(b))), a, b);
  return pack_bf16x2(a, b);
}

// The gate of 8 dims (bf16x8), or zeros when there is none.
__device__ __forceinline__ uint4 load_gate(const RowGqaParams& P, long long at) {
  return P.gate != nullptr ? *reinterpret_cast<const uint4*>(P.gate + at) : make_uint4(0u, 0u, 0u, 0u);
}

// out[8 dims] = bf16(x * sigmoid(gate)) of bf16 values x, or x without a gate.
__device__ __forceinline__ void store_gated(const RowGqaParams& P, long long at, uint4 x, uint4 g) {
  if (P.gate != nullptr) x = make_uint4(gated_pair(x.x, g.x), gated_pair(x.y, g.y), gated_pair(x.z, g.z), gated_pair(x.w, g.w));
  *reinterpret_cast<uint4*>(P.out + at) = x;
}
// The same of fp32 values, rounded to bf16 first (the sparse GQA stage's
// rounding before its gate).
__device__ __forceinline__ void store_gated8(const RowGqaParams& P, long long at, const float (&x)[8], uint4 g) {
  store_gated(P, at, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                pack_bf16x2(x[6], x[7])), g);
}

}  // namespace qsa
