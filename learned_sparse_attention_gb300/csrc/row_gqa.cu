// Attention of single rows over the paged KV cache: the packed selection over
// a cache with block scales (qsa_sparse_gqa_scaled) and window attention
// (qsa_window_gqa).
//
// Mathematics.  For row i and query head h of KV head h / G:
//   s_t = (q . k_t) * D^-1/2 * ks_t,  out = sum_t softmax(s)_t vs_t v_t
// over the row's tokens, ks_t / vs_t the scales of the token's block (or the
// cache's static scales, or 1), zero when the row sees nothing; then
// out = bf16(bf16(out) * sigmoid(gate)).  One pass over the tokens with the
// running maximum and sum in fp32.
//
// One CTA per (row, KV head); warps take the tokens in turn, a lane four
// dims of every head of the group; the warps are merged in shared memory.
#include "kv_scale.cuh"
#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int GM, int KVT>
__global__ void __launch_bounds__(kThreads) row_gqa_kernel(const RowGqaParams P) {
  __shared__ float s_m[kWarps][GM], s_l[kWarps][GM];
  __shared__ float s_o[kWarps][GM][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x / P.rows, row = blockIdx.x % P.rows;
  const int req = P.token_to_req[row];
  int n, ns = 0, lo = 0;
  const int32_t* prow = nullptr;
  if (P.packed != nullptr) {
    prow = P.packed + static_cast<long long>(row) * P.packed_width;
    n = prow[P.packed_width - 1];
    if (req < 0 || req >= P.reqs || n < 0 || n >= P.packed_width) {
      if (threadIdx.x == 0) flag_error(P.err);
      n = 0;
    }
  } else {
    if (req < 0 || req >= P.reqs || row < P.qsl[req] || row >= P.qsl[req + 1]) return;
    const int p = P.logical[row];
    ns = min(P.sinks, p + 1);
    lo = max(ns, p - P.window + 1);
    n = p < 0 ? 0 : ns + max(0, p + 1 - lo);
  }
  const int G = P.group;
  float q[GM][4], o[GM][4], m[GM], l[GM];
#pragma unroll
  for (int h = 0; h < GM; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    const uint16_t* qh = P.q + (static_cast<long long>(row) * P.hq + kvh * G + min(h, G - 1)) * 128 + 4 * lane;
    const uint2 v = *reinterpret_cast<const uint2*>(qh);
    q[h][0] = bf16_lo(v.x); q[h][1] = bf16_hi(v.x); q[h][2] = bf16_lo(v.y); q[h][3] = bf16_hi(v.y);
    o[h][0] = o[h][1] = o[h][2] = o[h][3] = 0.f;
  }
  bool bad = false;
  for (int i = warp; i < n; i += kWarps) {
    const int t = prow != nullptr ? prow[i] : i < ns ? i : lo + i - ns;
    const int blk = t < 0 ? -1 : t / P.page;
    const int pid = blk >= 0 && blk < P.bt_stride ? P.block_table[static_cast<long long>(req) * P.bt_stride + blk] : -1;
    if (pid < 0 || pid >= P.num_blocks) {
      bad = true;
      continue;
    }
    const long long r = (static_cast<long long>(pid) * P.hkv + kvh) * P.page + t % P.page;
    float k[4], v[4], ks = 1.f, vs = 1.f;
    if (KVT == QSA_DTYPE_BF16) {
      const uint16_t* x = static_cast<const uint16_t*>(P.kv) + r * 256 + 4 * lane;
      const uint2 a = *reinterpret_cast<const uint2*>(x), b = *reinterpret_cast<const uint2*>(x + 128);
      k[0] = bf16_lo(a.x); k[1] = bf16_hi(a.x); k[2] = bf16_lo(a.y); k[3] = bf16_hi(a.y);
      v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x); v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
    } else {
      const uint8_t* x = static_cast<const uint8_t*>(P.kv) + r * 256 + 4 * lane;
      uint32_t lo2, hi2;
      e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t*>(x), lo2, hi2);
      float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo2)), b = __half22float2(*reinterpret_cast<__half2*>(&hi2));
      k[0] = a.x; k[1] = a.y; k[2] = b.x; k[3] = b.y;
      e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t*>(x + 128), lo2, hi2);
      a = __half22float2(*reinterpret_cast<__half2*>(&lo2));
      b = __half22float2(*reinterpret_cast<__half2*>(&hi2));
      v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
      if (KVT == QSA_DTYPE_E4M3) {
        ks = P.k_scale;
        vs = P.v_scale;
      } else {
        const uint8_t* sc = P.scales + 2 * (r / P.scale_block);
        ks = exp2i(scale_exp(sc[0]));
        vs = exp2i(scale_exp(sc[1]));
      }
    }
    ks *= 0.08838834764831845f;
#pragma unroll
    for (int h = 0; h < GM; ++h) {
      float s = q[h][0] * k[0] + q[h][1] * k[1] + q[h][2] * k[2] + q[h][3] * k[3];
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= ks;
      const float mn = fmaxf(m[h], s);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float al = __expf(m[h] - ref), p = __expf(s - ref);
      m[h] = mn;
      l[h] = l[h] * al + p;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[h][e] = o[h][e] * al + p * vs * v[e];
    }
  }
  if (bad && lane == 0) flag_error(P.err);
#pragma unroll
  for (int h = 0; h < GM; ++h) {
    s_m[warp][h] = m[h];
    s_l[warp][h] = l[h];
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[warp][h][4 * lane + e] = o[h][e];
  }
  __syncthreads();
  for (int h = 0; h < G; ++h) {
    const int d = threadIdx.x;
    float M = -INFINITY, L = 0.f, a = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    if (M == -INFINITY) M = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float wt = __expf(s_m[w][h] - M);
      L += wt * s_l[w][h];
      a += wt * s_o[w][h][d];
    }
    const long long at = (static_cast<long long>(row) * P.hq + kvh * G + h) * 128 + d;
    // (a NaN sum is not an empty row)
    float y = bf16_round(L == 0.f ? 0.f : a / L);
    if (P.gate != nullptr) y = y / (1.0f + __expf(-__uint_as_float(static_cast<uint32_t>(P.gate[at]) << 16)));
    const __nv_bfloat16 b = __float2bfloat16_rn(y);
    P.out[at] = *reinterpret_cast<const uint16_t*>(&b);
  }
}

template <int GM>
cudaError_t launch_group(const RowGqaParams& p, cudaStream_t stream) {
  const dim3 grid(p.rows * p.hkv), block(kThreads);
  switch (p.kv_dtype) {
    case QSA_DTYPE_BF16: return launch_kernel(row_gqa_kernel<GM, QSA_DTYPE_BF16>, grid, block, 0, stream, false, p);
    case QSA_DTYPE_E4M3: return launch_kernel(row_gqa_kernel<GM, QSA_DTYPE_E4M3>, grid, block, 0, stream, false, p);
    default: return launch_kernel(row_gqa_kernel<GM, QSA_DTYPE_E4M3_BLOCK>, grid, block, 0, stream, false, p);
  }
}

}  // namespace

cudaError_t launch_row_gqa(const RowGqaParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  return p.group <= 8 ? launch_group<8>(p, stream) : launch_group<16>(p, stream);
}

}  // namespace qsa
