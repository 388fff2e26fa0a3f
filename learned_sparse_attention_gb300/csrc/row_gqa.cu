// Attention of single rows over the paged KV cache: the packed selection over
// a cache with block scales (qsa_sparse_gqa_scaled), window attention of few
// rows per request (qsa_window_gqa), and the same with capped or biased scores,
// documents and prefixes (qsa_biased_gqa).
//
// Mathematics.  For row i and query head h of KV head h / G, over the row's
// tokens t with scales ks_t, vs_t (of the token's block, static, or 1):
//   s_t = (q . k_t) * D^-1/2 * ks_t,   out = sum_t softmax(s)_t vs_t v_t,
// zero when the row sees nothing, then out = bf16(bf16(out) * sigmoid(gate)).
// One pass over the tokens.  The exponentials are taken against a reference m
// that moves only when a score passes it by a margin; with block scales the
// weight that meets v_t is p_t = 2^(s_t log2 e + log2 vs_t - m), and the sum
// of the softmax adds p_t / vs_t, so neither scale costs a multiplication of
// the K or V tile.
//
// e4m3 codes become f16 right before their MMA (exact, two a conversion), q is
// f16 times a power of two per head (exact but for elements 2^-28 below its
// largest), p is f16.  (m16n8k32 MMAs on the codes, with q and p as two e4m3
// terms, are correct too, but this part has none in hardware: 900
// instructions a slab instead of 400.)
//
// Bound: HBM (256 or 512 contiguous bytes of each token and KV head).  One CTA
// per (row, KV head, split), four warps, each with its own cp.async ring over
// slabs of 16 (bf16) or 32 tokens; a warp finds its slabs' cache rows itself,
// two slabs ahead of their copies, so the loop has no block barrier.  Both
// products have the heads on M (16: one or two blocks of 8) and the tokens
// (S = Q K^T) or dims (O = P V) on N, so a lane's scores are the P fragment it
// needs next.  Of e4m3 rows a lane holds 4 consecutive bytes where bf16 rows
// give it 2 + 2: dims (K) and tokens (V) are taken in that order, by q's
// fragments and by K's rows (tau, below).  Splits join in a fixed order: in a
// cluster, or as fp32 partials that a second kernel reads.
// Roundings.  Weights become bf16 (bf16 values) or f16 (e4m3 values) because an
// MMA's operands have one type; the softmax's sum adds them unrounded.  That is
// up to 2^-8 or 2^-11 of a weight, either way, where the output is rounded to
// 2^-8 of itself; a second term for the rest would double the products.  f16
// weights end at 2^-24 of the largest: with block scales a token whose weight
// times V scale is that far below the row's largest adds nothing to the output.
// The approximate exponential and reciprocal (2^-22) lie far below both.
// Measured, ten calls on ten sets of inputs: 64 rows of 32 query and 4 KV heads
// over block scales, the last 4100 tokens 48.0 us (5.6 TB/s; e4m3 decoded as two
// e4m3 terms 72 us), 2051 selected ones 35.8 us (3.8 TB/s; as many contiguous
// ones 34.6 us, and 28.8 as a window, which looks up no packed entries: what it
// waits for is the chain of lookups, not the runs of 1 KB); 8 rows of 64 and 8
// heads, 4103 selected tokens in 4 splits 23.7 us (18.7 with inputs in L2).
// Biased calls: a capped score takes one more exponential and a reciprocal, a
// distance one multiply-add; 64 rows of ~4100 to 8192 tokens over block scales 84
// us with masks alone, 83 with a cap, 87 with slopes, 88 with both (4.5 TB/s; the
// chains of eight warps an SM, unpacking among them, and the longest rows' CTAs
// bound it: static e4m3 79 us, 5.1 TB/s; bf16 130 us, 6.2).
#include <cooperative_groups.h>

#include "kv_scale.cuh"
#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"
#include "row_output.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kBadRow = 0xFFFFFFFFu;

// Two 16x16 byte matrices, transposed: lanes 0-15 point at the rows of the
// first, 16-31 of the second.  Lane (g, t) gets, of each, the four bytes of
// rows 4t .. 4t+3 in column g (r[0], r[2]) and in column g + 8 (r[1], r[3]).
__device__ __forceinline__ void ldmatrix_b8_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
// 4-byte asynchronous copy of src_bytes bytes, the rest zero.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(src_bytes)
               : "memory");
}

// Layout by cache type: KVT 0 bf16, 1 e4m3 with static scales, 2 e4m3 with
// block scales.  TS: tokens of a slab.
template <int KVT>
struct RowPlan {
  static constexpr bool kE4m3 = KVT != 0;
  static constexpr int TS = kE4m3 ? 32 : 16;
  static constexpr int kRowB = kE4m3 ? 128 : 256;     // bytes of a token's K (or V)
  static constexpr int kSlab = TS * kRowB * 2;        // 8 KB: K rows, then V rows
  static constexpr int kStages = 3;
  // the margin (log2) by which a weight may pass the reference
  static constexpr float kUp = 8.0f;
  static constexpr int kSmem = kWarps * kStages * kSlab;
};

// K rows are swizzled so that the 8 rows of one ldmatrix matrix (e4m3: rows
// tau(nb, 0..7)) fall on different banks, V rows by their own 8 neighbours.
template <int KVT>
__device__ __forceinline__ int swz_k(int tok) {
  return KVT == 0 ? tok & 7 : (tok & 1) | ((tok >> 1) & 6);
}

// HB: blocks of 8 query heads (groups of 16: 2), the halves of an M of 16.
// MOD: a biased call.  Its tokens come nearest to the row first, so that with a
// distance bias the reference does not have to follow the scores up.
template <int KVT, int HB, bool MOD>
__global__ void __launch_bounds__(kThreads, 2) row_gqa_kernel(const RowGqaParams P) {
  using RP = RowPlan<KVT>;
  constexpr int TS = RP::TS, ST = RP::kStages;
  constexpr int NBK = TS / 8;                // column blocks of S
  constexpr int NT = TS / 4;                 // tokens of a lane: 4 or 8
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_raw[kWarps][ST][KVT == 2 ? 32 : 1];  // scale words as copied
  __shared__ float4 s_scl[kWarps][3][KVT == 2 ? 8 : 1];      // ks, log2 vs, 1 / vs of a slab
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // KV-head-major order: rows of one request that share tokens meet in L2
  // (with clusters, the splits of a row and KV head are one)
  const int pair = P.cluster ? static_cast<int>(blockIdx.x) / P.splits : static_cast<int>(blockIdx.x);
  const int kvh = pair / P.rows, row = pair % P.rows;
  const int split = P.cluster ? static_cast<int>(blockIdx.x) % P.splits : static_cast<int>(blockIdx.y);
  const int G = P.group;
  const int req = P.token_to_req[row];
  griddep_launch_dependents();

  // ---- the row's tokens: entries of the packed row, or the sinks and the window
  int n, ns = 0, lo = 0;
  [[maybe_unused]] int pos = 0;
  const int32_t* prow = nullptr;
  if constexpr (MOD) {
    if (!row_live(P, row, req)) return;
    const Span span = biased_span(P, row);
    pos = span.p;
    lo = span.lo;
    n = max(0, min(span.hi, P.keys - 1) - lo + 1);
    if (span.sees() && span.hi >= P.keys && threadIdx.x == 0) flag_error(P.err);
  } else if (P.packed != nullptr) {
    prow = P.packed + static_cast<long long>(row) * P.packed_width;
    n = prow[P.packed_width - 1];
    if (req < 0 || req >= P.reqs || n < 0 || n >= P.packed_width) {
      if (threadIdx.x == 0) flag_error(P.err);
      n = 0;
    }
  } else {
    if (!row_live(P, row, req)) return;
    const int p = window_position(P, row);
    const int end = min(p + 1, P.keys);  // (a position may lie past the table)
    ns = min(P.sinks, end);
    lo = max(ns, p - P.window + 1);
    n = p < 0 ? 0 : ns + max(0, end - lo);
    if (p >= P.keys && threadIdx.x == 0 && (P.window > 0 || P.sinks > P.keys)) flag_error(P.err);
  }
  const int nslab = (n + TS - 1) / TS;
  const int per = (nslab + P.splits - 1) / P.splits;
  const int sb = split * per, se = min(nslab, sb + per);
  const int cnt = se > sb + warp ? (se - sb - warp + kWarps - 1) / kWarps : 0;  // slabs of this warp
  const int32_t* bt_row = P.block_table + static_cast<long long>(n > 0 ? req : 0) * P.bt_stride;
  // the tokens and pages of a warp's slab i: lane l < TS its l-th token
  auto fetch_tok = [&](int i) -> int {
    const int at = (sb + warp + kWarps * i) * TS + lane;
    if (i >= cnt || lane >= TS || at >= n) return -1;
    if constexpr (MOD) return lo + n - 1 - at;
    if (prow == nullptr) return at < ns ? at : lo + at - ns;
    const int e = prow[at];
    return e < 0 ? -2 : e;  // (-1: no token; -2: an entry that is none)
  };
  auto fetch_page = [&](int tok) -> int {
    if (tok < 0) return -1;
    const int blk = page_of(P, tok);
    return blk < P.bt_stride ? bt_row[blk] : -1;
  };
  bool bad = false;
  auto row_id = [&](int tok, int page) -> uint32_t {
    if (tok == -1) return kBadRow;
    if (tok < 0 || page < 0 || page >= P.num_blocks) {
      bad = true;
      return kBadRow;
    }
    return (static_cast<uint32_t>(page) * P.hkv + kvh) * static_cast<uint32_t>(P.page) + (tok - page_of(P, tok) * P.page);
  };
  int tok[ST + 1], pg[ST];
#pragma unroll
  for (int i = 0; i <= ST; ++i) tok[i] = fetch_tok(i);

  // ---- Q as A fragments, 16 dims each: row g is head g, row g + 8 head 8 + g.
  // qs: what a head's scores are multiplied by (D^-1/2 log2 e and, e4m3, the
  // power of two taken out of q and the static K scale; block scales come per
  // token)
  uint32_t qa[8][4];
  float qs[HB];
#pragma unroll
  for (int hb = 0; hb < 2; ++hb) {
    const int h = 8 * hb + g;
    const bool act = hb < HB && h < G;
    const uint16_t* qh = P.q + (static_cast<long long>(row) * P.hq + kvh * G + min(h, G - 1)) * 128;
    if (hb >= HB) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) qa[kk][hb] = qa[kk][2 + hb] = 0u;
    } else if constexpr (RP::kE4m3) {
      uint2 v[8];
      float peak = 0.f;
      bool odd = false;  // an infinity or a NaN
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        v[kk] = act ? *reinterpret_cast<const uint2*>(qh + 16 * kk + 4 * t) : make_uint2(0u, 0u);
        const float x[4] = {bf16_lo(v[kk].x), bf16_hi(v[kk].x), bf16_lo(v[kk].y), bf16_hi(v[kk].y)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          odd |= !(fabsf(x[e]) <= 3.39e38f);
          peak = fmaxf(peak, fabsf(x[e]));
        }
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
        odd |= __shfl_xor_sync(0xffffffffu, static_cast<int>(odd), o) != 0;
      }
      // a power of two that brings the head's largest |q| into [2^14, 2^15)
      // (two factors: 2^e itself may leave fp32)
      const int e = peak > 0.f ? max(__float_as_int(peak) >> 23, 1) - 127 - 14 : 0;
      const float f0 = exp2i(-(e / 2)), f1 = exp2i(-(e - e / 2));
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qa[kk][hb] = pack_f16x2(bf16_lo(v[kk].x) * f0 * f1, bf16_hi(v[kk].x) * f0 * f1);
        qa[kk][2 + hb] = pack_f16x2(bf16_lo(v[kk].y) * f0 * f1, bf16_hi(v[kk].y) * f0 * f1);
      }
      qs[hb < HB ? hb : 0] = odd ? __int_as_float(0x7fffffff)
                                 : exp2i(e / 2) * (0.08838834764831845f * kLog2e * (KVT == 1 ? P.k_scale : 1.0f)) * exp2i(e - e / 2);
    } else {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qa[kk][hb] = act ? *reinterpret_cast<const uint32_t*>(qh + 16 * kk + 2 * t) : 0u;
        qa[kk][2 + hb] = act ? *reinterpret_cast<const uint32_t*>(qh + 16 * kk + 8 + 2 * t) : 0u;
      }
      qs[hb < HB ? hb : 0] = 0.08838834764831845f * kLog2e;
    }
  }

  // biased calls: with a cap, scores become capped_exponent's argument; the cap's
  // and slopes' factors
  [[maybe_unused]] float cap2 = 0.f, slope2[HB];
  if constexpr (MOD) {
    cap2 = P.cap * kLog2e;
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      if (P.cap != 0.f) qs[hb] *= 2.0f / P.cap;
      slope2[hb] = P.slopes != nullptr ? P.slopes[kvh * G + min(8 * hb + g, G - 1)] * kLog2e : 0.f;
    }
  }

  // ---- the ring
  uint8_t* ring = smem + warp * ST * RP::kSlab;
  uint32_t vmask[ST];   // valid tokens of the slabs in flight, oldest first
  uint32_t odd_pair[ST];  // (block scales) which half of its scale word a token takes
  const uint8_t* kvb = static_cast<const uint8_t*>(P.kv);
  const long long scale_bytes =
      KVT == 2 ? 2ll * P.num_blocks * P.hkv * (P.page / P.scale_block) : 0;
  const int scale_shift = KVT == 2 ? __ffs(P.scale_block) - 1 : 0;
  auto issue = [&](int stage, uint32_t rid, uint32_t& vm, uint32_t& odd) {
    vm = __ballot_sync(0xffffffffu, rid != kBadRow);
    uint8_t* dst = ring + stage * RP::kSlab;
    // a lane copies 16 bytes of K or V of one token in each instruction
    constexpr int LPR = 2 * RP::kRowB / 16;  // lanes of a token's row: 32 or 16
    const int c = lane % LPR, is_v = c >= LPR / 2 ? 1 : 0, chunk = c % (LPR / 2), sub = lane / LPR;
    const uint8_t* src = kvb + c * 16;
    uint8_t* dl = dst + is_v * TS * RP::kRowB;
    constexpr uint32_t kFull = TS == 32 ? 0xffffffffu : 0xffffu;
    if (vm == kFull) {
#pragma unroll
      for (int j0 = 0; j0 < TS; j0 += 32 / LPR) {
        const int j = j0 + sub;
        const uint32_t r = __shfl_sync(0xffffffffu, rid, j);
        cp_async16_full(dl + j * RP::kRowB + ((chunk ^ (is_v ? j & 7 : swz_k<KVT>(j))) << 4),
                        src + static_cast<long long>(r) * (2 * RP::kRowB));
      }
    } else {  // masked tokens become zeros
#pragma unroll
      for (int j0 = 0; j0 < TS; j0 += 32 / LPR) {
        const int j = j0 + sub;
        const uint32_t r = __shfl_sync(0xffffffffu, rid, j);
        const bool ok = (vm >> j) & 1u;
        cp_async16(dl + j * RP::kRowB + ((chunk ^ (is_v ? j & 7 : swz_k<KVT>(j))) << 4),
                   src + static_cast<long long>(ok ? r : 0u) * (2 * RP::kRowB), ok ? 16u : 0u);
      }
    }
    if constexpr (KVT == 2) {
      // the aligned word around the token's two scale bytes (the last word of
      // an odd number of pairs holds one)
      const bool ok = rid != kBadRow;
      const uint32_t pair = ok ? rid >> scale_shift : 0u;
      const long long at = 2ll * (pair & ~1u);
      cp_async4(&s_raw[warp][stage][lane], P.scales + at,
                ok ? static_cast<uint32_t>(min(4ll, scale_bytes - at)) : 0u);
      odd = __ballot_sync(0xffffffffu, pair & 1u);
    }
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) pg[i] = fetch_page(tok[i]);
#pragma unroll
  for (int i = 0; i < ST; ++i) vmask[i] = odd_pair[i] = 0u;
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    if (i < cnt) issue(i, row_id(tok[i], pg[i]), vmask[i], odd_pair[i]);
    cp_async_commit();
  }
  // the slab to copy next, and the one after it
  int tok_n = tok[ST - 1], pg_n = pg[ST - 1], tok_nn = tok[ST];

  float o[16][4];
  float m[HB], l[HB];
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    m[hb] = -INFINITY;
    l[hb] = 0.f;
  }
#pragma unroll
  for (int nb = 0; nb < 16; ++nb) o[nb][0] = o[nb][1] = o[nb][2] = o[nb][3] = 0.f;

  int stage = 0;
  for (int it = 0; it < cnt; ++it) {
    cp_async_wait<ST - 2>();
    __syncwarp();  // slab it has landed for every lane; slab it - 1 is free
    {
      int nst = stage + ST - 1;
      if (nst >= ST) nst -= ST;
      if (it + ST - 1 < cnt) issue(nst, row_id(tok_n, pg_n), vmask[ST - 1], odd_pair[ST - 1]);
      cp_async_commit();
      tok_n = tok_nn;
      pg_n = fetch_page(tok_n);
      tok_nn = fetch_tok(it + ST + 1);
    }
    const uint8_t* sK = ring + stage * RP::kSlab;
    const uint8_t* sV = sK + TS * RP::kRowB;
    const uint32_t vm = vmask[0];
    float ks[NT], lv[NT], iv[NT];  // of the lane's tokens (block scales)
    if constexpr (KVT == 2) {
      const uint32_t w = s_raw[warp][stage][lane] >> ((odd_pair[0] >> lane & 1u) * 16);
      const int ek = scale_exp(w & 0xFFu), ev = scale_exp((w >> 8) & 0xFFu);
      reinterpret_cast<float*>(s_scl[warp][0])[lane] = exp2i(ek);
      reinterpret_cast<float*>(s_scl[warp][1])[lane] = static_cast<float>(ev);
      reinterpret_cast<float*>(s_scl[warp][2])[lane] = exp2i(-ev);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 a = s_scl[warp][0][4 * u + t], b = s_scl[warp][1][4 * u + t], c = s_scl[warp][2][4 * u + t];
        ks[4 * u] = a.x; ks[4 * u + 1] = a.y; ks[4 * u + 2] = a.z; ks[4 * u + 3] = a.w;
        lv[4 * u] = b.x; lv[4 * u + 1] = b.y; lv[4 * u + 2] = b.z; lv[4 * u + 3] = b.w;
        iv[4 * u] = c.x; iv[4 * u + 1] = c.y; iv[4 * u + 2] = c.z; iv[4 * u + 3] = c.w;
      }
    }

    // ---- S = Q K^T.  Column c of block nb is token tau(nb, c):
    //   bf16   8 nb + c;   e4m3  16 (nb / 2) + 4 (c / 2) + 2 (nb % 2) + c % 2
    // so that a lane's columns 2t, 2t + 1 are the tokens of its P fragment.
    float s[NBK][4];
#pragma unroll
    for (int nb = 0; nb < NBK; ++nb) {
      s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
      const int c = lane & 7;
      const int tk = RP::kE4m3 ? 16 * (nb >> 1) + 4 * (c >> 1) + 2 * (nb & 1) + (c & 1) : 8 * nb + c;
#pragma unroll
      for (int j = 0; j < RP::kRowB / 64; ++j) {  // four 16-byte chunks
        uint32_t b[4];
        ldmatrix_x4(b, sK + tk * RP::kRowB + (((4 * j + (lane >> 3)) ^ swz_k<KVT>(tk)) << 4));
        if constexpr (RP::kE4m3) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t f0, f1;
            e4m3x4_to_f16x2x2(b[u], f0, f1);
            mma_f16_16816(s[nb], qa[4 * j + u], f0, f1);
          }
        } else {
          mma_bf16_16816(s[nb], qa[2 * j], b[0], b[1]);
          mma_bf16_16816(s[nb], qa[2 * j + 1], b[2], b[3]);
        }
      }
    }

    // ---- weights.  Entry e of block nb: the lane's token number 2 nb + e
    uint32_t pa[TS / 16][4];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      float z[NT];  // exponents (log2) without the reference
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        z[i] = s[i >> 1][2 * hb + (i & 1)] * qs[hb];
        if constexpr (KVT == 2 && !MOD) z[i] = fmaf(z[i], ks[i], lv[i]);
        if constexpr (KVT == 2 && MOD) z[i] *= ks[i];
      }
      if constexpr (MOD) {
        if (P.cap != 0.f) {
#pragma unroll
          for (int i = 0; i < NT; ++i) z[i] = capped_exponent(z[i], cap2);
        }
        if (P.slopes != nullptr) {
          // token number tk of the slab lies at lo + n - 1 - at0 - tk
          const float off = static_cast<float>(pos - (lo + n - 1) + (sb + warp + kWarps * it) * TS);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int tk = RP::kE4m3 ? 16 * (i >> 2) + 4 * t + (i & 3) : 8 * (i >> 1) + 2 * t + (i & 1);
            z[i] = fmaf(-slope2[hb], fabsf(off + static_cast<float>(tk)), z[i]);
          }
        }
        if constexpr (KVT == 2) {
#pragma unroll
          for (int i = 0; i < NT; ++i) z[i] += lv[i];
        }
      }
      constexpr uint32_t kFull = TS == 32 ? 0xffffffffu : 0xffffu;
      if (vm != kFull) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int tk = RP::kE4m3 ? 16 * (i >> 2) + 4 * t + (i & 3) : 8 * (i >> 1) + 2 * t + (i & 1);
          if (!((vm >> tk) & 1u)) z[i] = -INFINITY;
        }
      }
      float mx = z[0];
#pragma unroll
      for (int i = 1; i < NT; ++i) mx = fmaxf(mx, z[i]);
      float& mr = m[hb];
      // (no reference yet: any score passes it)
      if (__any_sync(0xffffffffu, mx > mr + RP::kUp)) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(mr, mx);
        const float al = ex2_ftz(mr - (mn == -INFINITY ? 0.f : mn));
        l[hb] *= al;
#pragma unroll
        for (int nb = 0; nb < 16; ++nb) {
          o[nb][2 * hb] *= al;
          o[nb][2 * hb + 1] *= al;
        }
        mr = mn;
      }
      const float ref = mr == -INFINITY ? 0.f : mr;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        z[i] = ex2_ftz(z[i] - ref);
        sum = KVT == 2 ? fmaf(z[i], iv[i], sum) : sum + z[i];
      }
      l[hb] += sum;
#pragma unroll
      for (int u = 0; u < TS / 16; ++u) {
        pa[u][hb] = RP::kE4m3 ? pack_f16x2(z[4 * u], z[4 * u + 1]) : pack_bf16x2(z[4 * u], z[4 * u + 1]);
        pa[u][2 + hb] = RP::kE4m3 ? pack_f16x2(z[4 * u + 2], z[4 * u + 3]) : pack_bf16x2(z[4 * u + 2], z[4 * u + 3]);
        if constexpr (HB == 1) pa[u][1] = pa[u][3] = 0u;
      }
    }

    // ---- O += P V
#pragma unroll
    for (int d = 0; d < 8; ++d) {  // 16 dims
      uint32_t b[4];
      if constexpr (RP::kE4m3) {
        ldmatrix_b8_trans(b, sV + lane * 128 + ((d ^ (lane & 7)) << 4));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t f0, f1;
          e4m3x4_to_f16x2x2(b[u], f0, f1);
          mma_f16_16816(o[2 * d + (u & 1)], pa[u >> 1], f0, f1);
        }
      } else {
        const int tk = lane & 15;
        ldmatrix_x4_trans(b, sV + tk * 256 + (((2 * d + (lane >> 4)) ^ (tk & 7)) << 4));
        mma_bf16_16816(o[2 * d], pa[0], b[0], b[1]);
        mma_bf16_16816(o[2 * d + 1], pa[0], b[2], b[3]);
      }
    }
#pragma unroll
    for (int i = 0; i + 1 < ST; ++i) {
      vmask[i] = vmask[i + 1];
      odd_pair[i] = odd_pair[i + 1];
    }
    if (++stage == ST) stage = 0;
  }
  cp_async_wait<0>();
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_error(P.err);

  // ---- join the warps: [head][warp] references and sums, [warp][head][dim]
  __syncthreads();
  constexpr int HN = 8 * HB;
  constexpr int LD = 128 + 4;  // (head rows a few banks apart)
  float* cm = reinterpret_cast<float*>(smem);
  float* cl = cm + kWarps * HN;
  float* co = cl + kWarps * HN;
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    float sum = l[hb];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const int at = warp * HN + 8 * hb + g;
    if (t == 0) {
      cm[at] = m[hb];
      cl[at] = sum;
    }
#pragma unroll
    for (int nb = 0; nb < 16; ++nb)
      *reinterpret_cast<float2*>(co + at * LD + 8 * nb + 2 * t) = make_float2(o[nb][2 * hb], o[nb][2 * hb + 1]);
  }
  __syncthreads();
  float* fm = co + kWarps * HN * LD;  // with clusters: the CTA's own part, [head] and [head][dim]
  float* fl = fm + HN;
  float* fo = fl + HN;
  const int d0 = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    const int h = (threadIdx.x >> 4) + 8 * hb;
    if (h >= G) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cm[w * HN + h]);
    float L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = cm[w * HN + h];
      const float wt = mw == -INFINITY ? 0.f : ex2_ftz(mw - M);
      L = fmaf(cl[w * HN + h], wt, L);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(co[(w * HN + h) * LD + d0 + e], wt, acc[e]);
    }
    if (P.cluster) {
      if (d0 == 0) {
        fm[h] = M;
        fl[h] = L;
      }
#pragma unroll
      for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(fo + h * 128 + d0 + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      continue;
    }
    // (a NaN sum is not an empty row)
    const float inv = L == 0.f ? 0.f : (KVT == 1 ? P.v_scale : 1.0f) / L;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= inv;
    const long long head = static_cast<long long>(row) * P.hq + kvh * G + h;
    if (P.splits == 1) {
      store_gated8(P, head * 128 + d0, acc, load_gate(P, head * 128 + d0));
      continue;
    }
    const long long ph = static_cast<long long>(split) * P.rows * P.hq + head;
    float4* po = reinterpret_cast<float4*>(P.part_o + ph * 128 + d0);
    po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (d0 == 0) P.part_lse[ph] = L == 0.f ? -INFINITY : M + log2f(L);
  }
  if (!P.cluster) return;
  // ---- join the cluster's parts, 8 dims of a head a thread, over all its CTAs
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  cluster.sync();
  for (int it = split + P.splits * static_cast<int>(threadIdx.x); it < 16 * G; it += P.splits * kThreads) {
    const int h = it >> 4, d = (it & 15) * 8;
    const long long at = (static_cast<long long>(row) * P.hq + kvh * G + h) * 128 + d;
    const uint4 gate = load_gate(P, at);
    float M = -INFINITY;
    for (int q = 0; q < P.splits; ++q) M = fmaxf(M, cluster.map_shared_rank(fm, q)[h]);
    float L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < P.splits; ++q) {
      const float mq = cluster.map_shared_rank(fm, q)[h];
      const float wt = mq == -INFINITY ? 0.f : ex2_ftz(mq - M);
      L = fmaf(cluster.map_shared_rank(fl, q)[h], wt, L);
      const float4* o4 = reinterpret_cast<const float4*>(cluster.map_shared_rank(fo, q) + h * 128 + d);
      const float4 a = o4[0], b = o4[1];
      acc[0] = fmaf(a.x, wt, acc[0]); acc[1] = fmaf(a.y, wt, acc[1]);
      acc[2] = fmaf(a.z, wt, acc[2]); acc[3] = fmaf(a.w, wt, acc[3]);
      acc[4] = fmaf(b.x, wt, acc[4]); acc[5] = fmaf(b.y, wt, acc[5]);
      acc[6] = fmaf(b.z, wt, acc[6]); acc[7] = fmaf(b.w, wt, acc[7]);
    }
    const float inv = L == 0.f ? 0.f : (KVT == 1 ? P.v_scale : 1.0f) / L;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= inv;
    store_gated8(P, at, acc, gate);
  }
  cluster.sync();  // (a CTA's part is read until here)
}

// Joins the splits of each (row, head), 8 dims a thread, in split order.  A
// half-warp's lanes read the log-sum-exps of 16 splits at a time and the
// partials of 8 are on their way together (33 splits of one row, one after
// another, took 11 us of 19).
__global__ void __launch_bounds__(256) row_merge_kernel(const RowGqaParams P) {
  griddep_wait();  // every split's partials are written
  const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long head = idx >> 4;
  if (head >= static_cast<long long>(P.rows) * P.hq) return;
  const int lane16 = static_cast<int>(idx) & 15, row = static_cast<int>(head / P.hq), d0 = lane16 * 8;
  if (P.packed == nullptr && !row_live(P, row, P.token_to_req[row])) return;
  const unsigned half = 0xFFFFu << (threadIdx.x & 16);  // (as one from here on)
  const uint4 gate = load_gate(P, head * 128 + d0);
  const long long stride = static_cast<long long>(P.rows) * P.hq;
  constexpr int kMost = kMaxRowSplits / 16;
  float w[kMost];
  float M = -INFINITY, W = 0.f;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int s = 16 * k + lane16;
    w[k] = s < P.splits ? __ldcg(P.part_lse + s * stride + head) : -INFINITY;
    nan |= w[k] != w[k];
    M = fmaxf(M, w[k]);
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(half, M, o));
  nan = __any_sync(half, nan);
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    w[k] = w[k] == -INFINITY ? -1.f : ex2_ftz(w[k] - M);  // (-1: saw nothing)
    W += fmaxf(w[k], 0.f);
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) W += __shfl_xor_sync(half, W, o);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    if (16 * k >= P.splits) break;
#pragma unroll 1
    for (int i = 0; i < 16 && 16 * k + i < P.splits; i += 8) {
      float4 a[8], b[8];
      float ws[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        ws[u] = __shfl_sync(half, w[k], i + u, 16);
        a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        // (a split that saw nothing may not have written; one whose weight
        // vanishes still hands on what is not finite)
        if (ws[u] >= 0.f) {
          const float4* po = reinterpret_cast<const float4*>(P.part_o + ((16 * k + i + u) * stride + head) * 128 + d0);
          a[u] = __ldcg(po);
          b[u] = __ldcg(po + 1);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        acc[0] = fmaf(ws[u], a[u].x, acc[0]); acc[1] = fmaf(ws[u], a[u].y, acc[1]);
        acc[2] = fmaf(ws[u], a[u].z, acc[2]); acc[3] = fmaf(ws[u], a[u].w, acc[3]);
        acc[4] = fmaf(ws[u], b[u].x, acc[4]); acc[5] = fmaf(ws[u], b[u].y, acc[5]);
        acc[6] = fmaf(ws[u], b[u].z, acc[6]); acc[7] = fmaf(ws[u], b[u].w, acc[7]);
      }
    }
  }
  const float inv = nan ? __int_as_float(0x7fffffff) : W == 0.f ? 0.f : 1.0f / W;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= inv;
  store_gated8(P, head * 128 + d0, acc, gate);
}

template <int KVT, int HB, bool MOD>
cudaError_t launch_kind(const RowGqaParams& p, cudaStream_t stream) {
  using RP = RowPlan<KVT>;
  constexpr int kMerge = (kWarps * 8 * HB * (128 + 4 + 2) + 8 * HB * (128 + 2)) * 4;
  constexpr int kSmem = RP::kSmem > kMerge ? RP::kSmem : kMerge;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(row_gqa_kernel<KVT, HB, MOD>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  if (p.cluster)
    return launch_kernel_cluster(row_gqa_kernel<KVT, HB, MOD>, dim3(p.rows * p.hkv * p.splits), dim3(kThreads), kSmem,
                                 stream, false, p.splits, p);
  return launch_kernel(row_gqa_kernel<KVT, HB, MOD>, dim3(p.rows * p.hkv, p.splits), dim3(kThreads), kSmem,
                       stream, false, p);
}

template <int KVT>
cudaError_t launch_type(const RowGqaParams& p, cudaStream_t stream) {
  const bool wide = p.group > 8;
  if (p.biased) return wide ? launch_kind<KVT, 2, true>(p, stream) : launch_kind<KVT, 1, true>(p, stream);
  return wide ? launch_kind<KVT, 2, false>(p, stream) : launch_kind<KVT, 1, false>(p, stream);
}

}  // namespace

// As many splits as keep the CTAs in one wave at two per SM (shared memory): a
// second wave, or a row cut finer than that, costs more than it evens out (L2
// flushed before each call: 64 rows x 4 KV heads of 4100 tokens, e4m3, 1 split
// 65 us, 2 splits 73; 8 rows x 8 of 4103, 3 splits 34 us, 4 splits 32, 5 splits
// 40).  A warp has two slabs at the least, and the join, which reads a partial
// for each split, keeps their square to a twelfth of the tokens (one row and KV
// head of 4100 tokens, bf16: 4 splits 21.8 us, 8 to 22 splits 17.5, 33 splits
// 19.6).
int row_gqa_splits(int rows, int hkv, long long max_tokens, int kv_dtype, int sms) {
  const long long base = static_cast<long long>(rows) * hkv;
  if (base <= 0) return 1;
  const int least = (kv_dtype == QSA_DTYPE_BF16 ? 16 : 32) * kWarps * 2;
  long long s = 2ll * sms / base;
  const long long most = (max_tokens + least - 1) / least;
  if (s > most) s = most;
  if (s > kMaxRowSplits) s = kMaxRowSplits;
  while (s > 1 && 12 * s * s > max_tokens) --s;
  return s < 1 ? 1 : static_cast<int>(s);
}

// Up to eight splits of a row and KV head are a cluster and join through its
// shared memory, without the partials' way through memory and a second launch
// (8 rows x 8 KV heads in 4 splits 33.9 -> 31.9 us, two rows x 4 KV heads in 8
// splits 19.6 -> 17.6, L2 flushed before each call); not where the launch nearly
// fills the SMs, whose groups may then hold fewer clusters than single CTAs.
bool row_gqa_cluster(int rows, int hkv, int splits, int sms) {
  return splits > 1 && splits <= 8 && static_cast<long long>(rows) * hkv * splits <= 2 * sms * 85 / 100;
}

cudaError_t launch_row_gqa(const RowGqaParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  cudaError_t e;
  switch (p.kv_dtype) {
    case QSA_DTYPE_BF16: e = launch_type<0>(p, stream); break;
    case QSA_DTYPE_E4M3: e = launch_type<1>(p, stream); break;
    default: e = launch_type<2>(p, stream); break;
  }
  if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
  return launch_row_merge(p, stream);
}

cudaError_t launch_row_merge(const RowGqaParams& p, cudaStream_t stream) {
  const long long items = static_cast<long long>(p.rows) * p.hq * 16;
  return launch_kernel(row_merge_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, stream, true, p);
}

}  // namespace qsa
