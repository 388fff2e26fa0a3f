// The fused projection of the main attention and the indexer from 4-bit
// weights: y = x . w^T as in proj_gemm.cu, with the stacked weights held as
// e2m1 codes and a scale for each group of inputs (qsa_qkv_index_proj_w4).
//
// Mathematics.  w[c][k] = code(c, k) * s(c, k / group) * scale.  A code has 2
// significant bits and a scale 4 at the most (e4m3) or 1 (a power of two), so
// code * s is a bf16 value exactly, and y is an fp32 sum of exact products,
// times `scale`, rounded once.  An e2m1 code's exponent and mantissa placed on
// a bf16's (bits 6 .. 8) are that value times 2^-126, subnormals included; one
// bf16 multiplication by s * 2^111 makes it the weight times 2^-15, which the
// epilogue takes back: the factor has to be a bf16 value (so powers of two end at
// 2^16), sums of large inputs keep room below fp32's end, and only products below
// 2^-111 lose bits.
//
// Up to 8 rows: a warp takes 32 columns and every fourth stretch of 128 inputs.
// Its lanes load 32 consecutive codes of four columns each (64 bytes of a column
// together), unpack them to the A fragments of m16n8k16 MMAs and take x's
// fragments in the same order of inputs; the four warps of a CTA add up in
// shared memory, in order.  More rows: tcgen05 (below).
//
// Bound: few rows by waits for loads beside the instructions that unpack (17 for
// eight codes): 11 warps an SM with one stretch of codes ahead, issue slots 53 % used,
// DRAM 29 %, 2.4 of 3.1 stall cycles an issue waits for loads (HBM alone would take 4.6
// us for hidden 4096 and 13 440 columns, loads in this order alone 5.8); tiles of few
// rows by unpacking and fixed costs, prefill by the tensor cores.
// Measured there, ten calls on four sets of inputs: one row 11.1 us, 8 rows 12.7, 9
// to 64 rows 18 to 20, 128 rows 23, 256 rows 30, 2048 rows 156 (1.44 PFLOP/s); 3
// rows of hidden 1024 and 3456 columns 2.9.  Of the 20 us of 64 rows 8 remain
// without products and sums.  Unpacking by two shifts instead of a multiplication
// takes 18 cycles a word and scheduler instead of 15.6, by byte tables 20; more
// warps with fewer registers 13 to 17 us for one row.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <cmath>

#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"
#include "umma_elect.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;

// The eight codes of a word times m, in pairs: codes j and j + 4 in r[j].  A
// nibble times 2^12 + 2^6 (or 2^8 + 2^2, four bits on) has its sign where a
// bf16's is and its other bits at a bf16's last two exponent bits and first
// mantissa bit; no other bits of the two copies meet there.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t m, uint32_t* r) {
  const uint32_t v = w >> 8;
  r[0] = mul_bf16x2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, m);
  r[1] = mul_bf16x2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, m);
  r[2] = mul_bf16x2(((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, m);
  r[3] = mul_bf16x2(((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, m);
}

// Scales: FMT 0, powers of two (groups of 32); FMT 1, e4m3 (groups of 16).
template <int FMT>
constexpr int kGroup = FMT == 0 ? 32 : 16;
constexpr int kShift = 15;  // weights are held times 2^-kShift
constexpr int kMxLeast = 67, kMxMost = 143;  // scale bytes: 2^-60 .. 2^16
constexpr float kScaleUp = 2.596148429267414e33f;  // 2^111
// A scale byte as a bf16 pair, times 2^(126 - kShift).
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
  uint32_t hi;
  if constexpr (FMT == 0) {
    hi = (min(max(byte, static_cast<uint32_t>(kMxLeast)), static_cast<uint32_t>(kMxMost)) + 126 - kShift) << 23;
  } else {
    uint32_t f16, other;
    e4m3x4_to_f16x2x2(byte, f16, other);
    hi = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(f16))) * kScaleUp);
  }
  return prmt(hi, hi, 0x3232);
}

// A sum of products of inputs and held weights, as an output.  (A factor below 1
// comes first into the power of two, so that neither leaves fp32 early.)
__device__ __forceinline__ uint16_t output_of(float y, float scale) {
  constexpr float k = static_cast<float>(1 << kShift);
  const bool small = fabsf(scale) < 1.0f;
  const __nv_bfloat16 v = __float2bfloat16_rn(y * (small ? scale * k : k) * (small ? 1.0f : scale));
  return *reinterpret_cast<const uint16_t*>(&v);
}

// An output column's place.
struct Column {
  uint16_t* dst;
  int ld;
};
__device__ __forceinline__ Column column_of(const ProjW4Params& P, int col) {
  if (col < P.qkv_cols) return {P.qkv_out + col, P.qkv_cols};
  col -= P.qkv_cols;
  if (col < P.index_q_cols) return {P.index_q_out + col, P.index_q_cols};
  return {P.index_k_out + (col - P.index_q_cols), P.index_k_cols};
}

// Eight outputs of a row from column `col` on, those past the last column left
// out: one store where they lie side by side in one output, on 16 bytes.
__device__ __forceinline__ void store8(const ProjW4Params& P, int col, int row, uint4 v) {
  if (col + 8 <= P.ncols) {
    const Column a = column_of(P, col), b = column_of(P, col + 7);
    uint16_t* dst = a.dst + static_cast<long long>(row) * a.ld;
    if (a.ld == b.ld && b.dst - a.dst == 7 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
      *reinterpret_cast<uint4*>(dst) = v;
      return;
    }
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
  for (int e = 0; e < 8 && col + e < P.ncols; ++e) {
    const Column o = column_of(P, col + e);
    o.dst[static_cast<long long>(row) * o.ld] = static_cast<uint16_t>((e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3]) >> (16 * (e & 1)));
  }
}

// The scales of a lane's 32 inputs, as loaded, to factors of its four words.
template <int FMT>
__device__ __forceinline__ void factors(uint32_t bytes, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == 0) {
    lo = hi = scale_pair<FMT>(bytes);
  } else {
    uint32_t f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(f) : "r"(bytes));
    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&f));
    lo = prmt(__float_as_uint(s.x * kScaleUp), 0u, 0x3232);
    hi = prmt(__float_as_uint(s.y * kScaleUp), 0u, 0x3232);
  }
}

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32, 3) w4_rows_kernel(const ProjW4Params P) {
  constexpr int kStep = 128 * kWarps;
  __shared__ float part[kWarps][32][8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 32, r0 = blockIdx.y * 8;
  // offsets from the CTA's first column and row (columns and rows past the last
  // one repeat it; 32 bits, hidden < 2^24)
  const uint8_t* codes = P.codes + static_cast<long long>(n0) * (P.hidden / 2);
  const uint8_t* scales = P.scales + static_cast<long long>(n0) * (P.hidden / kGroup<FMT>);
  const uint16_t* x = P.x + static_cast<long long>(r0) * P.hidden;
  int w[4], s[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = min(g + 8 * c, P.ncols - 1 - n0);
    w[c] = col * (P.hidden / 2) + 64 * warp + 16 * t;
    s[c] = col * (P.hidden / kGroup<FMT>) + 128 / kGroup<FMT> * warp + 32 / kGroup<FMT> * t;
  }
  const int xr = min(g, P.rows - 1 - r0) * P.hidden + 128 * warp + 32 * t;
  float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  // a stretch's codes, scales and inputs; the next one's are on their way.  Lanes
  // past the last input read the row's last ones; their factors and inputs are
  // zeros.
  struct Codes {
    uint4 a[4];
    uint32_t s[4];
  };
  // a lane's stretch begins here at the latest (below 0 where the CTA's warps and
  // lanes have more room than there are inputs; the sums with w, s, xr are not)
  const int last = P.hidden - 128 * warp - 32 * t - 32;
  auto at = [](int sum) { return static_cast<uint32_t>(sum); };
  auto load_codes = [&](int k) {
    Codes v;
    const int from = min(k, last);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v.a[c] = __ldg(reinterpret_cast<const uint4*>(codes + at(w[c] + from / 2)));
      v.s[c] = FMT == 0 ? static_cast<uint32_t>(__ldg(scales + at(s[c] + from / 32)))
                        : static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(scales + at(s[c] + from / 16))));
    }
    return v;
  };
  struct Inputs {
    uint4 x[4];
  };
  auto load_inputs = [&](int k) {
    Inputs v;
    const int from = xr + min(k, last);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.x[i] = *reinterpret_cast<const uint4*>(x + at(from + 8 * i));
    return v;
  };
  const int steps = (P.hidden - 128 * warp + kStep - 1) / kStep;  // (<= 0: none)
  Codes next;
  Inputs ahead;
  if (steps > 0) {
    next = load_codes(0);
    ahead = load_inputs(0);
  }
  for (int j = 0; j < steps; ++j) {
    const int k = j * kStep;
    const Codes v = next;
    Inputs in = ahead;
    if (j + 1 < steps) {
      next = load_codes(k + kStep);
      ahead = load_inputs(k + kStep);
    }
    uint32_t m[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) factors<FMT>(v.s[c], m[c][0], m[c][1]);
    if (k > last) {  // (a ragged last stretch)
#pragma unroll
      for (int c = 0; c < 4; ++c) m[c][0] = m[c][1] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) in.x[i] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 xi = in.x[i];
      const uint32_t xb[4] = {prmt(xi.x, xi.z, 0x5410), prmt(xi.x, xi.z, 0x7632), prmt(xi.y, xi.w, 0x5410), prmt(xi.y, xi.w, 0x7632)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 16 columns
        auto word = [&](int c) { return i == 0 ? v.a[c].x : i == 1 ? v.a[c].y : i == 2 ? v.a[c].z : v.a[c].w; };
        uint32_t p0[4], p1[4];
        unpack8(word(2 * h), m[2 * h][i >> 1], p0);
        unpack8(word(2 * h + 1), m[2 * h + 1][i >> 1], p1);
        const uint32_t f0[4] = {p0[0], p1[0], p0[1], p1[1]}, f1[4] = {p0[2], p1[2], p0[3], p1[3]};
        mma_bf16_16816(acc[h], f0, xb[0], xb[1]);
        mma_bf16_16816(acc[h], f1, xb[2], xb[3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[warp][16 * (i >> 2) + g + 8 * ((i >> 1) & 1)][2 * t + (i & 1)] = acc[i >> 2][i & 3];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 8; i += kWarps * 32) {
    const int c = i & 31, r = i >> 5;
    if (n0 + c >= P.ncols || r0 + r >= P.rows) continue;
    float y = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) y += part[q][c][r];
    const Column o = column_of(P, n0 + c);
    o.dst[static_cast<long long>(r0 + r) * o.ld] = output_of(y, P.scale);
  }
}

// ---------------------------------------------------------------- tiles
// More rows: tcgen05, 128 columns (M) by BN rows (N) a CTA.
//   warp 0     TMA: x by blocks of 64 or 128 inputs, codes by stretches of 256
//              (128 bytes of a column);
//   warp 1     MMAs, weights from tensor memory (A), x from shared memory (B);
//   warps 2-9  a thread to a column: codes from shared memory, unpacked, to
//              tensor memory, every other block each half; at the end the
//              outputs.
// Every wait is bounded (mbar_wait); a timeout sets the error word, and the tile's
// outputs stay as they were, or are NaNs where a cluster joins its sums.
// kSplit: tiles of few rows leave the SMs without enough columns (13 440 make 105
// tiles), so that clusters of CTAs share a tile's inputs and join their sums
// through shared memory.  Measured: 64 rows with two CTAs a tile and two an SM 20.1
// us, with four and three 22.5 (blocks of 64 inputs, 64 registers a thread), 128
// rows unsplit 22.3; blocks of 128 inputs 22.3 us where blocks of 64 take 25.9 (128
// rows), but 173 us where those take 157 (256-row tiles, 2048 rows: fewer blocks
// fit).  The sums' way through shared memory to stores of 16 bytes took 64 rows
// from 23 to 20 us; 2-byte stores of columns cost 128 rows 3 us.
template <int BN>
struct Tile {
  static constexpr bool kSplit = BN <= 64;
  static constexpr int H = BN == 256 ? 1 : 2;     // 64 inputs each, of a block
  static constexpr int XS = BN == 256 ? 4 : 3;    // blocks of x
  static constexpr int CS = kSplit ? 2 : 3;       // stretches of 256 codes of a column
  static constexpr int AS = kSplit ? 3 : BN == 128 ? 2 : 8;  // blocks of weights in tensor memory, 32 H columns each
  static constexpr int kCols = BN == 256 ? 512 : 256;
  static constexpr int kX = H * BN * 128, kC = 128 * 128;
  static constexpr int kSmem = 1024 + XS * kX + CS * kC;
  static constexpr int kThreads = 320;
  static constexpr int kCtas = kSplit ? 2 : 1;    // of an SM
  static_assert(BN + 32 * H * AS <= kCols, "tensor memory");
  static_assert(BN * 128 * (kSplit ? 4 : 2) <= XS * kX, "the sums fit x's place");
};

// 32 codes of a column (four words, k ascending) to 16 pairs of bf16.
template <int FMT>
__device__ __forceinline__ void unpack32(uint4 v, uint32_t m0, uint32_t m1, uint32_t (&r)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = FMT == 1 && i >= 2 ? m1 : m0;
    uint32_t p[4];
    unpack8(w[i], m, p);
    r[4 * i] = prmt(p[0], p[1], 0x5410);
    r[4 * i + 1] = prmt(p[2], p[3], 0x5410);
    r[4 * i + 2] = prmt(p[0], p[1], 0x7632);
    r[4 * i + 3] = prmt(p[2], p[3], 0x7632);
  }
}

template <int FMT, int BN>
__global__ void __launch_bounds__(Tile<BN>::kThreads, Tile<BN>::kCtas)
    w4_tile_kernel(const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_x, const ProjW4Params P, int splits) {
  using T = Tile<BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t x_full[T::XS], x_empty[T::XS], c_full[T::CS], c_empty[T::CS], a_full[T::AS], a_empty[T::AS], acc_full;
  __shared__ uint32_t tmem_slot;
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sC = smem_raw + pad;
  uint8_t* sX = sC + T::CS * T::kC;
  bool done = true;  // (false: a wait gave up)
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int rank = T::kSplit ? static_cast<int>(blockIdx.x) % splits : 0;
  const int n0 = static_cast<int>(blockIdx.x) / (T::kSplit ? splits : 1) * 128, r0 = blockIdx.y * BN;
  const int rows = min(BN, P.rows - r0);
  // its blocks of 64 H inputs: nb from b0 on (a last half is filled up with zeros)
  constexpr int H = T::H, kPer = 4 / H;  // (blocks of a stretch of codes)
  const int blocks = (P.hidden + 64 * H - 1) / (64 * H), per = (blocks + splits - 1) / splits;
  const int b0 = T::kSplit ? rank * per : 0, nb = T::kSplit ? min(blocks - b0, per) : blocks;
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < T::XS; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], 1);
    }
    for (int i = 0; i < T::CS; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], 8);
    }
    for (int i = 0; i < T::AS; ++i) {
      mbar_init(&a_full[i], 4);
      mbar_init(&a_empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, T::kCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    for (int i = 0; i < nb; ++i) {
      if (i % kPer == 0) {
        const int cs = i / kPer % T::CS;
        done = all_ok(mbar_wait(&c_empty[cs], ((i / kPer / T::CS) & 1) ^ 1, P.err));
        if (!done) break;
        if (lane == 0) mbar_arrive_expect_tx(&c_full[cs], T::kC);
        __syncwarp();
        tma_box(sC + cs * T::kC, &tmap_c, (b0 + i) * 32 * H, n0, &c_full[cs]);
      }
      const int xs = i % T::XS;
      done = all_ok(mbar_wait(&x_empty[xs], ((i / T::XS) & 1) ^ 1, P.err));
      if (!done) break;
      if (lane == 0) mbar_arrive_expect_tx(&x_full[xs], T::kX);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < H; ++h)
        tma_box(sX + xs * T::kX + h * BN * 128, &tmap_x, ((b0 + i) * H + h) * 64, r0, &x_full[xs]);
    }
  } else if (warp == 1) {
    const uint32_t idesc = umma_idesc(1u, 128, BN);
    const uint32_t x0 = desc_lo(smem_addr(sX), 16);
    for (int i = 0; i < nb; ++i) {
      const int xs = i % T::XS, as = i % T::AS;
      done = all_ok(mbar_wait(&x_full[xs], (i / T::XS) & 1, P.err) && mbar_wait(&a_full[as], (i / T::AS) & 1, P.err));
      if (!done) break;
      tc_fence_after_sync();
#pragma unroll
      for (int kk = 0; kk < 4 * H; ++kk)
        mma_ts(tmem, tmem + BN + 32 * H * as + 8 * kk, x0 + ((xs * T::kX + (kk >> 2) * BN * 128 + 32 * (kk & 3)) >> 4), idesc,
               (i | kk) != 0 ? 1u : 0u);
      mma_commit(&x_empty[xs]);
      mma_commit(&a_empty[as]);
    }
    if (done) mma_commit(&acc_full);
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const int row = 32 * quad + lane, col = n0 + row;
    // a block's scale bytes: four (e4m3) or two for 64 inputs, zeros past the last
    const uint8_t* sp = P.scales + static_cast<long long>(min(col, P.ncols - 1)) * (P.hidden / kGroup<FMT>);
    struct Bytes {
      uint32_t b[H];
    };
    auto scale_bytes = [&](int i) -> Bytes {
      Bytes s;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int k = 64 * (H * (b0 + i) + h);
        s.b[h] = 0u;
        if (i >= nb || k >= P.hidden) continue;
        if constexpr (FMT == 0)
          s.b[h] = *reinterpret_cast<const uint16_t*>(sp + k / 32);
        else
          s.b[h] = *reinterpret_cast<const uint32_t*>(sp + k / 16);
      }
      return s;
    };
    constexpr int kAhead = 4 / H;
    Bytes sc[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) sc[u] = scale_bytes(half + 2 * u);
    bool ok = true;
    for (int i0 = half; i0 < nb && ok; i0 += 2 * kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + 2 * u;
        if (i >= nb || !ok) break;
        const Bytes s = sc[u];
        sc[u] = scale_bytes(i + 2 * kAhead);
        const int cs = i / kPer % T::CS, as = i % T::AS;
        ok = all_ok(mbar_wait(&c_full[cs], (i / kPer / T::CS) & 1, P.err));
        const uint8_t* src = sC + cs * T::kC + row * 128;
        const uint32_t dst = tmem + lanes + BN + 32 * H * as;
        uint4 v[2 * H];
#pragma unroll
        for (int q = 0; q < 2 * H; ++q) v[q] = *reinterpret_cast<const uint4*>(src + (((2 * H * (i % kPer) + q) ^ (row & 7)) << 4));
#pragma unroll
        for (int q = 0; q < 2 * H; ++q) {
          uint32_t m0, m1, r[16];
          if constexpr (FMT == 0)
            factors<FMT>((s.b[q >> 1] >> (8 * (q & 1))) & 0xFFu, m0, m1);
          else
            factors<FMT>(s.b[q >> 1] >> (16 * (q & 1)), m0, m1);
          unpack32<FMT>(v[q], m0, m1, r);
          if (q == 0) {
            ok = ok && all_ok(mbar_wait(&a_empty[as], ((i / T::AS) & 1) ^ 1, P.err));
            tc_fence_after_sync();
          }
          tmem_st16(dst + 16 * q, r);
        }
        // (this half's last block of the stretch)
        __syncwarp();
        if ((i % kPer >= kPer - 2 || i + 2 >= nb) && lane == 0) mbar_arrive(&c_empty[cs]);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[as]);
      }
    }
    // ---- sums: this thread's column, every other 16 rows each half, to shared
    // memory (x's place: every MMA is done), as fp32 where they are joined
    ok = ok && (nb <= 0 || all_ok(mbar_wait(&acc_full, 0, P.err)));
    tc_fence_after_sync();
#pragma unroll 1
    for (int c = 16 * half; c < BN && c < rows; c += 32) {
      uint32_t v[16];
      if (nb > 0) tmem_ld16(tmem + lanes + c, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float y = nb > 0 && ok ? __uint_as_float(v[j]) : 0.f;
        if constexpr (T::kSplit)
          reinterpret_cast<float*>(sX)[(c + j) * 128 + row] = y;
        else
          reinterpret_cast<uint16_t*>(sX)[(c + j) * 128 + row] = output_of(y, P.scale);
      }
    }
    done = ok;
  }
  tc_fence_before_sync();
  const bool good = __syncthreads_and(done);
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, T::kCols);
  }
  // ---- outputs, eight columns a thread
  if constexpr (T::kSplit) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    if (!good)  // (a wait gave up: no sum of these may pass for a result)
      for (int i = threadIdx.x; i < BN * 128; i += T::kThreads) reinterpret_cast<float*>(sX)[i] = __int_as_float(0x7fffffff);
    cluster.sync();
    // the cluster's sums, in order: every CTA its share of the rows
    const int items = (rows - rank + splits - 1) / splits * 16;
#pragma unroll 1
    for (int i = threadIdx.x; i < items; i += T::kThreads) {
      const int r = rank + (i >> 4) * splits, c = 8 * (i & 15);
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q0 = 0; q0 < 8; q0 += 4) {
        if (q0 >= splits) break;
        float4 a[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q0 + q >= splits) break;
          const float4* from = reinterpret_cast<const float4*>(cluster.map_shared_rank(reinterpret_cast<float*>(sX), q0 + q) + r * 128 + c);
          a[q] = from[0];
          b[q] = from[1];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q0 + q >= splits) break;
          y[0] += a[q].x; y[1] += a[q].y; y[2] += a[q].z; y[3] += a[q].w;
          y[4] += b[q].x; y[5] += b[q].y; y[6] += b[q].z; y[7] += b[q].w;
        }
      }
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = output_of(y[2 * e], P.scale) | (static_cast<uint32_t>(output_of(y[2 * e + 1], P.scale)) << 16);
      store8(P, n0 + c, r0 + r, make_uint4(v[0], v[1], v[2], v[3]));
    }
    cluster.sync();  // (a CTA's sums are read until here)
  } else if (good) {
    const Column first = column_of(P, n0), last = column_of(P, min(n0 + 127, P.ncols - 1));
    if (first.ld % 8 == 0 && last.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(first.dst) & 15) == 0) {
#pragma unroll 4
      for (int i = threadIdx.x; i < rows * 16; i += T::kThreads)
        store8(P, n0 + 8 * (i & 15), r0 + (i >> 4), reinterpret_cast<const uint4*>(sX)[i]);
    } else {
      // rows that begin anywhere: a warp to a row, neighbouring columns together
      // (945 rows, hidden 320, 5033 columns: 30 -> 14.6 us)
#pragma unroll 1
      for (int c = lane; c < 128 && n0 + c < P.ncols; c += 32) {
        const Column o = column_of(P, n0 + c);
#pragma unroll 4
        for (int r = warp; r < rows; r += T::kThreads / 32)
          o.dst[static_cast<long long>(r0 + r) * o.ld] = reinterpret_cast<const uint16_t*>(sX)[r * 128 + c];
      }
    }
  }
}

template <int FMT>
cudaError_t launch_rows(const ProjW4Params& p, cudaStream_t stream) {
  const dim3 grid((p.ncols + 31) / 32, (p.rows + 7) / 8);
  return launch_kernel(w4_rows_kernel<FMT>, grid, dim3(kWarps * 32), 0, stream, false, p);
}

// CTAs of a split tile: as many as find room at once, with two blocks each or more.
int split_count(long long tiles, int groups, int hidden, int sms) {
  int splits = 1;
  while (splits < 8 && 2 * splits * tiles * groups <= 2ll * sms && hidden / 64 >= 4 * splits) splits *= 2;
  return splits;
}

template <int FMT, int BN>
cudaError_t launch_tile(const ProjW4Params& p, const CUtensorMap& codes, const CUtensorMap& x, cudaStream_t stream) {
  using T = Tile<BN>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(w4_tile_kernel<FMT, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int tiles = (p.ncols + 127) / 128, groups = (p.rows + BN - 1) / BN;
  if constexpr (T::kSplit) {
    const int splits = split_count(tiles, groups, p.hidden, p.sms);
    return launch_kernel_cluster(w4_tile_kernel<FMT, BN>, dim3(tiles * splits, groups), dim3(T::kThreads), T::kSmem, stream, false, splits, codes,
                                 x, p, splits);
  }
  return launch_kernel(w4_tile_kernel<FMT, BN>, dim3(tiles, groups), dim3(T::kThreads), T::kSmem, stream, false, codes, x, p, 1);
}

template <int FMT>
cudaError_t launch_format(const ProjW4Params& p, const CUtensorMap& codes, const CUtensorMap& x, cudaStream_t stream) {
  switch (w4_tile_rows(p.rows, p.hidden, p.ncols, p.sms)) {
    case 0: return launch_rows<FMT>(p, stream);
    case 16: return launch_tile<FMT, 16>(p, codes, x, stream);
    case 64: return launch_tile<FMT, 64>(p, codes, x, stream);
    case 128: return launch_tile<FMT, 128>(p, codes, x, stream);
    default: return launch_tile<FMT, 256>(p, codes, x, stream);
  }
}

}  // namespace

// 8 rows take 12.7 us by warps and 17.3 in a tile of 16; 9 to 16 rows 18.3 in it,
// 20 in one of 64, and 21.7 by warps with fragments for 16 rows.  (hidden 4096, 13
// 440 columns; 3 rows of hidden 1024 and 3456 columns 2.9 us by warps.)
// More rows: the tile that they fill, or another one by estimates in us:
//   64   7.1 + 0.51 for each 128 inputs of a CTA and CTA of an SM, + 1.7 for each
//        CTA of an SM behind the first two, + 0.53 a split;
//   128  3.7 + 0.48 for each 128 inputs, for each CTA of an SM;
//   256  4.4 + 0.5 likewise;
// where one is 5 % faster (up to 64 rows, which tiles of 128 leave half empty, 34).
// Measured, tiles of 64 / 128 / 256 rows, us: hidden 4096, 1664 columns, 148 rows
// 13.3 / 18.9 / 23.6; 7296 columns, 212 rows 31.9 / 21.8 / 24.7, 335 rows 44.8 /
// 35.9 / 28.3; hidden 1152, 7296 columns, 64 rows 11.3 / 8.2 / 9.5, 256 rows 13.8 /
// 9.1 / 11.8, 570 rows 23.7 / 16.6 / 17.5; 13 440 columns, 148 rows 18.5 / 15.1 /
// 10.7.  Over 176 such sizes of 30 to 1319 rows the choice takes 1.005 of the fastest
// on average, 1.23 at worst; the tile that the rows fill 1.14 and 1.77.
int w4_tile_rows(int rows, int hidden, int ncols, int sms) {
  if (rows <= 16) return rows <= 8 ? 0 : 16;
  if (rows > 65535 * 64) return 256;  // (a grid's limit)
  const long long tiles = (ncols + 127ll) / 128;
  const double blocks = hidden / 128.0;
  auto per_sm = [&](long long ctas) { return static_cast<double>((ctas + sms - 1) / sms); };
  const int groups = (rows + 63) / 64, splits = split_count(tiles, groups, hidden, sms);
  const double ctas = per_sm(tiles * groups * splits);
  const double us[3] = {7.1 + 0.51 * std::ceil(blocks / splits) * ctas + 1.7 * std::fmax(ctas - 2.0, 0.0) + (splits > 1 ? 0.53 * splits : 0.0),
                        (3.7 + 0.48 * blocks) * per_sm(tiles * ((rows + 127) / 128)),
                        (4.4 + 0.5 * blocks) * per_sm(tiles * ((rows + 255) / 256))};
  const int filled = rows <= 64 ? 0 : rows <= 128 ? 1 : 2;
  int best = 0;
  for (int i = 1; i < 3; ++i)
    if (us[i] < us[best]) best = i;
  return 64 << (us[best] < (rows <= 64 ? 0.66 : 0.95) * us[filled] ? best : filled);
}

cudaError_t launch_proj_w4(const ProjW4Params& p, const CUtensorMap& codes, const CUtensorMap& x, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  return p.format == QSA_W4_MX ? launch_format<0>(p, codes, x, stream) : launch_format<1>(p, codes, x, stream);
}

}  // namespace qsa
