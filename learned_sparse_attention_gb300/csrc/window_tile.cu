// Window attention of many rows per request (prefill chunks, verify steps) on
// the tcgen05 tensor cores.
//
// Mathematics.  As in row_gqa.cu; here 128 (row, head) pairs of one request
// and KV head are the M rows of S = Q K^T and O += P V, R = 128 / G rows with
// their G heads, and a CTA runs two such tiles, A and B (rows r0 .. r0 + R - 1
// and the R after them), over one stream of 128-key tiles.  A thread owns one
// M row of S, so the softmax needs no exchange: it keeps the row's reference
// (moved only when a score passes it by 2^8) and sum in registers, and
// rescales the accumulator itself when the reference moves.
//
// Roles, 16 warps:
//   0-3, 4-7  softmax of tile A, B: S from TMEM, masks on the tiles that need
//             them, P back over S's columns, at the end the gated output;
//   8-11      load K and V tiles of 128 keys through the block table into a
//             ring (128-byte swizzle): bf16 by TMA or cp.async; e4m3 codes
//             through registers, as f16 (exact).  Keys that no row of the CTA sees
//             become zeros, whatever the cache holds there;
//   12        issues the MMAs: S_A(j+1) right after O_A(j), so the softmax of
//             one tile runs under the products of the other.
// TMEM: S_A, S_B, O_A, O_B of 128 columns each.  P is the A operand from
// TMEM; V is the N-major B operand of the ring tile as it is stored.
// e4m3 caches: Q enters as f16 times a power of two per row; K's block scales
// multiply the scores and V's enter the exponent, as in row_gqa.cu.
//
// A V element that is not finite in a tile that some rows do not see would
// reach them as 0 * inf: such elements are zeroed in the ring, remembered by
// key, and added to the rows that see them at the end.
// Every wait is bounded (mbar_wait); a timeout sets the error word.
#include <climits>

#include "kv_scale.cuh"
#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"
#include "row_output.cuh"
#include "stage_helpers.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kTileBytes = 128 * 256;  // 128 rows of 128 16-bit values, two 64-dim atoms
constexpr int kAtom = 128 * 128;
constexpr int kBufs = 4;
constexpr int kSlots = 4;        // tiles whose scales and page masks are kept
constexpr int kPoison = 32;      // masked tiles that can remember odd V elements
constexpr float kUp = 8.0f;
constexpr float kLeast = 1.2e-38f;  // a score's factor is never 0: masked scores are -inf

struct TileShared {
  uint64_t full[kBufs], empty[kBufs], info[kSlots], s_full[2], p_ready[2], o_full, loads_done;
  uint32_t tmem;
  int poison_n;
  int poison_tile[kPoison];        // first key
  uint32_t poison[kPoison][4];     // keys with an odd V element
  uint32_t valid[kSlots][4];       // keys on pages of the cache
  int check[kSlots];               // some key is not
  float4 scale[kSlots][8];         // ks, log2 vs, 1 / vs of each 16 keys
  float qs[256];                   // per M row: what its scores are multiplied by
  int pos[256];                    // its position (-1: before the start; INT_MIN: no row)
};
constexpr int kSmem = 1024 + 2 * kTileBytes + kBufs * kTileBytes + static_cast<int>(sizeof(TileShared));

// ---------------------------------------------------------------- tcgen05
// The MMAs and commits below are executed by a whole converged warp and issued
// by the lane that elect.sync names (always the same one): their operands
// then stay in uniform registers, and an issue costs a few cycles instead of
// the ~120 that a lone lane's took (measured: as long as the MMA itself).
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit inputs, fp32 accumulate
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar))
      : "memory");
}
// One box of a 2-D map, issued likewise.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ unsigned long long f32x2_fma(unsigned long long a, unsigned long long b,
                                                        unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ void f32x2_unpack(unsigned long long a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
          "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Registers of a warpgroup's threads, which together keep to the launch's 128
// a thread: all four warps of the group execute it.
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Byte of 16-byte chunk c (8 dims) of row r in a swizzled two-atom tile.
__device__ __forceinline__ int tile_byte(int r, int c) {
  return (c >> 3) * kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// The key tiles of a CTA: those of the sinks, then those of the window.
struct Tiles {
  int ns, w0, n;  // sink tiles, first window tile, all
  __device__ __forceinline__ int first_key(int j) const { return (j < ns ? j : w0 + j - ns) * 128; }
};

// KVT 0 bf16, 1 e4m3 with static scales, 2 e4m3 with block scales
template <int KVT>
__global__ void __launch_bounds__(kThreads, 1) window_tile_kernel(const __grid_constant__ CUtensorMap tmap, const RowGqaParams P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_pmin, s_pmax, s_neg;
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sQ = smem_raw + pad;
  uint8_t* sKV = sQ + 2 * kTileBytes;
  TileShared& sh = *reinterpret_cast<TileShared*>(sKV + kBufs * kTileBytes);
  constexpr int kSoftmaxRegs = KVT == 0 ? 192 : 176, kLoadRegs = KVT == 0 ? 80 : 112, kMmaRegs = 48;
  static_assert(2 * kSoftmaxRegs + kLoadRegs + kMmaRegs <= 4 * 128, "the launch's registers");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform)
  const int kvh = blockIdx.y, split = blockIdx.z;
  const int G = P.group, R = 128 / G;
  griddep_launch_dependents();
  const int4 grp = find_group(P.qsl, P.reqs, P.rows, 2 * R, blockIdx.x, P.err);
  if (grp.x < 0) return;
  const int row0 = grp.x, nrows = grp.y, req = grp.z;

  // ---- positions of the CTA's rows
  if (tid == 0) {
    s_pmin = INT_MAX;
    s_pmax = -1;
    s_neg = 0;
    sh.poison_n = 0;
  }
  if (tid < kPoison * 4) sh.poison[tid >> 2][tid & 3] = 0u;
  __syncthreads();
  if (tid < nrows) {
    const int p = P.logical[row0 + tid];
    if (p >= 0) {
      atomicMin(&s_pmin, p);
      atomicMax(&s_pmax, p);
    } else {
      s_neg = 1;
    }
  }
  __syncthreads();
  const int pmin = s_pmin, pmax = s_pmax;
  const bool neg = s_neg != 0;  // some row sees nothing
  const int wlo = pmax < 0 ? 0 : max(0, pmin - P.window + 1);     // first key of any window
  const int wlo_all = pmax < 0 ? 0 : max(0, pmax - P.window + 1); // of every window
  Tiles T;
  {
    const int sinks = min(P.sinks, pmax + 1);
    T.ns = (sinks + 127) >> 7;
    T.w0 = max(T.ns, wlo >> 7);
    const int end = P.window > 0 ? (pmax >> 7) + 1 : 0;
    T.n = pmax < 0 ? 0 : T.ns + max(0, end - T.w0);
  }
  const int per = (T.n + P.splits - 1) / P.splits;
  const int j0 = split * per, nt = max(0, min(T.n, j0 + per) - j0);
  const bool two = nrows > R;

  if (nt == 0) {  // nothing to see here: zeros, or an empty split
    for (int i = tid; i < nrows * G * 16; i += kThreads) {
      const int d0 = (i & 15) * 8, h = (i >> 4) % G, r = (i >> 4) / G;
      const long long head = static_cast<long long>(row0 + r) * P.hq + kvh * G + h;
      if (P.splits > 1) {
        if (d0 == 0) P.part_lse[static_cast<long long>(split) * P.rows * P.hq + head] = -INFINITY;
      } else {
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store_gated8(P, head * 128 + d0, z, load_gate(P, head * 128 + d0));
      }
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sh.full[i], 128);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 128);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&sh.info[i], 1);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.loads_done, 128);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  // ---- Q, a half-warp per M row
  for (int m = tid >> 4; m < 256; m += kThreads / 16) {
    const int lane16 = tid & 15, im = m & 127;
    const int r = (m >> 7) * R + im / G;
    const bool act = im < R * G && r < nrows;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (act)
      v = *reinterpret_cast<const uint4*>(P.q + (static_cast<long long>(row0 + r) * P.hq + kvh * G + im % G) * 128 + 8 * lane16);
    float qs = 0.08838834764831845f * kLog2e;
    if constexpr (KVT != 0) {
      // f16 times a power of two that brings the row's largest |q| into
      // [2^14, 2^15): exact down to 2^-28 of it
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[8], peak = 0.f;
      bool odd = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
        odd |= !(fabsf(x[e]) <= 3.39e38f);
        peak = fmaxf(peak, fabsf(x[e]));
      }
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) {
        peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
        odd |= __shfl_xor_sync(0xffffffffu, static_cast<int>(odd), o) != 0;
      }
      const int e = peak > 0.f ? max(__float_as_int(peak) >> 23, 1) - 127 - 14 : 0;
      const float f0 = exp2i(-(e / 2)), f1 = exp2i(-(e - e / 2));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = odd ? 0.f : x[i] * f0 * f1;
      v = make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]), pack_f16x2(x[6], x[7]));
      qs = fmaxf(exp2i(e / 2) * (qs * (KVT == 1 ? P.k_scale : 1.0f)) * exp2i(e - e / 2), kLeast);
      if (odd) qs = -1.0f;  // (the row's result is a NaN)
    }
    *reinterpret_cast<uint4*>(sQ + (m >> 7) * kTileBytes + tile_byte(im, lane16)) = v;
    if (lane16 == 0) {
      sh.qs[m] = qs;
      sh.pos[m] = act ? max(P.logical[row0 + r], -1) : INT_MIN;
    }
  }
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ loads
    regs_down<kLoadRegs>();
    const int lt = tid - 256;  // 0 .. 127
    const int32_t* bt_row = P.block_table + static_cast<long long>(req) * P.bt_stride;
    const uint8_t* kvb = static_cast<const uint8_t*>(P.kv);
    const bool page_pow2 = (P.page & (P.page - 1)) == 0;
    const int page_shift = __ffs(P.page) - 1;
    auto seen = [&](int key) { return key <= pmax && (key >= wlo || key < P.sinks); };
    // cache row of the first key of 16-key block (lane & 7) of tile j, or
    // kUnseen: nothing to see there, or kNoPage: a page that is none
    constexpr uint32_t kUnseen = 0xFFFFFFFFu, kNoPage = 0xFFFFFFFEu;
    auto fetch_rows = [&](int j) -> uint32_t {
      const int k0 = T.first_key(j) + 16 * (lane & 7);
      if (!(k0 <= pmax && (k0 + 15 >= wlo || k0 < P.sinks))) return kUnseen;
      const int blk = page_pow2 ? k0 >> page_shift : k0 / P.page;
      const int pid = blk < P.bt_stride ? bt_row[blk] : -1;
      if (pid < 0 || pid >= P.num_blocks) return kNoPage;
      return (static_cast<uint32_t>(pid) * P.hkv + kvh) * static_cast<uint32_t>(P.page) + (k0 - blk * P.page);
    };
    // the masks and scales of tile j, by one warp, before its K is announced
    auto publish = [&](int j, uint32_t rows) {
      const int slot = (j - j0) % kSlots;
      const unsigned bad = __ballot_sync(0xffffffffu, rows == kNoPage) & 0xFFu;
      if (lane < 4) {
        const unsigned two_blocks = (bad >> (2 * lane)) & 3u;
        sh.valid[slot][lane] = ~(((two_blocks & 1u) ? 0xFFFFu : 0u) | ((two_blocks & 2u) ? 0xFFFF0000u : 0u));
      }
      if (lane == 0) {
        sh.check[slot] = bad != 0u;
        if (bad) flag_error(P.err);
      }
      if (KVT == 2 && lane < 8) {
        int ek = 0, ev = 0;
        if (rows < kNoPage) {
          const uint16_t w = *reinterpret_cast<const uint16_t*>(P.scales + 2ll * (rows / P.scale_block));
          ek = scale_exp(w & 0xFF);
          ev = scale_exp(w >> 8);
        }
        sh.scale[slot][lane] = make_float4(exp2i(ek), static_cast<float>(ev), exp2i(-ev), 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.info[slot]);
    };
    // zeroes odd V elements of a masked tile and remembers their keys
    auto tile_masked = [&](int j) {
      const int kb = T.first_key(j);
      return neg || !((kb >= wlo_all || kb + 127 < P.sinks) && kb + 127 <= pmin);
    };
    int masked_n = 0;
    auto remember = [&](int slot, int key) {
      if (slot < kPoison) atomicOr(&sh.poison[slot][key >> 5], 1u << (key & 31));
      else flag_error(P.err);
    };
    auto open_poison = [&](int j) {  // (the same in every thread)
      if (lt == 0 && masked_n < kPoison) sh.poison_tile[masked_n] = T.first_key(j);
      return masked_n++;
    };

    if constexpr (KVT == 0) {
      // Tiles that every row sees come by TMA where a box holds at least 32
      // keys of a page (P.box; the SM's TMA unit takes ~90 cycles a box,
      // whatever its size, and a K and V tile have 2048 cycles between them);
      // the others by cp.async, which zeroes what is not seen.
      constexpr int LAG = 2;  // tiles in flight behind the one being issued
      uint32_t rows = fetch_rows(j0), rows_next = kUnseen;
      auto finish = [&](int s) {  // tile s has landed
        const int j = j0 + (s >> 1), b = s % kBufs;
        if ((s & 1) && tile_masked(j)) {
          const int slot = open_poison(j);
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            const int key = 8 * i + (lt >> 4);
            uint4* p = reinterpret_cast<uint4*>(sKV + b * kTileBytes + tile_byte(key, lt & 15));
            uint4 v = *p;
            uint32_t w[4] = {v.x, v.y, v.z, v.w}, odd = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7F80u) == 0x7F80u) {
                w[e] &= 0xFFFF0000u;
                odd = 1u;
              }
              if ((w[e] & 0x7F800000u) == 0x7F800000u) {
                w[e] &= 0xFFFFu;
                odd = 1u;
              }
            }
            if (odd) {
              *p = make_uint4(w[0], w[1], w[2], w[3]);
              remember(slot, key);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&sh.full[b]);
      };
      int done = 0;  // tiles announced
      const int dst0 = tile_byte(lt >> 4, lt & 15);
      for (int s = 0; s < 2 * nt; ++s) {
        const int j = j0 + (s >> 1), b = s % kBufs, is_v = s & 1;
        if (!is_v) {
          if (s > 0) rows = rows_next;
          rows_next = (s >> 1) + 1 < nt ? fetch_rows(j + 1) : kUnseen;
        }
        const int kb = T.first_key(j);
        const bool masked = tile_masked(j);
        const bool tma = P.box != 0 && !masked && __all_sync(0xffffffffu, rows < kNoPage);
        if (tma && done < s) {
          cp_async_wait<0>();
          for (; done < s; ++done) finish(done);
        }
        if (!all_ok(mbar_wait(&sh.empty[b], ((s / kBufs) & 1) ^ 1, P.err))) break;
        if (!is_v && warp == 8) publish(j, rows);
        uint8_t* dst = sKV + b * kTileBytes;
        if (tma) {
          if (lt == 0)
            mbar_arrive_expect_tx(&sh.full[b], kTileBytes);
          else
            mbar_arrive(&sh.full[b]);
          __syncwarp();
          if (warp == 8) {
            // boxes of 64 dims of P.box keys
            for (int k = 0; k < 128; k += P.box) {
              const int r = static_cast<int>(__shfl_sync(0xffffffffu, rows, k >> 4));
              tma_box(dst + k * 128, &tmap, is_v * 128, r, &sh.full[b]);
              tma_box(dst + kAtom + k * 128, &tmap, is_v * 128 + 64, r, &sh.full[b]);
            }
          }
          done = s + 1;
          continue;
        }
        const uint8_t* src = kvb + is_v * 256 + (lt & 15) * 16;
        uint32_t base[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) base[i] = __shfl_sync(0xffffffffu, rows, i);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = 8 * i + (lt >> 4);
          const uint32_t r = base[i >> 1];
          const bool ok = r < kNoPage && (!masked || seen(kb + key));
          cp_async16(dst + dst0 + i * 1024, src + static_cast<unsigned long long>(ok ? r + (key & 15) : 0u) * 512,
                     ok ? 16u : 0u);
        }
        cp_async_commit();
        if (s - done >= LAG) {
          cp_async_wait<LAG>();
          finish(done++);
        }
      }
      cp_async_wait<0>();
      for (; done < 2 * nt; ++done) finish(done);
    } else {
      // 16 codes a lane and load; the next tile's codes are in flight while
      // this one's are converted
      auto load = [&](int s, uint32_t rows, uint4 (&v)[8]) {
        const int j = j0 + (s >> 1), kb = T.first_key(j);
        const bool masked = tile_masked(j);
        const uint8_t* src = kvb + (s & 1) * 128 + (lt & 7) * 16;
        uint32_t base[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) base[i] = __shfl_sync(0xffffffffu, rows, i);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool ok = base[i] < kNoPage && (!masked || seen(kb + 16 * i + (lt >> 3)));
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (ok) v[i] = *reinterpret_cast<const uint4*>(src + static_cast<unsigned long long>(base[i] + (lt >> 3)) * 256);
        }
      };
      uint32_t rows = fetch_rows(j0), rows_next = nt > 1 ? fetch_rows(j0 + 1) : kUnseen;
      uint4 cur[8], nxt[8];
      load(0, rows, cur);
      const int dst0 = tile_byte(lt >> 3, 2 * (lt & 7)), dst1 = tile_byte(lt >> 3, 2 * (lt & 7) + 1);
      for (int s = 0; s < 2 * nt; ++s) {
        const int j = j0 + (s >> 1), b = s % kBufs, is_v = s & 1;
        const uint32_t rows_here = rows;
        if (is_v) {  // the next load is the next tile's K
          rows = rows_next;
          rows_next = (s >> 1) + 2 < nt ? fetch_rows(j + 2) : kUnseen;
        }
        if (s + 1 < 2 * nt) load(s + 1, rows, nxt);
        if (!all_ok(mbar_wait(&sh.empty[b], ((s / kBufs) & 1) ^ 1, P.err))) break;
        if (!is_v && warp == 8) publish(j, rows_here);
        int slot = -1;
        if (is_v && tile_masked(j)) slot = open_poison(j);
        uint8_t* dst = sKV + b * kTileBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = 16 * i + (lt >> 3);
          uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w}, h[8];
          if (slot >= 0) {
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int q = 0; q < 32; q += 8)
                if (((w[e] >> q) & 0x7Fu) == 0x7Fu) {
                  w[e] &= ~(0xFFu << q);
                  odd = true;
                }
            if (odd) remember(slot, key);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_f16x2x2(w[e], h[2 * e], h[2 * e + 1]);
          *reinterpret_cast<uint4*>(dst + dst0 + 2048 * i) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + dst1 + 2048 * i) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&sh.full[b]);
#pragma unroll
        for (int i = 0; i < 8; ++i) cur[i] = nxt[i];
      }
    }
    if (lt == 0) sh.poison_n = min(masked_n, kPoison);
    mbar_arrive(&sh.loads_done);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ MMA
    regs_down<kMmaRegs>();
    if (warp == 12) {
      constexpr uint32_t fmt = KVT == 0 ? 1u : 0u;  // bf16 or f16
      const uint32_t id_s = umma_idesc(fmt, 128, 128);
      const uint32_t id_o = id_s | (1u << 16);      // B is N-major
      const uint64_t q0 = umma_sdesc_sw128(smem_addr(sQ));
      const uint64_t k0 = umma_sdesc_sw128(smem_addr(sKV));
      // N-major: the second 64 dims one atom on, 8-key groups 1024 bytes apart
      const uint64_t v0 = (k0 & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(kAtom >> 4) << 16);
      auto scores = [&](int x, int s) {
        const uint64_t a = q0 + ((x * kTileBytes) >> 4), b = k0 + (((s % kBufs) * kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
          mma_ss(tmem + 128 * x, a + off, b + off, id_s, kk != 0 ? 1u : 0u);
        }
      };
      auto values = [&](int x, int s, bool first) {
        const uint64_t b = v0 + (((s % kBufs) * kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * kk, b + ((kk * 2048) >> 4), id_o,
                      first && kk == 0 ? 0u : 1u);
      };
      auto wait_full = [&](int s) {
        const bool ok = all_ok(mbar_wait(&sh.full[s % kBufs], (s / kBufs) & 1, P.err));
        tc_fence_after_sync();
        return ok;
      };
      bool ok = wait_full(0);
      if (ok) {
        scores(0, 0);
        mma_commit(&sh.s_full[0]);
        if (two) {
          scores(1, 0);
          mma_commit(&sh.s_full[1]);
        }
        mma_commit(&sh.empty[0]);
      }
      for (int j = 0; j < nt && ok; ++j) {
        const int sv = 2 * j + 1, sk = 2 * j + 2;
        const bool more = j + 1 < nt;
        ok = wait_full(sv) && all_ok(mbar_wait(&sh.p_ready[0], j & 1, P.err));
        if (!ok) break;
        tc_fence_after_sync();
        values(0, sv, j == 0);
        if (more) {
          ok = wait_full(sk);
          if (!ok) break;
          scores(0, sk);
          mma_commit(&sh.s_full[0]);
        }
        if (two) {
          ok = all_ok(mbar_wait(&sh.p_ready[1], j & 1, P.err));
          if (!ok) break;
          tc_fence_after_sync();
          values(1, sv, j == 0);
        }
        mma_commit(&sh.empty[sv % kBufs]);
        if (more) {
          if (two) {
            scores(1, sk);
            mma_commit(&sh.s_full[1]);
          }
          mma_commit(&sh.empty[sk % kBufs]);
        }
      }
      mma_commit(&sh.o_full);
    }
  } else if (warp < 4 || two) {
    // ------------------------------------------------------------ softmax
    regs_up<kSoftmaxRegs>();
    const int x = warp >> 2, m = tid;  // M row m & 127 of tile x
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + 128 * x + lanes, to = tmem + 256 + 128 * x + lanes;
    const float qs = fabsf(sh.qs[m]);
    const int p = sh.pos[m];
    // the tile's own bounds decide which key tiles need masks
    const int hi_all = __reduce_min_sync(0xffffffffu, p == INT_MIN ? INT_MAX : p);
    const int lo_all = __reduce_max_sync(0xffffffffu, p == INT_MIN ? INT_MIN : p - P.window + 1);
    float ref = -INFINITY, l = sh.qs[m] < 0.f ? __int_as_float(0x7fffffff) : 0.f;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      const int kb = T.first_key(j0 + j), slot = j % kSlots;
      // its masks and scales, then its scores.  (A slot's next tile is
      // published only after both softmaxes are done with this one: its K
      // waits for a ring buffer that S of tile j + 2 frees.)
      ok = all_ok(mbar_wait(&sh.info[slot], (j / kSlots) & 1, P.err) && mbar_wait(&sh.s_full[x], j & 1, P.err));
      if (!ok) break;
      tc_fence_after_sync();
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_issue(ts + 32 * c, r[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld32(r[c]);
      const bool plain = kb + 127 <= hi_all && (kb >= lo_all || kb + 127 < P.sinks) && sh.check[slot] == 0;
      if (!plain) {
        const int hi = p - kb, lo = p - P.window + 1 - kb, sk = P.sinks - kb;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t val = sh.valid[slot][c];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int k = 32 * c + i;
            const bool vis = k <= hi && (k >= lo || k < sk) && ((val >> i) & 1u);
            if (!vis) r[c][i] = 0xFF800000u;
          }
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const uint32_t* rr = &r[b >> 1][(b & 1) * 16];
        float bm = max3(__uint_as_float(rr[0]), __uint_as_float(rr[1]), __uint_as_float(rr[2]));
        float b2 = max3(__uint_as_float(rr[3]), __uint_as_float(rr[4]), __uint_as_float(rr[5]));
#pragma unroll
        for (int i = 6; i < 14; i += 4) {
          bm = max3(bm, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
          b2 = max3(b2, __uint_as_float(rr[i + 2]), __uint_as_float(rr[i + 3]));
        }
        bm = fmaxf(max3(bm, __uint_as_float(rr[14]), __uint_as_float(rr[15])), b2);
        if constexpr (KVT == 2) {
          const float4 sc = sh.scale[slot][b];
          bm = fmaf(bm, fmaxf(qs * sc.x, kLeast), sc.y);
        }
        mx = fmaxf(mx, bm);
      }
      if constexpr (KVT != 2) mx *= qs;
      if (__any_sync(0xffffffffu, mx > ref + kUp)) {
        const float mn = fmaxf(ref, mx);
        const float al = ex2_ftz(ref - (mn == -INFINITY ? 0.f : mn));
        l *= al;
        if (j > 0) {  // (S of this tile is complete, so O of the last one is)
          uint32_t o[32];
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tmem_ld32_issue(to + 32 * c, o);
            tmem_wait_ld32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tmem_st32(to + 32 * c, o);
          }
        }
        ref = mn;
      }
      const float neg = ref == -INFINITY ? 0.f : -ref;
      unsigned long long sum2 = 0ull;  // (two sums, of even and odd keys)
      float sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float c = qs, base = neg, inv_vs = 1.0f;
          if constexpr (KVT == 2) {
            const float4 sc = sh.scale[slot][4 * h + b];
            c = fmaxf(c * sc.x, kLeast);
            base += sc.y;
            inv_vs = sc.z;
          }
          const unsigned long long c2 = f32x2_pack(c, c), base2 = f32x2_pack(base, base);
          unsigned long long bs2 = KVT == 2 ? 0ull : sum2;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const uint32_t* rr = &r[2 * h + (b >> 1)][(b & 1) * 16 + i];
            float p0, p1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(rr[0]), __uint_as_float(rr[1])), c2, base2), p0, p1);
            p0 = ex2_ftz(p0);
            p1 = ex2_ftz(p1);
            bs2 = f32x2_add(bs2, f32x2_pack(p0, p1));
            pk[8 * b + (i >> 1)] = KVT == 0 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
          }
          if constexpr (KVT == 2)
            sum = fmaf(f32x2_hsum(bs2), inv_vs, sum);
          else
            sum2 = bs2;
        }
        tmem_st32(ts + 32 * h, pk);
      }
      l += KVT == 2 ? sum : f32x2_hsum(sum2);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&sh.p_ready[x]);
    }
    // ---- output
    ok = all_ok(ok && mbar_wait(&sh.o_full, 0, P.err) && mbar_wait(&sh.loads_done, 0, P.err));
    tc_fence_after_sync();
    const int im = m & 127, rr = x * R + im / G;
    const bool act = ok && im < R * G && rr < nrows;
    const long long head = static_cast<long long>(row0 + rr) * P.hq + kvh * G + im % G;
    // (a NaN sum is not an empty row)
    const float inv = l == 0.f ? 0.f : (KVT == 1 ? P.v_scale : 1.0f) / l;
    bool poisoned = false;
    for (int b = 0; b < sh.poison_n; ++b)
      poisoned |= (sh.poison[b][0] | sh.poison[b][1] | sh.poison[b][2] | sh.poison[b][3]) != 0u;
    const long long ph = static_cast<long long>(split) * P.rows * P.hq + head;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[32];
      tmem_ld32_issue(to + 32 * c, o);
      tmem_wait_ld32(o);
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
      if (!act) continue;
      if (poisoned) {  // what the row sees of the remembered elements
#pragma unroll 1
        for (int b = 0; b < sh.poison_n * 128; ++b) {
          if (!((sh.poison[b >> 7][(b >> 5) & 3] >> (b & 31)) & 1u)) continue;
          const int key = sh.poison_tile[b >> 7] + (b & 127);
          if (key > p || !(key > p - P.window || key < P.sinks)) continue;
          const int blk = key / P.page;
          const int pid = P.block_table[static_cast<long long>(req) * P.bt_stride + blk];
          const long long at = ((static_cast<long long>(pid) * P.hkv + kvh) * P.page + key - blk * P.page) * 256 + 128 + 32 * c;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float v = KVT == 0 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(P.kv)[at + i]) << 16)
                            : (static_cast<const uint8_t*>(P.kv)[at + i] & 0x7F) == 0x7F ? __int_as_float(0x7fffffff) : 0.f;
            if (!(fabsf(v) <= 3.39e38f)) f[i] += v;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float y[8] = {f[8 * q], f[8 * q + 1], f[8 * q + 2], f[8 * q + 3], f[8 * q + 4], f[8 * q + 5], f[8 * q + 6], f[8 * q + 7]};
        const int d0 = 32 * c + 8 * q;
        if (P.splits > 1) {
          float4* po = reinterpret_cast<float4*>(P.part_o + ph * 128 + d0);
          po[0] = make_float4(y[0], y[1], y[2], y[3]);
          po[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
          store_gated8(P, head * 128 + d0, y, load_gate(P, head * 128 + d0));
        }
      }
    }
    if (act && P.splits > 1) P.part_lse[ph] = l == 0.f ? -INFINITY : ref + log2f(l);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int KVT>
cudaError_t launch_kind(const RowGqaParams& p, const CUtensorMap& tmap, const dim3& grid, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(window_tile_kernel<KVT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_kernel(window_tile_kernel<KVT>, grid, dim3(kThreads), kSmem, stream, false, tmap, p);
}

}  // namespace

int window_tile_rows(int group) { return 2 * (128 / group); }

int window_tile_splits(int rows, int hkv, int group, long long max_tokens, int sms) {
  const int per = window_tile_rows(group);
  const long long ctas = static_cast<long long>((rows + per - 1) / per) * hkv;
  if (ctas <= 0) return 1;
  const long long tiles = (max_tokens + 127) / 128 + 1;
  long long s = sms / ctas;
  if (s > tiles / 2) s = tiles / 2;
  if (s > 64) s = 64;
  return s < 1 ? 1 : static_cast<int>(s);
}

cudaError_t launch_window_tile(const RowGqaParams& p, const CUtensorMap& tmap, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  long long groups = static_cast<long long>(p.rows) / window_tile_rows(p.group) + p.reqs;
  if (groups > p.rows) groups = p.rows;
  const dim3 grid(static_cast<unsigned>(groups), p.hkv, p.splits);
  cudaError_t e;
  switch (p.kv_dtype) {
    case QSA_DTYPE_BF16: e = launch_kind<0>(p, tmap, grid, stream); break;
    case QSA_DTYPE_E4M3: e = launch_kind<1>(p, tmap, grid, stream); break;
    default: e = launch_kind<2>(p, tmap, grid, stream); break;
  }
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_row_merge(p, stream);
}

}  // namespace qsa
