// Window attention of many rows per request (prefill chunks, verify steps) on
// the tcgen05 tensor cores.
//
// Mathematics.  As in row_gqa.cu; here 128 (row, head) pairs of one request
// and KV head are the M rows of S = Q K^T and O += P V, R = 128 / G rows with
// their G heads, and a CTA runs two such tiles, A and B (rows r0 .. r0 + R - 1
// and the R after them), over one stream of 128-key tiles.  Where the rows fit
// tile A, B takes the same rows over every other key tile (e4m3 caches), and
// A's warps join the two at the end.  Two threads share an M row, 64 keys each;
// both keep the row's reference and a sum of their own weights in registers.
//
// Roles, 20 warps:
//   0-7, 8-15 softmax of tile A, B: S from TMEM, masks on the tiles that need
//             them, P back over S's columns, at the end the gated output;
//   16        issues the MMAs: S_A(j+1) right after O_A(j), so the softmax of
//             one tile runs under the products of the other;
//   17        loads by TMA, in boxes that pages are multiples of;
//   18, 19    what needs a thread's hand: V of tiles that some row does not
//             see (keys that no row of the CTA sees become zeros, whatever the
//             cache holds there), V of e4m3 caches from codes to f16 (exact).
// Two warps to a row and tile because a warp alone on its scheduler issues an
// instruction every other cycle at best: with one, the ~550 instructions of a
// row's softmax took 1450 cycles, the two products 1060 a tile, and neither
// could hide the other.
// TMEM: S_A, S_B, O_A, O_B of 128 columns each.  P is the A operand from
// TMEM; V is the N-major B operand of the ring tile as it is stored.
// e4m3 caches: K's codes are multiplied as they are, by q split into two terms,
// hi in e4m3 and lo in e5m2, after a power of two per row that puts its largest
// |q| into [128, 256).  An element from 2^-6 up (2^-13 of the largest) is exact:
// hi takes 4 of its 8 bits and leaves at most 8 units of its last place (2^-13
// at the least), which 3 bits hold.  A smaller one leaves at most 2^-10 to lo,
// which is off by 2^-14 there, 2^-21 of the largest (with lo in e4m3, whose
// steps end at 2^-9: exact from 2^-9 of the largest, off by 2^-17).  P and V
// are f16.  K's block scales multiply the scores and
// V's enter the exponent, as in row_gqa.cu.
//
// A V element that is not finite in a tile that some rows do not see would
// reach them as 0 * inf: such elements are zeroed in the ring, remembered by
// key, and added to the rows that see them at the end.  Rows before their
// request's start see nothing and set no masks: their sums are not used.
// Every wait is bounded (mbar_wait); a timeout sets the error word.
//
// Roundings: as in row_gqa.cu (the A operand in TMEM has V's type).
//
// Bound: the tensor cores in the loop (a tile's S of 128 x 128 x 128 and its
// product with V take ~1270 cycles, and a row group's tile waits ~1600 for its
// weights while the other group's products take ~1060: 2900 cycles for two
// groups and 128 keys), fixed costs for short windows (~10 000 cycles to the
// first S, ~8 000 from the last weights to the end) and, at one CTA an SM, the
// last wave.  Measured, 32 query and 4 KV heads, window 4096, 4 sinks, ten calls
// on ten sets of inputs: 16 384 rows 813 us (1.35 PFLOP/s), 8192 rows 409 us on
// bf16 and 435 us with block scales; 32 requests of 4 rows 57 us on bf16 (4.8
// TB/s) and 49 us with block scales; 3 requests of ~1200 to 2011 rows, 24 query
// heads, window 1000: 109 us (484 CTAs, 3.2 waves that take four).
// Without the softmax the loads and products alone took 374 us for the 8192
// rows.
#include <cuda_fp16.h>

#include <climits>

#include "kv_scale.cuh"
#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"
#include "row_output.cuh"
#include "stage_helpers.cuh"

namespace qsa {
namespace {

constexpr int kSoftWarps = 16;
constexpr int kThreads = (kSoftWarps + 4) * 32;
constexpr int kTile = 128 * 256;  // bytes of 128 rows of 128 16-bit values, two 64-dim atoms
constexpr int kAtom = 128 * 128;
constexpr int kSlots = 8;        // tiles whose scales and page masks are kept
constexpr int kPoison = 32;      // tiles that can remember odd V elements
// A row's reference is moved when a weight has grown by 2^8 (bf16) or 2^10.
// bf16 weights: it is set so that the largest is 2^-7; that one has reached 2
// shows in the top bit of its exponent, so a tile is checked by or-ing its
// packed weights, half the instructions of a maximum.  f16 weights, whose
// subnormals begin at 2^-14, are set to 1 and their packed maximum is taken
// (the same trick with room for 2^5 moved references so often that a chunk
// took 560 instead of 536 us).
template <int KVT>
constexpr float kRoom = KVT == 0 ? 7.0f : 0.0f;
constexpr uint32_t kTwo = 0x40004000u;
constexpr float kFar = 1048576.f;  // 2^20: fp32 steps of 2^-3
constexpr float kLeast = 1.2e-38f;  // a score's factor is never 0: masked scores are -inf

// The rings.  e4m3 caches: K tiles stay codes, half the size, and V's codes
// have a ring of their own before they become f16.
template <int KVT>
struct Rings {
  static constexpr int NK = KVT == 0 ? 2 : 3, NV = 2, NR = KVT == 0 ? 0 : 2;
  static constexpr int kKey = KVT == 0 ? kTile : kAtom;
  static constexpr int kBytes = NK * kKey + NV * kTile + NR * kAtom;
  static_assert(kSlots > NK + 2, "a slot is rewritten only after its tile's softmax");
};

// A CTA's rows and the places of its keys, for the rare questions what they see.
struct Rows {
  const int32_t* positions;
  int n, window, sinks;
  int ns, shift;  // (of Tiles)
  bool apart;     // there may be keys between their windows that nobody sees
  unsigned long long* err;
};

struct TileShared {
  uint64_t kfull[3], kempty[3], vfull[2], vempty[2], vgo[2], rfull[2], rempty[2];
  uint64_t info[kSlots], s_full[2], p_ready[2], q_ready[2], o_full[2], loads_done;
  uint32_t tmem;
  int poison_tile[kPoison];        // its number times 128, or -1 from the first free entry on
  uint32_t poison[kPoison][4];     // keys with an odd V element
  uint32_t odd_keys[2][4];         // those of the tile that warp 18, 19 is at
  uint32_t valid[kSlots][4];       // keys on pages of the cache
  int check[kSlots];               // some key is not
  int first[kSlots][2];            // first key of each half, -1: of two stretches of keys, or not all on pages
  int ns, shift;                   // (of Tiles)
  Rows rows[3];                    // of the warps that load, one each
  alignas(16) uint32_t scale[kSlots][8];  // of each 16 keys, two bf16: ks, and log2 vs above it
  float qs[256];                   // per M row: what its scores are multiplied by (< 0: its scores are NaN)
  float pair[2][2][256];           // what a row's two threads tell each other
  float join[2][128];              // tile B's sums and references, where it has the same rows as A
};
template <int KVT>
constexpr int kSmem = 1024 + 2 * kTile + Rings<KVT>::kBytes + static_cast<int>(sizeof(TileShared));

// ---------------------------------------------------------------- tcgen05
// The MMAs and commits below are executed by a whole converged warp and issued
// by the lane that elect.sync names (always the same one): their operands
// then stay in uniform registers, and an issue costs a few cycles instead of
// the ~120 that a lone lane's took (measured: as long as the MMA itself).
// Matrix descriptors by their low words (address, leading offset): the high
// word (8-row groups 1024 bytes apart, 128-byte swizzle) is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
  return ((saddr >> 4) & 0x3FFFu) | ((leading >> 4) << 16);
}
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit inputs, fp32 accumulate
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Same for 8-bit inputs
__device__ __forceinline__ void mma_ss_f8(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
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
// 16 columns, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Registers of a warpgroup's threads, which together keep to the launch's 96
// a thread: all four warps of the group execute it.
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Two floats -> two e5m2 bytes (to nearest even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint16_t f32x2_to_e5m2x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}
// Byte of 16-byte chunk c (8 dims) of row r in a swizzled two-atom tile.
__device__ __forceinline__ constexpr int tile_byte(int r, int c) {
  return (c >> 3) * kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The two warps of a row meet (64 threads); with a vote, any's answer.
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0u;
}

// The n lowest bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
template <int N>
struct Int {
  static constexpr int value = N;
};
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// The keys of a CTA, in boxes: those of the sinks, ns of them, then those of the
// windows, `shift` on; n tiles of 128.
struct Tiles {
  int ns, shift, n;
  __device__ __forceinline__ int key(int v) const { return v < ns ? v : v + shift; }
};

// Whether one of the rows sees one of the keys a .. b (a warp's question).
__device__ __forceinline__ bool rows_see(const Rows* rows, int a, int b) {
  bool yes = false;
#pragma unroll 1
  for (int r = threadIdx.x & 31; r < rows->n; r += 32) {
    const int p = min(rows->positions[r], kMaxKeys);  // (as window_position; below 0 it sees none)
    yes |= p >= a && (a < rows->sinks || (rows->window > 0 && b > p - rows->window));
  }
  return __any_sync(0xffffffffu, yes);
}

// Counts an error where one of them sees a key of the 16-key blocks `blocks` of
// the tile from v on.
__device__ __noinline__ void count_blocks(const Rows* rows, int v, unsigned blocks) {
  bool seen = !rows->apart;
#pragma unroll 1
  for (; blocks != 0u && !seen; blocks &= blocks - 1u) {
    const int k0 = Tiles{rows->ns, rows->shift, 0}.key(v + 16 * (__ffs(blocks) - 1));
    seen = rows_see(rows, k0, k0 + 15);
  }
  if (seen && (threadIdx.x & 31) == 0) flag_error(rows->err);
}

// Files the odd keys that a warp has found in the tile from v on, but for those
// that nobody sees.
__device__ __noinline__ void file_poison(TileShared* sh, int which, int v) {
  const Rows* rows = &sh->rows[which];
  uint32_t* odd_keys = sh->odd_keys[which & 1];
  const Tiles T{rows->ns, rows->shift, 0};
  __syncwarp();
  uint32_t odd[4], any = 0u;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    odd[w] = odd_keys[w];
    const int k = v + 32 * w;
    if (rows->apart && odd[w] != 0u) {
      uint32_t look = rows_see(rows, T.key(k), T.key(k + 31)) ? odd[w] : 0u;
      odd[w] = 0u;
#pragma unroll 1
      for (; look != 0u; look &= look - 1u) {
        const int key = T.key(k + __ffs(look) - 1);
        if (rows_see(rows, key, key)) odd[w] |= look & -look;
      }
    }
    any |= odd[w];
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    int b = kPoison;
    if (any != 0u) {
      for (b = 0; b < kPoison; ++b) {
        const int was = atomicCAS(&sh->poison_tile[b], -1, v);
        if (was == -1 || was == v) break;
      }
      if (b == kPoison) flag_error(rows->err);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (b < kPoison) atomicOr(&sh->poison[b][w], odd[w]);
      odd_keys[w] = 0u;
    }
  }
  __syncwarp();
}

// KVT 0 bf16, 1 e4m3 with static scales, 2 e4m3 with block scales.
template <int KVT>
__global__ void __launch_bounds__(kThreads, 1) window_tile_kernel(const __grid_constant__ CUtensorMap tmap, const RowGqaParams P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_pmin, s_pmax;
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sQ = smem_raw + pad;
  using RG = Rings<KVT>;
  uint8_t* sK = sQ + 2 * kTile;
  uint8_t* sV = sK + RG::NK * RG::kKey;
  uint8_t* sR = sV + RG::NV * kTile;
  TileShared& sh = *reinterpret_cast<TileShared*>(sK + RG::kBytes);
  constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
  static_assert(4 * kSoftmaxRegs + kOtherRegs <= 5 * 96, "the launch's registers");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform)
  const int kvh = blockIdx.y, split = blockIdx.z;
  const int G = P.group, R = 128 / G;
  // the row and the head of an M row (below 256 + 16)
  const unsigned g_magic = 65536u / G + 1u;
  auto row_of = [&](int im) { return static_cast<int>(im * g_magic >> 16); };
  auto head_of = [&](int im) { return im - row_of(im) * G; };
  griddep_launch_dependents();
  // ---- barriers and TMEM, while the row group's loads are on their way
  if (tid == kThreads - 1) {
    // (vfull: a lane of each of warps 18 and 19, or the TMA warp's for both)
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.kfull[i], 1);
      mbar_init(&sh.kempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.vfull[i], 2);
      mbar_init(&sh.vempty[i], 1);
      mbar_init(&sh.vgo[i], 1);
      mbar_init(&sh.rfull[i], 1);
      mbar_init(&sh.rempty[i], 2);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 256);
      mbar_init(&sh.q_ready[i], 8);
      mbar_init(&sh.o_full[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&sh.info[i], 1);
    mbar_init(&sh.loads_done, 64);
    fence_barrier_init();
  }
  if (warp == kSoftWarps) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  const int4 grp = find_group(P.qsl, P.reqs, P.rows, 2 * R, blockIdx.x, P.err);
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  auto free_tmem = [&] {
    if (warp == kSoftWarps) tmem_dealloc(tmem, 512);
  };
  if (grp.x < 0) {
    free_tmem();
    return;
  }
  const int row0 = grp.x, nrows = grp.y, req = grp.z;

  // ---- positions of the CTA's rows, and behind them the Q rows on their way:
  // sixteen M rows a warp, a half-warp per row
  const int own_pos = tid < nrows ? window_position(P, row0 + tid) : -1;
  const bool two = nrows > R;  // tile B has rows of its own
  uint4 qv[8];
  if (warp < kSoftWarps) {
    const int im0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1) + (lane >> 4);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int im = im0 + 2 * u, r = (two ? warp >> 3 : 0) * R + row_of(im);
      qv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (im < R * G && r < nrows)
        qv[u] = *reinterpret_cast<const uint4*>(P.q + (static_cast<long long>(row0 + r) * P.hq + kvh * G + head_of(im)) * 128 + 8 * (lane & 15));
    }
  }
  if (tid == 0) {
    s_pmin = INT_MAX;
    s_pmax = -1;
  }
  if (tid < kPoison) sh.poison_tile[tid] = -1;
  if (tid < kPoison * 4) sh.poison[tid >> 2][tid & 3] = 0u;
  if (tid < 8) sh.odd_keys[tid >> 2][tid & 3] = 0u;
  __syncthreads();
  if (own_pos >= 0) {  // (others see nothing)
    atomicMin(&s_pmin, own_pos);
    atomicMax(&s_pmax, own_pos);
  }
  __syncthreads();
  const int pmin = s_pmin, pmax = s_pmax;
  const int wlo = pmax < 0 ? 0 : max(0, pmin - P.window + 1);     // first key of any window
  const int wlo_all = pmax < 0 ? 0 : max(0, pmax - P.window + 1); // of every window
  Tiles T;
  {
    const int keys = min(pmax + 1, P.keys);  // (a position may lie past the table)
    const int sinks = (min(P.sinks, keys) + P.box - 1) & -P.box, w0 = wlo & -P.box;
    const bool apart = P.window > 0 && w0 > sinks;
    T.ns = apart ? sinks : 0;
    T.shift = apart ? w0 - sinks : 0;
    // (windows that begin past the table hold none of its keys, the sinks stay)
    const int end = P.window > 0 ? max(keys - T.shift, T.ns) : sinks;
    T.n = pmax < 0 ? 0 : (end + 127) >> 7;
  }
  const int per = P.splits > 1 ? (T.n + P.splits - 1) / P.splits : T.n;
  const int j0 = split * per, nt = max(0, min(T.n, j0 + per) - j0);
  // Tile B without rows of its own takes every other key tile of A's: on e4m3
  // caches, whose bytes do not bound it (32 requests of 4 rows, 4100 tokens:
  // block scales 63 -> 51 us, bf16 58 -> 60 us).
  const bool duo = KVT != 0 && !two && nt > 1;

  if (pmax >= P.keys && tid == 0 && (P.window > 0 || P.sinks > P.keys)) flag_error(P.err);
  if (nt == 0) {  // nothing to see here: zeros, or an empty split
    for (int i = tid; i < nrows * G * 16; i += kThreads) {
      const int d0 = (i & 15) * 8, h = head_of(i >> 4), r = row_of(i >> 4);
      const long long head = static_cast<long long>(row0 + r) * P.hq + kvh * G + h;
      if (P.splits > 1) {
        if (d0 == 0) P.part_lse[static_cast<long long>(split) * P.rows * P.hq + head] = -INFINITY;
      } else {
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store_gated8(P, head * 128 + d0, z, load_gate(P, head * 128 + d0));
      }
    }
    free_tmem();
    return;
  }


  const int32_t* bt_row = P.block_table + static_cast<long long>(req) * P.bt_stride;
  const int scale_shift = KVT == 2 ? __ffs(P.scale_block) - 1 : 0;
  auto seen = [&](int key) { return key <= pmax && (key >= wlo || key < P.sinks); };
  // every row of the CTA sees keys a .. b; none does any of them
  auto all_seen = [&](int a, int b) { return b <= pmin && (a >= wlo_all || b < P.sinks); };
  // some row of the CTA does not see all of tile j
  auto tile_masked = [&](int j) {
    const int v = 128 * j, n = min(max(T.ns - v, 0), 128);
    return (n > 0 && !all_seen(v, v + n - 1)) || (n < 128 && !all_seen(v + n + T.shift, v + 127 + T.shift));
  };
  // Page id, then cache row, of the first key of 16-key block (lane & 7) of
  // tile j; kUnseen where there is nothing to see, kNoPage where the page is
  // none.
  constexpr uint32_t kUnseen = 0xFFFFFFFFu, kNoPage = 0xFFFFFFFEu;
  auto block_key = [&](int j) { return T.key(128 * j + 16 * (lane & 7)); };
  auto fetch_page = [&](int j) -> int {
    const int k0 = block_key(j);
    if (!(k0 <= pmax && (k0 + 15 >= wlo || k0 < P.sinks))) return -1;
    const int blk = page_of(P, k0);
    return blk < P.bt_stride ? bt_row[blk] : -1;
  };
  auto to_row = [&](int j, int page) -> uint32_t {
    const int k0 = block_key(j);
    if (!(k0 <= pmax && (k0 + 15 >= wlo || k0 < P.sinks))) return kUnseen;
    if (page < 0 || page >= P.num_blocks) return kNoPage;
    const int blk = page_of(P, k0);
    return (static_cast<uint32_t>(page) * P.hkv + kvh) * static_cast<uint32_t>(P.page) + (k0 - blk * P.page);
  };
  // V of a tile that some row does not see, or that lies on a page that is
  // none, has to be looked through (both loaders find the same answer)
  auto by_hand = [&](int j, uint32_t rows) { return tile_masked(j) || !all_ok(rows != kNoPage); };
  auto scale_word = [&](uint32_t rows) -> uint32_t {
    if (KVT != 2 || rows >= kNoPage) return 0x7F7Fu;
    return *reinterpret_cast<const uint16_t*>(P.scales + 2ll * (rows >> scale_shift));
  };
  // what the softmax needs to know of tile number i, before its K is announced
  auto publish = [&](int i, uint32_t rows, uint32_t scales) {
    const int slot = i % kSlots;
    const unsigned bad = __ballot_sync(0xffffffffu, rows == kNoPage) & 0xFFu;
    if (bad != 0u && lane < 4) {
      const unsigned two_blocks = (bad >> (2 * lane)) & 3u;
      sh.valid[slot][lane] = ~(((two_blocks & 1u) ? 0xFFFFu : 0u) | ((two_blocks & 2u) ? 0xFFFF0000u : 0u));
    }
    if (KVT == 2 && lane < 8) {
      const int ek = scale_exp(scales & 0xFF), ev = scale_exp(scales >> 8);
      sh.scale[slot][lane] = pack_bf16x2(exp2i(ek), static_cast<float>(ev));
    }
    if (lane < 2) {
      const int v = 128 * (j0 + i) + 64 * lane;
      sh.first[slot][lane] = bad != 0u || (v < T.ns && v + 63 >= T.ns) ? -1 : T.key(v);
    }
    // (counted where a row sees one of them)
    if (bad != 0u) count_blocks(&sh.rows[0], 128 * (j0 + i), bad);
    if (lane == 0) {
      sh.check[slot] = bad != 0u;
      sh.ns = T.ns;
      sh.shift = T.shift;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.info[slot]);
  };

  if (warp >= kSoftWarps) {
    regs_down<kOtherRegs>();
    if (warp > kSoftWarps) {
      // (windows that all meet leave no key out: the first and the last cover them)
      if (lane == 0)
        sh.rows[warp - (kSoftWarps + 1)] = {P.logical + row0, nrows, P.window, P.sinks, T.ns, T.shift, pmax - pmin >= P.window, P.err};
      __syncwarp();
    }
    if (warp >= kSoftWarps + 2) {
      // ---------------------------------------------------------- by hand
      const int lt = tid - (kSoftWarps + 2) * 32;  // 0 .. 63
      // an odd element at key `key` of a tile, and, once the warp is through
      // the tile (some is its lane's answer), the tile with its odd keys
      uint32_t* odd_keys = sh.odd_keys[(warp - (kSoftWarps + 1)) & 1];
      auto remember = [&](int key) { atomicOr(&odd_keys[key >> 5], 1u << (key & 31)); };
      auto file = [&](int v, bool some) {
        if (!__any_sync(0xffffffffu, some)) return;
        file_poison(&sh, warp - (kSoftWarps + 1), v);
      };
      auto announce = [&](uint64_t* bar) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      int page_n = nt > 1 ? fetch_page(j0 + 1) : -1;
      uint32_t rows = to_row(j0, fetch_page(j0));

      // Goes through tile j's V, whose 16-key blocks are on cache rows r: zeroes
      // for keys that no row sees or whose page is none; of keys that some rows
      // see and others do not, the elements that are not finite become zeros
      // and the key is remembered (check_key says whether it had some).  64 / S
      // threads take a key; the ranges of both kinds are few and short, and
      // found once (these two warps get few of their schedulers' slots).
      auto mask_tile = [&](int j, uint32_t r, auto stride, auto zero_key, auto check_key) {
        constexpr int S = decltype(stride)::value;
        const int v = 128 * j, k0 = lt / (64 / S);
        bool some = false;
        auto zero = [&](int from, int to) {
#pragma unroll 1
          for (int key = from + ((k0 - from) & (S - 1)); key < to; key += S) zero_key(key);
        };
        auto check = [&](int from, int to) {
#pragma unroll 1
          for (int key = from + ((k0 - from) & (S - 1)); key < to; key += S)
            if (check_key(key)) {
              remember(key);
              some = true;
            }
        };
        const unsigned there = __ballot_sync(0xffffffffu, r != kNoPage);
        if (there != 0xffffffffu) {  // blocks of 16 keys on no page: key by key
#pragma unroll 1
          for (int i = 0; i < 128; ++i) {
            const int key = T.key(v + i);
            if (!((there >> (i >> 4)) & 1u) || !seen(key))
              zero(i, i + 1);
            else if (!all_seen(key, key))
              check(i, i + 1);
          }
        } else {
          const int n = min(max(T.ns - v, 0), 128);  // (keys of the sinks)
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            // within the tile: the sinks end at s1; the windows begin at a0, all
            // of them have begun at a1, the first row ends at b0, the last at b1
            const int lo = part == 0 ? 0 : n, hi = part == 0 ? n : 128, kb = part == 0 ? v : v + T.shift;
            if (lo >= hi) continue;
            auto in = [&](int key) { return min(max(key - kb, lo), hi); };
            const int s1 = in(P.sinks), a0 = max(in(wlo), s1), a1 = max(in(wlo_all), s1);
            const int b0 = in(pmin + 1), b1 = in(pmax + 1);
            zero(s1, min(a0, b1));
            zero(b1, hi);
            check(b0, min(s1, b1));                    // sinks that lie ahead of some row
            check(a0, min(a1, b1));                    // keys that some window has left
            check(max(max(a0, b0), min(a1, b1)), b1);  // keys ahead of some row
          }
        }
        file(v, some);
      };
      if constexpr (KVT == 0) {
        // V of masked tiles as it has landed
        const int c = lt & 15;
        uint32_t turns = 0u;  // of each buffer, handed over by warp 17
        for (int i = 0; i < nt; ++i) {
          const int j = j0 + i, vbuf = i % RG::NV;
          const uint32_t here = rows;
          if (i + 1 < nt) rows = to_row(j + 1, page_n);
          page_n = i + 2 < nt ? fetch_page(j + 2) : -1;
          if (!by_hand(j, here)) continue;
          if (!all_ok(mbar_wait(&sh.vgo[vbuf], (turns >> vbuf) & 1u, P.err))) break;
          turns ^= 1u << vbuf;
          uint8_t* tile = sV + vbuf * kTile;
          mask_tile(
              j, here, Int<4>(),
              [&](int key) { *reinterpret_cast<uint4*>(tile + tile_byte(key, c)) = make_uint4(0u, 0u, 0u, 0u); },
              [&](int key) {
                uint4* at = reinterpret_cast<uint4*>(tile + tile_byte(key, c));
                const uint4 v = *at;
                uint32_t w[4] = {v.x, v.y, v.z, v.w}, odd = 0u;
                // an exponent of all ones carries into the sign's place
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= ((w[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                if (odd == 0u) return false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
                  if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
                return true;
              });
          announce(&sh.vfull[vbuf]);
        }
      } else {
        const int c = lt & 7, k0 = lt >> 3;
        for (int i = 0; i < nt; ++i) {
          const int j = j0 + i, vbuf = i % RG::NV, rbuf = i % RG::NR;
          const uint32_t here = rows;
          if (i + 1 < nt) rows = to_row(j + 1, page_n);
          page_n = i + 2 < nt ? fetch_page(j + 2) : -1;
          if (!all_ok(mbar_wait(&sh.rfull[rbuf], (i / RG::NR) & 1, P.err) &&
                      mbar_wait(&sh.vempty[vbuf], ((i / RG::NV) & 1) ^ 1, P.err)))
            break;
          const uint8_t* src = sR + rbuf * kAtom + tile_byte(k0, c);
          uint8_t* d0 = sV + vbuf * kTile + tile_byte(k0, 2 * c);
          uint8_t* d1 = sV + vbuf * kTile + tile_byte(k0, 2 * c + 1);
          auto convert = [&](int q, uint4 v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x2x2(w[e], f[2 * e], f[2 * e + 1]);
            *reinterpret_cast<uint4*>(d0 + 1024 * q) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(d1 + 1024 * q) = make_uint4(f[4], f[5], f[6], f[7]);
          };
#pragma unroll
          for (int q = 0; q < 16; q += 8) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const uint4*>(src + 1024 * (q + u));
#pragma unroll
            for (int u = 0; u < 8; ++u) convert(q + u, v[u]);
          }
          if (by_hand(j, here))  // (each thread the keys that it converted)
            mask_tile(
                j, here, Int<8>(),
                [&](int key) {
                  *reinterpret_cast<uint4*>(d0 + 1024 * (key >> 3)) = make_uint4(0u, 0u, 0u, 0u);
                  *reinterpret_cast<uint4*>(d1 + 1024 * (key >> 3)) = make_uint4(0u, 0u, 0u, 0u);
                },
                [&](int key) {
                  const uint4 v = *reinterpret_cast<const uint4*>(src + 1024 * (key >> 3));
                  uint32_t w[4] = {v.x, v.y, v.z, v.w}, odd = 0u;
                  // a NaN's seven ones carry into the sign's place
#pragma unroll
                  for (int e = 0; e < 4; ++e) odd |= ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                  if (odd == 0u) return false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t nan = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    w[e] &= ~(nan | (nan - (nan >> 7)));
                  }
                  convert(key >> 3, make_uint4(w[0], w[1], w[2], w[3]));
                  return true;
                });
          announce(&sh.vfull[vbuf]);
          if (lane == 0) mbar_arrive(&sh.rempty[rbuf]);
        }
      }
      mbar_arrive(&sh.loads_done);
    } else if (warp == kSoftWarps) {
      // ---------------------------------------------------------- MMA
      constexpr uint32_t fmt = KVT == 0 ? 1u : 0u;  // bf16 or f16
      const uint32_t id_s = umma_idesc(fmt, 128, 128);  // (format 0 is e4m3 among 8-bit operands, 1 e5m2)
      const uint32_t id_o = id_s | (1u << 16);          // B is N-major
      const uint32_t q0 = desc_lo(smem_addr(sQ), 16), k0 = desc_lo(smem_addr(sK), 16);
      // N-major: the second 64 dims one atom on
      const uint32_t v0 = desc_lo(smem_addr(sV), kAtom);
      auto scores = [&](int x, int i) {
        const uint32_t a = q0 + ((x * kTile) >> 4), b = k0 + (((i % RG::NK) * RG::kKey) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int off = (kk & 3) * 32, atom = (kk >> 2) * kAtom;
          if constexpr (KVT == 0)
            mma_ss(tmem + 128 * x, a + ((atom + off) >> 4), b + ((atom + off) >> 4), id_s, kk != 0 ? 1u : 0u);
          else  // the hi terms, then the lo terms (A in e5m2), over the same codes
            mma_ss_f8(tmem + 128 * x, a + ((atom + off) >> 4), b + (off >> 4), kk < 4 ? id_s : id_s | (1u << 7), kk != 0 ? 1u : 0u);
        }
      };
      // O += P V of tile number i
      auto values = [&](int x, int i) {
        const uint32_t b = v0 + (((i % RG::NV) * kTile) >> 4);
        const int own = duo ? i >> 1 : i;  // (of tile x)
        if (!all_ok(mbar_wait(&sh.p_ready[x], own & 1, P.err))) return false;
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * kk, b + ((kk * 2048) >> 4), id_o,
                 own == 0 && kk == 0 ? 0u : 1u);
        return true;
      };
      auto wait_k = [&](int i) {
        const bool ok = all_ok(mbar_wait(&sh.kfull[i % RG::NK], (i / RG::NK) & 1, P.err));
        tc_fence_after_sync();
        return ok;
      };
      auto start = [&](int x, int i) {
        scores(x, i);
        mma_commit(&sh.s_full[x]);
      };
      auto wait_v = [&](int i) { return all_ok(mbar_wait(&sh.vfull[i % RG::NV], (i / RG::NV) & 1, P.err)); };
      auto wait_q = [&](int x) {
        const bool ok = all_ok(mbar_wait(&sh.q_ready[x], 0, P.err));
        tc_fence_after_sync();
        return ok;
      };
      bool ok = wait_q(0) && wait_k(0);
      if (ok) {
        start(0, 0);
        if (two) {
          ok = wait_q(1);
          start(1, 0);
        }
        mma_commit(&sh.kempty[0]);
        if (duo) {
          ok = wait_q(1) && wait_k(1);
          start(1, 1);
          mma_commit(&sh.kempty[1]);
        }
      }
      // (x a constant where it can be: with one loop for all, 8192 rows took 412
      // instead of 405 us)
      for (int i = 0; i < nt && ok && !duo; ++i) {
        const bool more = i + 1 < nt;
        ok = wait_v(i) && values(0, i);
        if (!ok) break;
        if (more) {
          ok = wait_k(i + 1);
          if (!ok) break;
          start(0, i + 1);
        } else {
          mma_commit(&sh.o_full[0]);
        }
        if (two) {
          ok = values(1, i);
          if (!ok) break;
        }
        mma_commit(&sh.vempty[i % RG::NV]);
        if (more) {
          if (two) start(1, i + 1);
          mma_commit(&sh.kempty[(i + 1) % RG::NK]);
        } else {
          mma_commit(&sh.o_full[1]);
        }
      }
      for (int i = 0; i < nt && ok && duo; ++i) {
        ok = wait_v(i) && values(i & 1, i);
        if (!ok) break;
        mma_commit(&sh.vempty[i % RG::NV]);
        if (i + 2 < nt) {
          ok = wait_k(i + 2);
          if (!ok) break;
          start(i & 1, i + 2);
          mma_commit(&sh.kempty[(i + 2) % RG::NK]);
        } else {
          mma_commit(&sh.o_full[i & 1]);
        }
      }
    } else if (warp == kSoftWarps + 1) {
      // ---------------------------------------------------------- TMA
      int page_n = nt > 1 ? fetch_page(j0 + 1) : -1;
      uint32_t rows = to_row(j0, fetch_page(j0)), word = scale_word(rows);
      // The boxes of a tile that hold keys of the cache: a bit for each at its
      // first 16-key block, whose lane gets its cache row.
      auto find_boxes = [&](uint32_t r, int& y) {
        const unsigned there = __ballot_sync(0xffffffffu, r < kNoPage) & 0xFFu;
        const int per = P.box >> 4;  // blocks of a box
        const unsigned in = (there >> (lane & 7)) & ((1u << per) - 1u);
        // (its first block may be one that nothing sees: count back)
        const int first = in != 0u ? __ffs(in) - 1 : 0;
        y = static_cast<int>(__shfl_sync(0xffffffffu, r, (lane & 7) + first)) - 16 * first;
        return __ballot_sync(0xffffffffu, lane < 8 && (lane & (per - 1)) == 0 && in != 0u);
      };
      // them at columns x .. (atoms of 128 bytes) on `full` with `arrivals`
      // arrivals
      auto tile = [&](uint64_t* full, uint32_t arrivals, uint8_t* dst, unsigned boxes, int y, int x, int atoms) {
        if (lane == 0) {
          mbar_arrive_expect_tx(full, __popc(boxes) * atoms * P.box * 128);
          if (arrivals > 1) mbar_arrive(full);
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (!((boxes >> b) & 1u)) continue;
          const int yb = __shfl_sync(0xffffffffu, y, b);
          tma_box(dst + b * 2048, &tmap, x, yb, full);
          if (atoms == 2) tma_box(dst + kAtom + b * 2048, &tmap, x + 64, yb, full);
        }
      };
      for (int i = 0; i < nt; ++i) {
        const int j = j0 + i, kbuf = i % RG::NK, vbuf = i % RG::NV;
        const uint32_t here = rows, word_here = word;
        if (i + 1 < nt) {
          rows = to_row(j + 1, page_n);
          word = scale_word(rows);
        }
        page_n = i + 2 < nt ? fetch_page(j + 2) : -1;
        int y;
        const unsigned boxes = find_boxes(here, y);
        if (!all_ok(mbar_wait(&sh.kempty[kbuf], ((i / RG::NK) & 1) ^ 1, P.err))) break;
        publish(i, here, word_here);
        tile(&sh.kfull[kbuf], 1, sK + kbuf * RG::kKey, boxes, y, 0, KVT == 0 ? 2 : 1);
        if constexpr (KVT == 0) {
          if (!all_ok(mbar_wait(&sh.vempty[vbuf], ((i / RG::NV) & 1) ^ 1, P.err))) break;
          if (by_hand(j, here)) {
            tile(&sh.vgo[vbuf], 1, sV + vbuf * kTile, boxes, y, 128, 2);
          } else {
            tile(&sh.vfull[vbuf], 2, sV + vbuf * kTile, boxes, y, 128, 2);
          }
        } else {
          const int rbuf = i % RG::NR;
          if (!all_ok(mbar_wait(&sh.rempty[rbuf], ((i / RG::NR) & 1) ^ 1, P.err))) break;
          tile(&sh.rfull[rbuf], 1, sR + rbuf * kAtom, boxes, y, 128, 1);
        }
      }
    }
  } else if (warp < 8 || two || duo) {
    // ------------------------------------------------------------ softmax
    regs_up<kSoftmaxRegs>();
    // M row im of tile x; this thread's 64 keys (at the end: dims) of it
    const int x = warp >> 3, hf = (warp >> 2) & 1, im = 32 * (warp & 3) + lane, m = 128 * x + im;
    const int pair = 1 + 4 * x + (warp & 3);  // the barrier of the row's two warps
    const int r0 = two ? row0 + x * R : row0;  // first row
    const bool live = im < R * G && r0 + row_of(im) < row0 + nrows;
    // its position; a row before the start computes what it likes and is
    // zero at the end
    auto position = [&] { return live ? window_position(P, r0 + row_of(im)) : -1; };
    const int pos = position(), p = max(pos, 0);
    // ---- Q of the two warps' 32 M rows, sixteen each, a half-warp per row
    {
      uint8_t* tile = sQ + x * kTile;
      const int lane16 = lane & 15, im0 = 32 * (warp & 3) + 16 * hf + (lane >> 4);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int im = im0 + 2 * u;
        float qs = 0.08838834764831845f * kLog2e;
        if constexpr (KVT == 0) {
          *reinterpret_cast<uint4*>(tile + tile_byte(im, lane16)) = qv[u];
        } else {
          const uint32_t w[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
          // the largest |q| as bf16 bits (0x7F80 and more: not finite)
          uint32_t top = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max_u16x2(top, w[e] & 0x7FFF7FFFu);
          top = max_u16x2(top, top >> 16);
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
          const uint32_t peak = top & 0xFFFFu;
          // (a row below 2^-119 keeps fewer bits: its scores are 0 beside 1)
          const int e = peak != 0u ? max(static_cast<int>(peak >> 7) - 127 - 7, -126) : 0;
          const float f0 = exp2i(-e);
          float f[8];
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = (i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1])) * f0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t h0 = f32x2_to_e4m3x2(f[4 * i], f[4 * i + 1]), h1 = f32x2_to_e4m3x2(f[4 * i + 2], f[4 * i + 3]);
            hi[i] = h0 | (h1 << 16);
            uint32_t b0, b1;
            e4m3x4_to_f16x2x2(hi[i], b0, b1);
            const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&b0));
            const float2 y1 = __half22float2(*reinterpret_cast<const __half2*>(&b1));
            lo[i] = static_cast<uint32_t>(f32x2_to_e5m2x2(f[4 * i] - y0.x, f[4 * i + 1] - y0.y)) |
                    (static_cast<uint32_t>(f32x2_to_e5m2x2(f[4 * i + 2] - y1.x, f[4 * i + 3] - y1.y)) << 16);
          }
          qs = fmaxf(qs * (KVT == 1 ? P.k_scale : 1.0f) * exp2i(e), kLeast);
          if (peak >= 0x7F80u) {  // not finite: NaN codes, which make every score that is seen a NaN
            qs = -1.0f;
            hi[0] = hi[1] = 0x7F7F7F7Fu;
          }
          // the hi terms' atom, then the lo terms'
          uint8_t* dst = tile + im * 128 + (((lane16 >> 1) ^ (im & 7)) << 4) + (lane16 & 1) * 8;
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(dst + kAtom) = make_uint2(lo[0], lo[1]);
        }
        if (lane16 == 0) sh.qs[128 * x + im] = qs;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready[x]);
    // (the gate's half row into L2 while there is time)
    if (live && (x == 0 || two) && P.gate != nullptr && P.splits == 1)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          P.gate + (static_cast<long long>(r0 + row_of(im)) * P.hq + kvh * G + head_of(im)) * 128 + 64 * hf));
    pair_sync(pair);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + 128 * x + lanes, to = tmem + 256 + 128 * x + 64 * hf + lanes;
    const float qs = fabsf(sh.qs[m]);
    // the 32 rows' own bounds decide which key tiles need masks
    const int hi_all = __reduce_min_sync(0xffffffffu, pos >= 0 ? p : INT_MAX);
    const int lo_all = __reduce_max_sync(0xffffffffu, pos >= 0 ? p - P.window + 1 : INT_MIN);
    // (a row that sees nothing never asks for a reference)
    float ref = pos >= 0 && sh.qs[m] > 0.f ? -INFINITY : 0.f, l = 0.f;
    // (a wait that gives up ends the waiting, not the loop: the two warps
    // always meet)
    bool ok = true;
    const int both = duo ? 1 : 0;  // (tile x's own key tiles: all, or every other)
    int own = 0;
#pragma unroll 1
    for (int j = both & x; j < nt; j += 1 + both, ++own) {
      const int slot = j % kSlots;
      // the tile's masks and scales, then its scores.  (A slot's next tile is
      // published only after both softmaxes are done with this one: its K
      // waits for a ring buffer that S of a later tile frees.)
      ok = all_ok(ok && mbar_wait(&sh.info[slot], (j / kSlots) & 1, P.err) && mbar_wait(&sh.s_full[x], own & 1, P.err));
      tc_fence_after_sync();
      const int kb = sh.first[slot][hf];
      const bool plain = kb >= 0 && kb + 63 <= hi_all && (kb >= lo_all || kb + 63 < P.sinks);
      uint32_t sc[4];  // (block scales)
      if constexpr (KVT == 2) {
        const uint4 a = *reinterpret_cast<const uint4*>(&sh.scale[slot][4 * hf]);
        sc[0] = a.x; sc[1] = a.y; sc[2] = a.z; sc[3] = a.w;
      }
      // the largest of 16 scores
      auto max16 = [&](const uint32_t* rr) {
        float bm = max3(__uint_as_float(rr[0]), __uint_as_float(rr[1]), __uint_as_float(rr[2]));
        float b2 = max3(__uint_as_float(rr[3]), __uint_as_float(rr[4]), __uint_as_float(rr[5]));
#pragma unroll
        for (int i = 6; i < 14; i += 4) {
          bm = max3(bm, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
          b2 = max3(b2, __uint_as_float(rr[i + 2]), __uint_as_float(rr[i + 3]));
        }
        bm = max3(bm, __uint_as_float(rr[14]), __uint_as_float(rr[15]));
        return fmaxf(bm, b2);
      };
      // its exponent (log2), without the reference
      auto exponent = [&](float bm, int b) {
        if constexpr (KVT == 2) return fmaf(bm, fmaxf(qs * bf16_lo(sc[b]), kLeast), bf16_hi(sc[b]));
        return bm * qs;
      };
      // The weights are taken against the reference as it stands; only where
      // one of the row's has grown too large (or a row has no reference yet)
      // is it moved and the tile done again.  (S is in place until P is
      // stored, and P is stored only after the two warps have met: the second
      // half's lies over the first half's S.)
      // A reference beyond 2^20 is looked at in every tile.
      bool moved = __any_sync(0xffffffffu, !(fabsf(ref) <= kFar));
      uint32_t pk[32];
      float sum;
#pragma unroll 1
      while (true) {
        uint32_t r[2][32];
        tmem_ld32_issue(ts + 64 * hf, r[0]);
        tmem_ld32_issue(ts + 64 * hf + 32, r[1]);
        tmem_wait_ld32(r[0]);
        tmem_wait_ld32(r[1]);
        if (!plain) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            auto sees_of = [&](int k0) {
              return low_bits(p + 1 - k0) & (~low_bits(p - P.window + 1 - k0) | low_bits(P.sinks - k0));
            };
            const int v0 = 128 * (j0 + j) + 64 * hf + 32 * c;
            const uint32_t first = low_bits(sh.ns - v0);
            uint32_t vis = (sees_of(v0) & first) | (sees_of(v0 + sh.shift) & ~first);
            if (sh.check[slot] != 0) vis &= sh.valid[slot][2 * hf + c];
#pragma unroll
            for (int i = 0; i < 32; ++i) r[c][i] = (vis & (1u << i)) != 0u ? r[c][i] : 0xFF800000u;
          }
        }
        bool far = false;
        if (moved) {
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < 4; ++b) mx = fmaxf(mx, exponent(max16(&r[b >> 1][16 * (b & 1)]), b));
          sh.pair[own & 1][hf][m] = mx;
          pair_sync(pair);
          mx = fmaxf(mx, sh.pair[own & 1][hf ^ 1][m]);
          // moves the reference up, the sums with it
          const float mn = fmaxf(ref, mx + kRoom<KVT>);
          const float al = ex2_ftz(ref - (mn == -INFINITY ? 0.f : mn));
          l *= al;
          if (own > 0) {  // (S of this tile is complete, so O of the last one is)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[16];
              tmem_ld16(to + 16 * c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tmem_st16(to + 16 * c, o);
            }
          }
          ref = mn;
          // Further out an unrounded product less the rounded reference leaves a
          // weight's range: exponents are rounded first, as the reference was.
          far = __any_sync(0xffffffffu, fabsf(ref) > kFar && ref != -INFINITY);
          if (far) {
#pragma unroll
            for (int i = 0; i < 64; ++i) r[i >> 5][i & 31] = __float_as_uint(exponent(__uint_as_float(r[i >> 5][i & 31]), i >> 4));
          }
        }
        const float neg_ref = ref == -INFINITY ? 0.f : -ref;
        unsigned long long sum2 = 0ull;  // (two sums, of even and odd keys)
        uint32_t any_bits = 0u;
        __half2 top = __float2half2_rn(0.f);
        sum = 0.f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t* rr = &r[b >> 1][16 * (b & 1)];
          float f = far ? 1.0f : qs, base = neg_ref, inv_vs = 1.0f;
          if constexpr (KVT == 2) {
            if (!far) {
              f = fmaxf(f * bf16_lo(sc[b]), kLeast);
              base += bf16_hi(sc[b]);
            }
            inv_vs = ex2_ftz(-bf16_hi(sc[b]));
          }
          const unsigned long long f2 = f32x2_pack(f, f), base2 = f32x2_pack(base, base);
          unsigned long long bs2 = KVT == 2 ? 0ull : sum2;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float p0, p1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1])), f2, base2), p0, p1);
            p0 = ex2_ftz(p0);
            p1 = ex2_ftz(p1);
            bs2 = f32x2_add(bs2, f32x2_pack(p0, p1));
            pk[8 * b + (i >> 1)] = KVT == 0 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint32_t a = pk[8 * b + i], c = pk[8 * b + i + 1];
            if constexpr (KVT == 0)
              any_bits |= a | c;
            else
              top = __hmax2(top, __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&c)));
          }
          if constexpr (KVT == 2)
            sum = fmaf(f32x2_hsum(bs2), inv_vs, sum);
          else
            sum2 = bs2;
        }
        if constexpr (KVT != 2) sum = f32x2_hsum(sum2);
        const bool large = KVT == 0 ? (any_bits & kTwo) != 0u
                                    : __hgt(__hmax(__low2half(top), __high2half(top)), __float2half(1024.f));
        if (moved || !pair_any(pair, large)) break;
        moved = true;
      }
      l += sum;
      tmem_st32(ts + 32 * hf, pk);
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&sh.p_ready[x]);
    }
    // ---- output
    sh.pair[own & 1][hf][m] = l;
    pair_sync(pair);
    l += sh.pair[own & 1][hf ^ 1][m];
    ok = all_ok(ok && mbar_wait(&sh.o_full[x], 0, P.err) && mbar_wait(&sh.loads_done, 0, P.err));
    float other = 0.f;  // what tile B's O is multiplied by
    float self = 1.f;
    if (duo) {
      if (x == 1) {
        sh.join[0][im] = l;  // (twice the same)
        sh.join[1][im] = ref;
        asm volatile("bar.arrive 9, 512;" ::: "memory");
      } else {
        ok = all_ok(ok && mbar_wait(&sh.o_full[1], 0, P.err));
        asm volatile("bar.sync 9, 512;" ::: "memory");
        const float lb = sh.join[0][im], rb = sh.join[1][im], top = fmaxf(ref, rb);
        self = ref == -INFINITY ? 0.f : ex2_ftz(ref - top);
        other = rb == -INFINITY ? 0.f : ex2_ftz(rb - top);
        l = l * self + lb * other;
        ref = top;
      }
    }
    tc_fence_after_sync();
    if (x == 0 || two) {  // (tile B's part has joined A's)
      const long long head = static_cast<long long>(r0 + row_of(im)) * P.hq + kvh * G + head_of(im);
      const long long ph = static_cast<long long>(split) * P.rows * P.hq + head;
      // (a NaN sum is not an empty row)
      const bool sees = position() >= 0, empty = !sees || l == 0.f;
      const float inv = (KVT == 1 ? P.v_scale : 1.0f) / l;
      self *= inv;
      other *= inv;
      // the warp's 32 rows and 64 dims cross to coalesced stores through their
      // own place in the Q tile, which no MMA reads any more
      uint8_t* tile = sQ + x * kTile;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t o[32];
        tmem_ld32_issue(to + 32 * c, o);
        tmem_wait_ld32(o);
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = empty ? 0.f : __uint_as_float(o[i]) * self;
        if (duo) {
          tmem_ld32_issue(to + 128 + 32 * c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = empty ? 0.f : fmaf(__uint_as_float(o[i]), other, f[i]);
        }
        if (sees && ok) {  // what the row sees of the remembered elements
#pragma unroll 1
          for (int b = 0; b < kPoison * 128 && sh.poison_tile[b >> 7] >= 0; ++b) {
            if (!((sh.poison[b >> 7][(b >> 5) & 3] >> (b & 31)) & 1u)) continue;
            const int key = T.key(sh.poison_tile[b >> 7] + (b & 127));
            if (key > p || !(key > p - P.window || key < P.sinks)) continue;
            const int blk = page_of(P, key);
            const int pid = P.block_table[static_cast<long long>(req) * P.bt_stride + blk];
            const long long at = ((static_cast<long long>(pid) * P.hkv + kvh) * P.page + key - blk * P.page) * 256 + 128 + 64 * hf + 32 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float v = KVT == 0 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(P.kv)[at + i]) << 16)
                              : (static_cast<const uint8_t*>(P.kv)[at + i] & 0x7F) == 0x7F ? __int_as_float(0x7fffffff) : 0.f;
              if (!(fabsf(v) <= 3.39e38f)) f[i] += v;
            }
          }
        }
        if (P.splits > 1) {
          if (!live || !ok) continue;
          float4* po = reinterpret_cast<float4*>(P.part_o + ph * 128 + 64 * hf + 32 * c);
#pragma unroll
          for (int q = 0; q < 8; ++q) po[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(tile + tile_byte(im, 8 * hf + 4 * c + q)) =
                make_uint4(pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                           pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7]));
        }
      }
      if (P.splits > 1) {
        if (live && ok && hf == 0) P.part_lse[ph] = empty ? -INFINITY : ref + log2f(l);
      } else if (ok) {
        __syncwarp();
        // four rows at a time, eight lanes each
        const int c8 = 8 * hf + (lane & 7), im0 = 32 * (warp & 3) + (lane >> 3);
        uint4 gate[8];
        auto at = [&](int i2) {
          return (static_cast<long long>(r0 + row_of(i2)) * P.hq + kvh * G + head_of(i2)) * 128 + 8 * c8;
        };
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i2 = im0 + 4 * u;
          gate[u] = i2 < R * G && r0 + row_of(i2) < row0 + nrows ? load_gate(P, at(i2)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i2 = im0 + 4 * u;
          if (i2 < R * G && r0 + row_of(i2) < row0 + nrows)
            store_gated(P, at(i2), *reinterpret_cast<const uint4*>(tile + tile_byte(i2, c8)), gate[u]);
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  free_tmem();
}

template <int KVT>
cudaError_t launch_kind(const RowGqaParams& p, const CUtensorMap& tmap, const dim3& grid, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(window_tile_kernel<KVT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<KVT>);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_kernel(window_tile_kernel<KVT>, grid, dim3(kThreads), kSmem<KVT>, stream, false, tmap, p);
}

}  // namespace

int window_tile_rows(int group) { return 2 * (128 / group); }

// (at the least: a request's last group may be a part of one)
long long window_tile_groups(int rows, int reqs, int group) {
  const int per = window_tile_rows(group);
  const long long groups = (static_cast<long long>(rows) + per - 1) / per;
  return groups < reqs ? (reqs < rows ? reqs : rows) : groups;
}

// As many splits as keep to one wave with four tiles each or more (one request
// of 32 rows and 4100 tokens, 4 KV heads: 25 us, with two tiles or more 30 us).
int window_tile_splits(int rows, int reqs, int hkv, int group, long long max_tokens, int sms) {
  const long long ctas = window_tile_groups(rows, reqs, group) * hkv;
  if (ctas <= 0) return 1;
  const long long tiles = (max_tokens + 127) / 128 + 1;
  long long s = sms / ctas;
  if (s > tiles / 4) s = tiles / 4;
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
