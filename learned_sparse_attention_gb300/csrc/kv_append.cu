// qsa_kv_append: a step's keys and values into the paged KV cache, with the
// norm and the position rotation applied on the way, and the main attention's
// q and gate beside them when asked for.
//
// Mathematics.  Per row and KV head: k = RoPE(GemmaRMSNorm(k)), v as it is
// (qsa_rope.cuh, fp32, one rounding to the cache's type).  bf16 caches store
// them as they are, e4m3 caches with a static scale store e4m3(x / scale).
// With block scales a run -- consecutive rows whose slots ascend inside one
// block of B tokens -- shares one power of two for K and one for V of each KV
// head: with a = max |x| over the run (finite values),
//   e_new = the smallest e with a <= 448 * 2^e, within [-40, 40];
//   e     = e_new if the run begins the block, else max(e_old, e_new);
//   code  = e4m3(x * 2^-e), and the codes before the run become
//           e4m3(code * 2^(e_old - e)) when e > e_old.
// A power of two makes the re-encoding a shift of the exponent, exact but for
// codes that fall among e4m3's subnormals, so a block that grows token by
// token loses nothing to its history that one write would have kept.
//
// Bound: memory.  A row is read once and written once; the arithmetic is an
// eighth of an instruction a byte.  Layout: half-warps hold a 128-dim head
// (16 bytes a lane).  With block scales a CTA holds a run's keys and values
// of one KV head in registers between the maximum and the rounding (2, 4 or 8
// tokens a half-warp), so they are read once.
// Measured, 32 query and 4 KV heads, blocks of 32, ten calls on ten sets of
// inputs: 16 384 rows with queries 114 us (5.1 TB/s of reads and writes), 64 rows
// 4.0 us, 128 rows 6.4 us.
#include "kv_scale.cuh"
#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"
#include "qsa_rope.cuh"

namespace qsa {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 128;
constexpr int kHalves = kThreads / 16;  // half-warps of a CTA

__device__ __forceinline__ RopeParams rope_of(const AppendParams& P) {
  return RopeParams{P.cos_sin, P.max_pos, P.mrope, P.sec_h, P.sec_w, P.err};
}

__device__ __forceinline__ void load_pos(const AppendParams& P, int row, int64_t (&pos)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) pos[k] = P.positions[static_cast<long long>(row) * 3 + (P.mrope ? k : 0)];
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float s) {
  uint2 v;
  v.x = static_cast<uint32_t>(f32x2_to_e4m3x2(x[0] * s, x[1] * s)) |
        (static_cast<uint32_t>(f32x2_to_e4m3x2(x[2] * s, x[3] * s)) << 16);
  v.y = static_cast<uint32_t>(f32x2_to_e4m3x2(x[4] * s, x[5] * s)) |
        (static_cast<uint32_t>(f32x2_to_e4m3x2(x[6] * s, x[7] * s)) << 16);
  return v;
}

__device__ __forceinline__ void load_gain(const uint16_t* w, int lane16, float (&g)[8]) {
  load8_bf16(w + 8 * lane16, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] += 1.0f;
}

// q = RoPE(GemmaRMSNorm(q)) and the gate of rows row0, row0 + step, ...: each
// half-warp takes two heads at a time, and the next two's loads (and the
// next row's position) are on the way while these are worked on.
__device__ __forceinline__ void query_rows(const AppendParams& P, int row0, int step) {
  constexpr int U = 2;
  const int hw = threadIdx.x >> 4, lane16 = threadIdx.x & 15;
  float g[8];
  load_gain(P.q_norm_w, lane16, g);
  auto load = [&](int row, int base, uint4 (&q)[U], uint4 (&gate)[U]) {
    const uint16_t* x = P.qkv + static_cast<long long>(row) * (2 * P.hq + 2 * P.hkv) * kD + 8 * lane16;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + hw + kHalves * u;
      q[u] = gate[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < P.rows && h < P.hq) {
        q[u] = *reinterpret_cast<const uint4*>(x + (2 * h) * kD);
        gate[u] = *reinterpret_cast<const uint4*>(x + (2 * h + 1) * kD);
      }
    }
  };
  uint4 q[U], gate[U];
  load(row0, 0, q, gate);
  int64_t pos[3];
  load_pos(P, row0, pos);
  for (int row = row0; row < P.rows; row += step) {
    float c[8], s[8];
    rope_coeffs(rope_of(P), lane16, pos, c, s);
    if (row + step < P.rows) load_pos(P, row + step, pos);
    for (int base = 0; base < P.hq; base += kHalves * U) {  // (the norm's shuffles span the warp)
      uint4 nq[U], ngate[U];
      const bool last = base + kHalves * U >= P.hq;
      load(last ? row + step : row, last ? 0 : base + kHalves * U, nq, ngate);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = base + hw + kHalves * u;
        if (base + kHalves * u < P.hq) {  // (the same for the whole CTA)
          float f[8];
          unpack8(q[u], f);
          norm_rope(f, g, P.eps, lane16, c, s);
          if (h < P.hq) {
            const long long o = (static_cast<long long>(row) * P.hq + h) * kD + 8 * lane16;
            *reinterpret_cast<uint4*>(P.q_out + o) = pack8_bf16(f);
            *reinterpret_cast<uint4*>(P.gate_out + o) = gate[u];
          }
        }
        q[u] = nq[u];
        gate[u] = ngate[u];
      }
    }
  }
}

// K and V rows of a bf16 or statically scaled cache: one row, all KV heads.
__device__ __forceinline__ void plain_kv_row(const AppendParams& P, int row) {
  const int hw = threadIdx.x >> 4, lane16 = threadIdx.x & 15;
  const long long slot = P.slots[row];
  if (slot < 0) return;
  const long long blk = slot / P.page, off = slot - blk * P.page;
  if (blk >= P.num_blocks) {
    if (threadIdx.x == 0) flag_error(P.err);
    return;
  }
  const uint16_t* x = P.qkv + (static_cast<long long>(row) * (2 * P.hq + 2 * P.hkv) + 2 * P.hq) * kD;
  int64_t pos[3];
  load_pos(P, row, pos);
  float c[8], s[8], g[8];
  rope_coeffs(rope_of(P), lane16, pos, c, s);
  load_gain(P.k_norm_w, lane16, g);
  for (int base = 0; base < P.hkv; base += kHalves) {
    const int h = base + hw;
    const bool act = h < P.hkv;
    float xk[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4 vv = make_uint4(0u, 0u, 0u, 0u);
    if (act) {
      load8_bf16(x + h * kD + 8 * lane16, xk);
      vv = *reinterpret_cast<const uint4*>(x + (P.hkv + h) * kD + 8 * lane16);
    }
    norm_rope(xk, g, P.eps, lane16, c, s);
    if (!act) continue;
    const long long r = (blk * P.hkv + h) * P.page + off;
    if (P.kv_dtype == QSA_DTYPE_BF16) {
      uint16_t* dst = static_cast<uint16_t*>(P.kv) + r * 256;
      *reinterpret_cast<uint4*>(dst + 8 * lane16) = pack8_bf16(xk);
      *reinterpret_cast<uint4*>(dst + 128 + 8 * lane16) = vv;
    } else {
      uint8_t* dst = static_cast<uint8_t*>(P.kv) + r * 256;
      float xv[8];
      unpack8(vv, xv);
      *reinterpret_cast<uint2*>(dst + 8 * lane16) = pack8_e4m3(xk, 1.0f / P.k_scale);
      *reinterpret_cast<uint2*>(dst + 128 + 8 * lane16) = pack8_e4m3(xv, 1.0f / P.v_scale);
    }
  }
}

// Whether row i + 1 goes on with row i's run (blocks of kHalves * NT tokens).
template <int NT>
__device__ __forceinline__ bool goes_on(const AppendParams& P, int i) {
  if (i < 0 || i + 1 >= P.rows) return false;
  const long long a = P.slots[i], b = P.slots[i + 1];
  return a >= 0 && b > a && ((a ^ b) & ~(static_cast<long long>(kHalves) * NT - 1)) == 0;
}

// The run that begins at row i, one KV head, into a cache with block scales.
// NT: tokens of a block per half-warp.
template <int NT>
__device__ __forceinline__ void scaled_run(const AppendParams& P, int i, int h, const float (&g)[8]) {
  __shared__ float s_peak[kHalves][2];
  const int hw = threadIdx.x >> 4, lane16 = threadIdx.x & 15, lane = threadIdx.x & 31;
  constexpr int B = kHalves * NT;
  const long long slot = P.slots[i];
  const long long blk = slot / P.page;
  if (blk >= P.num_blocks) {
    if (h == 0 && threadIdx.x == 0) flag_error(P.err);
    return;
  }
  const long long past = lane < i ? P.slots[i - 1 - lane] : -1;
  // the run's length: every warp looks at all B rows
  int m = 0;
#pragma unroll
  for (int w = 0; w < (B + 31) / 32; ++w) {
    const unsigned on = __ballot_sync(0xffffffffu, goes_on<NT>(P, i + 32 * w + lane));
    if (m == 32 * w) m += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
  }
  m = min(m + 1, B);
  const int off = static_cast<int>(slot - blk * P.page), f = off % B;
  const long long row0 = (blk * P.hkv + h) * P.page + off;
  uint8_t* sc = static_cast<uint8_t*>(P.scales) + 2 * ((row0 - f) / B);
  uint8_t* kv = static_cast<uint8_t*>(P.kv);
  const int ek_old = scale_exp(sc[0]), ev_old = scale_exp(sc[1]);

  // the run's keys, values and positions, all asked for before any is used
  uint4 kr[NT], v[NT];
  int64_t pos[NT][3];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    if (kHalves * u >= m) continue;  // (the same for the whole CTA)
    const int row = i + min(hw + kHalves * u, m - 1);
    const uint16_t* x = P.qkv + (static_cast<long long>(row) * (2 * P.hq + 2 * P.hkv) + 2 * P.hq + h) * kD + 8 * lane16;
    kr[u] = *reinterpret_cast<const uint4*>(x);
    v[u] = *reinterpret_cast<const uint4*>(x + P.hkv * kD);
    load_pos(P, row, pos[u]);
  }
  // a run in the block of the last row before it (it repeats or steps back, or
  // padding parts it from that row) would race with that row's run
  const unsigned rows = __ballot_sync(0xffffffffu, past >= 0 && past < static_cast<long long>(P.num_blocks) * P.page);
  const long long last = __shfl_sync(0xffffffffu, past, rows != 0u ? __ffs(rows) - 1 : 0);
  if (rows != 0u && ((last ^ slot) & ~(B - 1ll)) == 0) {
    if (h == 0 && threadIdx.x == 0) flag_error(P.err);
    return;
  }
  float k[NT][8];
  float pk = 0.f, pv = 0.f;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    if (kHalves * u >= m) continue;
    float c[8], s[8], xv[8];
    rope_coeffs(rope_of(P), lane16, pos[u], c, s);
    unpack8(kr[u], k[u]);
    norm_rope(k[u], g, P.eps, lane16, c, s);
    unpack8(v[u], xv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pk = fmaxf(pk, finite_abs(k[u][e]));
      pv = fmaxf(pv, finite_abs(xv[e]));
    }
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    pk = fmaxf(pk, __shfl_xor_sync(0xffffffffu, pk, o));
    pv = fmaxf(pv, __shfl_xor_sync(0xffffffffu, pv, o));
  }
  __syncthreads();  // the previous run's peaks are read
  if (lane16 == 0) {
    s_peak[hw][0] = pk;
    s_peak[hw][1] = pv;
  }
  __syncthreads();  // (also: every thread has read the old scales)
#pragma unroll
  for (int w = 0; w < kHalves; ++w) {
    pk = fmaxf(pk, s_peak[w][0]);
    pv = fmaxf(pv, s_peak[w][1]);
  }
  int ek = scale_exp_for(pk), ev = scale_exp_for(pv);
  if (f > 0) {
    ek = max(ek, ek_old);
    ev = max(ev, ev_old);
    if (ek > ek_old || ev > ev_old) {  // the block's earlier tokens, 16 codes a thread
      const float fk = exp2i(ek_old - ek), fv = exp2i(ev_old - ev);
      for (int c = threadIdx.x; c < f * 16; c += kThreads) {
        uint4* p = reinterpret_cast<uint4*>(kv + (row0 - f) * 256) + c;
        *p = rescale16((c & 15) < 8 ? fk : fv, *p);
      }
    }
  }
  if (threadIdx.x == 0) {
    sc[0] = static_cast<uint8_t>(ek + 127);
    sc[1] = static_cast<uint8_t>(ev + 127);
  }
  const float sk = exp2i(-ek), sv = exp2i(-ev);
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int j = hw + kHalves * u;
    if (j >= m) continue;
    // (ascending slots inside the block, not necessarily adjacent)
    const long long r = row0 + (P.slots[i + j] - slot);
    float xv[8];
    unpack8(v[u], xv);
    *reinterpret_cast<uint2*>(kv + r * 256 + 8 * lane16) = pack8_e4m3(k[u], sk);
    *reinterpret_cast<uint2*>(kv + r * 256 + 128 + 8 * lane16) = pack8_e4m3(xv, sv);
  }
}

// Queries alone, row by row.
__global__ void __launch_bounds__(kThreads, 5) query_kernel(const AppendParams P) {
  griddep_launch_dependents();
  query_rows(P, blockIdx.x, P.q_ctas);
}

// CTAs [0, kv_ctas) write K and V: with block scales CTA (c, h, part) every
// parts-th run of KV head h of those that begin in rows [c * chunk, (c + 1) *
// chunk), otherwise CTA c those rows.  The others prepare queries, a row each.  Where the queries have
// a launch of their own (`beside`), this one runs beside it and needs nothing
// of it; its last CTA waits for that one's end, so that this kernel's end is
// both's.
// NT: B / kHalves with block scales, 0 without.
template <int NT>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams P) {
  const int lane16 = threadIdx.x & 15;
  int cta = blockIdx.x;
  griddep_launch_dependents();
  if (cta < P.kv_ctas) {
    const int h = NT > 0 ? cta % P.hkv : 0;
    const int part = NT > 0 ? cta / P.hkv % P.parts : 0;
    const int i0 = (NT > 0 ? cta / P.hkv / P.parts : cta) * P.chunk;
    const int i1 = min(i0 + P.chunk, P.rows);
    if constexpr (NT > 0) {
      float g[8];
      load_gain(P.k_norm_w, lane16, g);
      int turn = part;                      // runs until this CTA's next one
      for (int b = i0; b < i1; b += 32) {  // 32 rows at a time: where runs begin
        const int i = b + (threadIdx.x & 31);
        unsigned first = __ballot_sync(0xffffffffu, i < i1 && P.slots[i] >= 0 && !goes_on<NT>(P, i - 1));
        for (; first != 0u; first &= first - 1u) {
          if (turn-- != 0) continue;
          turn = P.parts - 1;
          scaled_run<NT>(P, b + __ffs(first) - 1, h, g);
        }
      }
    } else {
      for (int i = i0; i < i1; ++i) plain_kv_row(P, i);
    }
    if (P.beside && blockIdx.x == gridDim.x - 1) griddep_wait();
    return;
  }
  query_rows(P, cta - P.kv_ctas, P.rows);
}

template <int NT>
cudaError_t launch_nt(AppendParams p, cudaStream_t stream) {
  // From 1024 rows on the queries have a launch of their own, three CTAs an SM
  // that run through many rows, and K and V another that fills the rest of each
  // SM, a CTA for each block of rows and KV head (16 384 rows, 32 q and 4 KV
  // heads: 113 us, 5.2 TB/s; K and V first 129 us, four or five query CTAs an
  // SM 113 and 126 us).  One kernel's registers would keep queries from having
  // their loads in flight, and a CTA for each of 16 384 rows and heads takes
  // longer to start than to run (250 us).  Below, where a launch weighs more,
  // one launch of a CTA per row (and KV head).  Two launches / one, us (inputs in
  // L2): 512 rows of one sequence 9.1 / 9.2 and of 512 sequences 16.0 / 15.6,
  // 1024 rows 11.5 / 15.7 and 25.6 / 28.7.
  const bool many = p.rows >= 1024;
  p.chunk = NT > 0 && many ? kHalves * NT : 1;
  const int chunks = (p.rows + p.chunk - 1) / p.chunk;
  // (a chunk may be one run or, in a decode batch, a run a row: while there is
  // room, several CTAs share its runs; 1024 sequences of a row 47 -> 25.6 us with
  // inputs in L2, 32.5 without)
  const int parts = many ? 6 * sm_count() / (chunks * p.hkv) : 1;
  p.parts = parts < 1 ? 1 : parts > 16 ? 16 : parts;
  p.kv_ctas = NT > 0 ? chunks * p.hkv * p.parts : chunks;
  p.q_ctas = p.q_out == nullptr ? 0 : p.rows;
  if (!many)
    return launch_kernel(append_kernel<NT>, dim3(p.kv_ctas + p.q_ctas), dim3(kThreads), 0, stream, false, p);
  p.beside = p.q_ctas != 0;
  if (p.q_ctas != 0) {
    const int most = sm_count() * 3;
    if (p.q_ctas > most) p.q_ctas = most;
    const cudaError_t e = launch_kernel(query_kernel, dim3(p.q_ctas), dim3(kThreads), 0, stream, false, p);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(append_kernel<NT>, dim3(p.kv_ctas), dim3(kThreads), 0, stream, p.beside != 0, p);
}

}  // namespace

cudaError_t launch_kv_append(AppendParams p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  switch (p.kv_dtype == QSA_DTYPE_E4M3_BLOCK ? p.scale_block : 0) {
    case 0: return launch_nt<0>(p, stream);
    case 16: return launch_nt<2>(p, stream);
    case 32: return launch_nt<4>(p, stream);
    case 64: return launch_nt<8>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qsa
