// The pages of a paged cache on the device: sequences are forked, extended and
// freed, the pool is packed, pages are copied (qsa_pages_*).
//
// State, the caller's: refs[page] (how many sequences hold it; free iff 0),
// block_table[req][] and lengths[req] (tokens).  With pages(L) = ceil(L / page):
//   fork     child := parent: its full pages are shared (refs + 1), the last,
//            part-filled one is copied to a free page, its used units only;
//   extend   request r gets pages(L + n) - pages(L) free pages and n positions
//            and slots;
//   free     refs - 1 for each page, length 0, table row -1;
//   compact  with L live pages, the k-th free page below L takes the contents
//            and references of the k-th live page from L on.
// Free pages are given out in ascending order, to the requests (or forks) in
// the order of the call: there is no free list to keep, results do not depend
// on timing, and the pool stays dense.  A page's rank among the free ones is a
// scan over refs; a request's first rank is a scan over the needs, kept in
// shared memory, where the owner of a rank is found by bisection.
//
// A planner is one cluster of up to 8 CTAs of 1024 threads (each reads 4 pages'
// refs a turn; the CTAs exchange one total a turn through distributed shared
// memory), so that it needs no scratch and no second launch; copies, table rows
// and shared pages' counts follow in a grid of their own.  Every kernel starts
// while the one before it in the stream ends and waits for it before it reads
// anything; planners let their followers start at once (two children 16.4 -> 14.6
// us, now 15.3; copies that do so too left it at 15.5).
//
// Bound: planners by latency (a few dependent loads, two scans, the cluster's
// barriers), copies by HBM.  Measured: fork, a ring's copy, extend and free of two
// children of a small model 15.3 us (five launches; the calls take the host 22), of
// 240 children of 16 prompts of ~10 000 to 20 000 tokens 33 us, 15 of them the
// copies of 66 MB of last pages (static e4m3 27.5, block scales 33: half the bytes, more
// planes); half of a pool of 48 sequences of ~4500 to 9000
// tokens packed in 246 us (1.32 GB read and written, 5.6 TB/s behind a planner of 9
// us; 4 to 16 accesses of a thread in flight, 2 to 8 CTAs an SM and parts of 16 to
// 128 KB took 246 to 294, streaming loads 263).  A planner that makes the copies
// of few and small forks itself saves a launch, but one CTA takes longer over them
// than the launch did (17 -> 20 us at the time).
#include <cooperative_groups.h>

#include <climits>



#include "qsa_device.cuh"
#include "qsa_kernels.h"
#include "qsa_launch.cuh"

namespace cg = cooperative_groups;

namespace qsa {
namespace {

constexpr int kPlan = 1024;       // threads of a planner's CTA
constexpr int kCopy = 256;        // threads of a copying CTA
constexpr int kFlight = 8;        // accesses of a thread on their way together
constexpr int kChunk = 64 << 10;  // bytes that a copying CTA takes at the least
constexpr int kPlanSmem = 200 << 10;

struct Plane {
  uint8_t* base;
  long long page_bytes, seg_bytes;
  int segments, per, unit_bytes;  // per: tokens of a unit
  int whole, part;                // log2 of the access width for whole pages, and for parts of their segments
};
// (by value in the launch: short lists keep it small)
template <int N>
struct Planes {
  Plane p[N];
  int n;
};

struct Pool {
  int num_blocks, page, reqs, bt_stride;
  int capacity;  // tokens of a table row
  int32_t* refs;
  int32_t* table;
  int32_t* lengths;
  unsigned long long* err;
  __device__ __forceinline__ int pages(int tokens) const {
    return static_cast<int>((static_cast<unsigned>(tokens) + page - 1u) / static_cast<unsigned>(page));
  }
  __device__ __forceinline__ int32_t* row(int r) const { return table + static_cast<long long>(r) * bt_stride; }
};

// Exclusive sum over the block's threads of a pair of counts (low and high 32
// bits) or of one 64-bit count; total: everyone's.
__device__ __forceinline__ long long block_scan(long long v, long long* total, long long (&warps)[33]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();  // (the last scan's sums have been read)
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const long long mine = lane < kPlan / 32 ? warps[lane] : 0;
    long long w = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warps[lane] = w - mine;
    if (lane == 31) warps[32] = w;
  }
  __syncthreads();
  *total = warps[32];
  return warps[warp] + s - v;
}

// The same over the cluster's blocks, in the order of their ranks.  `slot`: two
// totals in turn, so that one barrier a turn is enough.
__device__ __forceinline__ long long cluster_scan(long long v, long long* total, long long (&warps)[33],
                                                  long long (&slot)[2], int turn) {
  cg::cluster_group cluster = cg::this_cluster();
  long long mine;
  long long at = block_scan(v, &mine, warps);
  if (threadIdx.x == 0) slot[turn & 1] = mine;
  cluster.sync();
  long long sum = 0;
  const unsigned rank = cluster.block_rank(), blocks = cluster.num_blocks();
  for (unsigned b = 0; b < blocks; ++b) {
    const long long t = *cluster.map_shared_rank(&slot[turn & 1], b);
    if (b < rank) at += t;
    sum += t;
  }
  *total = sum;
  return at;
}

// The references of the four pages from p on (1 for pages past the pool).
__device__ __forceinline__ int4 load_refs(const Pool& P, long long p) {
  int4 v = make_int4(1, 1, 1, 1);
  if (p + 3 < P.num_blocks && (reinterpret_cast<uintptr_t>(P.refs) & 15) == 0) {
    v = *reinterpret_cast<const int4*>(P.refs + p);
  } else {
    if (p < P.num_blocks) v.x = P.refs[p];
    if (p + 1 < P.num_blocks) v.y = P.refs[p + 1];
    if (p + 2 < P.num_blocks) v.z = P.refs[p + 2];
    if (p + 3 < P.num_blocks) v.w = P.refs[p + 3];
  }
  return v;
}

// Hands out the free pages in ascending order, rank 0 up to `need` - 1, to
// take(rank, page) with their reference set to 1.  Returns how many there were
// (at the most `need`).  All the cluster's threads call it; at least one
// cluster barrier passes.
template <typename F>
__device__ __forceinline__ long long take_free(const Pool& P, long long need, long long (&warps)[33], long long (&slot)[2], F&& take) {
  cg::cluster_group cluster = cg::this_cluster();
  const long long step = 4ll * kPlan * cluster.num_blocks();
  long long found = 0;
  int turn = 0;
  long long p = 4ll * (kPlan * static_cast<long long>(cluster.block_rank()) + threadIdx.x);
  if (need == 0) cluster.sync();
  for (long long base = 0; base < P.num_blocks && found < need; base += step, p += step, ++turn) {
    const int4 v = load_refs(P, p);
    const int free4[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
    long long total;
    long long rank = found + cluster_scan(free4[0] + free4[1] + free4[2] + free4[3], &total, warps, slot, turn);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!free4[k]) continue;
      if (rank < need) {
        P.refs[p + k] = 1;
        take(rank, static_cast<int>(p + k));
      }
      ++rank;
    }
    found += total;
  }
  return found < need ? found : need;
}

// The first of n ascending sums that is above `rank`.
template <typename T>
__device__ __forceinline__ int owner(const T* sums, int n, long long rank) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > rank)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- copies
template <typename T>
__device__ __forceinline__ void copy_run(const uint8_t* src, uint8_t* dst, long long first, long long last) {
  // elements first .. last - 1, eight of a thread on their way together
  const T* s = reinterpret_cast<const T*>(src);
  T* d = reinterpret_cast<T*>(dst);
  for (long long i = first + threadIdx.x; i < last; i += kFlight * kCopy) {
    T v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (i + u * kCopy < last) v[u] = s[i + u * kCopy];
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (i + u * kCopy < last) __stcs(d + i + u * kCopy, v[u]);
  }
}
template <typename T>
__device__ __forceinline__ void copy_segments(const uint8_t* src, uint8_t* dst, long long seg_bytes, int per_seg, long long first, long long last) {
  // the first per_seg elements of each segment, elements first .. last - 1 of all of them
  const int stride = static_cast<int>(seg_bytes / static_cast<int>(sizeof(T)));
  const T* s = reinterpret_cast<const T*>(src);
  T* d = reinterpret_cast<T*>(dst);
  for (long long i0 = first + threadIdx.x; i0 < last; i0 += kFlight * kCopy) {
    T v[kFlight];
    int at[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const unsigned i = static_cast<unsigned>(i0 + u * kCopy);
      if (i >= last) break;
      const unsigned seg = i / static_cast<unsigned>(per_seg);
      at[u] = static_cast<int>(seg * stride + (i - seg * per_seg));  // (within a page: below 2^30)
      v[u] = __ldcs(s + at[u]);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (i0 + u * kCopy >= last) break;
      __stcs(d + at[u], v[u]);
    }
  }
}

// Part `part` of `parts` of the first `units` units of each segment of a page
// (units < 0: the whole page).
__device__ __forceinline__ void copy_page(const Plane& L, int from, int to, int units, int part, int parts) {
  const uint8_t* s = L.base + from * L.page_bytes;
  uint8_t* d = L.base + to * L.page_bytes;
  const long long seg = units < 0 ? L.seg_bytes : static_cast<long long>(units) * L.unit_bytes;
  const bool whole = seg == L.seg_bytes;
  const int w = whole ? L.whole : L.part;
  const long long n = (whole ? L.page_bytes : seg * L.segments) >> w;  // (below 2^31)
  // parts on borders of 32 elements
  const long long per = ((n + parts - 1) / parts + 31) & ~31ll;
  const long long first = part * per, last = first + per < n ? first + per : n;
  if (first >= last) return;
  if (whole) {
    switch (w) {
      case 4: copy_run<uint4>(s, d, first, last); break;
      case 3: copy_run<uint2>(s, d, first, last); break;
      case 2: copy_run<uint32_t>(s, d, first, last); break;
      case 1: copy_run<uint16_t>(s, d, first, last); break;
      default: copy_run<uint8_t>(s, d, first, last); break;
    }
  } else {
    const int per_seg = static_cast<int>(seg >> w);
    switch (w) {
      case 4: copy_segments<uint4>(s, d, L.seg_bytes, per_seg, first, last); break;
      case 3: copy_segments<uint2>(s, d, L.seg_bytes, per_seg, first, last); break;
      case 2: copy_segments<uint32_t>(s, d, L.seg_bytes, per_seg, first, last); break;
      case 1: copy_segments<uint16_t>(s, d, L.seg_bytes, per_seg, first, last); break;
      default: copy_segments<uint8_t>(s, d, L.seg_bytes, per_seg, first, last); break;
    }
  }
}

// ---------------------------------------------------------------- fork
// tails[i]: the page of the child's own copy of the last page, -1 none needed
// (or padding, or the parent's is no page of the pool), -2 refused.
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const Pool P, const int32_t* parents, const int32_t* children, int n, int32_t* tails) {
  extern __shared__ int32_t sm[];
  __shared__ long long warps[33], slot[2];
  int32_t* claim = sm;           // [reqs]: the first fork that names it as its child
  int32_t* sums = sm + P.reqs;   // [n]: forks up to this one that need a page
  int32_t* len = sums + n;       // [n]: tokens, -1 padding, -2 refused
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < P.reqs; i += kPlan) claim[i] = INT_MAX;
  griddep_wait();
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int c = children[i];
    if (parents[i] >= 0 && c >= 0 && c < P.reqs) atomicMin(&claim[c], i);
  }
  __syncthreads();
  long long needed = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int l = -1, need = 0;
    if (i < n) {
      const int a = parents[i], c = children[i];
      if (a >= 0 && c >= 0) {
        l = -2;
        if (a < P.reqs && c < P.reqs) {
          const int t = P.lengths[a], u = P.lengths[c];
          if (claim[c] == i && u == 0 && t >= 0 && t <= P.capacity) l = t;
        }
      }
      len[i] = l;
      if (l > 0 && l % P.page != 0) {  // (a last page outside the pool is not copied)
        const int last = P.row(a)[l / P.page];
        need = last >= 0 && last < P.num_blocks;
      }
    }
    long long total;
    const long long at = block_scan(need, &total, warps);
    if (i < n) sums[i] = static_cast<int32_t>(needed + at + need);
    needed += total;
  }
  __syncthreads();
  const long long got = take_free(P, needed, warps, slot, [&](long long rank, int page) {
    const int i = owner(sums, n, rank);
    tails[i] = page;
    P.row(children[i])[len[i] / P.page] = page;
  });
  // (every CTA has read the lengths by now)
  cg::cluster_group cluster = cg::this_cluster();
  if (cluster.block_rank() == 0) {
    for (int i = threadIdx.x; i < n; i += kPlan) {
      const int l = len[i];
      const bool need = sums[i] > (i > 0 ? sums[i - 1] : 0);
      if (l == -2 || (need && sums[i] > got)) {
        tails[i] = -2;
        flag_error(P.err);
        continue;
      }
      if (!need) tails[i] = -1;
      if (l >= 0) P.lengths[children[i]] = l;
    }
  }
  cluster.sync();  // (a CTA's totals are read until here)
}

// Fork i = blockIdx.x: blockIdx.y < planes.n copies its last page there, the
// last y its table row and the shared pages' references.
template <int N>
__global__ void __launch_bounds__(kCopy, 4) fork_copy_kernel(const Pool P, const __grid_constant__ Planes<N> L, const int32_t* parents,
                                                             const int32_t* children, const int32_t* tails) {
  const int i = blockIdx.x, plane = blockIdx.y;
  griddep_wait();
  const int a = parents[i], c = children[i];
  const int tail = tails[i];
  if (tail == -2 || a < 0 || c < 0) return;  // (the planner has checked the others)
  const int l = P.lengths[c], full = l / P.page, used = l - full * P.page;
  const int32_t* from = P.row(a);
  if (plane < L.n) {
    if (used == 0 || tail < 0) return;
    const Plane& pl = L.p[plane];
    copy_page(pl, from[full], tail, (used + pl.per - 1) / pl.per, blockIdx.z, gridDim.z);
    return;
  }
  int32_t* to = P.row(c);
  for (int k = blockIdx.z * kCopy + threadIdx.x; k < P.bt_stride; k += gridDim.z * kCopy) {
    if (k == full && tail >= 0) continue;  // (the planner's)
    int page = -1;
    if (k == full && used != 0) {  // (the planner found no page of the pool there)
      flag_error(P.err);
    } else if (k < full) {
      page = from[k];
      if (page < 0 || page >= P.num_blocks) {
        page = -1;
        flag_error(P.err);
      } else {
        atomicAdd(&P.refs[page], 1);
      }
    }
    to[k] = page;
  }
}

// Pair i = blockIdx.x: page src[i] to dst[i] in plane blockIdx.y.  A pair whose
// dst an earlier pair has too, or that is another pair's src, would race: it is
// left out.  Every CTA of the pair asks that itself (n <= kMaxPairs): without a
// second launch or scratch, but n^2 reads.  Measured: 256 pages of 128 KB 15 us, 4096
// 201 (5.3 TB/s); 256 rings of 2 KB 2.9 us, 4096 34, 16 384 428, where the reads of the
// list are nearly all.
template <int N>
__global__ void __launch_bounds__(kCopy, 4) copy_kernel(const __grid_constant__ Planes<N> L, int num_blocks, const int32_t* src, const int32_t* dst,
                                                     int n, unsigned long long* err) {
  const int i = blockIdx.x;
  griddep_wait();
  const int s = src[i], d = dst[i];
  if (s < 0 || d < 0) return;
  bool bad = s >= num_blocks || d >= num_blocks;
  for (int j = threadIdx.x; j < n; j += kCopy)
    if (j != i) {
      const int sj = src[j], dj = dst[j];
      bad |= sj >= 0 && dj >= 0 && (sj == d || (j < i && dj == d));
    }
  if (__syncthreads_or(bad)) {
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) flag_error(err);
    return;
  }
  if (s != d) copy_page(L.p[blockIdx.y], s, d, -1, blockIdx.z, gridDim.z);
}

// ---------------------------------------------------------------- extend
__global__ void __launch_bounds__(kPlan) extend_kernel(const Pool P, const int32_t* qsl, const int32_t* token_to_req, int rows, int32_t* positions,
                                                       int64_t* slots) {
  extern __shared__ long long sums[];  // [reqs]: pages needed up to this request
  __shared__ long long warps[33], slot[2];
  cg::cluster_group cluster = cg::this_cluster();
  griddep_launch_dependents();
  griddep_wait();
  // a request's new tokens, -1: refused; and the pages they need
  auto wanted = [&](int r, int* need) {
    const int q0 = qsl[r], q1 = qsl[r + 1], l = P.lengths[r];
    *need = 0;
    if (q0 < 0 || q1 < q0 || q1 > rows || l < 0 || static_cast<long long>(l) + (q1 - q0) > P.capacity) return -1;
    *need = P.pages(l + (q1 - q0)) - P.pages(l);
    return q1 - q0;
  };
  long long needed = 0;
  for (int r0 = 0; r0 < P.reqs; r0 += kPlan) {
    const int r = r0 + threadIdx.x;
    int need = 0;
    if (r < P.reqs) wanted(r, &need);
    long long total;
    const long long at = block_scan(need, &total, warps);
    if (r < P.reqs) sums[r] = needed + at + need;
    needed += total;
  }
  __syncthreads();
  const long long got = take_free(P, needed, warps, slot, [&](long long rank, int page) {
    const int r = owner(sums, P.reqs, rank);
    const long long first = r > 0 ? sums[r - 1] : 0;
    P.row(r)[P.pages(P.lengths[r]) + static_cast<int>(rank - first)] = page;
  });
  cluster.sync();  // the table is complete, for every CTA
  for (int i = cluster.block_rank() * kPlan + threadIdx.x; i < rows; i += kPlan * cluster.num_blocks()) {
    const int r = token_to_req[i];
    int pos = -1;
    long long at = -1;
    if (r >= 0 && r < P.reqs && i >= qsl[r] && i < qsl[r + 1]) {
      int need;
      if (wanted(r, &need) >= 0 && (need == 0 || sums[r] <= got)) {
        pos = P.lengths[r] + (i - qsl[r]);
        const int page = P.row(r)[pos / P.page];
        if (page < 0 || page >= P.num_blocks)
          flag_error(P.err);
        else
          at = static_cast<long long>(page) * P.page + pos % P.page;
      }
    }
    positions[i] = pos;
    slots[i] = at;
  }
  cluster.sync();  // the lengths and totals have been read
  if (cluster.block_rank() != 0) return;
  for (int r = threadIdx.x; r < P.reqs; r += kPlan) {
    int need;
    const int count = wanted(r, &need);
    if (count >= 0 && (need == 0 || sums[r] <= got)) {
      if (count > 0) P.lengths[r] += count;
      continue;
    }
    flag_error(P.err);
    // what it was given before the free pages ran out goes back
    const long long first = sums[r] - need;
    const int have = count >= 0 ? P.pages(P.lengths[r]) : 0;
    for (long long k = first; k < got && k < sums[r]; ++k) {
      int32_t* e = P.row(r) + have + (k - first);
      P.refs[*e] = 0;
      *e = -1;
    }
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kCopy) free_kernel(const Pool P, const int32_t* requests) {
  __shared__ int tokens;
  griddep_launch_dependents();
  griddep_wait();
  const int r = requests[blockIdx.x];
  if (r < 0) return;
  if (threadIdx.x == 0) {
    tokens = 0;
    if (r >= P.reqs)
      flag_error(P.err);
    else
      tokens = atomicExch(&P.lengths[r], 0);  // (a request named twice: once)
  }
  __syncthreads();
  if (tokens < 0 || tokens > P.capacity) {
    if (threadIdx.x == 0) flag_error(P.err);
    return;
  }
  const int n = P.pages(tokens);
  int32_t* row = P.row(r < P.reqs ? r : 0);
  for (int k = threadIdx.x; k < n; k += kCopy) {
    const int page = row[k];
    row[k] = -1;
    bool bad = page < 0 || page >= P.num_blocks;
    if (!bad && atomicSub(&P.refs[page], 1) <= 0) {  // held by nobody
      atomicAdd(&P.refs[page], 1);
      bad = true;
    }
    if (bad) flag_error(P.err);
  }
}

// ---------------------------------------------------------------- compact
struct Moves {
  int32_t* count;   // pages that move
  int32_t* to;      // [num_blocks]: where a page is afterwards (-1: free now), from a 16-byte border on
  int32_t* movers;  // [num_blocks / 2 + 1], and where they go
  int32_t* holes;
};

__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Pool P, const Moves M, int32_t* live_out) {
  __shared__ long long warps[33], slot[2];
  cg::cluster_group cluster = cg::this_cluster();
  const long long step = 4ll * kPlan * cluster.num_blocks();
  const long long p0 = 4ll * (kPlan * static_cast<long long>(cluster.block_rank()) + threadIdx.x);
  griddep_launch_dependents();
  griddep_wait();
  int turn = 0;
  long long count = 0, live;
  const int4 first = load_refs(P, p0);
  for (long long p = p0; p < P.num_blocks; p += step) {
    const int4 v = p == p0 ? first : load_refs(P, p);
    count += (v.x > 0) + (v.y > 0 && p + 1 < P.num_blocks) + (v.z > 0 && p + 2 < P.num_blocks) + (v.w > 0 && p + 3 < P.num_blocks);
  }
  cluster_scan(count, &live, warps, slot, turn++);
  // ranks of holes (low half) and movers (high half)
  long long found = 0;
  long long p = p0;
  for (long long base = 0; base < P.num_blocks; base += step, p += step, ++turn) {
    const int4 v4 = base == 0 ? first : load_refs(P, p);
    const int v[4] = {v4.x, v4.y, v4.z, v4.w};
    long long mine = 0;
    int kind[4], to[4];  // 1: a hole, 2: a mover
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool low = p + k < live;
      kind[k] = p + k >= P.num_blocks ? 0 : low && v[k] <= 0 ? 1 : !low && v[k] > 0 ? 2 : 0;
      mine += kind[k] == 1 ? 1ll : kind[k] == 2 ? 1ll << 32 : 0ll;
      to[k] = low && v[k] > 0 ? static_cast<int>(p + k) : -1;  // (movers' below)
    }
    if (p + 3 < P.num_blocks) {
      *reinterpret_cast<int4*>(M.to + p) = make_int4(to[0], to[1], to[2], to[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < P.num_blocks) M.to[p + k] = to[k];
    }
    long long total;
    long long rank = found + cluster_scan(mine, &total, warps, slot, turn);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (kind[k] == 1) {
        M.holes[rank & 0x7fffffff] = static_cast<int>(p + k);
        rank += 1;
      } else if (kind[k] == 2) {
        M.movers[rank >> 32] = static_cast<int>(p + k);
        rank += 1ll << 32;
      }
    }
    found += total;
  }
  cluster.sync();  // both lists are complete, and M.to but for movers
  const int moves = static_cast<int>(found >> 32);
  for (int k = cluster.block_rank() * kPlan + threadIdx.x; k < moves; k += kPlan * cluster.num_blocks()) M.to[M.movers[k]] = M.holes[k];
  if (cluster.block_rank() == 0 && threadIdx.x == 0) {
    *M.count = moves;
    *live_out = static_cast<int32_t>(live);
  }
}

template <int N>
__global__ void __launch_bounds__(kCopy, 4) compact_move_kernel(const Pool P, const __grid_constant__ Planes<N> L, const Moves M, int parts) {
  griddep_wait();
  const int moves = *M.count;
  const long long ctas = gridDim.x;
  const long long items = static_cast<long long>(moves) * parts;
  for (int plane = 0; plane < L.n; ++plane)
    for (long long i = blockIdx.x; i < items; i += ctas) {
      const int k = static_cast<int>(i / parts);
      copy_page(L.p[plane], M.movers[k], M.holes[k], -1, static_cast<int>(i - static_cast<long long>(k) * parts), parts);
    }
  // (references and table rows from the last CTAs on, which may have had no copies)
  const long long back = ctas - 1 - blockIdx.x;
  for (long long k = back * kCopy + threadIdx.x; k < moves; k += ctas * kCopy) {
    const int from = M.movers[k];
    P.refs[M.holes[k]] = P.refs[from];
    P.refs[from] = 0;
  }
  for (long long r = back; r < P.reqs; r += ctas) {
    const int l = P.lengths[r];
    if (l < 0 || l > P.capacity) {
      if (threadIdx.x == 0) flag_error(P.err);
      continue;
    }
    int32_t* row = P.row(static_cast<int>(r));
    const int n = P.pages(l);
    for (int k = threadIdx.x; k < n; k += kCopy) {
      const int page = row[k];
      const int to = page >= 0 && page < P.num_blocks ? M.to[page] : -1;
      if (to < 0)  // (no used page: below `live` it may hold another sequence's tokens now)
        flag_error(P.err);
      else if (to != page)
        row[k] = to;
    }
  }
}

// ---------------------------------------------------------------- host
int log2_width(uintptr_t bits) {
  int w = 0;
  while (w < 4 && ((bits >> w) & 1) == 0) ++w;
  return w;
}

qsa_status check_planes(const qsa_page_plane* planes, int n, int page_size, long long* page_bytes) {
  if (n < 0) return QSA_ERR_SHAPE;
  if (n > QSA_MAX_PAGE_PLANES) return QSA_ERR_UNSUPPORTED;
  if (n > 0 && planes == nullptr) return QSA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0) return QSA_ERR_SHAPE;
  *page_bytes = 0;
  for (int i = 0; i < n; ++i) {
    const qsa_page_plane& s = planes[i];
    if (s.base == nullptr) return QSA_ERR_INVALID_ARG;
    if (s.segments < 1 || s.unit_bytes < 1 || s.tokens_per_unit < 1 || page_size % s.tokens_per_unit != 0) return QSA_ERR_SHAPE;
    const long long seg = static_cast<long long>(page_size / s.tokens_per_unit) * s.unit_bytes;
    if (seg > (1ll << 30) / s.segments) return QSA_ERR_SHAPE;  // (a page of a plane: 1 GiB)
    if (seg * s.segments > *page_bytes) *page_bytes = seg * s.segments;
  }
  return QSA_OK;
}

template <int N>
void fill_planes(Planes<N>* out, const qsa_page_plane* planes, int n, int page_size) {
  out->n = n;
  for (int i = 0; i < n; ++i) {
    const qsa_page_plane& s = planes[i];
    Plane& p = out->p[i];
    p.base = static_cast<uint8_t*>(s.base);
    p.segments = s.segments;
    p.per = s.tokens_per_unit;
    p.unit_bytes = s.unit_bytes;
    p.seg_bytes = static_cast<long long>(page_size / s.tokens_per_unit) * s.unit_bytes;
    p.page_bytes = p.seg_bytes * s.segments;
    const uintptr_t whole = reinterpret_cast<uintptr_t>(s.base) | static_cast<uintptr_t>(p.page_bytes);
    p.whole = log2_width(whole);
    p.part = log2_width(whole | static_cast<uintptr_t>(p.seg_bytes) | static_cast<uintptr_t>(s.unit_bytes));
  }
}
// f with the planes in a list of the length that fits
template <typename F>
cudaError_t with_planes(const qsa_page_plane* planes, int n, int page_size, F&& f) {
  if (n <= 8) {
    Planes<8> l;
    fill_planes(&l, planes, n, page_size);
    return f(l);
  }
  Planes<QSA_MAX_PAGE_PLANES> l;
  fill_planes(&l, planes, n, page_size);
  return f(l);
}

qsa_status check_pool(const qsa_page_pool* pool, Pool* P, long long* page_bytes) {
  if (pool == nullptr) return QSA_ERR_INVALID_ARG;
  const qsa_status st = check_planes(pool->planes, pool->n_planes, pool->page_size, page_bytes);
  if (st != QSA_OK) return st;
  if (pool->num_blocks < 1 || pool->reqs < 1 || pool->bt_stride < 1) return QSA_ERR_SHAPE;
  if (!pool->refs || !pool->block_table || !pool->lengths) return QSA_ERR_INVALID_ARG;
  const uintptr_t a4 = reinterpret_cast<uintptr_t>(pool->refs) | reinterpret_cast<uintptr_t>(pool->block_table) |
                       reinterpret_cast<uintptr_t>(pool->lengths);
  if (a4 & 3) return QSA_ERR_INVALID_ARG;
  P->num_blocks = pool->num_blocks;
  P->page = pool->page_size;
  P->reqs = pool->reqs;
  P->bt_stride = pool->bt_stride;
  const long long tokens = static_cast<long long>(pool->bt_stride) * pool->page_size;
  P->capacity = static_cast<int>(tokens < kMaxKeys ? tokens : kMaxKeys);
  P->refs = pool->refs;
  P->table = pool->block_table;
  P->lengths = pool->lengths;
  return QSA_OK;
}

bool words(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// CTAs of a planner: as many as find something to read in one turn.
int plan_ctas(int num_blocks, long long other) {
  int c = 1;
  while (c < 8 && (num_blocks > 4 * kPlan * c || other > 4ll * kPlan * c)) c *= 2;
  return c;
}

// A planner's shared memory, allowed once a device.
template <typename K>
cudaError_t allow_smem(K* kernel, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// CTAs that share a page's copy: enough of them all for the SMs, none with less
// than kChunk bytes.
int copy_parts(long long pages, long long page_bytes, int sms) {
  const long long most = (page_bytes + kChunk - 1) / kChunk;
  long long parts = pages > 0 ? (8ll * sms + pages - 1) / pages : 1;
  if (parts > most) parts = most;
  if (parts > 1024) parts = 1024;
  return parts < 1 ? 1 : static_cast<int>(parts);
}

constexpr int kMaxPairs = 16384;

qsa_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

qsa_status do_fork(const qsa_page_pool* pool, const int32_t* parents, const int32_t* children, int n, int32_t* tails, cudaStream_t stream) {
  Pool P{};
  long long page_bytes;
  const qsa_status st = check_pool(pool, &P, &page_bytes);
  if (st != QSA_OK) return st;
  if (n < 0) return QSA_ERR_SHAPE;
  if (n == 0) return QSA_OK;
  if (!words(parents) || !words(children) || !words(tails)) return QSA_ERR_INVALID_ARG;
  const long long smem = 4ll * (static_cast<long long>(P.reqs) + 2ll * n);
  if (smem > kPlanSmem) return QSA_ERR_UNSUPPORTED;
  P.err = internal_error_word();
  if (P.err == nullptr) return QSA_ERR_CUDA;
  static bool allowed[64] = {};
  cudaError_t e = allow_smem(fork_plan_kernel, allowed);
  if (e != cudaSuccess) return QSA_ERR_CUDA;
  const int ctas = plan_ctas(P.num_blocks, 0);
  e = launch_kernel_cluster(fork_plan_kernel, dim3(ctas), dim3(kPlan), static_cast<size_t>(smem), stream, true, ctas, P, parents, children, n, tails);
  if (e != cudaSuccess) return QSA_ERR_CUDA;
  const int parts = copy_parts(static_cast<long long>(n) * (pool->n_planes > 0 ? pool->n_planes : 1), page_bytes, sm_count());
  return cuda_ok(with_planes(pool->planes, pool->n_planes, pool->page_size, [&](const auto& planes) {
    auto kernel = fork_copy_kernel<sizeof(planes.p) / sizeof(Plane)>;
    return launch_kernel(kernel, dim3(n, pool->n_planes + 1, parts), dim3(kCopy), 0, stream, true, P, planes, parents, children,
                         static_cast<const int32_t*>(tails));
  }));
}

qsa_status do_extend(const qsa_page_pool* pool, const int32_t* qsl, const int32_t* token_to_req, int rows, int32_t* positions, int64_t* slots,
                     cudaStream_t stream) {
  Pool P{};
  long long page_bytes;
  const qsa_status st = check_pool(pool, &P, &page_bytes);
  if (st != QSA_OK) return st;
  if (rows < 0) return QSA_ERR_SHAPE;
  if (rows == 0) return QSA_OK;
  if (!words(qsl) || !words(token_to_req) || !words(positions) || slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7))
    return QSA_ERR_INVALID_ARG;
  const long long smem = 8ll * P.reqs;
  if (smem > kPlanSmem) return QSA_ERR_UNSUPPORTED;
  P.err = internal_error_word();
  if (P.err == nullptr) return QSA_ERR_CUDA;
  static bool allowed[64] = {};
  if (allow_smem(extend_kernel, allowed) != cudaSuccess) return QSA_ERR_CUDA;
  const int ctas = plan_ctas(P.num_blocks, rows);
  return cuda_ok(launch_kernel_cluster(extend_kernel, dim3(ctas), dim3(kPlan), static_cast<size_t>(smem), stream, true, ctas, P, qsl, token_to_req,
                                       rows, positions, slots));
}

qsa_status do_free(const qsa_page_pool* pool, const int32_t* requests, int n, cudaStream_t stream) {
  Pool P{};
  long long page_bytes;
  const qsa_status st = check_pool(pool, &P, &page_bytes);
  if (st != QSA_OK) return st;
  if (n < 0) return QSA_ERR_SHAPE;
  if (n == 0) return QSA_OK;
  if (!words(requests)) return QSA_ERR_INVALID_ARG;
  P.err = internal_error_word();
  if (P.err == nullptr) return QSA_ERR_CUDA;
  return cuda_ok(launch_kernel(free_kernel, dim3(n), dim3(kCopy), 0, stream, true, P, requests));
}

size_t compact_bytes(const Pool& P) { return 4 * (4 + static_cast<size_t>(P.num_blocks) + 2 * (static_cast<size_t>(P.num_blocks) / 2 + 1)); }

qsa_status do_compact(const qsa_page_pool* pool, int32_t* live, void* ws, size_t ws_bytes, cudaStream_t stream) {
  Pool P{};
  long long page_bytes;
  const qsa_status st = check_pool(pool, &P, &page_bytes);
  if (st != QSA_OK) return st;
  if (!words(live)) return QSA_ERR_INVALID_ARG;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < compact_bytes(P)) return QSA_ERR_WORKSPACE;
  P.err = internal_error_word();
  if (P.err == nullptr) return QSA_ERR_CUDA;
  Moves M{};
  M.count = static_cast<int32_t*>(ws);
  M.to = M.count + 4;
  M.movers = M.to + P.num_blocks;
  M.holes = M.movers + P.num_blocks / 2 + 1;
  const int ctas = plan_ctas(P.num_blocks, 0), sms = sm_count();
  cudaError_t e = launch_kernel_cluster(compact_plan_kernel, dim3(ctas), dim3(kPlan), 0, stream, true, ctas, P, M, live);
  if (e != cudaSuccess) return QSA_ERR_CUDA;
  const long long most = (page_bytes + kChunk - 1) / kChunk;
  const int parts = most < 1 ? 1 : most > 1024 ? 1024 : static_cast<int>(most);
  // (no more CTAs than the pool can have things to move)
  long long grid = (P.num_blocks / 2 + 1ll) * parts;
  if (grid < P.reqs) grid = P.reqs;
  if (grid > 4ll * sms) grid = 4ll * sms;
  return cuda_ok(with_planes(pool->planes, pool->n_planes, pool->page_size, [&](const auto& planes) {
    auto kernel = compact_move_kernel<sizeof(planes.p) / sizeof(Plane)>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopy), 0, stream, true, P, planes, M, parts);
  }));
}

qsa_status do_copy(const qsa_page_plane* planes, int n_planes, int page_size, int num_blocks, const int32_t* src, const int32_t* dst, int n,
                   cudaStream_t stream) {
  long long page_bytes;
  const qsa_status st = check_planes(planes, n_planes, page_size, &page_bytes);
  if (st != QSA_OK) return st;
  if (n < 0 || num_blocks < 1) return QSA_ERR_SHAPE;
  if (n > kMaxPairs) return QSA_ERR_UNSUPPORTED;
  if (n == 0 || n_planes == 0) return QSA_OK;
  if (!words(src) || !words(dst)) return QSA_ERR_INVALID_ARG;
  unsigned long long* err = internal_error_word();
  if (err == nullptr) return QSA_ERR_CUDA;
  const int parts = copy_parts(static_cast<long long>(n) * n_planes, page_bytes, sm_count());
  return cuda_ok(with_planes(planes, n_planes, page_size, [&](const auto& list) {
    auto kernel = copy_kernel<sizeof(list.p) / sizeof(Plane)>;
    return launch_kernel(kernel, dim3(n, n_planes, parts), dim3(kCopy), 0, stream, true, list, num_blocks, src, dst, n, err);
  }));
}

}  // namespace
}  // namespace qsa

using namespace qsa;

extern "C" {

qsa_status qsa_pages_fork(const qsa_page_pool* pool, const int32_t* parents, const int32_t* children, int32_t n, int32_t* tails, void* stream) {
  return no_throw([&] { return do_fork(pool, parents, children, n, tails, static_cast<cudaStream_t>(stream)); });
}

qsa_status qsa_pages_extend(const qsa_page_pool* pool, const int32_t* query_start_loc, const int32_t* token_to_req, int32_t rows,
                            int32_t* logical_positions, int64_t* slot_mapping, void* stream) {
  return no_throw([&] {
    return do_extend(pool, query_start_loc, token_to_req, rows, logical_positions, slot_mapping, static_cast<cudaStream_t>(stream));
  });
}

qsa_status qsa_pages_free(const qsa_page_pool* pool, const int32_t* requests, int32_t n, void* stream) {
  return no_throw([&] { return do_free(pool, requests, n, static_cast<cudaStream_t>(stream)); });
}

qsa_status qsa_pages_compact(const qsa_page_pool* pool, int32_t* live, void* ws, size_t ws_bytes, void* stream) {
  return no_throw([&] { return do_compact(pool, live, ws, ws_bytes, static_cast<cudaStream_t>(stream)); });
}

size_t qsa_pages_workspace_bytes(const qsa_page_pool* pool) {
  Pool P{};
  long long page_bytes;
  return check_pool(pool, &P, &page_bytes) == QSA_OK ? compact_bytes(P) : 0;
}

qsa_status qsa_pages_copy(const qsa_page_plane* planes, int32_t n_planes, int32_t page_size, int32_t num_blocks, const int32_t* src,
                          const int32_t* dst, int32_t n, void* stream) {
  return no_throw([&] { return do_copy(planes, n_planes, page_size, num_blocks, src, dst, n, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
