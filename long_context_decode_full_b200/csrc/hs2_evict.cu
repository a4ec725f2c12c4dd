// hs2_evict.cu -- keeping the cache: the accepted path of a drafted tree moves
// to the front of the draft, and a cache over its budget keeps the tokens with
// the largest accumulated attention weight.
//
// Both move rows within a unit's own positions, toward the front, in place.
#include <cooperative_groups.h>
#include <limits.h>

#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_select_common.cuh"

namespace hs2 {

namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ int64_t evict_slot(const int32_t *pt, int max_pages, int ps, int64_t num_slots, int b, int pos) {
  const int64_t s = pt == nullptr ? (int64_t)b * ps + pos
                                  : (int64_t)__ldg(pt + (int64_t)b * max_pages + pos / ps) * ps + pos % ps;
  return s >= 0 && s < num_slots ? s : -1;
}

// ------------------------------------------------------------------ accept
// Rows T - n + path[i] -> T - n + i, i < path_len.  One CTA per (sequence, K or
// V, 256 bytes of a row) and one per sequence for the E4M3 scales: every row is
// read before any is written, so the path may come in any order.  Bound by
// latency: two dependent loads (page table, row) and a store, 4.5 us for 4 sequences
// and 5.4 us for 64 of 64 drafts, below the 10 us that a call takes on the host.
constexpr int kAcceptThreads = 256;
constexpr int kAcceptCols = 256;  // bytes of a row per CTA: 16 threads x 16 bytes
constexpr int kAcceptRounds = kMaxDraft * kAcceptCols / 16 / kAcceptThreads;

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams p) {
  __shared__ int64_t sh_src[kMaxDraft], sh_dst[kMaxDraft];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, job = blockIdx.x;
  const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
  const int n = clamp_len(p.num_draft ? __ldg(p.num_draft + b) : p.M, min(kMaxDraft, T));  // a path may be narrower
  const int a = clamp_len(__ldg(p.path_len + b), min(n, p.M));
  const int first = T - n;
  if ((int)threadIdx.x < a) {
    const int j = __ldg(p.path + (int64_t)b * p.M + threadIdx.x);
    int64_t src = -1, dst = -1;
    if (j >= 0 && j < n && j != (int)threadIdx.x) {
      src = evict_slot(p.page_table, p.max_pages, p.page_size, p.num_slots, b, first + j);
      dst = evict_slot(p.page_table, p.max_pages, p.page_size, p.num_slots, b, first + threadIdx.x);
    }
    sh_src[threadIdx.x] = dst >= 0 ? src : -1;  // -1: stays where it is
    sh_dst[threadIdx.x] = dst;
  }
  if (job == 0 && threadIdx.x == 0) p.lens_out[b] = first + a;
  __syncthreads();
  const int chunks = (p.row_bytes + kAcceptCols - 1) / kAcceptCols;
  if (job < 2 * chunks) {
    uint8_t *x = static_cast<uint8_t *>(job < chunks ? p.k : p.v);
    const int col = (job % chunks) * kAcceptCols + (threadIdx.x & 15) * 16;
    uint4 r[kAcceptRounds];
#pragma unroll
    for (int k = 0; k < kAcceptRounds; ++k) {
      const int i = k * (kAcceptThreads / 16) + (threadIdx.x >> 4);
      if (i < a && sh_src[i] >= 0 && col < p.row_bytes)
        r[k] = __ldcg(reinterpret_cast<const uint4 *>(x + sh_src[i] * p.row_bytes + col));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kAcceptRounds; ++k) {
      const int i = k * (kAcceptThreads / 16) + (threadIdx.x >> 4);
      if (i < a && sh_src[i] >= 0 && col < p.row_bytes)
        *reinterpret_cast<uint4 *>(x + sh_dst[i] * p.row_bytes + col) = r[k];
    }
    return;
  }
  // E4M3: the scales of this job's heads, kAcceptScaleHeads at a time
  const int h0 = (job - 2 * chunks) * kAcceptScaleHeads, nh = min(kAcceptScaleHeads, p.Hkv - h0);
  float ks[kMaxDraft * kAcceptScaleHeads / kAcceptThreads], vs[kMaxDraft * kAcceptScaleHeads / kAcceptThreads];
#pragma unroll
  for (int k = 0; k < kMaxDraft * kAcceptScaleHeads / kAcceptThreads; ++k) {
    const int e = k * kAcceptThreads + threadIdx.x, i = e / kAcceptScaleHeads, h = e % kAcceptScaleHeads;
    if (i < a && h < nh && sh_src[i] >= 0) {
      ks[k] = __ldcg(p.k_scale + sh_src[i] * p.Hkv + h0 + h);
      vs[k] = __ldcg(p.v_scale + sh_src[i] * p.Hkv + h0 + h);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMaxDraft * kAcceptScaleHeads / kAcceptThreads; ++k) {
    const int e = k * kAcceptThreads + threadIdx.x, i = e / kAcceptScaleHeads, h = e % kAcceptScaleHeads;
    if (i < a && h < nh && sh_src[i] >= 0) {
      p.k_scale[sh_dst[i] * p.Hkv + h0 + h] = ks[k];
      p.v_scale[sh_dst[i] * p.Hkv + h0 + h] = vs[k];
    }
  }
}

// ------------------------------------------------------------------ select
// The kept positions of a unit (sequence, kv head) over its budget K: of the
// positions below T - W the K - W with the largest sums (ties to the lower
// position, NaN below everything), then the window.  A cluster of CTAs per unit
// takes equal shares of the positions: three radix passes (11, 11, 10 bits of an
// order-preserving key) find the exact key of the last one taken, then each share
// writes its positions behind the earlier shares' counts.  A pass counts into shared
// memory; each CTA adds its part of the bins over the cluster and hands the sums to
// all (distributed shared memory), so every CTA finds the bin itself.  A share's
// keys stay in registers where they fit; a unit of one CTA needs no cluster.  Up to
// 512 positions are ranked by counting instead, each thread's key against all.
// Bound by seven cluster barriers: 27 us for
// 16 units of 65,536 (37 us with one warp vote per key, which takes ~190 cycles, and
// keys read again in every pass).
constexpr int kPickBins = 2048;
constexpr int kPickKeys = 16;  // of a thread, in registers
constexpr int kPickRank = 512;  // positions ranked by counting: n^2 comparisons, 2 us at 512 and 8 at 1,024, where the passes take 8

__device__ __forceinline__ uint32_t sum_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  if (x == 0.f) return 0x80000000u;  // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int kPickThreads>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const EvictParams p) {
  __shared__ __align__(16) uint32_t sh_hist[kPickBins], sh_tot[kPickBins];
  __shared__ int sh_warp[33], sh_res[2];
  __shared__ int2 sh_counts[8];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  griddep_wait();
  griddep_launch_dependents();
  const int u = blockIdx.x / C, b = u / p.Hkv, kvh = u % p.Hkv;
  const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
  const int K = p.budget, tid = threadIdx.x;
  int32_t *kept = p.kept + (int64_t)u * K;
  if (rank == 0 && tid == 0 && kvh == 0) p.lens_out[b] = min(T, K);
  if (T <= K) {  // everything stays (the same for the whole cluster)
    for (int i = rank * kPickThreads + tid; i < K; i += C * kPickThreads) kept[i] = i < T ? i : -1;
    return;
  }
  const int W = min(p.window, K), n = T - W, take = K - W;
  const float *acc = p.acc + (int64_t)u * p.acc_stride;
  for (int i = rank * kPickThreads + tid; i < W; i += C * kPickThreads) kept[take + i] = n + i;
  if (take == 0) return;
  if (n <= kPickRank) {  // the same for the cluster
    if (rank != 0) return;
    const uint32_t key = tid < n ? sum_key(__ldg(acc + tid)) : 0u;
    sh_tot[tid] = key;
    __syncthreads();
    // sums before this one: larger ones, and equal ones at lower positions
    const uint4 *all = reinterpret_cast<const uint4 *>(sh_tot);
    const int mine = tid / 32 * 8, end = (n + 3) / 4;  // the warp's own keys
    int before = 0;
    if (mine < end) {  // not for the warps behind the last position
    for (int j = 0; j < mine; ++j) {
      const uint4 x = all[j];
      before += (x.x >= key) + (x.y >= key) + (x.z >= key) + (x.w >= key);
    }
    for (int j = mine; j < min(mine + 8, end); ++j) {
      const uint4 x = all[j];
      const int t = 4 * j;
      before += (x.x > key || (x.x == key && t < tid)) + (x.y > key || (x.y == key && t + 1 < tid)) +
                (x.z > key || (x.z == key && t + 2 < tid)) + (x.w > key || (x.w == key && t + 3 < tid));
    }
    for (int j = mine + 8; j < end; ++j) {
      const uint4 x = all[j];
      before += (x.x > key) + (x.y > key) + (x.z > key) + (x.w > key);
    }
    }
    const bool taken = tid < n && before < take;
    int tot;
    const int at = block_exclusive_scan(taken, sh_warp, &tot);
    if (taken) kept[at] = tid;
    return;
  }
  auto meet = [&]() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  const int share = (n + C - 1) / C, c0 = min(n, rank * share), c1 = min(n, c0 + share);
  const bool held = share <= kPickKeys * kPickThreads;
  uint32_t keys[kPickKeys];
  if (held) {
#pragma unroll
    for (int k = 0; k < kPickKeys; ++k) {
      const int t = c0 + k * kPickThreads + tid;
      keys[k] = t < c1 ? sum_key(__ldg(acc + t)) : 0u;
    }
  }
  uint32_t prefix = 0;
  int need = take;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11, nb = 1 << bits;
    for (int i = tid; i < nb; i += kPickThreads) sh_hist[i] = 0u;
    __syncthreads();
    const int top = shift + bits;
    auto count = [&](int t, uint32_t key) {
      if (t < c1 && (pass == 0 || (key >> top) == (prefix >> top))) atomicAdd(&sh_hist[(key >> shift) & (nb - 1)], 1u);
    };
    if (held) {
#pragma unroll
      for (int k = 0; k < kPickKeys; ++k) count(c0 + k * kPickThreads + tid, keys[k]);
    } else {
      constexpr int kLoads = 8;
      for (int t0 = c0; t0 < c1; t0 += kLoads * kPickThreads) {
        float x[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int t = t0 + k * kPickThreads + tid;
          x[k] = t < c1 ? __ldg(acc + t) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) count(t0 + k * kPickThreads + tid, sum_key(x[k]));
      }
    }
    meet();
    if (C > 1) {
      const int per = nb / C;  // C is a power of two up to 8
      for (int i = tid; i < per; i += kPickThreads) {
        uint32_t sum = 0;
#pragma unroll 4
        for (int r = 0; r < C; ++r) sum += cluster.map_shared_rank(sh_hist, r)[rank * per + i];
#pragma unroll 4
        for (int r = 0; r < C; ++r) cluster.map_shared_rank(sh_tot, r)[rank * per + i] = sum;
      }
      cluster.sync();
    }
    int above;
    const int bin = find_threshold_bin(C > 1 ? sh_tot : sh_hist, nb, need, &above, sh_warp, sh_res);
    prefix |= (uint32_t)bin << shift;
    need -= above;
  }
  // Keys above `prefix` are all taken, `need` of the equal ones from the front. Both counts go in one word: at most
  // 16,384 each of a share whose keys are held; a longer share counts its totals first and walks its positions again.
  const int warp = tid >> 5, lane = tid & 31;
  const uint32_t below = (1u << lane) - 1u;
  constexpr int kPickWarps = kPickThreads / 32;
  int tot_gt, tot_eq;
  if (held) {
#pragma unroll
    for (int k = 0; k < kPickKeys; ++k) {
      const bool in = c0 + k * kPickThreads + tid < c1;
      const uint32_t mg = __ballot_sync(0xffffffffu, in && keys[k] > prefix), me = __ballot_sync(0xffffffffu, in && keys[k] == prefix);
      if (lane == 0) sh_tot[k * kPickWarps + warp] = (uint32_t)(__popc(mg) | (__popc(me) << 16));
    }
    __syncthreads();
    int tot;
    const int x = tid < kPickKeys * kPickWarps ? (int)sh_tot[tid] : 0, before = block_exclusive_scan(x, sh_warp, &tot);
    if (tid < kPickKeys * kPickWarps) sh_tot[tid] = (uint32_t)before;
    tot_gt = tot & 0xffff;
    tot_eq = tot >> 16;
  } else {
    int gt = 0, eq = 0;
    for (int t = c0 + tid; t < c1; t += kPickThreads) {
      const uint32_t key = sum_key(__ldg(acc + t));
      gt += key > prefix;
      eq += key == prefix;
    }
    block_exclusive_scan(gt, sh_warp, &tot_gt);
    block_exclusive_scan(eq, sh_warp, &tot_eq);
  }
  if (tid < C) cluster.map_shared_rank(sh_counts, tid)[rank] = make_int2(tot_gt, tot_eq);
  meet();
  int gt0 = 0, eq0 = 0;
  for (int r = 0; r < rank; ++r) {
    gt0 += sh_counts[r].x;
    eq0 += sh_counts[r].y;
  }
  if (held) {
#pragma unroll
    for (int k = 0; k < kPickKeys; ++k) {
      const int t = c0 + k * kPickThreads + tid;
      const bool is_gt = t < c1 && keys[k] > prefix, is_eq = t < c1 && keys[k] == prefix;
      const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq), before = sh_tot[k * kPickWarps + warp];
      const int g = gt0 + (int)(before & 0xffffu) + __popc(mg & below), e = eq0 + (int)(before >> 16) + __popc(me & below);
      if (is_gt || (is_eq && e < need)) kept[g + min(e, need)] = t;
    }
    return;
  }
  // in position order: a warp takes 128 positions as 4 rounds of 32 lanes
  constexpr int kTile = kPickThreads * 4;
  for (int t0 = c0; t0 < c1; t0 += kTile) {
    uint32_t mg[4], me[4];
    int cg_ = 0, ce = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + warp * 128 + 32 * r + lane;
      const uint32_t key = t < c1 ? sum_key(__ldg(acc + t)) : 0u;
      mg[r] = __ballot_sync(0xffffffffu, t < c1 && key > prefix);
      me[r] = __ballot_sync(0xffffffffu, t < c1 && key == prefix);
      cg_ += __popc(mg[r]);
      ce += __popc(me[r]);
    }
    int tot;  // both counts in one scan: at most 4096 each
    const int scan = block_exclusive_scan(lane == 0 ? cg_ | (ce << 16) : 0, sh_warp, &tot);
    const int base = __shfl_sync(0xffffffffu, scan, 0);
    int g = gt0 + (base & 0xffff), e = eq0 + (base >> 16);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + warp * 128 + 32 * r + lane;
      const int ge = e + __popc(me[r] & below), gg = g + __popc(mg[r] & below);
      const bool is_eq = (me[r] >> lane) & 1u, is_gt = (mg[r] >> lane) & 1u;
      if (is_gt || (is_eq && ge < need)) kept[gg + min(ge, need)] = t;
      g += __popc(mg[r]);
      e += __popc(me[r]);
    }
    gt0 += tot & 0xffff;
    eq0 += tot >> 16;
  }
}

// ------------------------------------------------------------------ move
// Row kept[j] -> j of one unit, j ascending, in place: kept[j] >= j, so rows that
// are read in runs, each before it is written, are never overwritten unread.  A
// cluster of CTAs moves one unit's K rows (V rows, sums, scales), each a part of
// every run, whole rows each (32-byte columns of the same rows, a CTA each, took
// 110 us for halving 4 x 65,536 tokens: DRAM reads 64 bytes at a time); a cluster
// barrier stands between a run's reads and its writes.  Rows wait for their turn in
// a ring in shared memory, so some 100 KB per SM are on the way without a register.
// A row's two places are found once, by one thread, steps ahead of its copy.  Halving
// 4 x 65,536 tokens of 4 heads (bf16) takes 129 us with the selection, 4.2 TB/s; bound
// by the steps' latency, 1.2 us each.
constexpr int kMoveThreads = 256;
constexpr int kMoveRuns = 5;  // in the ring: one written, one awaited, three on the way
constexpr int kMoveRows = 256;  // rows of a CTA's part of a run, at most (8 loads of 32 rows: a head has 128 bytes or more)

template <int LOADS>
struct MoveRing {
  uint4 data[kMoveRuns][LOADS * kMoveThreads];
  int32_t from[2][kMoveRows];        // of the run that is copied next, and the one after it
  int32_t to[kMoveRuns][kMoveRows];  // -1: nothing moves
};

template <typename V>
__device__ __forceinline__ void copy_async(uint32_t dst, const V *src) {
  if constexpr (sizeof(V) == 16) cp_async_16(dst, src);
  else cp_async_4(dst, src);
}

// LOADS elements per thread and run; `lanes` elements per row
template <typename V, int LOADS, typename Ring>
__device__ __forceinline__ void move_rows(uint8_t *base, int64_t row_bytes, int lanes, int col, const int32_t *kept, int K,
                                          const EvictParams &p, int b, bool sums, Ring &ring) {
  cg::cluster_group cluster = cg::this_cluster();
  const int per = kMoveThreads / lanes, rows = per * LOADS, run = rows * (int)cluster.num_blocks();
  const int tid = threadIdx.x, r0 = tid / lanes, j_first = (int)cluster.block_rank() * rows;
  const int32_t *pt = p.page_table && !sums ? p.page_table + (int64_t)b * p.max_pages : nullptr;
  const uint32_t ps = (uint32_t)p.page_size;
  // This thread's row of a run: its kept position, then the page numbers of both places, are fetched a step before they
  // are looked at.
  int t_far = -1, t = -1, pg_from = 0, pg_to = 0;
  auto look = [&](int j0) {
    const int j = j0 + j_first + tid;
    t_far = tid < rows && j < K ? __ldcg(kept + j) : -1;
  };
  auto pages = [&](int j0) {
    const int j = j0 + j_first + tid;
    t = t_far == j ? -1 : t_far;
    if (pt && t >= 0) {
      pg_from = __ldg(pt + (uint32_t)t / ps);
      pg_to = __ldg(pt + (uint32_t)j / ps);
    }
  };
  auto places = [&](int j0, int at, int at2) {
    if (tid >= rows) return;
    int64_t from = t, to = j0 + j_first + tid;
    if (!sums && t >= 0) {
      from = pt ? (int64_t)pg_from * ps + (uint32_t)t % ps : (int64_t)b * ps + t;
      to = pt ? (int64_t)pg_to * ps + (uint32_t)to % ps : (int64_t)b * ps + to;
      if (from < 0 || from >= p.num_slots || to < 0 || to >= p.num_slots) to = -1;
    }
    ring.from[at2][tid] = (int32_t)from;
    ring.to[at][tid] = t >= 0 ? (int32_t)to : -1;
  };
  V *data = reinterpret_cast<V *>(ring.data);
  auto fetch = [&](int at, int at2) {
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int r = k * per + r0;
      if (ring.to[at][r] >= 0)
        copy_async(smem_u32(data + (at * LOADS + k) * kMoveThreads + tid),
                   reinterpret_cast<const V *>(base + ring.from[at2][r] * row_bytes + col));
    }
    cp_async_commit();
  };
  auto write = [&](int at) {
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int to = ring.to[at][k * per + r0];
      if (to >= 0) *reinterpret_cast<V *>(base + to * row_bytes + col) = data[(at * LOADS + k) * kMoveThreads + tid];
    }
  };
  {  // places of runs 0 to 3, copies of runs 0 to 2: all of a kind at once
    int kept_of[kMoveRuns + 1], from_of[kMoveRuns], to_of[kMoveRuns];
#pragma unroll
    for (int i = 0; i <= kMoveRuns; ++i) {
      look(i * run);
      kept_of[i] = t_far;
    }
#pragma unroll
    for (int i = 0; i < kMoveRuns; ++i) {
      t_far = kept_of[i];
      pages(i * run);
      from_of[i] = pg_from, to_of[i] = pg_to;
    }
#pragma unroll
    for (int i = 0; i < kMoveRuns - 1; ++i) {
      const int j = i * run + j_first + tid;
      t = kept_of[i] == j ? -1 : kept_of[i];
      pg_from = from_of[i], pg_to = to_of[i];
      places(i * run, i, i & 1);
      __syncthreads();
      if (i < kMoveRuns - 2) fetch(i, i & 1);
    }
    const int j = (kMoveRuns - 1) * run + j_first + tid;
    t = kept_of[kMoveRuns - 1] == j ? -1 : kept_of[kMoveRuns - 1];
    pg_from = from_of[kMoveRuns - 1], pg_to = to_of[kMoveRuns - 1];
    t_far = kept_of[kMoveRuns];
  }
  int at = 0, i = 0;  // the run that is awaited: its place, its number
  for (int j0 = 0; j0 < K; j0 += run, ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kMoveRuns - 3) : "memory");
    if (j0 > 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // This CTA's part of the run is read: it is in shared memory, so the barrier has nothing to order (a release would
    // wait for the last run's writes, 1.5 us a step).
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int before = at == 0 ? kMoveRuns - 1 : at - 1, next = at < 2 ? at + 3 : at - 2;  // runs i - 1 and i + 3
    if (j0 > 0) write(before);
    __syncthreads();  // run i + 3's places are there, and run i - 1 has left its own: run i + 4's
    fetch(next, (i + 3) & 1);
    places(j0 + (kMoveRuns - 1) * run, before, i & 1);
    pages(j0 + kMoveRuns * run);
    look(j0 + (kMoveRuns + 1) * run);
    at = at == kMoveRuns - 1 ? 0 : at + 1;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  write(at == 0 ? kMoveRuns - 1 : at - 1);
  cp_async_wait_all();
}
template <int LOADS>
__global__ void __launch_bounds__(kMoveThreads, 2) move_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint8_t move_smem[];
  MoveRing<LOADS> &move_ring = *reinterpret_cast<MoveRing<LOADS> *>(move_smem);
  griddep_wait();
  griddep_launch_dependents();
  const int u = blockIdx.x / (int)cg::this_cluster().num_blocks(), b = u / p.Hkv, kvh = u % p.Hkv, job = blockIdx.y;
  const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
  if (T <= p.budget) return;  // the same for the cluster
  const int32_t *kept = p.kept + (int64_t)u * p.budget;
  const int64_t row_bytes = (int64_t)p.Hkv * p.head_bytes;
  if (job < 2) {
    const int lanes = p.head_bytes / 16;
    move_rows<uint4, LOADS>(static_cast<uint8_t *>(job == 0 ? p.k : p.v), row_bytes, lanes, kvh * p.head_bytes + (threadIdx.x % lanes) * 16,
                     kept, p.budget, p, b, false, move_ring);
  } else if (job == 2) {
    move_rows<float, 1>(reinterpret_cast<uint8_t *>(p.acc + (int64_t)u * p.acc_stride), 4, 1, 0, kept, p.budget, p, b, true, move_ring);
  } else {
    move_rows<float, 1>(reinterpret_cast<uint8_t *>(job == 3 ? p.k_scale : p.v_scale), (int64_t)p.Hkv * 4, 1, kvh * 4, kept, p.budget,
                     p, b, false, move_ring);
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptParams &p, bool scales, cudaStream_t s) {
  const int jobs = 2 * ((p.row_bytes + kAcceptCols - 1) / kAcceptCols) +
                   (scales ? (p.Hkv + kAcceptScaleHeads - 1) / kAcceptScaleHeads : 0);
  return launch_ex(accept_kernel, dim3(jobs, p.B), dim3(kAcceptThreads), 0, s, 0, p);
}

cudaError_t launch_evict(const EvictParams &p0, bool scales, int sms, cudaStream_t s) {
  EvictParams p = p0;
  const int units = p.B * p.Hkv;
  int C = 1;  // shares of at least 2,048 positions, and no more CTAs than SMs
  while (C < 8 && p.t_cap > (int64_t)C * 4096 && (int64_t)units * C * 2 <= sms) C *= 2;
  cudaError_t e;
  // 16 positions per thread: two CTAs of 512 threads per SM for short sequences
  e = p.t_cap <= 512 * kPickKeys ? launch_ex(pick_kernel<512>, dim3((unsigned)(units * C)), dim3(512), 0, s, C, p)
                                 : launch_ex(pick_kernel<1024>, dim3((unsigned)(units * C)), dim3(1024), 0, s, C, p);
  if (e != cudaSuccess) return e;
  // CTAs per unit and job: no more for K's and V's rows than fit beside each other (two
  // per SM), and a run of theirs (at least 32 rows each) no longer than the budget.  The
  // jobs of the sums and scales come behind in the grid and take places that are left or
  // become free, in rings of the rows' size: 24 sequences of 4 heads in E4M3 launch 480 CTAs
  // on 296 places.
  C = 1;
  const int jobs = scales ? 5 : 3;
  while (C < 8 && (int64_t)units * 2 * C * 2 <= 2 * sms && p.budget > C * 64) C *= 2;
  auto move = [&](auto kern, size_t bytes) {
    const cudaError_t err = set_smem_once(reinterpret_cast<const void *>(kern), (int)bytes);
    return err != cudaSuccess ? err : launch_ex(kern, dim3((unsigned)(units * C), jobs), dim3(kMoveThreads), bytes, s, C, p);
  };
  // Where one CTA per SM is enough for K and V, twice the rows per step: a step takes 1.2 us whatever it moves.
  if ((int64_t)units * 2 * C <= sms) return move(move_kernel<8>, sizeof(MoveRing<8>));
  return move(move_kernel<4>, sizeof(MoveRing<4>));
}

}  // namespace hs2
