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
// latency: two dependent loads (page table, row) and a store.
constexpr int kAcceptThreads = 256;
constexpr int kAcceptCols = 256;  // bytes of a row per CTA: 16 threads x 16 bytes
constexpr int kAcceptRounds = kMaxDraft * kAcceptCols / 16 / kAcceptThreads;

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams p) {
  __shared__ int64_t sh_src[kMaxDraft], sh_dst[kMaxDraft];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, job = blockIdx.x;
  const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
  const int n = clamp_len(p.num_draft ? __ldg(p.num_draft + b) : p.M, min(min(p.M, kMaxDraft), T));
  const int a = clamp_len(__ldg(p.path_len + b), n);
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
// takes equal shares of the positions: three radix passes (11, 11, 10 bits of
// an order-preserving key; histograms in shared memory, added over the cluster
// through distributed shared memory) find the exact key of the last one taken,
// then each share writes its positions behind the earlier shares' counts.
// Bound by reading the sums four times from L2 and by nine cluster barriers.
constexpr int kPickThreads = 512;
constexpr int kPickBins = 2048;

__device__ __forceinline__ uint32_t sum_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  if (x == 0.f) return 0x80000000u;  // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const EvictParams p) {
  __shared__ uint32_t sh_hist[kPickBins], sh_tot[kPickBins];
  __shared__ int sh_warp[33], sh_res[2], sh_found[2];
  __shared__ int2 sh_counts[16];
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
  const int share = (n + C - 1) / C, c0 = min(n, rank * share), c1 = min(n, c0 + share);
  uint32_t prefix = 0;
  int need = take;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11, nb = 1 << bits;
    for (int i = tid; i < nb; i += kPickThreads) sh_hist[i] = 0u;
    __syncthreads();
    const int top = shift + bits;
    constexpr int kLoads = 8;
    for (int t0 = c0; t0 < c1; t0 += kLoads * kPickThreads) {
      float x[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int t = t0 + k * kPickThreads + tid;
        x[k] = t < c1 ? __ldg(acc + t) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const uint32_t key = sum_key(x[k]);
        const bool in = t0 + k * kPickThreads + tid < c1 && (pass == 0 || (key >> top) == (prefix >> top));
        const uint32_t bin = (key >> shift) & (nb - 1);
        // many sums are equal (zeros): one add per warp and bin
        const uint32_t peers = __match_any_sync(0xffffffffu, in ? bin : 0xffffffffu);
        if (in && (tid & 31) == __ffs(peers) - 1) atomicAdd(&sh_hist[bin], (uint32_t)__popc(peers));
      }
    }
    cluster.sync();
    const int per = nb / C;  // C is a power of two up to 16
    for (int i = tid; i < per; i += kPickThreads) {
      uint32_t s = 0;
      for (int r = 0; r < C; ++r) s += cluster.map_shared_rank(sh_hist, r)[rank * per + i];
      cluster.map_shared_rank(sh_tot, 0)[rank * per + i] = s;
    }
    cluster.sync();
    if (rank == 0) {
      int above;
      const int bin = find_threshold_bin(sh_tot, nb, need, &above, sh_warp, sh_res);
      if (tid < C) {
        int *f = cluster.map_shared_rank(sh_found, tid);
        f[0] = bin;
        f[1] = above;
      }
    }
    cluster.sync();
    prefix |= (uint32_t)sh_found[0] << shift;
    need -= sh_found[1];
  }
  // keys above `prefix` are all taken, `need` of the equal ones from the front
  int gt = 0, eq = 0;
  for (int t = c0 + tid; t < c1; t += kPickThreads) {
    const uint32_t key = sum_key(__ldg(acc + t));
    gt += key > prefix;
    eq += key == prefix;
  }
  int tot_gt, tot_eq;
  block_exclusive_scan(gt, sh_warp, &tot_gt);
  block_exclusive_scan(eq, sh_warp, &tot_eq);
  if (tid < C) cluster.map_shared_rank(sh_counts, tid)[rank] = make_int2(tot_gt, tot_eq);
  cluster.sync();
  int gt0 = 0, eq0 = 0;
  for (int r = 0; r < rank; ++r) {
    gt0 += sh_counts[r].x;
    eq0 += sh_counts[r].y;
  }
  // in position order: a warp takes 128 positions as 4 rounds of 32 lanes
  constexpr int kTile = kPickThreads * 4;
  const int warp = tid >> 5, lane = tid & 31;
  const uint32_t below = (1u << lane) - 1u;
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
    int tot;  // both counts in one scan: at most 2048 each
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
// Row kept[j] -> j of one unit, j ascending, in place: kept[j] >= j, so a CTA
// that reads a run of rows before it writes them never overwrites a row that
// is still to be read.  The rows cannot be dealt over CTAs without such an
// order between them, but a row's columns can: a CTA owns `cols` bytes of one
// unit's K or V rows (or its sums, or its scales) and walks all of them.
constexpr int kMoveThreads = 512;
constexpr int kMoveLoads = 4;

template <typename V>
__device__ __forceinline__ void move_rows(uint8_t *base, int64_t row_bytes, int lanes, int col, const int32_t *kept, int K,
                                          const EvictParams &p, int b, bool sums) {
  const int per = kMoveThreads / lanes, tile = per * kMoveLoads;  // rows per round of loads, per tile
  const int r0 = threadIdx.x / lanes;
  for (int j0 = 0; j0 < K; j0 += tile) {
    V x[kMoveLoads];
    int64_t dst[kMoveLoads];
#pragma unroll
    for (int k = 0; k < kMoveLoads; ++k) {
      const int j = j0 + k * per + r0;
      dst[k] = -1;
      if (j < K) {
        const int t = __ldcg(kept + j);
        if (t != j) {
          const int64_t from = sums ? t : evict_slot(p.page_table, p.max_pages, p.page_size, p.num_slots, b, t);
          const int64_t to = sums ? j : evict_slot(p.page_table, p.max_pages, p.page_size, p.num_slots, b, j);
          if (from >= 0 && to >= 0) {
            x[k] = __ldcg(reinterpret_cast<const V *>(base + from * row_bytes + col));
            dst[k] = to;
          }
        }
      }
    }
    __syncthreads();  // every row of the tile is read
#pragma unroll
    for (int k = 0; k < kMoveLoads; ++k)
      if (dst[k] >= 0) *reinterpret_cast<V *>(base + dst[k] * row_bytes + col) = x[k];
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int u = blockIdx.x, b = u / p.Hkv, kvh = u % p.Hkv;
  const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
  if (T <= p.budget) return;
  const int32_t *kept = p.kept + (int64_t)u * p.budget;
  const int chunks = p.head_bytes / p.cols, job = blockIdx.y;
  if (job < 2 * chunks) {
    uint8_t *x = static_cast<uint8_t *>(job < chunks ? p.k : p.v);
    const int lanes = p.cols / 16;
    move_rows<uint4>(x, (int64_t)p.Hkv * p.head_bytes, lanes,
                     kvh * p.head_bytes + (job % chunks) * p.cols + (threadIdx.x % lanes) * 16, kept, p.budget, p, b, false);
  } else if (job == 2 * chunks) {
    move_rows<float>(reinterpret_cast<uint8_t *>(p.acc + (int64_t)u * p.acc_stride), 4, 1, 0, kept, p.budget, p, b, true);
  } else {
    move_rows<float>(reinterpret_cast<uint8_t *>(job == 2 * chunks + 1 ? p.k_scale : p.v_scale), (int64_t)p.Hkv * 4, 1,
                     kvh * 4, kept, p.budget, p, b, false);
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
  int C = 1;  // shares of at least 2,048 positions, and no more CTAs than fit beside each other
  while (C < 16 && p.t_cap > (int64_t)C * 4096 && (int64_t)units * C * 2 <= 4 * sms) C *= 2;
  cudaError_t e;
  if (C > 8 && (e = allow_wide_clusters_once(reinterpret_cast<const void *>(pick_kernel))) != cudaSuccess) return e;
  e = launch_ex(pick_kernel, dim3((unsigned)(units * C)), dim3(kPickThreads), 0, s, C, p);
  if (e != cudaSuccess) return e;
  // columns per CTA: whole rows when the units alone fill the GPU, down to a
  // 32-byte sector when there are few
  p.cols = p.head_bytes;
  while (p.cols > 32 && (int64_t)units * 2 * (p.head_bytes / p.cols) < 2 * sms) p.cols /= 2;
  const int jobs = 2 * (p.head_bytes / p.cols) + 1 + (scales ? 2 : 0);
  return launch_ex(move_kernel, dim3((unsigned)units, jobs), dim3(kMoveThreads), 0, s, 0, p);
}

}  // namespace hs2
