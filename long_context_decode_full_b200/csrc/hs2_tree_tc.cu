// hs2_tree_tc.cu -- attention of a tree of drafted tokens over a bf16 or E4M3
// cache on the tensor cores (tcgen05, accumulators in tensor memory).
//
// A CTA walks the tiles of its share (hs2_tree_common.cuh) with two streams, a
// warpgroup each, a thread per query row.  Stream s holds 128 logits columns
// S_s and D output columns O_s of tensor memory and repeats, per tile of 128
// positions,
//   S_s = Q_s K^T                       (tcgen05.mma, Q and K in shared memory)
//   P_s = 2^(c2 S_s - m), l += sum P_s  (registers; P_s as bf16 over S_s's columns)
//   O_s += P_s V                        (tcgen05.mma, P from tensor memory).
// While one stream's warpgroup is at its exponentials the tensor cores work for
// the other.  A block of more than 128 rows gives each stream 128 of them, and
// both take every tile; with 128 rows or fewer both hold the same rows and take
// every other tile, so a memory-bound call has two warpgroups at work, too; the
// joining kernel adds their sums.
//
// m moves only when a row's maximum passes it by more than 8 (in base-2
// exponents): weights stay below 2^8, which bf16 and fp32 sums hold as well as
// weights below 1, and O_s is rescaled a few times per unit instead of per tile.
//
// E4M3 caches.  S_s uses the codes as they are: the query row, scaled by a power
// of two to at most 448, is split into two E4M3 terms hi + lo (a bf16 value has
// 8 significand bits, each term holds 4, and the remainder of rounding to 4 bits
// fits the other 4), so S_s = hi K^T + lo K^T at E4M3's double rate costs what one
// bf16 product does; below 2^-6 of E4M3's range the terms are off by 2^-10 of it.
// The key's scale multiplies the logit.  V's codes are converted to bf16 (exact)
// by a warpgroup of its own, and its scale joins the weight before it is rounded.
//
// Roles: warps 0-3 and 4-7 the streams, 8-11 the values (conversion, and rows
// that must not be multiplied, below), 12 the TMA loads, 13 the MMA issue.
//
// Rows of V that a query row must not see, whatever they hold: weight 0 times
// NaN is NaN in a matrix product, so the values warpgroup clears the rows behind
// the sequence, and drafts' rows with a non-finite element; the latter are added
// to the rows that do see them one by one (add_bad_rows).
#include <type_traits>

#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_tc.cuh"
#include "hs2_tree_common.cuh"

namespace hs2 {

namespace {

constexpr int kKeys = 128;       // positions per tile
constexpr int kStreamRows = 128;
constexpr int kThreads = 512;
constexpr int kTmemCols = 512;
// 65,536 registers: 2 x 128 threads x 200 and 2 x 128 x 56
constexpr int kRegsStream = 200, kRegsOther = 56;
constexpr float kMaxGrowth = 8.f;

template <int D, bool FP8>
struct TreeTc {
  static constexpr int kQ = FP8 ? 2 * kStreamRows * D : kStreamRows * D * 2;  // a stream's query
  static constexpr int kTile = kKeys * D * (FP8 ? 1 : 2);                     // a K or V tile as it is in the cache
  static constexpr int kVals = FP8 ? kKeys * D * 2 : 0;                       // a converted V tile
  static constexpr int kPanel = kKeys * 128;                                  // 128 bytes of every row
  static constexpr int kPanels = kTile / kPanel;
  static constexpr int kStages = FP8 ? 5 : (D == 128 ? 5 : 8);
  static constexpr size_t oStage = 2 * kQ, oVals = oStage + (size_t)kStages * kTile, oScale = oVals + 2 * kVals,
                          oBar = oScale + (FP8 ? 2 * 2 * kKeys * 4 : 0);
  // full[S], empty[S], q_full[2], s_full[2], p_full[2], o_full[2], v_ready[2], v_free[2], scale_full[2], v_landed[2], done
  static constexpr int kBars = 2 * kStages + 17;
  static constexpr size_t oBad = oBar + (size_t)((kBars * 8 + 15) / 16 * 16), oInfo = oBad + 16, kBytes = oInfo + 64 + 1024;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

struct TreeInfo {       // shared
  int64_t total, base;  // tiles; tiles before sequence b0
  int32_t b0;           // the sequence in which the share begins
  uint32_t tmem;
  int32_t abort;
};

// One unit's part in a share.
struct TreeSeg {
  int b, kvh, i0, i1, T, n, first, nr;
  bool pair, begins, whole;
};

struct TreeWalk {
  int64_t g, g0, g1, base;
  int b;
  __device__ __forceinline__ TreeWalk(const TreeInfo &in, const TreeShare &share, int64_t group)
      : g(share.start(group)), g0(g), g1(share.start(group + 1)), base(in.base), b(in.b0) {}
  // The next segment that has rows for this CTA.
  __device__ __forceinline__ bool next(const TreeParams &p, int block, TreeSeg &s) {
    while (g < g1 && b < p.B) {
      s.T = tree_len(p, b);
      const int nb = (s.T + kKeys - 1) / kKeys;
      const int64_t r = g - base;
      if (r >= (int64_t)p.Hkv * nb) {
        base += (int64_t)p.Hkv * nb;
        ++b;
        continue;
      }
      s.b = b;
      s.kvh = (int)(r / nb);
      s.i0 = (int)(r % nb);
      s.i1 = (int)min((int64_t)nb, s.i0 + (g1 - g));
      s.n = tree_drafts(p, b, s.T);
      s.first = s.T - s.n;
      s.begins = g == g0;
      s.whole = s.i0 == 0 && s.i1 == nb;
      g += s.i1 - s.i0;
      s.nr = min(2 * kStreamRows, s.n * p.G - block * 2 * kStreamRows);
      s.pair = s.nr > kStreamRows;
      if (s.nr > 0) return true;
    }
    return false;
  }
};

// The loads of a segment: K of the first `ahead` tiles, then V of tile i and K of
// tile i + ahead; and the stages that hold them.  bf16: one ring in this order.
// E4M3: a ring for K (3 stages) and one for V (2), because the values warpgroup
// waits for V alone, and a waiter that misses a stage's phases cannot tell them apart.
template <bool FP8, int S>
struct TreeOrder {
  int nt, ahead;
  uint32_t before;  // tiles of the CTA's earlier segments
  __device__ __forceinline__ TreeOrder(const TreeSeg &s, uint32_t tiles)
      : nt(s.i1 - s.i0), ahead(min(s.pair ? 1 : 2, nt)), before(tiles) {}
  struct Place {
    uint32_t stage, parity;
  };
  __device__ __forceinline__ Place v(int i) const {
    if constexpr (FP8) return {3u + ((before + i) & 1u), ((before + i) >> 1) & 1u};
    const uint32_t at = 2 * before + ahead + i + min(i, nt - ahead);
    return {at % S, (at / S) & 1u};
  }
  __device__ __forceinline__ Place k(int i) const {
    if constexpr (FP8) return {(before + i) % 3u, ((before + i) / 3u) & 1u};
    const uint32_t at = 2 * before + (i < ahead ? i : i + 1 + min(i - ahead, nt - ahead));
    return {at % S, (at / S) & 1u};
  }
};

__device__ __forceinline__ void wait_or_abort(uint64_t *bar, uint32_t parity, volatile int32_t *abort, uint32_t *err,
                                              uint32_t bit) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (*abort) return;
    if (clock64() - t0 > kSpinLimitCycles) {
      *abort = 1;
      set_error(err, bit);
      return;
    }
  }
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// one column of this thread's lane
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr) : "memory");
  return r;
}
// 32 columns of packed weights
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B with A (bf16) in tensor memory
__device__ __forceinline__ void mma_ts_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(1u)
      : "memory");
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

// the drafts' bits of 64 columns of a tile, the first draft at column r
__device__ __forceinline__ uint64_t shift_bits(uint64_t bits, int r) {
  return r >= 64 ? 0ull : (r >= 0 ? bits << r : (r > -64 ? bits >> -r : 0ull));
}
// columns before r of 64
__device__ __forceinline__ uint64_t below(int r) { return r >= 64 ? ~0ull : (r <= 0 ? 0ull : (1ull << r) - 1ull); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// two E4M3 codes of four to bf16 pairs (exact)
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  uint32_t a, b;
  e4m3x4_to_f16x2x2(w, a, b);
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  const float2 fx = __half22float2(x), fy = __half22float2(y);
  lo = pack_bf16(fx.x, fx.y);
  hi = pack_bf16(fy.x, fy.y);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const TreeParams p) {
  using C = TreeTc<D, FP8>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::oBar);
  uint64_t *full = bars, *empty = bars + S, *q_full = bars + 2 * S, *s_full = q_full + 2, *p_full = q_full + 4,
           *o_full = q_full + 6, *v_ready = q_full + 8, *v_free = q_full + 10, *scale_full = q_full + 12, *v_landed = q_full + 14, *done = q_full + 16;
  volatile uint64_t *bad_rows = reinterpret_cast<volatile uint64_t *>(smem + C::oBad);
  TreeInfo *info = reinterpret_cast<TreeInfo *>(smem + C::oInfo);
  volatile int32_t *abort = &info->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int block = blockIdx.x % p.blocks;
  const int64_t group = blockIdx.x / p.blocks;
  if (tid == 0) {
    for (int i = 0; i < C::kBars; ++i) mbar_init(bars + i, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 4);
      mbar_init(p_full + s, 4);
      mbar_init(scale_full + s, 128);
    }
    fence_mbar_init();
    info->abort = 0;
    info->total = 0;
  }
  if (warp == 12 && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {  // the tiles of all sequences, then the sequence where the share begins
    int64_t total = 0;
    for (int b = lane; b < p.B; b += 32) total += (tree_len(p, b) + kKeys - 1) / kKeys;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.Hkv;
    if (total > 0) {
      const TreeShare share{total, p.groups};
      const int64_t g0 = share.start(group);
      int64_t carry = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int64_t x = b0 + lane < p.B ? (int64_t)p.Hkv * ((tree_len(p, b0 + lane) + kKeys - 1) / kKeys) : 0;
        int64_t sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        sum += carry;
        if (sum - x <= g0 && g0 < sum) {  // one lane of one round, if the share is not empty
          info->base = sum - x;
          info->b0 = b0 + lane;
        }
        carry = __shfl_sync(0xffffffffu, sum, 31);
        if (carry > g0) break;
      }
      if (lane == 0) info->total = share.start(group + 1) > g0 ? total : 0;
    }
    if (blockIdx.x == 0) tree_prefix(p, p.prefix);
  }
  __syncthreads();
  if (info->total == 0) return;  // no tiles for this CTA
  if (warp == 13) {
    tc::tmem_alloc(&info->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = info->tmem;
  const TreeShare share{info->total, p.groups};
  TreeWalk walk(*info, share, group);
  TreeSeg seg;
  const int wg = warp >> 2;

  if (wg < 2) {
    // ------------------------------------------------------------ a stream
    regs_inc<kRegsStream>();
    const int s = wg, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + (uint32_t)(s * kKeys), to = tmem + lanes + 256u + (uint32_t)(s * D);
    uint8_t *sq = smem + s * C::kQ;
    uint32_t ns = 0, handled0 = 0;  // tiles of this stream; tiles handled by the values warpgroup before the segment
    while (walk.next(p, block, seg)) {
      const int nt = seg.i1 - seg.i0;
      const int special0 = max(seg.i0, min(seg.i1, seg.first / kKeys));  // first tile with a draft (or the tail)
      const uint32_t handled_here = FP8 ? nt : seg.i1 - special0;
      if (!seg.pair && s >= nt) {  // one tile: the other stream has it
        handled0 += handled_here;
        continue;
      }
      const int r = block * 2 * kStreamRows + (seg.pair ? s * kStreamRows : 0) + row;
      const bool mine = r < seg.n * p.G, busy = __any_sync(0xffffffffu, mine);
      const int tok = r / p.G, head = seg.kvh * p.G + r % p.G;
      const uint64_t bits = mine ? tree_bits(p, seg.b, tok, seg.n) : 0ull;
      float c2 = p.c2;
      // the query row to shared memory, 128-byte swizzle
      if (mine) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                           ((int64_t)seg.b * p.N + tok) * p.q_stride + (int64_t)head * D);
        uint4 x[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = __ldg(src + c);
        if constexpr (!FP8) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4 *>(sq + (c >> 3) * (kStreamRows * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[c];
        } else {
          float top = 0.f;
          bool finite = true;
          const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
#pragma unroll
          for (int e = 0; e < D / 2; ++e) {
            const float a = fabsf(bf16_lo(w[e])), b = fabsf(bf16_hi(w[e]));
            top = fmaxf(top, fmaxf(a, b));
            finite = finite && a <= 3.4e38f && b <= 3.4e38f;
          }
          // the largest power of two that takes the row to at most 448
          const uint32_t tb = __float_as_uint(top);
          const int k = min(126, 8 + 127 - (int)(tb >> 23) - ((tb & 0x7FFFFFu) > 0x600000u));
          const float up = __uint_as_float((uint32_t)(k + 127) << 23);
          c2 = finite ? p.c2 * __uint_as_float((uint32_t)(127 - k) << 23) : __int_as_float(0x7FC00000);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {  // 16 codes of each term
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              hi[e] = lo[e] = 0;
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const uint32_t u = w[8 * c + 2 * e + f];
                const float2 v = make_float2(bf16_lo(u) * up, bf16_hi(u) * up);
                const uint32_t h = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
                const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
                const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(v.x - back.x, v.y - back.y), __NV_SATFINITE, __NV_E4M3);
                hi[e] |= h << (16 * f);
                lo[e] |= l << (16 * f);
              }
            }
            uint8_t *dst = sq + row * 128 + ((c ^ (row & 7)) << 4);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(dst + kStreamRows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      __syncwarp();
      {
        const float zero[32] = {};
#pragma unroll
        for (int c = 0; c < D; c += 32) tc::st32(to + c, zero);
      }
      tc::fence_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + s);

      const float growth = kMaxGrowth / c2;
      float m = -INFINITY, l = 0.f;
      bool first_tile = true;
      for (int i = seg.pair ? 0 : s; i < nt; i += seg.pair ? 1 : 2) {
        const int t0 = (seg.i0 + i) * kKeys;
        const bool special = seg.i0 + i >= special0;
        const uint32_t hc = handled0 + (FP8 ? i : seg.i0 + i - special0);  // this tile among the handled ones
        wait_or_abort(s_full + s, ns & 1, abort, p.err, kErrFullWait);
        tc::fence_after();
        if (FP8) wait_or_abort(scale_full + (hc & 1), (hc >> 1) & 1, abort, p.err, kErrFullWait);
        if (special) wait_or_abort(v_ready + (hc & 1), (hc >> 1) & 1, abort, p.err, kErrFullWait);
        if (busy) {
          float x[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::ld32(ts + 32 * c, x[c]);
          const float *ks = reinterpret_cast<const float *>(smem + C::oScale) + (hc & 1) * 2 * kKeys, *vs = ks + kKeys;
          if constexpr (FP8) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(ks + 32 * c + e);
                x[c][e] *= f.x, x[c][e + 1] *= f.y, x[c][e + 2] *= f.z, x[c][e + 3] *= f.w;
              }
          }
          uint64_t seen[2] = {~0ull, ~0ull};
          if (special) {
            const int rel = seg.first - t0;
            seen[0] = below(rel) | shift_bits(bits, rel);
            seen[1] = below(rel - 64) | shift_bits(bits, rel - 64);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w = (uint32_t)(seen[c >> 1] >> (32 * (c & 1)));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((w >> e) & 1u)) x[c][e] = -INFINITY;
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = x[c][0];
#pragma unroll
            for (int e = 1; e < 32; ++e) mx[c] = fmaxf(mx[c], x[c][e]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool grow = m == -INFINITY ? top > -INFINITY : top > m + growth;
          const uint64_t bad = special ? bad_rows[hc & 1] : 0ull;
          if (__any_sync(0xffffffffu, grow) || bad) {
            float alpha = 1.f;
            if (grow) {
              alpha = m == -INFINITY ? 0.f : ex2_approx((m - top) * c2);
              m = top;
              l *= alpha;
            }
            __syncwarp();
            if (!first_tile) {
              wait_or_abort(o_full + s, (ns - 1) & 1, abort, p.err, kErrFullWait);  // the last product is in O
              tc::fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tc::ld32(to + c, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                tc::st32(to + c, o);
              }
            }
          }
          const float shift = m == -INFINITY ? 0.f : -m * c2;  // nothing seen yet: weights 0
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float a = ex2_approx(fmaf(x[2 * h + (e >> 5)][e & 31], c2, shift));
              float b = ex2_approx(fmaf(x[2 * h + (e >> 5)][(e & 31) + 1], c2, shift));
              sum[(e >> 1) & 3] += a + b;
              if constexpr (FP8) {
                const float2 f = *reinterpret_cast<const float2 *>(vs + 64 * h + e);
                a *= f.x, b *= f.y;
                if (special) {  // a scale that is not seen may be anything
                  a = (seen[h] >> e) & 1ull ? a : 0.f;
                  b = (seen[h] >> (e + 1)) & 1ull ? b : 0.f;
                }
              }
              w[e >> 1] = pack_bf16(a, b);
            }
            tmem_st32(ts + 32 * h, w);
          }
          tmem_wait_st();
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          if (bad) {  // rare: drafts whose values are not finite, for the rows that see them
            for (uint64_t rest = bad; rest; rest &= rest - 1) {
              const int j = __ffsll((long long)rest) - 1, c = seg.first + j - t0;
              const uint32_t pw = tmem_ld1(ts + (c >> 1));
              const float w = c & 1 ? bf16_hi(pw) : bf16_lo(pw);
              const bool sees = (bits >> j) & 1ull;
              const int64_t slot = tree_slot(p, seg.b, seg.first + j);
              const int64_t at = (slot * p.Hkv + seg.kvh) * D;
              if (slot < 0) continue;  // the same for the warp
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                float o[32];
                tc::ld32(to + d, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  float v;
                  if constexpr (FP8) {
                    const __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p.v)[at + d + e], __NV_E4M3);
                    v = __half2float(*reinterpret_cast<const __half *>(&hr));
                  } else {
                    v = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.v)[at + d + e]);
                  }
                  if (sees) o[e] = fmaf(w, v, o[e]);
                }
                tc::st32(to + d, o);
              }
            }
          }
          tc::fence_before();
        }
        first_tile = false;
        ++ns;
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + s);
      }
      handled0 += handled_here;
      wait_or_abort(o_full + s, (ns - 1) & 1, abort, p.err, kErrFullWait);
      tc::fence_after();
      if (busy) {
        const bool direct = seg.whole && (seg.pair || nt == 1);
        float *rec = tree_record(p, group, seg.begins ? 0 : 1, block, s);
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // nothing seen: zeros
        if (mine && !direct) {
          rec[row] = m * c2;
          rec[kStreamRows + row] = l;
        }
        __syncwarp();
        float4 *ro = reinterpret_cast<float4 *>(rec + 2 * kStreamRows) + row;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                               ((int64_t)seg.b * p.N + tok) * p.out_stride + (int64_t)head * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tc::ld32(to + c, o);
          if (mine && direct) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              dst[(c + e) / 8] = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                            pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              ro[(size_t)((c + e) / 4) * kStreamRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
    }
  } else if (wg == 2) {
    // ------------------------------------------------------------ values
    regs_dec<kRegsOther>();
    const int r = tid & 127;
    uint32_t tiles = 0, hc = 0;
    while (walk.next(p, block, seg)) {
      const TreeOrder<FP8, S> order(seg, tiles);
      const int special0 = max(seg.i0, min(seg.i1, seg.first / kKeys));
      for (int i = FP8 ? 0 : special0 - seg.i0; i < order.nt; ++i, ++hc) {
        const int t = (seg.i0 + i) * kKeys + r, slot_id = hc & 1;
        const bool live = t < seg.T;
        const auto at = order.v(i);
        const bool special = seg.i0 + i >= special0;
        float ks = 0.f, vs = 0.f;
        if constexpr (FP8) {
          const int64_t slot = live ? tree_slot(p, seg.b, t) : -1;
          if (slot >= 0) {
            ks = __ldg(p.k_scale + slot * p.Hkv + seg.kvh);
            vs = __ldg(p.v_scale + slot * p.Hkv + seg.kvh);
          }
        }
        wait_or_abort(v_free + slot_id, ((hc >> 1) & 1) ^ 1, abort, p.err, kErrEmptyWait);
        if (r == 0) bad_rows[slot_id] = 0ull;
        if constexpr (FP8) {
          float *sc = reinterpret_cast<float *>(smem + C::oScale) + slot_id * 2 * kKeys;
          sc[r] = ks;
          sc[kKeys + r] = vs;
          mbar_arrive(scale_full + slot_id);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!FP8) wait_or_abort(v_landed + slot_id, (hc >> 1) & 1, abort, p.err, kErrFullWait);
        wait_or_abort(full + at.stage, at.parity, abort, p.err, kErrFullWait);
        uint8_t *tile = smem + C::oStage + (size_t)at.stage * C::kTile;
        bool clear = !live, bad = false;
        const bool draft = live && t >= seg.first;
        if constexpr (FP8) {
          uint8_t *vals = smem + C::oVals + (size_t)slot_id * C::kVals;
          if (special && draft) {
            for (int c = 0; c < 8; ++c) {
              uint32_t w[4];
              lds128(w, smem_u32(tile) + r * 128 + c * 16);
#pragma unroll
              for (int e = 0; e < 4; ++e)  // a byte of 0x7F but for the sign: NaN
                bad = bad || __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
            }
          }
          clear = clear || bad;
#pragma unroll 2
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4], o[8];
            lds128(w, smem_u32(tile) + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(clear ? 0u : w[e], o[2 * e], o[2 * e + 1]);
            uint8_t *dst = vals + (c >> 2) * (kKeys * 128) + r * 128;
            *reinterpret_cast<uint4 *>(dst + (((2 * c & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + (((2 * c + 1 & 7) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        } else {
          if (draft) {
            for (int c = 0; c < D / 8; ++c) {
              uint32_t w[4];
              lds128(w, smem_u32(tile) + (c >> 3) * C::kPanel + r * 128 + (c & 7) * 16);
#pragma unroll
              for (int e = 0; e < 4; ++e)  // an exponent of ones: infinity or NaN
                bad = bad || (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
            }
          }
          if (clear || bad)
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4 *>(tile + (c >> 3) * C::kPanel + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        if (bad) atomicOr(reinterpret_cast<unsigned long long *>(smem + C::oBad) + slot_id, 1ull << (t - seg.first));
        tc::fence_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (r == 0) {
          mbar_arrive(v_ready + slot_id);
          if (FP8) mbar_arrive(empty + at.stage);
        }
      }
      tiles += order.nt;
    }
  } else {
    regs_dec<kRegsOther>();
    if (warp == 12) {
      // ---------------------------------------------------------- loads
      uint32_t tiles = 0;
      const int box = p.box, nbox = kKeys / box;
      while (walk.next(p, block, seg)) {
        const TreeOrder<FP8, S> order(seg, tiles);
        // lane's box of tile i: its first slot in the cache; a page outside it reads as zeros
        auto first_slot = [&](int i) {
          const int64_t pos = (int64_t)(seg.i0 + i) * kKeys + lane % nbox * box;
          if (i >= order.nt || pos >= seg.T) return 0;
          const int64_t slot = tree_slot(p, seg.b, pos);
          return slot < 0 ? (int)p.num_slots : (int)slot;
        };
        auto load = [&](const CUtensorMap &map, int i, int z, auto at) {
          const uint32_t st = at.stage;
          wait_or_abort(empty + st, at.parity ^ 1u, abort, p.err, kErrEmptyWait);
          if (__any_sync(0xffffffffu, *abort)) return;
          const int rows = min(kKeys, seg.T - (seg.i0 + i) * kKeys), boxes = (rows + box - 1) / box;
          if (lane == 0) mbar_arrive_expect_tx(full + st, (uint32_t)(boxes * box * 128 * C::kPanels));
          __syncwarp();
          const int k = lane % nbox, pn = lane / nbox;
          if (pn < C::kPanels && k < boxes)
            tma_load_3d(smem_u32(smem + C::oStage + (size_t)st * C::kTile + pn * C::kPanel + k * box * 128), &map, full + st,
                        pn * (FP8 ? 128 : 64), seg.kvh, z);
        };
        int z[4] = {first_slot(0), first_slot(1), first_slot(2), 0};
        for (int i = 0; i < order.ahead; ++i) load(tmk, i, z[i], order.k(i));
        for (int i = 0; i < order.nt; ++i) {
          z[3] = first_slot(i + 3);  // its page number is on the way while this tile is loaded
          load(tmv, i, z[0], order.v(i));
          if (i + order.ahead < order.nt) load(tmk, i + order.ahead, order.ahead == 1 ? z[1] : z[2], order.k(i + order.ahead));
          z[0] = z[1], z[1] = z[2], z[2] = z[3];
        }
        tiles += order.nt;
      }
      // Every copy has landed when the values and the products have used it; after an abort this waits for both
      // phases of every stage, as long as a copy may take.
      if (__any_sync(0xffffffffu, *abort))
        for (int st = 0; st < 2 * S; ++st) mbar_wait(full + st / 2, st & 1, kSpinLimitCycles / 100);
    } else if (warp == 13) {
      if (lane == 0) {
      // ---------------------------------------------------------- MMA issue
      const uint32_t id_s = tc::idesc(kStreamRows, kKeys, FP8 ? 0 : 1, 0, 0), id_o = tc::idesc(kStreamRows, D, 1, 0, 1);
      const uint32_t stage0 = smem_u32(smem + C::oStage), vals0 = smem_u32(smem + C::oVals), q0 = smem_u32(smem);
      uint32_t tiles = 0, hc = 0, np[2] = {0, 0}, nq[2] = {0, 0};
      auto logits = [&](int s, auto at) {  // S_s = Q_s K^T
        const uint32_t k = stage0 + at.stage * (uint32_t)C::kTile, q = q0 + (uint32_t)(s * C::kQ);
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            mma_e4m3(tmem + (uint32_t)(s * kKeys), tc::sdesc(q + (uint32_t)((e >> 2) * kStreamRows * 128 + (e & 3) * 32), 16, 1024, 2),
                     tc::sdesc(k + (uint32_t)((e & 3) * 32), 16, 1024, 2), id_s, e > 0);
        } else {
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            tc::mma_f16(tmem + (uint32_t)(s * kKeys), tc::sdesc(q + (uint32_t)((e >> 2) * kStreamRows * 128 + (e & 3) * 32), 16, 1024, 2),
                        tc::sdesc(k + (uint32_t)((e >> 2) * C::kPanel + (e & 3) * 32), 16, 1024, 2), id_s, e > 0);
        }
        tc::commit(s_full + s);
      };
      auto wait_full = [&](auto at) {
        wait_or_abort(full + at.stage, at.parity, abort, p.err, kErrFullWait);
        tc::fence_after();
      };
      while (walk.next(p, block, seg)) {
        const TreeOrder<FP8, S> order(seg, tiles);
        const int special0 = max(seg.i0, min(seg.i1, seg.first / kKeys));
        const int streams = seg.pair ? 2 : min(2, order.nt);
        for (int s = 0; s < streams; ++s) {
          wait_or_abort(q_full + s, nq[s]++ & 1, abort, p.err, kErrFullWait);
          tc::fence_after();
          const auto at = order.k(seg.pair ? 0 : s);
          if (!seg.pair || s == 0) wait_full(at);
          logits(s, at);
          if (!seg.pair || s == 1) tc::commit(empty + at.stage);
        }
        for (int i = 0; i < order.nt; ++i) {
          const auto at = order.v(i);
          const bool handled = FP8 || seg.i0 + i >= special0;
          if (!FP8) wait_full(at);
          if (handled) {
            if (!FP8) mbar_arrive(v_landed + (hc & 1));
            wait_or_abort(v_ready + (hc & 1), (hc >> 1) & 1, abort, p.err, kErrFullWait);
            tc::fence_after();
          }
          const uint32_t v = FP8 ? vals0 + (hc & 1) * (uint32_t)C::kVals : stage0 + at.stage * (uint32_t)C::kTile;
          const int s0 = seg.pair ? 0 : i & 1, s1 = seg.pair ? 1 : s0;
          for (int s = s0; s <= s1; ++s) {
            wait_or_abort(p_full + s, np[s]++ & 1, abort, p.err, kErrFullWait);
            tc::fence_after();
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)  // O_s += P_s V
              mma_ts_f16(tmem + 256u + (uint32_t)(s * D), tmem + (uint32_t)(s * kKeys + e * 8),
                         tc::sdesc(v + (uint32_t)e * 2048u, kKeys * 128, 1024, 2), id_o);
            tc::commit(o_full + s);
            if (s == s1) {
              if (!FP8) tc::commit(empty + at.stage);
              if (handled) tc::commit(v_free + (hc & 1));
            }
            const int k = i + (seg.pair ? 1 : 2);  // this stream's next tile
            if (k < order.nt) {
              if (s == s0) wait_full(order.k(k));
              logits(s, order.k(k));
              if (s == s1) tc::commit(empty + order.k(k).stage);
            }
          }
          hc += handled;
        }
        tiles += order.nt;
      }
      tc::commit(done);
      mbar_wait(done, 0);  // no product in flight when the tensor memory is freed
      }
      __syncwarp();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 13) tc::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

int tree_tc_rows() { return kStreamRows; }
int tree_tc_tile() { return kKeys; }

cudaError_t launch_tree_tc(const TreeParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, int kv_dtype, cudaStream_t s) {
  auto run = [&](auto kern, size_t bytes) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (int)bytes);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3((unsigned)(p.groups * p.blocks)), dim3(kThreads), bytes, s, 0, tmk, tmv, p);
  };
  if (kv_dtype == HS2_E4M3) return run(tree_tc_kernel<128, true>, TreeTc<128, true>::kBytes);
  return p.D == 64 ? run(tree_tc_kernel<64, false>, TreeTc<64, false>::kBytes)
                   : run(tree_tc_kernel<128, false>, TreeTc<128, false>::kBytes);
}

}  // namespace hs2
