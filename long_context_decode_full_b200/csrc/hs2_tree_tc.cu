// hs2_tree_tc.cu -- attention of a tree of drafted tokens over a bf16 or E4M3
// cache on the tensor cores (tcgen05, accumulators in tensor memory).
//
// A CTA walks the tiles of its share (hs2_tree_common.cuh) with two streams, a
// warpgroup each, a thread per query row.  Stream s holds 128 logits columns S_s
// and D output columns O_s of tensor memory and repeats, per tile of 128 positions,
//   S_s = Q_s K^T                     (tcgen05.mma, Q and K in shared memory)
//   P_s = 2^(c2 S_s - m), l += sum P  (registers; P as bf16 over S's columns)
//   O_s += P_s V                      (tcgen05.mma, P from tensor memory).
// While one stream's warpgroup is at its exponentials the tensor cores work for
// the other.  A block of more than 128 rows gives each stream 128 of them, and both
// take every tile; with 128 rows or fewer both hold the same rows and take every
// other tile, so a memory-bound call has two warpgroups at work, too; their sums
// are joined at the end.
//
// A stream works on 64 columns at a time, so the first half's product is under way
// during the second half's exponentials.  m is the maximum of a row's first columns
// and moves only when later weights pass it far (their sum over 64 columns passes
// 2^15): weights that stay below need no maximum, so an ordinary tile is read from
// tensor memory once, and O_s is rescaled a few times per unit instead of per tile.
// bf16 and fp32 sums hold such weights as well as weights below 1.
//
// E4M3 caches.  S_s uses the codes as they are: the query row, scaled by a power
// of two to at most 448, is split into two E4M3 terms hi + lo (a bf16 value has
// 8 significand bits, each term holds 4, and the remainder of rounding to 4 bits
// fits the other 4), so S_s = hi K^T + lo K^T at E4M3's double rate costs what one
// bf16 product does; below 2^-6 of E4M3's range the terms are off by 2^-10 of it.
// The key's scale multiplies the logit.  V's codes are converted to bf16 (exact)
// by a warpgroup of its own, and its scale joins the weight before it is rounded.
//
// Weights are rounded to bf16 for the product with V (2^-8 at most of each; their
// sum l takes them unrounded), which with the output's own rounding leaves 0.0024 of
// an output's size where exact weights leave 0.0017 (random rows).  Over a bf16
// cache the product has no other type for them.  Over E4M3 fp16 would hold three more
// bits, as the decode step's kernels do, but only of weights times scales within
// 2^-14 of the largest, and nothing below 2^-24: a million rows 2^-30 below one that
// dominates (a first row without a value of its own) would be lost, where bf16 keeps
// them as exact as any.
//
// Roles: warps 0-3 and 4-7 the streams, 8-11 the values (conversion, and rows
// that must not be multiplied, below), 12 the TMA loads, 13 the MMA issue, 14-15
// E4M3's scales.  Register shares follow the roles.
//
// Rows of V that a query row must not see, whatever they hold: weight 0 times
// NaN is NaN in a matrix product, so the values warpgroup clears the rows behind
// the sequence, and drafts' rows with a non-finite element; the latter are added
// to the rows that do see them one by one.
//
// Bounds and figures (one B200).  The products run at the tensor cores' full rate
// (65 cycles per 128 x 128 x 16 step, bf16, from shared or tensor memory, and per
// 128 x 128 x 32 step of E4M3).  Under sustained load the card is at its 1000 W cap
// and the SM clock falls to 1.1-1.6 GHz, so work that is not needed costs time even
// where it is hidden: blocks of at most 64 rows take M = 64 products (8 drafts over
// 256K x 4 sequences, bf16: 404 -> 371 us; 5.8 TB/s), and weights need no maximum.
//   8 x 8 rows, 4 x 262,144 tokens, bf16    355 us sustained (a launch alone 323 us: memory)
//   64 x 8 rows, 8 x 32,768, bf16           313 us sustained, 0.81 PFLOP/s
//   16 x 8 rows, 1 x 1,048,576, E4M3        419 us sustained (a launch alone 360 us)
// The last two are bound by a stream's chain: logits product, exponentials, weights'
// product, about 3,500 cycles per tile of both streams where the products need 2,048.
// Measured and dropped, against 371 / 326 / 440 at that step (us, in this order of
// cases; cards differ by up to 10%): tiles of 64 positions with two
// sets of logits columns 449 / 341 / 609 (a step with N = 64 takes as long as one with
// N = 128); two warpgroups per stream 399 / 317 / 498; two passes, maximum first,
// 397 / 315 / 640; a quarter of the exponentials as a polynomial on the FMA units
// 406 / 326 / 456; eight conversion warps (E4M3) 460.
#include <type_traits>

#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_pair.cuh"
#include "hs2_tc.cuh"
#include "hs2_tree_common.cuh"

namespace hs2 {

namespace {

constexpr int kKeys = 128;       // positions per tile
constexpr int kStreamRows = 128;
constexpr int kThreads = 512;
constexpr int kTmemCols = 512;
// 65,536 registers: 2 x 128 threads x 176 and 2 x 128 x 80
constexpr int kRegsStream = 176, kRegsOther = 80;
constexpr float kMaxGrowth = 8.f, kMaxSum = 32768.f;

template <int D, bool FP8>
struct TreeTc {
  static constexpr int kQ = FP8 ? 2 * kStreamRows * D : kStreamRows * D * 2;  // a stream's query
  static constexpr int kTile = kKeys * D * (FP8 ? 1 : 2);                     // a K or V tile as it is in the cache
  static constexpr int kVals = FP8 ? kKeys * D * 2 : 0;                       // a converted V tile
  static constexpr int kPanel = kKeys * 128;                                  // 128 bytes of every row
  static constexpr int kPanels = kTile / kPanel;
  static constexpr int kStagesK = FP8 ? 3 : (D == 128 ? 5 : 8), kStagesV = FP8 ? 2 : 0;  // bf16: V has no ring of its own
  static constexpr int kStages = kStagesK + kStagesV;
  static constexpr int kSlots = 2;   // tiles in the values warpgroup's hands
  static constexpr int kScales = 8;  // tiles whose scales are there or on the way: their fetch takes longer than a tile's logits
  static constexpr size_t oStage = 2 * kQ, oVals = oStage + (size_t)kStages * kTile, oScale = oVals + kSlots * kVals,
                          oQScale = oScale + (FP8 ? kScales * 2 * kKeys * 4 : 0),
                          oBar = oQScale + (FP8 ? 2 * kStreamRows * 4 : 0);
  // p_full and o_full: a stream's halves of a tile
  // full[S], empty[S], q_full[2], s_full[2], p_full[2][2], o_full[2][2], and per slot v_ready, v_free, v_landed; scale_full[8], scale_free[8]; done
  static constexpr int kBars = 2 * kStages + 12 + 3 * kSlots + 2 * kScales + 1;
  static constexpr size_t oBad = oBar + (size_t)((kBars * 8 + 15) / 16 * 16), oInfo = oBad + 8 * kSlots, kBytes = oInfo + 64 + 1024;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

struct TreeInfo {  // shared
  int32_t g0, g1;  // the share's tiles
  int32_t b0, base;  // the sequence in which it begins, and the tiles before that
  uint32_t tmem;
  int32_t abort;
};

// One unit's part in a share.
struct TreeSeg {
  int b, kvh, i0, i1, T, first, nr, special0;  // special0: the first tile with a draft, or rows behind the sequence
  bool pair, few, begins, whole;  // few: at most 64 rows
};

// Tiles are numbered in 32 bits: the entry points keep them below 2^31.
struct TreeWalk {
  int g, g0, g1, base, b;
  __device__ __forceinline__ explicit TreeWalk(const TreeInfo &in) : g(in.g0), g0(in.g0), g1(in.g1), base(in.base), b(in.b0) {}
  // The next segment that has rows for this CTA.
  __device__ __forceinline__ bool next(const TreeParams &p, int block, TreeSeg &s) {
    while (g < g1 && b < p.B) {
      s.T = tree_len(p, b);
      const int given = tree_given_drafts(p, b);  // fetched together
      const int nb = (s.T + kKeys - 1) / kKeys, r = g - base;
      if ((int64_t)r >= (int64_t)p.Hkv * nb) {
        base += p.Hkv * nb;
        ++b;
        continue;
      }
      s.b = b;
      s.kvh = r / nb;
      s.i0 = r - s.kvh * nb;
      s.i1 = min(nb, s.i0 + (g1 - g));
      const int n = clamp_len(given, min(p.N, s.T));
      s.first = s.T - n;
      s.special0 = max(s.i0, min(s.i1, s.first / kKeys));
      s.begins = g == g0;
      s.whole = s.i0 == 0 && s.i1 == nb;
      g += s.i1 - s.i0;
      s.nr = min(2 * kStreamRows, n * p.G - block * 2 * kStreamRows);
      s.pair = s.nr > kStreamRows;
      s.few = s.nr <= kStreamRows / 2;
      if (s.nr > 0) return true;
    }
    return false;
  }
};

// The pages of one row of every tile of a sequence, in tile order; the page numbers are fetched apart from their use.
struct TreePages {
  const int32_t *row;  // the next tile's page number
  int off, pos;        // the row's place in its page, and in the sequence
  __device__ __forceinline__ TreePages(const TreeParams &p, const TreeSeg &s, int first) : pos(s.i0 * kKeys + first) {
    const int page = pos / p.page_size;
    off = pos - page * p.page_size;
    row = p.page_table ? p.page_table + (int64_t)s.b * p.max_pages + page : nullptr;
  }
  struct Row {
    int page, off;  // off < 0: behind the sequence
  };
  __device__ __forceinline__ Row next(const TreeParams &p, int T) {
    Row r{0, off};
    if (pos >= T) r.off = -1;
    else if (row) r.page = __ldg(row);
    pos += kKeys;
    off += p.page_off;
    if (row) row += p.page_step;
    if (off >= p.page_size) {
      off -= p.page_size;
      if (row) ++row;
    }
    return r;
  }
  // the slot in the cache, or -1
  static __device__ __forceinline__ int64_t slot(const TreeParams &p, const TreeSeg &s, Row r) {
    const int64_t x = (int64_t)(p.page_table ? r.page : s.b) * p.page_size + r.off;
    return r.off >= 0 && x >= 0 && x < p.num_slots ? x : -1;
  }
};

// The loads of a segment, and the order in which the products use them: K of the
// first `ahead` tiles, then V of tile i and K of tile i + ahead.  bf16: one ring of
// stages in this order.  E4M3: a ring for K and one for V, because
// the values warpgroup waits for V alone, and a waiter that misses a stage's phases
// cannot tell them apart.
struct TreeRing {
  uint32_t stage, parity;
  template <int FIRST, int STAGES>
  __device__ __forceinline__ void next() {
    if (++stage == FIRST + STAGES) stage = FIRST, parity ^= 1u;
  }
};
__device__ __forceinline__ int tree_ahead(const TreeSeg &s) { return min(s.pair ? 1 : 2, s.i1 - s.i0); }

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
// 4 bytes, or zeros with bytes = 0
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// shared loads that stay where they are written
__device__ __forceinline__ float4 lds_float4(const float *p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ float2 lds_float2(const float *p) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(smem_u32(p)));
  return v;
}
// 64 columns
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%2"
      "7,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%5"
      "2,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
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

// Shared-memory descriptors of 128-byte-swizzled operands (hs2_tc.cuh) as two
// words: the upper one is the same for all (1 KB between groups of 8 rows), the
// lower one holds the address and, for an MN-major operand, the panels' distance.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t panel) { return (addr >> 4) | (panel >> 4) << 16; }
// The whole warp gets here and one lane issues: addresses stay in uniform registers.
__device__ __forceinline__ void mma_ts_f16(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0x7fffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(one), "r"(kDescHi)
      : "memory");
}
template <bool E4M3>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t one) {
  if constexpr (E4M3)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(one), "r"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(one), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

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
  constexpr int kSlots = C::kSlots, kScales = C::kScales, SK = C::kStagesK, SV = C::kStagesV;
  uint64_t *full = bars, *empty = bars + S, *q_full = bars + 2 * S, *s_full = q_full + 2, *p_full = q_full + 4,
           *o_full = q_full + 8, *v_ready = q_full + 12, *v_free = v_ready + kSlots, *v_landed = v_free + kSlots,
           *scale_full = v_landed + kSlots, *scale_free = scale_full + kScales, *done = scale_free + kScales;
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
      mbar_init(p_full + 2 * s, 4);
      mbar_init(p_full + 2 * s + 1, 4);
    }
    for (int s = 0; s < kScales; ++s) mbar_init(scale_full + s, 64);
    fence_mbar_init();
    info->abort = 0;
    info->g0 = info->g1 = 0;
  }
  if (warp == 12 && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  if (warp == 13) {
    tc::tmem_alloc(&info->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = info->tmem;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {  // the tiles of all sequences, then the sequence where the share begins
    int64_t total = 0;
    for (int b = lane; b < p.B; b += 32) total += (tree_len(p, b) + kKeys - 1) / kKeys;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.Hkv;
    if (total > 0) {
      const TreeShare share(total, p.groups);
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
          info->base = (int32_t)(sum - x);
          info->b0 = b0 + lane;
        }
        carry = __shfl_sync(0xffffffffu, sum, 31);
        if (carry > g0) break;
      }
      if (lane == 0) {
        info->g0 = (int32_t)g0;
        info->g1 = (int32_t)share.start(group + 1);
      }
    }
    if (blockIdx.x == 0) tree_prefix(p, p.prefix);
  }
  __syncthreads();
  if (info->g0 >= info->g1) {  // no tiles for this CTA
    if (warp == 13) tc::tmem_dealloc(tmem, kTmemCols);
    return;
  }
  TreeWalk walk(*info);
  TreeSeg seg;
  const int wg = warp >> 2;

  if (wg < 2) {
    // ------------------------------------------------------------ a stream
    regs_inc<kRegsStream>();
    const int s = wg;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + (uint32_t)(s * kKeys), to = tmem + lanes + 256u + (uint32_t)(s * D);
    uint8_t *sq = smem + s * C::kQ;
    bool handed = false;  // a record of sums that stream 0 may still read
    uint32_t ns = 0, handled0 = 0;  // tiles of this stream; tiles handled by the values warpgroup before the segment
    while (walk.next(p, block, seg)) {
      const int nt = seg.i1 - seg.i0;
      const uint32_t handled_here = FP8 ? nt : seg.i1 - seg.special0;
      if (!seg.pair && s >= nt) {  // one tile: the other stream has it
        handled0 += handled_here;
        continue;
      }
      // with M = 64 the product leaves 16 rows in the first half of each warp's lanes
      const int row = seg.few ? (warp & 3) * 16 + (lane & 15) : tid & 127;
      const int r = block * 2 * kStreamRows + (seg.pair ? s * kStreamRows : 0) + row;
      const int n = seg.T - seg.first;
      const bool mine = r < n * p.G && !(seg.few && lane >= 16), busy = __any_sync(0xffffffffu, mine);
      const int tok = r / p.G, head = seg.kvh * p.G + r % p.G;
      const uint64_t bits = mine ? tree_bits(p, seg.b, tok, n) : 0ull;
      float c2 = p.c2;
      // the query rows to shared memory, 128-byte swizzle
      if constexpr (!FP8) {
        if (mine) {
          const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                             ((int64_t)seg.b * p.N + tok) * p.q_stride + (int64_t)head * D);
          uint4 x[D / 8];
#pragma unroll
          for (int c = 0; c < D / 8; ++c) x[c] = __ldg(src + c);
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4 *>(sq + (c >> 3) * (kStreamRows * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[c];
        }
      } else {
        // eight neighbouring threads split a row into its terms, 16 elements each, and the row's own thread takes its scale
        constexpr int kPer = D / 16;
        const int r_first = block * 2 * kStreamRows + (seg.pair ? s * kStreamRows : 0);
        const int rows = min(kStreamRows, n * p.G - r_first), c = lane % kPer;
        float *scales = reinterpret_cast<float *>(smem + C::oQScale) + s * kStreamRows;
#pragma unroll 1
        for (int y = (tid & 127) / kPer; y < ((rows + 3) & ~3); y += 128 / kPer) {  // the same number of rounds for a warp
          const int rr = r_first + min(y, rows - 1), hh = seg.kvh * p.G + rr % p.G;
          const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                             ((int64_t)seg.b * p.N + rr / p.G) * p.q_stride + (int64_t)hh * D) + 2 * c;
          const uint4 x0 = __ldg(src), x1 = __ldg(src + 1);
          const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          float top = 0.f;
          bool finite = true;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = fabsf(bf16_lo(w[e])), b = fabsf(bf16_hi(w[e]));
            top = fmaxf(top, fmaxf(a, b));
            finite = finite && a <= 3.4e38f && b <= 3.4e38f;
          }
#pragma unroll
          for (int o = kPer / 2; o; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) && finite;
          }
          // the largest power of two that takes the row to at most 448
          const uint32_t tb = __float_as_uint(top);
          const int k = min(126, 8 + 127 - (int)(tb >> 23) - ((tb & 0x7FFFFFu) > 0x600000u));
          const float up = __uint_as_float((uint32_t)(k + 127) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            hi[e] = lo[e] = 0;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint32_t u = w[2 * e + f];
              const float2 v = make_float2(bf16_lo(u) * up, bf16_hi(u) * up);
              const uint32_t h = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
              const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
              const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
              const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(v.x - back.x, v.y - back.y), __NV_SATFINITE, __NV_E4M3);
              hi[e] |= h << (16 * f);
              lo[e] |= l << (16 * f);
            }
          }
          if (y < rows) {
            uint8_t *dst = sq + y * 128 + ((c ^ (y & 7)) << 4);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(dst + kStreamRows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (c == 0) scales[y] = finite ? p.c2 * __uint_as_float((uint32_t)(127 - k) << 23) : __int_as_float(0x7FC00000);
          }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(4 + s) : "memory");
        if (mine) c2 = scales[row];
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
      bool any_product = false;  // whether O holds a product
      for (int i = seg.pair ? 0 : s; i < nt; i += seg.pair ? 1 : 2) {
        const int t0 = (seg.i0 + i) * kKeys;
        const bool special = seg.i0 + i >= seg.special0;
        const uint32_t hc = handled0 + (FP8 ? i : seg.i0 + i - seg.special0);  // this tile among the handled ones
        const uint32_t slot_id = hc % kSlots, slot_parity = hc / kSlots & 1u;
        wait_or_abort(s_full + s, ns & 1u, abort, p.err, kErrFullWait);
        tc::fence_after();
        if (FP8) wait_or_abort(scale_full + hc % kScales, hc / kScales & 1u, abort, p.err, kErrFullWait);
        if (special) wait_or_abort(v_ready + slot_id, slot_parity, abort, p.err, kErrFullWait);
        const float *ks = reinterpret_cast<const float *>(smem + C::oScale) + hc % kScales * 2 * kKeys, *vs = ks + kKeys;
        const uint64_t bad = special ? bad_rows[slot_id] : 0ull;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t tx = ts + 64 * h;  // this half's logits, and its weights over them
          // O after the last product, times alpha
          auto rescale = [&](float alpha) {
            wait_or_abort(o_full + 2 * s + (h ^ 1), (h ? ns : ns - 1) & 1u, abort, p.err, kErrFullWait);
            tc::fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tc::ld32(to + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tc::st32(to + c, o);
            }
          };
          if (busy) {
            uint64_t bad_here = 0;
            uint32_t w[32];
            float sum;
            bool look = special || __any_sync(0xffffffffu, mine && m == -INFINITY);
            if (!look) {  // all is seen, and m is near
              const float2 cc = make_float2(c2, c2), sh = make_float2(-m * c2, -m * c2);
              float x[64];
              float2 sums[2] = {{0.f, 0.f}, {0.f, 0.f}};
              tmem_ld64(tx, x);
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                float2 k0 = cc, k1 = cc, v0, v1;
                if constexpr (FP8) {
                  const float4 f = lds_float4(ks + 64 * h + e), g = lds_float4(vs + 64 * h + e);
                  k0 = mul2(cc, make_float2(f.x, f.y)), k1 = mul2(cc, make_float2(f.z, f.w));
                  v0 = make_float2(g.x, g.y), v1 = make_float2(g.z, g.w);
                }
                float2 a = fma2(make_float2(x[e], x[e + 1]), k0, sh), b = fma2(make_float2(x[e + 2], x[e + 3]), k1, sh);
                a.x = ex2_approx(a.x), a.y = ex2_approx(a.y), b.x = ex2_approx(b.x), b.y = ex2_approx(b.y);
                sums[0] = add2(sums[0], a), sums[1] = add2(sums[1], b);
                if constexpr (FP8) a = mul2(a, v0), b = mul2(b, v1);
                w[e >> 1] = pack_bf16(a.x, a.y);
                w[(e >> 1) + 1] = pack_bf16(b.x, b.y);
              }
              const float2 both = add2(sums[0], sums[1]);
              sum = both.x + both.y;
              look = __any_sync(0xffffffffu, mine && sum > kMaxSum);
            }
            if (look) {
              const int j0 = t0 + 64 * h - seg.first;  // the draft in the half's first column
              const uint64_t seen = special ? below(-j0) | shift_bits(bits, -j0) : ~0ull;
              bad_here = bad & ~below(j0) & below(j0 + 64);
              // 32 logits from column c of the half on, times the keys' scales, the hidden ones at -infinity
              auto load_logits = [&](int c, float(&x)[32]) {
                tc::ld32(tx + c, x);
                if constexpr (FP8) {
#pragma unroll
                  for (int e = 0; e < 32; e += 2) {
                    const float2 u = mul2(make_float2(x[e], x[e + 1]), lds_float2(ks + 64 * h + c + e));
                    x[e] = u.x, x[e + 1] = u.y;
                  }
                }
                if (special) {
                  const uint32_t see = (uint32_t)(seen >> c);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!((see >> e) & 1u)) x[e] = -INFINITY;
                }
              };
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 64; c += 32) {
                float x[32];
                load_logits(c, x);
#pragma unroll
                for (int e = 0; e < 32; e += 8)
#pragma unroll
                  for (int f = 0; f < 4; ++f) mx[f] = fmaxf(fmaxf(mx[f], x[e + f]), x[e + f + 4]);
              }
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
              float alpha = 1.f;
              if (m == -INFINITY ? top > -INFINITY : top > m + growth) {
                alpha = m == -INFINITY ? 0.f : ex2_approx((m - top) * c2);
                m = top;
                l *= alpha;
              }
              __syncwarp();
              if (any_product && (bad_here || __any_sync(0xffffffffu, alpha != 1.f))) rescale(alpha);
              const float shift = m == -INFINITY ? 0.f : -m * c2;  // nothing seen yet: weights 0
              float2 sums = make_float2(0.f, 0.f);
#pragma unroll
              for (int c = 0; c < 64; c += 32) {
                float x[32];
                load_logits(c, x);
                const uint32_t see = (uint32_t)(seen >> c);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float2 a = make_float2(ex2_approx(fmaf(x[e], c2, shift)), ex2_approx(fmaf(x[e + 1], c2, shift)));
                  sums = add2(sums, a);
                  if constexpr (FP8) {  // a scale that is not seen may be anything
                    a = mul2(a, lds_float2(vs + 64 * h + c + e));
                    a.x = (see >> e) & 1u ? a.x : 0.f;
                    a.y = (see >> (e + 1)) & 1u ? a.y : 0.f;
                  }
                  w[(c + e) >> 1] = pack_bf16(a.x, a.y);
                }
              }
              sum = sums.x + sums.y;
            }
            l += sum;
            tmem_st32(tx, w);
            tmem_wait_st();
            if (bad_here) {  // rare: drafts whose values are not finite, for the rows that see them
              for (uint64_t rest = bad_here; rest; rest &= rest - 1) {
                const int j = __ffsll((long long)rest) - 1, c = seg.first + j - t0 - 64 * h;
                const uint32_t pw = tmem_ld1(tx + (c >> 1));
                const float wj = c & 1 ? bf16_hi(pw) : bf16_lo(pw);
                const bool sees = (bits >> j) & 1ull;
                const int64_t slot = tree_slot(p, seg.b, seg.first + j);
                if (slot < 0) continue;  // the same for the warp
                const int64_t at = (slot * p.Hkv + seg.kvh) * D;
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
                    if (sees) o[e] = fmaf(wj, v, o[e]);
                  }
                  tc::st32(to + d, o);
                }
              }
            }
            tc::fence_before();
          }
          any_product = true;
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 2 * s + h);
        }
        ++ns;
      }
      handled0 += handled_here;
      wait_or_abort(o_full + 2 * s + 1, (ns - 1) & 1u, abort, p.err, kErrFullWait);
      tc::fence_after();
      // A unit inside the share is finished here, by stream 0: of a unit whose tiles both streams took, stream 1 hands
      // its sums over in a record of their own, which stream 0 has read before stream 1 writes the next.
      const bool join = seg.whole && !seg.pair && nt > 1, finish = seg.whole && !(join && s == 1);
      if (join && s == 1 && handed) asm volatile("bar.sync 3, 256;" ::: "memory");
      float *rec = tree_record(p, group, join ? 2 : (seg.begins ? 0 : 1), block, join ? 1 : s);
      float4 *ro = reinterpret_cast<float4 *>(rec + 2 * kStreamRows) + row;
      if (busy && !finish) {
        if (mine) {
          rec[row] = m * c2;
          rec[kStreamRows + row] = l;
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tc::ld32(to + c, o);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              ro[(size_t)((c + e) / 4) * kStreamRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      if (join && s == 1) asm volatile("bar.arrive 2, 256;" ::: "memory");
      if (join && s == 0) asm volatile("bar.sync 2, 256;" ::: "memory");
      if (busy && finish) {
        float w0 = 1.f, w1 = 0.f, sum = l;
        if (join && mine) {
          const float m0 = m * c2, m1 = __ldcg(rec + row), M = fmaxf(m0, m1), at = M == -INFINITY ? 0.f : M;
          w0 = ex2_approx(m0 - at);
          w1 = ex2_approx(m1 - at);
          sum = w0 * l + w1 * __ldcg(rec + kStreamRows + row);
        }
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // nothing seen: zeros
        w0 *= inv, w1 *= inv;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                               ((int64_t)seg.b * p.N + tok) * p.out_stride + (int64_t)head * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();
          tc::ld32(to + c, o);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= w0;
            if (join) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = __ldcg(ro + (size_t)((c + e) / 4) * kStreamRows);
                o[e] = fmaf(w1, v.x, o[e]), o[e + 1] = fmaf(w1, v.y, o[e + 1]);
                o[e + 2] = fmaf(w1, v.z, o[e + 2]), o[e + 3] = fmaf(w1, v.w, o[e + 3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              dst[(c + e) / 8] = make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]),
                                            pack_bf16(o[e + 4], o[e + 5]), pack_bf16(o[e + 6], o[e + 7]));
          }
        }
      }
      if (join && s == 0) asm volatile("bar.arrive 3, 256;" ::: "memory");
      handed = handed || (join && s == 1);
    }
    if (handed) asm volatile("bar.sync 3, 256;" ::: "memory");
  } else if (wg == 2) {
    // ------------------------------------------------------------ values
    regs_dec<kRegsOther>();
    const int r = tid & (kKeys - 1);
    uint32_t tiles = 0, hc = 0;
    TreeRing ring{SK, 0};
    while (walk.next(p, block, seg)) {
      const int nt = seg.i1 - seg.i0, ahead = tree_ahead(seg);
      for (int i = FP8 ? 0 : seg.special0 - seg.i0; i < nt; ++i, ++hc) {
        const int t = (seg.i0 + i) * kKeys + r;
        const uint32_t slot_id = hc % kSlots, slot_parity = hc / kSlots & 1u;
        const bool live = t < seg.T, draft = live && t >= seg.first;
        if (!FP8) {  // V of tile i in the one ring
          const uint32_t at = 2 * tiles + ahead + i + min(i, nt - ahead);
          ring.stage = at % S, ring.parity = at / S & 1u;
        }
        wait_or_abort(v_free + slot_id, slot_parity ^ 1u, abort, p.err, kErrEmptyWait);
        if (tid == 2 * 128) bad_rows[slot_id] = 0ull;
        if (!FP8) wait_or_abort(v_landed + slot_id, slot_parity, abort, p.err, kErrFullWait);
        wait_or_abort(full + ring.stage, ring.parity, abort, p.err, kErrFullWait);
        uint8_t *tile = smem + C::oStage + (size_t)ring.stage * C::kTile;
        bool bad = false;
        if (draft) {  // the largest magnitude of the row's codes: NaN (E4M3), infinity and NaN (bf16) lie above all others
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < C::kPanels * 8; ++c) {
            uint32_t w[4];
            lds128(w, smem_u32(tile) + (c >> 3) * C::kPanel + r * 128 + (c & 7) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (FP8) top = __vmaxu4(top, w[e] & 0x7F7F7F7Fu);
              else top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
            }
          }
          if constexpr (FP8) bad = __vcmpeq4(top, 0x7F7F7F7Fu) != 0u;
          else bad = __vcmpgeu2(top, 0x7F807F80u) != 0u;
        }
        const bool clear = !live || bad;
        if (seg.i0 + i >= seg.special0) {  // the mask is clear, and every row has been looked at
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (bad)
            atomicOr(reinterpret_cast<unsigned long long *>(smem + C::oBad) + slot_id, 1ull << (t - seg.first));
        }
        if constexpr (FP8) {
          uint8_t *dst0 = smem + C::oVals + (size_t)slot_id * C::kVals + r * 128;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint8_t *dst = dst0 + half * (kKeys * 128);
            uint32_t w[4][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) lds128(w[c], smem_u32(tile) + r * 128 + (((4 * half + c) ^ (r & 7)) << 4));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(clear ? 0u : w[c][e], o[2 * e], o[2 * e + 1]);
              *reinterpret_cast<uint4 *>(dst + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4 *>(dst + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        } else if (clear) {
#pragma unroll
          for (int c = 0; c < C::kPanels * 8; ++c)
            *reinterpret_cast<uint4 *>(tile + (c >> 3) * C::kPanel + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_async_smem();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (tid == 2 * 128) {
          mbar_arrive(v_ready + slot_id);
          if (FP8) mbar_arrive(empty + ring.stage);
        }
        if (FP8) ring.next<SK, SV>();
      }
      tiles += nt;
    }
  } else {
    regs_dec<kRegsOther>();
    if (warp == 12) {
      // ---------------------------------------------------------- loads
      const int box = p.box, nbox = kKeys / box, k = lane % nbox, pn = lane / nbox;  // this lane's box of a tile
      const uint32_t to = smem_u32(smem + C::oStage) + pn * C::kPanel + k * box * 128;
      TreeRing ring_k{0, 0}, ring_v{SK, 0};
      auto load = [&](const CUtensorMap &map, TreeRing r, int z, int left) {  // `left` rows of the sequence
        wait_or_abort(empty + r.stage, r.parity ^ 1u, abort, p.err, kErrEmptyWait);
        if (__any_sync(0xffffffffu, *abort)) return;
        const int boxes = left >= kKeys ? nbox : (left + box - 1) / box;
        if (lane == 0) mbar_arrive_expect_tx(full + r.stage, (uint32_t)(boxes * box * 128 * C::kPanels));
        __syncwarp();
        if (pn < C::kPanels && k < boxes) tma_load_3d(to + r.stage * C::kTile, &map, full + r.stage, pn * (FP8 ? 128 : 64), seg.kvh, z);
      };
      auto load_k = [&](int z, int left) {
        load(tmk, ring_k, z, left);
        ring_k.next<0, SK>();
      };
      auto load_v = [&](int z, int left) {
        load(tmv, FP8 ? ring_v : ring_k, z, left);
        if (FP8) ring_v.next<SK, SV>();
        else ring_k.next<0, SK>();
      };
      while (walk.next(p, block, seg)) {
        const int nt = seg.i1 - seg.i0, ahead = tree_ahead(seg);
        TreePages pages(p, seg, k * box);
        int left = seg.T - seg.i0 * kKeys;  // rows from tile i on
        TreePages::Row next[3] = {};        // of tiles i + ahead to i + ahead + 2: fetched before they are needed
        int z[2] = {};                      // first slots of tiles i to i + ahead - 1; a page outside the cache reads as zeros
        auto take = [&]() {
          const int64_t x = TreePages::slot(p, seg, next[0]);
          next[0] = next[1], next[1] = next[2];
          next[2] = pages.next(p, seg.T);
          return x < 0 ? (int)p.num_slots : (int)x;
        };
#pragma unroll
        for (int e = 0; e < 3; ++e) next[e] = pages.next(p, seg.T);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (e < ahead) load_k(z[e] = take(), left - e * kKeys);
        for (int i = 0; i < nt; ++i, left -= kKeys) {
          load_v(z[0], left);
          const int z_new = take();
          if (i + ahead < nt) load_k(z_new, left - ahead * kKeys);
          z[0] = ahead == 2 ? z[1] : z_new;
          z[1] = z_new;
        }
      }
      // Every copy has landed when the values and the products have used it; after an abort this waits for both
      // phases of every stage, as long as a copy may take.
      if (__any_sync(0xffffffffu, *abort))
        for (int st = 0; st < 2 * S; ++st) mbar_wait(full + st / 2, st & 1, kSpinLimitCycles / 100);
    } else if (warp == 13) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t kTileLo = C::kTile >> 4, kPanelLo = C::kPanel >> 4, kRowsLo = kStreamRows * 128 >> 4;
      const uint32_t one = elect_one();
      const uint32_t id_s128 = tc::idesc(kStreamRows, kKeys, FP8 ? 0 : 1, 0, 0), id_o128 = tc::idesc(kStreamRows, D, 1, 0, 1);
      const uint32_t id_s64 = tc::idesc(kStreamRows / 2, kKeys, FP8 ? 0 : 1, 0, 0), id_o64 = tc::idesc(kStreamRows / 2, D, 1, 0, 1);
      uint32_t id_s = id_s128, id_o = id_o128;
      const uint32_t base = smem_u32(smem), bar = smem_u32(bars), tm = uniform(tmem);
      const uint32_t q0 = desc_lo(base, 16), k0 = desc_lo(base + (uint32_t)C::oStage, 16),
                     v0 = desc_lo(base + (uint32_t)(FP8 ? C::oVals : C::oStage), kKeys * 128);
      const uint32_t b_empty = bar + 8 * S, b_s = bar + 8 * (2 * S + 2), b_o = bar + 8 * (2 * S + 8), b_free = bar + 8 * (2 * S + 12 + kSlots),
                     b_scale = bar + 8 * (2 * S + 12 + 3 * kSlots + kScales);
      uint32_t hc = 0;
      TreeRing ring{0, 0};
      uint32_t np = 0, nq = 0;  // parities of each stream's weights and queries, a bit each
      auto flip = [](uint32_t &n, int s) {
        const uint32_t x = n >> s & 1u;
        n ^= 1u << s;
        return x;
      };
      auto logits = [&](uint32_t s, uint32_t stage) {  // S_s = Q_s K^T
        const uint32_t q = q0 + s * (C::kQ >> 4), k = k0 + stage * kTileLo;
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) mma_ss<true>(tm + s * kKeys, q + (e >> 2) * kRowsLo + (e & 3) * 2, k + (e & 3) * 2, id_s, e > 0, one);
        } else {
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            mma_ss<false>(tm + s * kKeys, q + (e >> 2) * kRowsLo + (e & 3) * 2, k + (e >> 2) * kPanelLo + (e & 3) * 2, id_s, e > 0, one);
        }
        commit_one(b_s + 8 * s, one);
      };
      auto wait_full = [&]() {  // for the next stage of the ring
        wait_or_abort(full + ring.stage, ring.parity, abort, p.err, kErrFullWait);
        tc::fence_after();
        const uint32_t stage = uniform(ring.stage);
        ring.next<0, SK>();
        return stage;
      };
      while (walk.next(p, block, seg)) {
        const int nt = seg.i1 - seg.i0, ahead = tree_ahead(seg), streams = seg.pair ? 2 : min(2, nt);
        id_s = uniform(seg.few ? id_s64 : id_s128), id_o = uniform(seg.few ? id_o64 : id_o128);
        for (int s = 0; s < streams; ++s) wait_or_abort(q_full + s, flip(nq, s), abort, p.err, kErrFullWait);
        tc::fence_after();
        for (int k = 0; k < ahead; ++k) {
          const uint32_t stage = wait_full();
          logits(k, stage);
          if (seg.pair) logits(1, stage);
          commit_one(b_empty + 8 * stage, one);
        }
        for (int i = 0; i < nt; ++i) {
          const bool handled = FP8 || seg.i0 + i >= seg.special0;
          const uint32_t slot = uniform(hc % kSlots), scale_slot = uniform(hc % kScales), stage = FP8 ? 0 : wait_full();
          if (handled) {
            if (!FP8 && lane == 0) mbar_arrive(v_landed + slot);
            wait_or_abort(v_ready + slot, hc / kSlots & 1u, abort, p.err, kErrFullWait);
            tc::fence_after();
          }
          const uint32_t v = v0 + (FP8 ? slot * (C::kVals >> 4) : stage * kTileLo);
          uint32_t next = 0;
          auto product = [&](uint32_t s, bool first, bool last) {  // O_s += P_s V, then the logits of the stream's next tile
            const uint32_t parity = flip(np, s);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              wait_or_abort(p_full + 2 * s + h, parity, abort, p.err, kErrFullWait);
              tc::fence_after();
#pragma unroll
              for (int e = 0; e < kKeys / 32; ++e)
                mma_ts_f16(tm + 256u + s * D, tm + s * kKeys + (uint32_t)(h * 64 + e * 8), v + (h * 4 + e) * (2048u >> 4), id_o, one);
              commit_one(b_o + 8 * (2 * s + h), one);
            }
            if (last && !FP8) commit_one(b_empty + 8 * stage, one);
            if (last && handled) commit_one(b_free + 8 * slot, one);
            if (last && FP8) commit_one(b_scale + 8 * scale_slot, one);
            if (i + ahead < nt) {
              if (first) next = wait_full();
              logits(s, next);
              if (last) commit_one(b_empty + 8 * next, one);
            }
          };
          if (seg.pair) {
            product(0, true, false);
            product(1, false, true);
          } else {
            product(uniform(i & 1), true, true);
          }
          hc += handled;
        }
      }
      commit_one(smem_u32(done), one);
      mbar_wait(done, 0);  // no product in flight when the tensor memory is freed
    } else if (FP8 && warp >= 14) {
      // ---------------------------------------------------------- scales
      float *sc = reinterpret_cast<float *>(smem + C::oScale);
      uint32_t hc = 0;
      while (walk.next(p, block, seg)) {
        const int nt = seg.i1 - seg.i0;
        const int r0 = (warp - 14) * 64 + lane;  // and the row 32 further
        TreePages pages[2] = {TreePages(p, seg, r0), TreePages(p, seg, r0 + 32)};
        TreePages::Row next[2][2];  // of tiles i and i + 1
#pragma unroll
        for (int k = 0; k < 2; ++k) next[k][0] = pages[k].next(p, seg.T), next[k][1] = pages[k].next(p, seg.T);
        for (int i = 0; i < nt; ++i, ++hc) {
          const uint32_t slot_id = hc % kScales;
          wait_or_abort(scale_free + slot_id, (hc / kScales & 1u) ^ 1u, abort, p.err, kErrEmptyWait);
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // rows that are not there get 0
            const int64_t at = TreePages::slot(p, seg, next[k][0]);
            const uint32_t dst = smem_u32(sc + slot_id * 2 * kKeys + r0 + 32 * k), bytes = at >= 0 ? 4u : 0u;
            const int64_t e = at >= 0 ? at * p.Hkv + seg.kvh : 0;
            cp_async_4_or_zero(dst, p.k_scale + e, bytes);
            cp_async_4_or_zero(dst + kKeys * 4, p.v_scale + e, bytes);
            next[k][0] = next[k][1];
            next[k][1] = pages[k].next(p, seg.T);
          }
          cp_async_mbar_arrive_noinc(scale_full + slot_id);
        }
      }
      cp_async_wait_all();
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
