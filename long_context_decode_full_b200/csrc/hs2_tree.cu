// hs2_tree.cu -- attention of a tree of drafted tokens over the cache: the
// kernel of fp32 caches, and the one that joins the records of cut units.
//
// Token i of sequence b (n drafted tokens, the last n of T rows) attends to the
// T - n rows of the context and to the drafts j with bit j of its mask set:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = 2^(c2 q.k_t - m),  m the running max.
//
// fp32 caches keep fp32 products on the CUDA cores (tensor cores would round
// the operands): a CTA of 16 x 16 threads takes 64 rows x 64 positions, each
// thread a 4 x 4 block of the logits and 4 rows x D / 16 columns of the output
// in registers (half the rows where a unit has at most 32, and half the positions
// where the tiles would not fill the GPU; at most 16 rows have a kernel of their own,
// below); Q, K, V and the weights are in shared memory, K's and Q's rows
// padded by 16 bytes so that 16-byte reads of 8 rows meet 32 banks.  Bound by
// latency on short caches: 5 drafts x 4 heads over 2,048 tokens take 14.8 us with the
// joining kernel (64-row, 64-position shapes and shares without tiles: 53 us).  Long
// ones run at 20 to 22 TFLOP/s, 0.3 of what the FMA units could (every 16-byte read of
// shared memory feeds 8 of their operations, and one tile's loads, logits and product
// wait for one another): 64 x 8 rows over 2 x 16,384 tokens 1.55 ms, 8 x 8 rows over
// 8 x 20,000 0.94 ms, 4 x 8 rows of the same 0.51 ms (4 KV heads, d 128).
#include <type_traits>

#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_rows.cuh"
#include "hs2_tree_common.cuh"

namespace hs2 {

namespace {

constexpr int kThreads = 256;

template <int D, int kRows, int kKeys>
struct TreeF32Smem {
  static constexpr int QS = D + 4, PS = kKeys + 4;
  static constexpr size_t kQ = 0, kK = kQ + (size_t)kRows * QS * 4, kV = kK + (size_t)kKeys * QS * 4,
                          kP = kV + (size_t)kKeys * D * 4, kBits = kP + (size_t)kRows * PS * 4,
                          kSlots = kBits + kRows * 8, kPrefix = kSlots + kKeys * 8;
  static size_t bytes(int B) { return kPrefix + (size_t)(B + 1) * 4; }
};

template <int D, int kRows, int kKeys>
__global__ void __launch_bounds__(kThreads) tree_f32_kernel(const TreeParams p) {
  using S = TreeF32Smem<D, kRows, kKeys>;
  constexpr int R = kRows / 16, K = kKeys / 16;  // rows and positions of a thread
  extern __shared__ __align__(16) uint8_t smem[];
  float *sq = reinterpret_cast<float *>(smem + S::kQ), *sk = reinterpret_cast<float *>(smem + S::kK);
  float *sv = reinterpret_cast<float *>(smem + S::kV), *sp = reinterpret_cast<float *>(smem + S::kP);
  uint64_t *bits = reinterpret_cast<uint64_t *>(smem + S::kBits);
  int64_t *slots = reinterpret_cast<int64_t *>(smem + S::kSlots);  // of the tile's positions, -1: none
  int32_t *prefix = reinterpret_cast<int32_t *>(smem + S::kPrefix);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int block = blockIdx.x % p.blocks;
  const int64_t group = blockIdx.x / p.blocks;
  griddep_wait();
  griddep_launch_dependents();
  if (tid < 32) tree_prefix(p, prefix);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = tid; i <= p.B; i += kThreads) p.prefix[i] = prefix[i];
  const int64_t total = (int64_t)p.Hkv * prefix[p.B];
  if (total == 0) return;
  const TreeShare share(total, p.groups);
  const int64_t g1 = share.start(group + 1);
  for (int64_t g = share.start(group); g < g1;) {
    // one segment: tiles [i0, i1) of unit (b, kvh)
    const int b = tree_seq(prefix, p.B, p.Hkv, g), nb = prefix[b + 1] - prefix[b];
    const int64_t r = g - (int64_t)p.Hkv * prefix[b];
    const int kvh = (int)(r / nb), i0 = (int)(r % nb), i1 = (int)min((int64_t)nb, i0 + (g1 - g));
    g += i1 - i0;
    const int T = tree_len(p, b), n = tree_drafts(p, b, T), first = T - n;
    const int row0 = block * kRows, nrows = min(kRows, n * p.G - row0);
    if (nrows <= 0) continue;  // the same for the whole CTA
    __syncthreads();           // the last segment's shared memory is free
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
      const int row = e / (D / 4), d = (e % (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < nrows) {
        const int i = (row0 + row) / p.G, h = kvh * p.G + (row0 + row) % p.G;
        x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + ((int64_t)b * p.N + i) * p.q_stride +
                                                   (int64_t)h * D + d));
      }
      *reinterpret_cast<float4 *>(sq + row * S::QS + d) = x;
    }
    for (int row = tid; row < kRows; row += kThreads)
      bits[row] = row < nrows ? tree_bits(p, b, (row0 + row) / p.G, n) : 0ull;
    float o[R][D / 16], m[R], l[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) o[i][k] = 0.f;
    }
    for (int it = i0; it < i1; ++it) {
      const int p0 = it * kKeys;
      if (tid < kKeys) slots[tid] = p0 + tid < T ? tree_slot(p, b, p0 + tid) : -1;
      __syncthreads();  // and the last tile's K, V and weights are read
#pragma unroll 4
      for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
        const int row = e / (D / 4), d = (e % (D / 4)) * 4;
        float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
        const int64_t slot = slots[row];
        if (slot >= 0) {
          const int64_t hrow = slot * p.Hkv + kvh;
          k4 = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + hrow * D + d));
          v4 = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.v) + hrow * D + d));
        }
        *reinterpret_cast<float4 *>(sk + row * S::QS + d) = k4;
        *reinterpret_cast<float4 *>(sv + row * D + d) = v4;
      }
      __syncthreads();
      float s[R][K];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[R], k4[K];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty * R + i) * S::QS + d);
#pragma unroll
        for (int j = 0; j < K; ++j) k4[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * S::QS + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < K; ++j)
            s[i][j] = fmaf(a[i].x, k4[j].x, fmaf(a[i].y, k4[j].y, fmaf(a[i].z, k4[j].z, fmaf(a[i].w, k4[j].w, s[i][j]))));
      }
      const bool plain = p0 + kKeys <= first;  // a tile of the context alone: all of it is seen
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint64_t mk = bits[ty * R + i];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          s[i][j] *= p.c2;
          if (!plain) {
            const int t = p0 + tx + 16 * j;
            if (!(t < first || (t < T && ((mk >> (t - first)) & 1ull)))) s[i][j] = -INFINITY;
          }
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float m_new = fmaxf(m[i], mx), at = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: weights 0
        const float alpha = m[i] == m_new ? 1.f : exp2f(m[i] - at);
        m[i] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const float w = exp2f(s[i][j] - at);
          sum += w;
          sp[(ty * R + i) * S::PS + tx + 16 * j] = w;
        }
#pragma unroll
        for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[i] = l[i] * alpha + sum;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) o[i][k] *= alpha;
      }
      __syncthreads();
      // in the draft, a value that a row does not see must not reach it, not even as 0 * NaN
      auto add_values = [&](auto hide) {
#pragma unroll 2
        for (int t = 0; t < kKeys; t += 4) {
          float w[R][4];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(sp + (ty * R + i) * S::PS + t);
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
          }
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
              const float4 v4 = *reinterpret_cast<const float4 *>(sv + (t + tt) * D + k * 64 + tx * 4);
              const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
              for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float x = decltype(hide)::value && w[i][tt] == 0.f ? 0.f : v[e];
                  o[i][4 * k + e] = fmaf(w[i][tt], x, o[i][4 * k + e]);
                }
            }
        }
      };
      if (plain) add_values(std::false_type{});
      else add_values(std::true_type{});
    }
    const bool whole = i0 == 0 && i1 == nb;
    const bool begins_share = g - (i1 - i0) == share.start(group);
    float *rec = whole ? nullptr : tree_record(p, group, begins_share ? 0 : 1, block, 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = ty * R + i;
      if (row >= nrows) continue;
      if (whole) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;  // nothing seen: zeros
        const int tok = (row0 + row) / p.G, h = kvh * p.G + (row0 + row) % p.G;
        const int64_t at = ((int64_t)b * p.N + tok) * p.out_stride + h * D;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float4 x = make_float4(o[i][4 * k] * inv, o[i][4 * k + 1] * inv, o[i][4 * k + 2] * inv, o[i][4 * k + 3] * inv);
          *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + k * 64 + tx * 4) = x;
        }
      } else {
        if (tx == 0) {
          rec[row] = m[i];
          rec[kRows + row] = l[i];
        }
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
          reinterpret_cast<float4 *>(rec + 2 * kRows)[(size_t)(k * 16 + tx) * kRows + row] =
              make_float4(o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]);
      }
    }
  }
}

// ------------------------------------------------------------------ few rows
// fp32 caches and at most 16 query rows of a unit, in blocks of 8: too little work
// per byte for tiles that pass through shared memory.  A warp takes 8 positions of
// every tile for all 8 rows, its lanes D / 32 dimensions each, and K, V, Q and the
// output stay in registers; while it works on four positions the next four are on
// their way.  The products' partial sums are added by halving exchanges, which leave
// lane 8 j + r with the logit of row r at position j; the weights return through shared
// memory, and the warps' sums are joined at a segment's end.
//   1 draft x 8 heads over 60,000 tokens, 4 KV heads, D 128: 78.5 us (the tiled kernel 213)
//   2 x 8 of the same: 135 us (213); 4 x 4, 2,500 tokens, 8 KV heads: 22.4 us (36.0)
//   D 64, 8 sequences of 20,000, 4 x 4: 266 us (290); 4 of 979: 16.9 us (15.9)
// 8 rows over 27 x 10,575 tokens take 313 us (3.7 TB/s), 16 rows 594 us (882): each block
// reads K and V, so three blocks would take what the tiled kernel does.  Bound by the
// issue of two warps per scheduler (0.48 instructions a cycle, a quarter of the waiting
// for loads): 566 instructions per four positions, 256 of them products.
constexpr int kFewRows = 8, kFewWarps = 8, kFewKeys = 64, kWarpKeys = kFewKeys / kFewWarps, kStepKeys = 4;

template <int D>
__global__ void __launch_bounds__(32 * kFewWarps, 1) tree_f32_few_kernel(const TreeParams p) {
  extern __shared__ int32_t few_prefix[];
  constexpr int R = kFewRows, NV = D / 32, NS = kStepKeys * R;
  static_assert(NS == 32 && kWarpKeys == 2 * kStepKeys, "a sum per lane, two steps a tile");
  __shared__ __align__(16) float sh_s[kFewWarps][NS];
  __shared__ float sh_m[kFewWarps][R], sh_l[kFewWarps][R], sh_o[kFewWarps][R * D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x % p.blocks;
  const int64_t group = blockIdx.x / p.blocks;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) tree_prefix(p, few_prefix);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.B; i += 32 * kFewWarps) p.prefix[i] = few_prefix[i];
  const int64_t total = (int64_t)p.Hkv * few_prefix[p.B];
  if (total == 0) return;
  const TreeShare share(total, p.groups);
  const int64_t g0 = share.start(group), g1 = share.start(group + 1);
  for (int64_t g = g0; g < g1;) {
    const int b = tree_seq(few_prefix, p.B, p.Hkv, g), nb = few_prefix[b + 1] - few_prefix[b];
    const int64_t at0 = g - (int64_t)p.Hkv * few_prefix[b];
    const int kvh = (int)(at0 / nb), i0 = (int)(at0 % nb), i1 = (int)min((int64_t)nb, i0 + (g1 - g));
    const bool begins = g == g0;
    g += i1 - i0;
    const int T = tree_len(p, b), n = tree_drafts(p, b, T), first = T - n;
    const int row0 = block * R, nrows = min(R, n * p.G - row0);
    if (nrows <= 0) continue;  // the same for the whole CTA
    RowVec<NV> q[R];
    float m = -INFINITY, l = 0.f, o[R][NV];  // m of row lane % R; l over this lane's positions alone
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + min(r, nrows - 1), h = kvh * p.G + row % p.G;
      q[r].load(static_cast<const float *>(p.q) + ((int64_t)b * p.N + row / p.G) * p.q_stride + (int64_t)h * D + lane * NV);
#pragma unroll
      for (int e = 0; e < NV; ++e) o[r][e] = 0.f;
    }
    // the slots of a warp's positions in tile i, one per lane
    auto look = [&](int i) -> int64_t {
      const int t = i * kFewKeys + warp * kWarpKeys + lane % kWarpKeys;
      return i < i1 && t < T ? tree_slot(p, b, t) : -1;
    };
    auto fetch = [&](RowVec<NV> *k, RowVec<NV> *v, int64_t mine, int half) {
      const int64_t row = (max(mine, (int64_t)0) * p.Hkv + kvh) * D;
#pragma unroll
      for (int j = 0; j < kStepKeys; ++j) {
        const int64_t at = __shfl_sync(0xffffffffu, row, half * kStepKeys + j) + lane * NV;
        k[j].load(static_cast<const float *>(p.k) + at);
        v[j].load(static_cast<const float *>(p.v) + at);
      }
    };
    auto step = [&](RowVec<NV> *k, RowVec<NV> *v, int64_t mine, int half, int t0) {
      if (__any_sync(0xffffffffu, mine < 0)) {  // no position, or no such page: zeros
#pragma unroll
        for (int j = 0; j < kStepKeys; ++j) {
          if (__shfl_sync(0xffffffffu, mine, half * kStepKeys + j) < 0) {
#pragma unroll
            for (int e = 0; e < NV; ++e) k[j].x[e] = v[j].x[e] = 0.f;
          }
        }
      }
      float s[NS];
#pragma unroll
      for (int j = 0; j < kStepKeys; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float a = 0.f;
#pragma unroll
          for (int e = 0; e < NV; ++e) a = fmaf(q[r].x[e], k[j].x[e], a);
          s[j * R + r] = a;
        }
      sum_over_lanes<NS>(s, lane);
      const bool plain = t0 + kStepKeys <= first;  // positions of the context alone: all are seen
      float x = s[0] * p.c2;                       // of row lane % R at position t0 + lane / R
      if (!plain) {
        const int t = t0 + lane / R, r = lane % R;
        if (t >= first) x = t < T && r < nrows && ((tree_bits(p, b, (row0 + r) / p.G, n) >> (t - first)) & 1ull) ? x : -INFINITY;
      }
      float top = fmaxf(m, x);
#pragma unroll
      for (int d = R; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float at = top == -INFINITY ? 0.f : top, alpha = m == top ? 1.f : exp2f(m - at), w = exp2f(x - at);
      m = top;
      l = fmaf(l, alpha, w);
      sh_s[warp][lane] = w;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = __shfl_sync(0xffffffffu, alpha, r);
#pragma unroll
          for (int e = 0; e < NV; ++e) o[r][e] *= f;
        }
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < NS; e += 4) {
        const float4 y = *reinterpret_cast<const float4 *>(&sh_s[warp][e]);
        s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
      }
      __syncwarp();
      // in the draft, a value that a row does not see must not reach it, not even as 0 * NaN
      if (plain) {
#pragma unroll
        for (int j = 0; j < kStepKeys; ++j)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < NV; ++e) o[r][e] = fmaf(s[j * R + r], v[j].x[e], o[r][e]);
      } else {
#pragma unroll
        for (int j = 0; j < kStepKeys; ++j)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < NV; ++e) o[r][e] = s[j * R + r] == 0.f ? o[r][e] : fmaf(s[j * R + r], v[j].x[e], o[r][e]);
      }
    };
    // while four positions are worked on, the next four are on their way
    RowVec<NV> k0[kStepKeys], v0[kStepKeys], k1[kStepKeys], v1[kStepKeys];
    int64_t mine = look(i0), next = look(i0 + 1);
    fetch(k0, v0, mine, 0);
    for (int i = i0; i < i1; ++i) {
      const int t0 = i * kFewKeys + warp * kWarpKeys;
      fetch(k1, v1, mine, 1);
      step(k0, v0, mine, 0, t0);
      fetch(k0, v0, next, 0);
      step(k1, v1, mine, 1, t0 + kStepKeys);
      mine = next, next = look(i + 2);
    }
#pragma unroll
    for (int d = R; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane < R) sh_m[warp][lane] = m, sh_l[warp][lane] = l;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < NV; ++e) sh_o[warp][r * D + lane * NV + e] = o[r][e];
    __syncthreads();
    const bool whole = i0 == 0 && i1 == nb;
    float *rec = tree_record(p, group, begins ? 0 : 1, block, 0);
    for (int e = threadIdx.x; e < nrows * D; e += 32 * kFewWarps) {
      const int r = e / D, dim = e % D;
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, sh_m[w][r]);
      const float at = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float f = exp2f(sh_m[w][r] - at);
        L = fmaf(f, sh_l[w][r], L);
        O = fmaf(f, sh_o[w][e], O);
      }
      if (whole) {
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // nothing seen: zeros
        const int row = row0 + r, h = kvh * p.G + row % p.G;
        static_cast<float *>(p.out)[((int64_t)b * p.N + row / p.G) * p.out_stride + (int64_t)h * D + dim] = O * inv;
      } else {
        if (dim == 0) rec[r] = M, rec[R + r] = L;
        rec[2 * R + ((dim / 4) * R + r) * 4 + dim % 4] = O;
      }
    }
    __syncthreads();  // shared memory is free for the next segment
  }
}

// ------------------------------------------------------------------ combine
// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the records s of a
// cut unit, in the order of its shares.
// A warp takes 32 rows and 4 columns, a CTA 32 rows and 32 columns; the records'
// places are listed in shared memory first.
constexpr int kCombineWarps = 8;

template <int D, bool F32>
__global__ void __launch_bounds__(32 * kCombineWarps) tree_combine_kernel(const TreeParams p) {
  __shared__ int64_t sh_at[2 * kMaxTreeGroups];  // records in floats from the first, -1: none
  griddep_wait();
  griddep_launch_dependents();
  const int kvh = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x / (D / 32) * 32, col4 = blockIdx.x % (D / 32) * kCombineWarps + (threadIdx.x >> 5);
  const int T = tree_len(p, b), n = tree_drafts(p, b, T), before = p.prefix[b], nb = p.prefix[b + 1] - before;
  const int64_t total = (int64_t)p.Hkv * p.prefix[p.B];  // all fetched together
  // Two calls that use one workspace at once (which the caller has to rule out) leave another call's tiles here: the
  // outputs are theirs to lose, but every place that follows from the tiles has to lie in this workspace's records.
  if (row0 >= n * p.G || nb <= 0 || before < 0 || total <= 0) return;
  const TreeShare share(total, p.groups);
  const int64_t U0 = (int64_t)p.Hkv * before + (int64_t)kvh * nb;
  const int64_t last = share.groups - 1, c0 = min(share.owner(U0), last), c1 = min(share.owner(U0 + nb - 1), last);
  // 32 rows lie in one block and in one stream's rows, or in several blocks of fewer rows
  const int per_block = p.rows * p.streams, block = row0 / per_block, in_block = row0 % per_block;
  const bool dealt = min(per_block, n * p.G - block * per_block) > p.rows;  // the streams have rows of their own
  const int streams = dealt ? 1 : p.streams, s0 = dealt ? in_block / p.rows : 0;
  const int row_here = min(row0 + lane, n * p.G - 1), r = row_here % (dealt ? p.rows : per_block);
  const int64_t shift = (int64_t)(row_here / per_block - block) * p.streams * p.rows * (p.D + 2);
  if (c0 == c1) return;  // finished by its CTA
  const int records = (int)(c1 - c0 + 1) * streams;
  for (int i = threadIdx.x; i < records; i += 32 * kCombineWarps) {
    const int64_t c = c0 + i / streams, g0 = share.start(c), g1 = share.start(c + 1);
    const int64_t tiles = min(g1, U0 + nb) - max(g0, U0);  // of the unit in this share
    sh_at[i] = tiles > i % streams ? (int64_t)tree_record_at(p, c, g0 < U0 ? 1 : 0, block, s0 + i % streams) : -1;
  }
  __syncthreads();
  // a batch of records at a time, so that their loads are in flight together
  constexpr int kBatch = 16;
  float M = -INFINITY, L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < records; i0 += kBatch) {
    float m[kBatch], l[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t x = i0 + k < records ? sh_at[i0 + k] : -1;
      m[k] = -INFINITY, l[k] = 0.f, v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x >= 0) {
        const float *rec = p.records + x + shift;
        m[k] = __ldcg(rec + r);
        l[k] = __ldcg(rec + p.rows + r);
        v[k] = __ldcg(reinterpret_cast<const float4 *>(rec + 2 * p.rows) + (size_t)col4 * p.rows + r);
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, m[k]);
    const float at = top == -INFINITY ? 0.f : top, alpha = exp2f(M - at);  // the first batch: 0 times 0
    M = top;
    L *= alpha;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= alpha;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = exp2f(m[k] - at);
      L = fmaf(w, l[k], L);
      o[0] = fmaf(w, v[k].x, o[0]), o[1] = fmaf(w, v[k].y, o[1]), o[2] = fmaf(w, v[k].z, o[2]), o[3] = fmaf(w, v[k].w, o[3]);
    }
  }
  const int row = row0 + lane;
  if (row >= n * p.G) return;
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  const int64_t e = ((int64_t)b * p.N + row / p.G) * p.out_stride + (int64_t)(kvh * p.G + row % p.G) * D + col4 * 4;
  if constexpr (F32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + e) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + e) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
}

}  // namespace

int tree_f32_few_rows() { return kFewRows; }
int tree_f32_ctas_per_sm(int D, int rows, int keys) {
  if (rows == kFewRows) return 1;
  if (D == 64) return rows == 32 && keys == 32 ? 3 : 2;
  return rows == 32 ? 2 : 1;
}

cudaError_t launch_tree_f32(const TreeParams &p, cudaStream_t s) {
  auto run = [&](auto kern, size_t bytes) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (int)bytes);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3((unsigned)(p.groups * p.blocks)), dim3(kThreads), bytes, s, 0, p);
  };
  auto shape = [&](auto rows, auto keys) {
    constexpr int R = decltype(rows)::value, K = decltype(keys)::value;
    return p.D == 64 ? run(tree_f32_kernel<64, R, K>, TreeF32Smem<64, R, K>::bytes(p.B))
                     : run(tree_f32_kernel<128, R, K>, TreeF32Smem<128, R, K>::bytes(p.B));
  };
  using S32 = std::integral_constant<int, 32>;
  using S64 = std::integral_constant<int, 64>;
  if (p.rows == kFewRows) {
    auto few = [&](auto kern) {
      const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (kMaxBatchSmem + 1) * 4);
      return e != cudaSuccess ? e : launch_ex(kern, dim3((unsigned)(p.groups * p.blocks)), dim3(32 * kFewWarps), (size_t)(p.B + 1) * 4, s, 0, p);
    };
    return p.D == 64 ? few(tree_f32_few_kernel<64>) : few(tree_f32_few_kernel<128>);
  }
  if (p.rows == 32) return p.tile == 32 ? shape(S32{}, S32{}) : shape(S32{}, S64{});
  return shape(S64{}, S64{});
}

cudaError_t launch_tree_combine(const TreeParams &p, bool f32, cudaStream_t s) {
  const dim3 grid((unsigned)((p.N * p.G + 31) / 32 * (p.D / 32)), (unsigned)p.Hkv, (unsigned)p.B), block(32 * kCombineWarps);
  if (f32)
    return p.D == 64 ? launch_ex(tree_combine_kernel<64, true>, grid, block, 0, s, 0, p)
                     : launch_ex(tree_combine_kernel<128, true>, grid, block, 0, s, 0, p);
  return p.D == 64 ? launch_ex(tree_combine_kernel<64, false>, grid, block, 0, s, 0, p)
                   : launch_ex(tree_combine_kernel<128, false>, grid, block, 0, s, 0, p);
}

}  // namespace hs2
