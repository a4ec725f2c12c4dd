// hs2_tree.cu -- attention of a tree of drafted tokens over the cache: the
// CUDA-core kernel, and the kernel that joins the records of cut units.
//
// Token i of sequence b (n drafted tokens, the last n of T rows) attends to the
// T - n rows of the context and to the drafts j with bit j of its mask set:
//   o = sum_t p_t v_t / sum_t p_t,  p_t = 2^(c2 q.k_t - m),  m the running max.
//
// fp32 caches keep fp32 products on the CUDA cores (tensor cores would round
// the operands): a CTA of 16 x 16 threads takes 64 rows x 64 positions, each
// thread a 4 x 4 block of the logits and 4 rows x D / 16 columns of the output
// in registers; Q, K, V and the weights are in shared memory, K's and Q's rows
// padded by 16 bytes so that 16-byte reads of 8 rows meet 32 banks.
#include <type_traits>

#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_tree_common.cuh"

namespace hs2 {

namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;

template <int D>
struct TreeF32Smem {
  static constexpr int QS = D + 4, PS = kKeys + 4;
  static constexpr size_t kQ = 0, kK = kQ + (size_t)kRows * QS * 4, kV = kK + (size_t)kKeys * QS * 4,
                          kP = kV + (size_t)kKeys * D * 4, kBits = kP + (size_t)kRows * PS * 4,
                          kPrefix = kBits + kRows * 8;
  static size_t bytes(int B) { return kPrefix + (size_t)(B + 1) * 4; }
};

// 4 elements of a cache row as fp32
template <int DT>
__device__ __forceinline__ float4 load_kv4(const void *x, int64_t e, float scale) {
  if constexpr (DT == HS2_F32) {
    return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(x) + e));
  } else if constexpr (DT == HS2_BF16) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(x) + e));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(x) + e));
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(w, lo, hi);
    __half2 a, b;
    memcpy(&a, &lo, 4);
    memcpy(&b, &hi, 4);
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    return make_float4(fa.x * scale, fa.y * scale, fb.x * scale, fb.y * scale);
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) tree_cuda_core_kernel(const TreeParams p) {
  using S = TreeF32Smem<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *sq = reinterpret_cast<float *>(smem + S::kQ), *sk = reinterpret_cast<float *>(smem + S::kK);
  float *sv = reinterpret_cast<float *>(smem + S::kV), *sp = reinterpret_cast<float *>(smem + S::kP);
  uint64_t *bits = reinterpret_cast<uint64_t *>(smem + S::kBits);
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
  const TreeShare share{total, p.groups};
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
        x = load_kv4<DT == HS2_F32 ? HS2_F32 : HS2_BF16>(p.q, ((int64_t)b * p.N + i) * p.q_stride + h * D + d, 1.f);
      }
      *reinterpret_cast<float4 *>(sq + row * S::QS + d) = x;
    }
    for (int row = tid; row < kRows; row += kThreads)
      bits[row] = row < nrows ? tree_bits(p, b, (row0 + row) / p.G, n) : 0ull;
    float o[4][D / 16], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) o[i][k] = 0.f;
    }
    for (int it = i0; it < i1; ++it) {
      const int p0 = it * kKeys;
      __syncthreads();  // the last tile's K, V and weights are read
      for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
        const int row = e / (D / 4), d = (e % (D / 4)) * 4;
        float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
        const int64_t slot = p0 + row < T ? tree_slot(p, b, p0 + row) : -1;
        if (slot >= 0) {
          const int64_t hrow = slot * p.Hkv + kvh;
          k4 = load_kv4<DT>(p.k, hrow * D + d, DT == HS2_E4M3 ? __ldg(p.k_scale + hrow) : 1.f);
          v4 = load_kv4<DT>(p.v, hrow * D + d, DT == HS2_E4M3 ? __ldg(p.v_scale + hrow) : 1.f);
        }
        *reinterpret_cast<float4 *>(sk + row * S::QS + d) = k4;
        *reinterpret_cast<float4 *>(sv + row * D + d) = v4;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], k4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + i) * S::QS + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * S::QS + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(a[i].x, k4[j].x, fmaf(a[i].y, k4[j].y, fmaf(a[i].z, k4[j].z, fmaf(a[i].w, k4[j].w, s[i][j]))));
      }
      const bool plain = p0 + kKeys <= first;  // a tile of the context alone: all of it is seen
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t mk = bits[ty * 4 + i];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
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
        for (int j = 0; j < 4; ++j) {
          const float w = exp2f(s[i][j] - at);
          sum += w;
          sp[(ty * 4 + i) * S::PS + tx + 16 * j] = w;
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
          float w[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(sp + (ty * 4 + i) * S::PS + t);
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
          }
#pragma unroll
          for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
              const float4 v4 = *reinterpret_cast<const float4 *>(sv + (t + tt) * D + k * 64 + tx * 4);
              const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
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
    float *rec = whole ? nullptr : tree_record(p, group, begins_share ? 0 : 1, block);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = ty * 4 + i;
      if (row >= nrows) continue;
      if (whole) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;  // nothing seen: zeros
        const int tok = (row0 + row) / p.G, h = kvh * p.G + (row0 + row) % p.G;
        const int64_t at = ((int64_t)b * p.N + tok) * p.out_stride + h * D;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float4 x = make_float4(o[i][4 * k] * inv, o[i][4 * k + 1] * inv, o[i][4 * k + 2] * inv, o[i][4 * k + 3] * inv);
          if constexpr (DT == HS2_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + k * 64 + tx * 4) = x;
          } else {
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at + k * 64 + tx * 4) =
                make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
          }
        }
      } else {
        if (tx == 0) {
          rec[row] = m[i];
          rec[kRows + row] = l[i];
        }
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
          *reinterpret_cast<float4 *>(rec + 2 * kRows + (size_t)row * D + k * 64 + tx * 4) =
              make_float4(o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]);
      }
    }
  }
}

// ------------------------------------------------------------------ combine
// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the shares s of a
// cut unit, in share order; one warp per row.
constexpr int kCombineWarps = 8;

template <int D, bool F32>
__global__ void __launch_bounds__(32 * kCombineWarps) tree_combine_kernel(const TreeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int kvh = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  const int T = tree_len(p, b), n = tree_drafts(p, b, T);
  if (row >= n * p.G) return;
  const int64_t total = (int64_t)p.Hkv * p.prefix[p.B];
  const int nb = p.prefix[b + 1] - p.prefix[b];
  if (nb == 0 || total == 0) return;
  const TreeShare share{total, p.groups};
  const int64_t U0 = (int64_t)p.Hkv * p.prefix[b] + (int64_t)kvh * nb;
  const int64_t c0 = share.owner(U0), c1 = share.owner(U0 + nb - 1);
  if (c0 == c1) return;  // finished by its CTA
  const int block = row / p.rows, r = row % p.rows;
  auto record = [&](int64_t c) { return tree_record(p, c, c == c0 && share.start(c) < U0 ? 1 : 0, block); };
  auto holds = [&](int64_t c) { return share.start(c + 1) > share.start(c); };
  float M = -INFINITY;
  for (int64_t c = c0 + lane; c <= c1; c += 32)
    if (holds(c)) M = fmaxf(M, __ldcg(record(c) + r));
  M = warp_max(M);
  const float at = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
#pragma unroll 4
  for (int64_t c = c0; c <= c1; ++c) {
    if (!holds(c)) continue;
    const float *rec = record(c);
    const float w = exp2f(__ldcg(rec + r) - at);
    L += w * __ldcg(rec + p.rows + r);
    const float *x = rec + 2 * p.rows + (size_t)r * D + lane * (D / 32);
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(x));
      o[0] += w * v.x, o[1] += w * v.y, o[2] += w * v.z, o[3] += w * v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2 *>(x));
      o[0] += w * v.x, o[1] += w * v.y;
    }
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  const int64_t e = ((int64_t)b * p.N + row / p.G) * p.out_stride + (kvh * p.G + row % p.G) * D + lane * (D / 32);
#pragma unroll
  for (int k = 0; k < D / 32; k += 2) {
    if constexpr (F32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + e + k) = make_float2(o[k] * inv, o[k + 1] * inv);
    else *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + e + k) = pack_bf16(o[k] * inv, o[k + 1] * inv);
  }
}

}  // namespace

int tree_f32_rows() { return kRows; }
int tree_f32_tile() { return kKeys; }
int tree_f32_ctas_per_sm(int D) { return D == 64 ? 3 : 1; }

cudaError_t launch_tree_f32(const TreeParams &p, int kv_dtype, cudaStream_t s) {
  auto run = [&](auto kern, size_t bytes) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (int)bytes);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3((unsigned)(p.groups * p.blocks)), dim3(kThreads), bytes, s, 0, p);
  };
  if (kv_dtype == HS2_E4M3) return run(tree_cuda_core_kernel<HS2_E4M3, 128>, TreeF32Smem<128>::bytes(p.B));
  if (kv_dtype == HS2_BF16)
    return p.D == 64 ? run(tree_cuda_core_kernel<HS2_BF16, 64>, TreeF32Smem<64>::bytes(p.B))
                     : run(tree_cuda_core_kernel<HS2_BF16, 128>, TreeF32Smem<128>::bytes(p.B));
  return p.D == 64 ? run(tree_cuda_core_kernel<HS2_F32, 64>, TreeF32Smem<64>::bytes(p.B))
                   : run(tree_cuda_core_kernel<HS2_F32, 128>, TreeF32Smem<128>::bytes(p.B));
}

cudaError_t launch_tree_combine(const TreeParams &p, bool f32, cudaStream_t s) {
  const dim3 grid((unsigned)((p.N * p.G + kCombineWarps - 1) / kCombineWarps), (unsigned)p.Hkv, (unsigned)p.B), block(32 * kCombineWarps);
  if (f32)
    return p.D == 64 ? launch_ex(tree_combine_kernel<64, true>, grid, block, 0, s, 0, p)
                     : launch_ex(tree_combine_kernel<128, true>, grid, block, 0, s, 0, p);
  return p.D == 64 ? launch_ex(tree_combine_kernel<64, false>, grid, block, 0, s, 0, p)
                   : launch_ex(tree_combine_kernel<128, false>, grid, block, 0, s, 0, p);
}

}  // namespace hs2
