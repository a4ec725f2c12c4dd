// hs2_rope.cu -- rotary positions on new tokens' queries and keys, and the
// append of their K/V rows to the paged cache.
//
// For a token at position p, pair i of a head's first `rot` elements turns by
// the angle p f_i:  (x, y) -> s (x cos - y sin, y cos + x sin), s the table's
// factor; the other elements and the values pass through.
//
// Angles: the table holds F_i = round(f_i / 2 pi * 2^64), so p F_i mod 2^64 is
// the angle's fraction of a turn with no reduction error at any position
// (fp32 angles are wrong by ~0.1 rad at position 10^6), and one sincospi per
// (token, pair) serves every head of the token.
//
// Bound by reading q, k, v once and writing q and the rows once.  A CTA takes
// 1 or 4 tokens: their sines go to shared memory first, then each thread
// moves 16 elements of a head -- both ends of 8 pairs, so the rotation needs
// no exchange -- as 16-byte loads and stores.  The D / 16 threads of a head are
// neighbours in a warp, so an E4M3 row's maximum is a shuffle reduction.
#include "hs2.h"
#include "hs2_internal.h"

namespace hs2 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens per CTA of a large call

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// codes nearest x / scale, ties to even, saturated at +-448
__device__ __forceinline__ void store8_e4m3(uint8_t *p, const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __nv_fp8_e4m3 c0(x[4 * k] / scale), c1(x[4 * k + 1] / scale), c2(x[4 * k + 2] / scale), c3(x[4 * k + 3] / scale);
    w[k] = (uint32_t)c0.__x | ((uint32_t)c1.__x << 8) | ((uint32_t)c2.__x << 16) | ((uint32_t)c3.__x << 24);
  }
  *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 sh_cs[kRopeTokens][D / 2];
  __shared__ int64_t sh_slot[kRopeTokens];  // the token's cache row, -1: none, -2: no such token
  constexpr int LPH = D / 16;               // threads per head
  griddep_wait();
  griddep_launch_dependents();
  const int tok0 = blockIdx.x * p.tokens_per_cta;
  const int ntok = min(p.tokens_per_cta, p.B * p.N - tok0);
  const int half = p.rot / 2;
  if ((int)threadIdx.x < ntok) {
    const int b = (tok0 + threadIdx.x) / p.N, i = (tok0 + threadIdx.x) % p.N;
    const int len = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
    const int n = clamp_len(p.num_new ? __ldg(p.num_new + b) : p.N, min(p.N, len));
    int64_t slot = -2;
    if (i < n) {
      const int pos = len - n + i;
      slot = p.page_table == nullptr
                 ? (int64_t)b * p.page_size + pos
                 : (int64_t)__ldg(p.page_table + (int64_t)b * p.max_pages + pos / p.page_size) * p.page_size +
                       pos % p.page_size;
      if (slot < 0 || slot >= p.num_slots) slot = -1;  // a page outside the cache: no row is written
    }
    sh_slot[threadIdx.x] = slot;
  }
  for (int e = threadIdx.x; e < ntok * half; e += kRopeThreads) {
    const int t = e / half, i = e % half;
    const uint64_t a = (uint64_t)(int64_t)__ldg(p.positions + tok0 + t) * __ldg(p.table + i);
    float s, c;
    sincospif((float)(int64_t)a * 0x1p-63f, &s, &c);  // half turns in [-1, 1)
    sh_cs[t][i] = make_float2(c * p.mscale, s * p.mscale);
  }
  __syncthreads();
  const int heads = p.Hq + 2 * p.Hkv, per_tok = heads * LPH;
  const int total = ntok * per_tok, step = kRopeThreads * gridDim.y;
  for (int e0 = blockIdx.y * kRopeThreads + (threadIdx.x & ~31); e0 < total; e0 += step) {
    const bool idle = e0 + (int)(threadIdx.x & 31) >= total;  // past the end: only takes part in the shuffles
    const int e = idle ? total - 1 : e0 + (int)(threadIdx.x & 31);
    const int t = e / per_tok, h = (e % per_tok) / LPH, l = e % LPH;
    const int64_t slot = sh_slot[t], tok = tok0 + t;
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    const int kvh = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
    const T *src = is_q   ? static_cast<const T *>(p.q) + tok * p.q_stride + (int64_t)h * D
                   : is_v ? static_cast<const T *>(p.v) + tok * p.v_stride + (int64_t)kvh * D
                          : static_cast<const T *>(p.k) + tok * p.k_stride + (int64_t)kvh * D;
    const bool turn = !is_v && 16 * l < p.rot;
    // the two runs of 8 elements: both ends of 8 pairs (half layout), or 16 in a row
    const int ea = turn && !p.interleaved ? 8 * l : 16 * l;
    const int eb = turn && !p.interleaved ? half + 8 * l : 16 * l + 8;
    const bool here = !idle && slot != -2 && (is_q ? p.q != nullptr : slot >= 0);
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
    if (here) {
      load8(src + ea, a);
      load8(src + eb, b);
    }
    if (turn) {
      if (!p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 cs = sh_cs[t][8 * l + i];
          const float x = a[i], y = b[i];
          a[i] = x * cs.x - y * cs.y;
          b[i] = y * cs.x + x * cs.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 ca = sh_cs[t][8 * l + i], cb = sh_cs[t][8 * l + 4 + i];
          const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
          a[2 * i] = x * ca.x - y * ca.y;
          a[2 * i + 1] = y * ca.x + x * ca.y;
          b[2 * i] = z * cb.x - w * cb.y;
          b[2 * i + 1] = w * cb.x + z * cb.y;
        }
      }
    }
    if constexpr (FP8) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
      for (int o = LPH / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (here && !is_q) {
        const float scale = amax / 448.f > 0.f ? amax / 448.f : 1.f;
        uint8_t *dst = static_cast<uint8_t *>(is_v ? p.cv : p.ck) + (slot * p.Hkv + kvh) * D;
        store8_e4m3(dst + ea, a, scale);
        store8_e4m3(dst + eb, b, scale);
        if (l == 0) (is_v ? p.v_scale : p.k_scale)[slot * p.Hkv + kvh] = scale;
      }
    } else if (here && !is_q) {
      T *dst = static_cast<T *>(is_v ? p.cv : p.ck) + (slot * p.Hkv + kvh) * D;
      store8(dst + ea, a);
      store8(dst + eb, b);
    }
    if (here && is_q) {
      T *dst = static_cast<T *>(p.q_out) + tok * (int64_t)p.Hq * D + (int64_t)h * D;
      store8(dst + ea, a);
      store8(dst + eb, b);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p0, int sms, cudaStream_t s) {
  RopeParams p = p0;
  const int64_t tokens = (int64_t)p.B * p.N;
  const int items = (p.Hq + 2 * p.Hkv) * (p.D / 16);
  // one token per CTA, its heads dealt over as many CTAs as there are items
  // for, while the tokens alone do not fill the GPU
  p.tokens_per_cta = tokens >= 8 * sms ? kRopeTokens : 1;
  const int gy = p.tokens_per_cta > 1 || tokens >= 2 * sms ? 1 : (items + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid((unsigned)((tokens + p.tokens_per_cta - 1) / p.tokens_per_cta), gy), block(kRopeThreads);
  if (p.kv_dtype == HS2_E4M3) return launch_ex(rope_kernel<__nv_bfloat16, 128, true>, grid, block, 0, s, 0, p);
  if (p.kv_dtype == HS2_BF16)
    return p.D == 64 ? launch_ex(rope_kernel<__nv_bfloat16, 64, false>, grid, block, 0, s, 0, p)
                     : launch_ex(rope_kernel<__nv_bfloat16, 128, false>, grid, block, 0, s, 0, p);
  return p.D == 64 ? launch_ex(rope_kernel<float, 64, false>, grid, block, 0, s, 0, p)
                   : launch_ex(rope_kernel<float, 128, false>, grid, block, 0, s, 0, p);
}

}  // namespace hs2
