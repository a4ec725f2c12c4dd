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
// Bound by reading q, k, v once and writing q and the rows once.  A CTA takes a
// run of tokens, 32 at a time: their sines go to shared memory, then each
// thread takes 16 elements of a head -- both ends of 8 pairs, so the rotation needs
// no exchange -- of one token after the other, the next one's loads under way.
// The D / 16 threads of a head are neighbours in a warp, so an E4M3 row's maximum
// is a shuffle reduction.  (A thread per token and head: twice the instructions,
// 50 us for 12,003 tokens into an E4M3 cache; four tokens in registers at once: too
// few threads, 64 us.)
#include "hs2.h"
#include "hs2_internal.h"
#include "hs2_pair.cuh"

namespace hs2 {

namespace {

constexpr int kRopeThreads = 320;  // at most
constexpr int kRopeTokens = 32;  // whose sines are in shared memory

// 8 elements as they are in memory, and as fp32
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = sizeof(T) == 4 ? __uint_as_float(u[i]) : __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
  }
};
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// x / scale as a division rounds it, for 16 elements of one scale: the product with the
// rounded reciprocal, corrected twice by its remainder.  A remainder x - q scale is exact in
// one fused operation; the first correction leaves q within a unit in the last place, from
// where the second one gives the rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990).
// The reciprocal alone is off by up to a unit and a half, and a quotient next to the middle
// of two codes took the other one.  (16 divisions a thread made the two warps of keys and
// values the last of ten: 48 us for 12,003 tokens into an E4M3 cache.)
struct RowScale {
  float scale, by, minus_inverse;  // the row's scale; the divisor and its reciprocal for elements times 2^64 or 1
  bool tiny;
  __device__ __forceinline__ explicit RowScale(float amax) {
    scale = amax / 448.f > 0.f ? amax / 448.f : 1.f;
    tiny = scale < 0x1p-60f;  // remainders would be subnormal: elements and scale times 2^64
    by = tiny ? scale * 0x1p64f : scale;
    minus_inverse = -1.f / by;
    if (by == INFINITY) by = 0.f;  // finite elements give 0, infinite ones NaN
  }
  __device__ __forceinline__ float2 quotient(float2 x) const {
    const float2 n = make_float2(minus_inverse, minus_inverse), d = make_float2(by, by), m = make_float2(-x.x, -x.y);
    float2 q = mul2(m, n);
    q = fma2(fma2(q, d, m), n, q);
    return fma2(fma2(q, d, m), n, q);
  }
};
// The codes nearest x / scale, ties to even, saturated at +-448.
__device__ __forceinline__ void store8_e4m3(uint8_t *p, float (&x)[8], const RowScale &s) {
  if (s.tiny) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(s.quotient(make_float2(x[4 * k], x[4 * k + 1])), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(s.quotient(make_float2(x[4 * k + 2], x[4 * k + 3])), __NV_SATFINITE, __NV_E4M3);
    w[k] = lo | hi << 16;
  }
  *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 ? 3 : 2) rope_kernel(const RopeParams p) {
  __shared__ float2 sh_cs[kRopeTokens][D / 2];
  __shared__ int64_t sh_slot[kRopeTokens];  // the token's cache row, -1: none, -2: no such token
  constexpr int LPH = D / 16;               // threads per head
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tokens = (int64_t)p.B * p.N;
  const int begin = (int)(blockIdx.x * tokens / gridDim.x), end = (int)((blockIdx.x + 1) * tokens / gridDim.x);
  const int half = p.rot / 2;
  const int items = (p.Hq + 2 * p.Hkv) * LPH;  // of one token: 16 elements each
  struct Item {
    int h, l, kvh, ea, eb;
    bool is_q, is_v, turn;
  };
  auto item = [&](int e) {
    Item x;
    x.h = e / LPH, x.l = e % LPH;
    x.is_q = x.h < p.Hq, x.is_v = x.h >= p.Hq + p.Hkv;
    x.kvh = x.is_v ? x.h - p.Hq - p.Hkv : x.h - p.Hq;
    x.turn = !x.is_v && 16 * x.l < p.rot;
    // the two runs of 8 elements: both ends of 8 pairs (half layout), or 16 in a row
    x.ea = x.turn && !p.interleaved ? 8 * x.l : 16 * x.l;
    x.eb = x.turn && !p.interleaved ? half + 8 * x.l : 16 * x.l + 8;
    return x;
  };
  auto stride_of = [&](const Item &x) { return x.is_q ? p.q_stride : (x.is_v ? p.v_stride : p.k_stride); };
  auto source = [&](const Item &x, int64_t tok) {
    return static_cast<const T *>(x.is_q ? p.q : (x.is_v ? p.v : p.k)) + tok * stride_of(x) + (x.is_q ? x.h : x.kvh) * D;
  };
  const int first = blockIdx.y * blockDim.x + threadIdx.x;
  for (int tok0 = begin; tok0 < end; tok0 += kRopeTokens) {
  const int ntok = min(kRopeTokens, end - tok0);
  Raw8<T> ra, rb;
  if (first < items) {  // the first token's elements are on the way during the sines
    const Item x = item(first);
    const T *src = source(x, tok0);
    ra.load(src + x.ea);
    rb.load(src + x.eb);
  }
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
  for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
    const int t = e / half, i = e % half;
    const uint64_t a = (uint64_t)(int64_t)__ldg(p.positions + tok0 + t) * __ldg(p.table + i);
    float s, c;
    sincospif((float)(int64_t)a * 0x1p-63f, &s, &c);  // half turns in [-1, 1)
    sh_cs[t][i] = make_float2(c * p.mscale, s * p.mscale);
  }
  __syncthreads();
  for (int e0 = first & ~31; e0 < items; e0 += blockDim.x * gridDim.y) {
    const bool idle = e0 + (int)(threadIdx.x & 31) >= items;  // past the end: only takes part in the shuffles
    const Item x = item(idle ? items - 1 : e0 + (int)(threadIdx.x & 31));
    const int h = x.h, l = x.l, kvh = x.kvh, ea = x.ea, eb = x.eb;
    const bool is_q = x.is_q, is_v = x.is_v, turn = x.turn;
    const int64_t stride = stride_of(x);
    const T *src = source(x, tok0);
    if (e0 != (first & ~31)) {
      ra.load(src + ea);
      rb.load(src + eb);
    }
    const bool rows = __any_sync(0xffffffffu, !is_q);  // the warp writes to the cache
    for (int t = 0; t < ntok; ++t) {
      const int64_t slot = sh_slot[t];
      const bool here = !idle && slot != -2 && (is_q || slot >= 0);
      float a[8], b[8];
      ra.get(a);
      rb.get(b);
      if (t + 1 < ntok) {  // tokens that a sequence does not have are read, too, and dropped
        ra.load(src + (t + 1) * stride + ea);
        rb.load(src + (t + 1) * stride + eb);
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
      if (rows) {
        const int64_t at = slot * p.Hkv + kvh;
        if constexpr (FP8) {
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          if (here && !is_q) {
            const RowScale s(amax);
            uint8_t *dst = static_cast<uint8_t *>(is_v ? p.cv : p.ck) + at * D;
            store8_e4m3(dst + ea, a, s);
            store8_e4m3(dst + eb, b, s);
            if (l == 0) (is_v ? p.v_scale : p.k_scale)[at] = s.scale;
          }
        } else if (here && !is_q) {
          T *dst = static_cast<T *>(is_v ? p.cv : p.ck) + at * D;
          store8(dst + ea, a);
          store8(dst + eb, b);
        }
      }
      if (here && is_q) {
        T *dst = static_cast<T *>(p.q_out) + ((tok0 + t) * (int64_t)p.Hq + h) * D;
        store8(dst + ea, a);
        store8(dst + eb, b);
      }
    }
  }
  __syncthreads();  // the sines and places are used
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int sms, cudaStream_t s) {
  const int64_t tokens = (int64_t)p.B * p.N;
  const int items = (p.Hq + 2 * p.Hkv) * (p.D / 16);
  // one token per CTA, its heads dealt over CTAs of 128 threads, while the tokens alone do not fill the GPU; else as
  // many CTAs as fit beside each other, with equal runs of tokens
  const bool few = tokens < 2 * sms;
  const int passes = (items + kRopeThreads - 1) / kRopeThreads;
  const int threads = few ? 128 : ((items + passes - 1) / passes + 31) / 32 * 32;
  const int64_t fit = (int64_t)sms * (p.kv_dtype == HS2_F32 ? 2 : 3) * (threads <= 160 ? 2 : 1);
  const int64_t gx = few || tokens < fit ? tokens : fit, gy = few ? (items + 127) / 128 : 1;
  const dim3 grid((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535)), block(threads);
  if (p.kv_dtype == HS2_E4M3) return launch_ex(rope_kernel<__nv_bfloat16, 128, true>, grid, block, 0, s, 0, p);
  if (p.kv_dtype == HS2_BF16)
    return p.D == 64 ? launch_ex(rope_kernel<__nv_bfloat16, 64, false>, grid, block, 0, s, 0, p)
                     : launch_ex(rope_kernel<__nv_bfloat16, 128, false>, grid, block, 0, s, 0, p);
  return p.D == 64 ? launch_ex(rope_kernel<float, 64, false>, grid, block, 0, s, 0, p)
                   : launch_ex(rope_kernel<float, 128, false>, grid, block, 0, s, 0, p);
}

}  // namespace hs2
