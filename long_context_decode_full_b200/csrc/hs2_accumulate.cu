// hs2_accumulate.cu -- running sums of the full layer's attention weights.
//
// After the attention kernel has left the raw logits s_{h,t} and the segment
// records, acc[t] = decay * acc[t] + sum_h 2^(a s_{h,t} - b_h) with a = c
// log2(e) and b_h = LSE_h log2(e); the newest `fresh` tokens (of each sequence, as
// many as it has gained since the last call) start at their first weight.  a and b_h are carried as float pairs, so the exponent's one
// rounding of consequence is the fused multiply-add's (below 2^-20 for weights
// above 2^-16).
//
// Bound by reading the logits (from L2 as far as they fit: the attention kernel
// marks them evict-last) and by reading and writing the sums once: 34 us beside the
// attention's 350 at 4 x 262,144 tokens, 8 heads a group, 6.5 TB/s with the logits'
// write.  The grid is
// one wave of position chunks, plus the CTAs that join the records into the
// attention output.
#include "hs2_internal.h"
#include "hs2_rows.cuh"
#include "hs2_select_common.cuh"

namespace hs2 {

namespace {

constexpr int kAccThreads = 256;

template <int G, int D>
__global__ void __launch_bounds__(kAccThreads) accumulate_kernel(const AccumulateParams ap) {
  __shared__ uint32_t sh_weights[kHistBins];  // combine CTAs: the records' weights
  __shared__ double sh_red[kAccThreads];
  __shared__ double sh_lse[G];
  __shared__ float sh_M[G], sh_L[G];
  __shared__ uint8_t sh_ok[kMaxRecords];
  constexpr int RS = G * (D + 2);
  const ScoreParams &p = ap.sp;
  griddep_wait();
  griddep_launch_dependents();
  const int chunk = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int comb = chunk - ((int)gridDim.x - p.ncomb);
  UnitInfo ui = unit_info(p, b, kvh);
  const int t0 = chunk * p.score_chunk, t1 = min(ui.T, t0 + p.score_chunk);
  if (comb < 0 && t0 >= ui.T) return;
  const int64_t u = (int64_t)b * p.Hkv + kvh;
  mark_records(ui, sh_ok);
  unit_lse<G, D>(p.ws.records + (size_t)u * p.R * RS, ui, p.c, sh_lse, sh_M, sh_L, sh_red);
  if (comb >= 0) {
    combine_unit<G, D>(p, ui, u, comb, sh_M, sh_L, sh_weights);
    return;
  }
  const double ad = (double)p.c * kLog2e;
  const float a_hi = (float)ad, a_lo = (float)(ad - (double)a_hi);
  float b_hi[G], b_lo[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const double bd = sh_lse[h] * kLog2e;
    b_hi[h] = (float)bd;
    b_lo[h] = (float)(bd - (double)b_hi[h]);
  }
  const float *lg = p.ws.logits + (size_t)u * p.ustride * G;
  float *acc = ap.acc + (size_t)u * ap.acc_stride;
  const int old_end = ui.T - (ap.fresh_each ? clamp_len(__ldg(ap.fresh_each + b), ui.T) : ap.fresh);  // sums below go on
  constexpr int Q = G >= 16 ? 1 : (G >= 8 ? 2 : 4);  // positions of a thread in flight
  for (int tb = t0 + (int)threadIdx.x; tb < t1; tb += Q * kAccThreads) {
    float raw[Q][G], old[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int t = tb + q * kAccThreads;
      old[q] = 0.f;
      if (t >= t1) continue;
      if (t < old_end) old[q] = __ldcs(acc + t);
      if constexpr (G % 4 == 0) {
#pragma unroll
        for (int h4 = 0; h4 < G / 4; ++h4) {
          const float4 v4 = __ldcs(reinterpret_cast<const float4 *>(lg + (size_t)t * G) + h4);
          raw[q][4 * h4] = v4.x;
          raw[q][4 * h4 + 1] = v4.y;
          raw[q][4 * h4 + 2] = v4.z;
          raw[q][4 * h4 + 3] = v4.w;
        }
      } else {
#pragma unroll
        for (int h = 0; h < G; ++h) raw[q][h] = __ldcs(lg + (size_t)t * G + h);
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int t = tb + q * kAccThreads;
      if (t >= t1) continue;
      float w[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float y = fmaf(raw[q][h], a_hi, -b_hi[h]), low = fmaf(raw[q][h], a_lo, -b_lo[h]);
        w[h] = exp2f(y + low);
      }
#pragma unroll
      for (int s = 1; s < G; s <<= 1)
#pragma unroll
        for (int h = 0; h + s < G; h += 2 * s) w[h] += w[h + s];
      acc[t] = t < old_end ? fmaf(ap.decay, old[q], w[0]) : w[0];
    }
  }
}

// ------------------------------------------------------------------ fp32 caches
// The attention of the call over an fp32 cache: logits and segment records as
// full_attn_f32_kernel leaves them (the same shares of 64-position tiles).  A warp
// takes 8 rows of every tile for all heads of the group: a lane has D / 32
// neighbouring dimensions, so a row of K or V is one 512- or 256-byte load; the
// 8 G products' partial sums are added over the lanes by halving exchanges and
// passed to all lanes through shared memory; the warps' sums are joined at a
// segment's end.  Bound by reading K and V (8 warps of 8 rows: 64 KB per CTA on the
// way).  One warp per head, as in that kernel, leaves most of an SM idle for small
// groups: 10 sequences of up to 17,430 tokens, 8 kv heads of one query head, d 128,
// take 140 us with the update (525 us with that kernel; the bytes' floor is 111).
constexpr int kRowWarps = 8, kRowTile = 64, kWarpRows = kRowTile / kRowWarps;

template <int G, int D>
__global__ void __launch_bounds__(32 * kRowWarps) rows_attn_f32_kernel(const FullParams p) {
  extern __shared__ int32_t sh_prefix[];
  __shared__ __align__(16) float sh_s[kRowWarps][kWarpRows * G];
  __shared__ float sh_m[kRowWarps][G], sh_l[kRowWarps][G], sh_o[kRowWarps][G * D];
  constexpr int NV = D / 32, NS = kWarpRows * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int x = b < p.B ? (clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap) + kRowTile - 1) / kRowTile : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.B) sh_prefix[b + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) sh_prefix[0] = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.B; i += 32 * kRowWarps) p.ws.prefix[i] = sh_prefix[i];
  const int64_t total = (int64_t)p.Hkv * sh_prefix[p.B];
  if (total == 0) return;
  const Partition part{total, p.N};
  const int64_t g1 = part.start(blockIdx.x + 1);
  const float cl = p.c * 1.4426950408889634f;
  for (int64_t g = part.start(blockIdx.x); g < g1;) {
    int lo = 0, hi = p.B - 1;  // the sequence of tile g
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)p.Hkv * sh_prefix[mid] <= g) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, nb = sh_prefix[b + 1] - sh_prefix[b];
    const int64_t r = g - (int64_t)p.Hkv * sh_prefix[b];
    const int kvh = (int)(r / nb), i0 = (int)(r % nb), i1 = (int)min((int64_t)nb, i0 + (g1 - g));
    const int64_t u = (int64_t)b * p.Hkv + kvh, U = (int64_t)p.Hkv * sh_prefix[b] + (int64_t)kvh * nb;
    g += i1 - i0;
    const int T = clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
    RowVec<NV> q[G];
    float m[G], l[G], o[G][NV];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      q[h].load(static_cast<const float *>(p.q) + (u * G + h) * D + lane * NV);
      m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < NV; ++e) o[h][e] = 0.f;
    }
    for (int i = i0; i < i1; ++i) {
      const int t0 = i * kRowTile + warp * kWarpRows;
      int64_t mine = -1;  // lane's row's place
      if (lane < kWarpRows && t0 + lane < T) {
        const int pos = t0 + lane;
        mine = p.page_table == nullptr ? (int64_t)b * p.page_size + pos
                                       : (int64_t)__ldg(p.page_table + (int64_t)b * p.max_pages + pos / p.page_size) * p.page_size +
                                             pos % p.page_size;
        if (mine < 0 || mine >= p.num_slots) mine = -1;
      }
      RowVec<NV> k[kWarpRows], v[kWarpRows];
#pragma unroll
      for (int j = 0; j < kWarpRows; ++j) {
        const int64_t slot = __shfl_sync(0xffffffffu, mine, j);
        if (slot >= 0) {
          const int64_t at = (slot * p.Hkv + kvh) * D + lane * NV;
          k[j].load(static_cast<const float *>(p.k) + at);
          v[j].load(static_cast<const float *>(p.v) + at);
        } else {
#pragma unroll
          for (int e = 0; e < NV; ++e) k[j].x[e] = v[j].x[e] = 0.f;
        }
      }
      float s[NS];
#pragma unroll
      for (int j = 0; j < kWarpRows; ++j)
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float a = 0.f;
#pragma unroll
          for (int e = 0; e < NV; ++e) a = fmaf(q[h].x[e], k[j].x[e], a);
          s[j * G + h] = a;
        }
      sum_over_lanes<NS>(s, lane);
      constexpr int kPer = NS >= 32 ? NS / 32 : 1, kShare = NS >= 32 ? 1 : 32 / NS;  // sums of a lane, lanes of a sum
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int at = lane / kShare * kPer + e, j = at / G;
        if (lane % kShare == 0) {
          sh_s[warp][at] = t0 + j < T ? s[e] : -INFINITY;
          if (t0 + j < T) p.ws.logits[(u * p.ustride + t0 + j) * G + at % G] = s[e];
        }
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < NS; e += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(&sh_s[warp][e]);
        s[e] = x.x, s[e + 1] = x.y, s[e + 2] = x.z, s[e + 3] = x.w;
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float top = m[h];
#pragma unroll
        for (int j = 0; j < kWarpRows; ++j) top = fmaxf(top, s[j * G + h]);
        const float at = top == -INFINITY ? 0.f : top, alpha = m[h] == top ? 1.f : exp2f((m[h] - at) * cl);
        m[h] = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kWarpRows; ++j) {
          s[j * G + h] = exp2f((s[j * G + h] - at) * cl);
          sum += s[j * G + h];
        }
        l[h] = fmaf(l[h], alpha, sum);
#pragma unroll
        for (int e = 0; e < NV; ++e) {
          float a = o[h][e] * alpha;
#pragma unroll
          for (int j = 0; j < kWarpRows; ++j) a = fmaf(s[j * G + h], v[j].x[e], a);
          o[h][e] = a;
        }
      }
    }
    // the warps' sums to the segment's record
#pragma unroll
    for (int h = 0; h < G; ++h) {
      if (lane == 0) sh_m[warp][h] = m[h], sh_l[warp][h] = l[h];
#pragma unroll
      for (int e = 0; e < NV; ++e) sh_o[warp][h * D + lane * NV + e] = o[h][e];
    }
    __syncthreads();
    const int64_t rec_at = blockIdx.x - part.cfirst(U);
    if (rec_at < 0 || rec_at >= p.R) {
      if (threadIdx.x == 0) set_error(p.ws.err, kErrRecord);
    } else {
      float *rec = p.ws.records + (size_t)(u * p.R + rec_at) * G * (D + 2);
      for (int e = threadIdx.x; e < G * D; e += 32 * kRowWarps) {
        const int h = e / D;
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, sh_m[w][h]);
        const float at = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
          const float f = exp2f((sh_m[w][h] - at) * cl);
          L = fmaf(f, sh_l[w][h], L);
          O = fmaf(f, sh_o[w][e], O);
        }
        if (e % D == 0) rec[h] = M, rec[G + h] = L;
        rec[2 * G + e] = O;
      }
    }
    __syncthreads();  // shared memory is free for the next segment
  }
}

template <int D>
cudaError_t run_rows(const FullParams &p, int grid, cudaStream_t s) {
  const size_t smem = (size_t)(p.B + 1) * 4;
  auto go = [&](auto kern) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), (kMaxBatchSmem + 1) * 4);
    return e != cudaSuccess ? e : launch_ex(kern, dim3(grid), dim3(32 * kRowWarps), smem, s, 0, p);
  };
  switch (p.G) {
    case 1: return go(rows_attn_f32_kernel<1, D>);
    case 2: return go(rows_attn_f32_kernel<2, D>);
    case 4: return go(rows_attn_f32_kernel<4, D>);
    default: return go(rows_attn_f32_kernel<8, D>);
  }
}

template <int D>
cudaError_t run(const AccumulateParams &p, cudaStream_t s) {
  const ScoreParams &sp = p.sp;
  const dim3 grid((unsigned)((sp.t_cap + sp.score_chunk - 1) / sp.score_chunk + sp.ncomb), sp.Hkv, sp.B), block(kAccThreads);
  switch (sp.G) {
    case 1: return launch_ex(accumulate_kernel<1, D>, grid, block, 0, s, 0, p);
    case 2: return launch_ex(accumulate_kernel<2, D>, grid, block, 0, s, 0, p);
    case 4: return launch_ex(accumulate_kernel<4, D>, grid, block, 0, s, 0, p);
    case 8: return launch_ex(accumulate_kernel<8, D>, grid, block, 0, s, 0, p);
    case 16: return launch_ex(accumulate_kernel<16, D>, grid, block, 0, s, 0, p);
    default: return launch_ex(accumulate_kernel<32, D>, grid, block, 0, s, 0, p);
  }
}

}  // namespace

cudaError_t launch_rows_f32(const FullParams &p, int grid, cudaStream_t s) {
  if (p.tile != kRowTile) return cudaErrorInvalidValue;  // the shares that the update reads back
  return p.D == 64 ? run_rows<64>(p, grid, s) : run_rows<128>(p, grid, s);
}

cudaError_t launch_accumulate(const AccumulateParams &p, cudaStream_t s) {
  return p.sp.D == 64 ? run<64>(p, s) : run<128>(p, s);
}

}  // namespace hs2
