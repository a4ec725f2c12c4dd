// hs2_accumulate.cu -- running sums of the full layer's attention weights.
//
// After the attention kernel has left the raw logits s_{h,t} and the segment
// records, acc[t] = decay * acc[t] + sum_h 2^(a s_{h,t} - b_h) with a = c
// log2(e) and b_h = LSE_h log2(e); the newest `fresh` tokens start at their
// first weight.  a and b_h are carried as float pairs, so the exponent's one
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
  constexpr int Q = G >= 16 ? 1 : (G >= 8 ? 2 : 4);  // positions of a thread in flight
  for (int tb = t0 + (int)threadIdx.x; tb < t1; tb += Q * kAccThreads) {
    float raw[Q][G], old[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int t = tb + q * kAccThreads;
      old[q] = 0.f;
      if (t >= t1) continue;
      if (t < ui.T - ap.fresh) old[q] = __ldcs(acc + t);
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
      acc[t] = t < ui.T - ap.fresh ? fmaf(ap.decay, old[q], w[0]) : w[0];
    }
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

cudaError_t launch_accumulate(const AccumulateParams &p, cudaStream_t s) {
  return p.sp.D == 64 ? run<64>(p, s) : run<128>(p, s);
}

}  // namespace hs2
