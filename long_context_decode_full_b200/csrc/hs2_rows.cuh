// hs2_rows.cuh -- fp32 rows of K and V held across a warp: a lane has D / 32
// neighbouring dimensions, so a row is one coalesced load and needs no shared
// memory.
#pragma once

#include "hs2_common.cuh"

namespace hs2 {

namespace {

template <int N>
struct RowVec {
  float x[N];
  __device__ __forceinline__ void load(const float *p) {
    if constexpr (N == 4) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
      x[0] = v.x, x[1] = v.y;
    }
  }
};

// Sums of N values over the 32 lanes: halves are exchanged while there are two or
// more, so value i ends in the lanes whose upper log2 N bits are i (N <= 32), or in
// the lane i / (N / 32), N / 32 values each.
template <int N>
__device__ __forceinline__ void sum_over_lanes(float *x, int lane) {
  int o = 16;
#pragma unroll
  for (int n = N; n > 1 && o > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? x[i] : x[i + n / 2], keep = up ? x[i + n / 2] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o > 0; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
}

}  // namespace

}  // namespace hs2
