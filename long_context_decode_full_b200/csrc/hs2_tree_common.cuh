// hs2_tree_common.cuh -- what the kernels of the drafted-tree attention agree
// on: the balanced partition of the tiles, a unit's rows and masks, and the
// records of units that are cut.
//
// A unit is a (sequence, kv head); its query rows are the n drafted tokens'
// heads of the group, row r = token r / G, head r % G, in blocks of p.rows x
// p.streams.  Tiles of p.tile positions are ordered by (sequence, kv head, tile)
// and cut into p.groups equal shares; the p.blocks CTAs of a share walk the same
// tiles with a row block each, side by side, so the later ones find K and V in L2.
//
// A CTA has p.streams sets of p.rows running sums.  A block of more than p.rows
// rows deals its rows to the streams, a smaller one its tiles.  A unit inside one
// share is finished by its CTA; of one that is cut, each stream with tiles leaves
// a record (m, l, o) per share, rows in base-2 exponents: slot 0 if the unit begins
// the share, else slot 1 (a share cuts at most the unit it begins with and the one
// it ends with; slot 2 is the CTA's own, to join its streams).  A record is
// m[rows], l[rows] and o as [D / 4][rows] groups of 4 columns, so that
// neighbouring rows are written and read side by side.
#pragma once

#include "hs2_internal.h"

namespace hs2 {

namespace {

// The tiles of every share; with fewer tiles than shares the last shares are empty.
struct TreeShare {
  int64_t total;  // Hkv * sum_b tiles
  int32_t groups;
  __device__ __forceinline__ TreeShare(int64_t tiles, int32_t shares)
      : total(tiles), groups((int32_t)min((int64_t)shares, tiles > 0 ? tiles : 1)) {}
  __device__ __forceinline__ int64_t start(int64_t c) const { return min(c, (int64_t)groups) * total / groups; }
  __device__ __forceinline__ int64_t owner(int64_t x) const { return ((x + 1) * groups - 1) / total; }
};

__device__ __forceinline__ int tree_len(const TreeParams &p, int b) {
  return clamp_len(__ldg(p.seq_lens + b), (int)p.t_cap);
}
// drafted tokens of sequence b, the last n of its T rows
__device__ __forceinline__ int tree_given_drafts(const TreeParams &p, int b) {
  return p.num_draft ? __ldg(p.num_draft + b) : p.N;
}
__device__ __forceinline__ int tree_drafts(const TreeParams &p, int b, int T) {
  return clamp_len(tree_given_drafts(p, b), min(p.N, T));
}
// the drafts that token i of sequence b sees
__device__ __forceinline__ uint64_t tree_bits(const TreeParams &p, int b, int i, int n) {
  const uint64_t m = p.mask ? __ldg(p.mask + (int64_t)b * p.N + i) : (2ull << i) - 1ull;
  return n >= 64 ? m : m & ((1ull << n) - 1ull);
}
// prefix[b] = tiles before sequence b, by one warp
__device__ __forceinline__ void tree_prefix(const TreeParams &p, int32_t *prefix) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int b = base + lane;
    int x = b < p.B ? (tree_len(p, b) + p.tile - 1) / p.tile : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (b < p.B) prefix[b + 1] = carry + x;
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) prefix[0] = 0;
}
// last sequence b with Hkv * prefix[b] <= x
__device__ __forceinline__ int tree_seq(const int32_t *prefix, int B, int Hkv, int64_t x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)Hkv * prefix[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int64_t tree_slot(const TreeParams &p, int b, int64_t pos) {
  const uint32_t at = (uint32_t)pos, ps = (uint32_t)p.page_size;  // lengths fit 31 bits
  const int64_t s = p.page_table == nullptr ? (int64_t)b * p.page_size + pos
                                            : (int64_t)__ldg(p.page_table + (int64_t)b * p.max_pages + at / ps) * ps + at % ps;
  return s >= 0 && s < p.num_slots ? s : -1;
}
__device__ __forceinline__ size_t tree_record_at(const TreeParams &p, int64_t group, int slot, int block, int stream) {
  return ((((size_t)group * kTreeSlots + slot) * p.blocks + block) * p.streams + stream) * (size_t)p.rows * (p.D + 2);
}
__device__ __forceinline__ float *tree_record(const TreeParams &p, int64_t group, int slot, int block, int stream) {
  return p.records + tree_record_at(p, group, slot, block, stream);
}

}  // namespace

}  // namespace hs2
