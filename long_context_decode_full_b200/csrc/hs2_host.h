// hs2_host.h -- host-side helpers of the C-ABI layer shared by its translation
// units (not part of the public ABI): error texts, argument checks and the
// cached tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hs2.h"

namespace hs2 {

// Sets the thread's hs2_last_error() text and returns `code`.
int fail(int code, const char *fmt, ...);
int cuda_fail(cudaError_t e, const char *what);
int sm_count();  // of the current device

bool aligned16(const void *p);
bool group_ok(int G);
int check_caches(const hs2_cache *k, const hs2_cache *v);
// A q / out descriptor against the cache; `what` names it in errors.
int check_heads(const hs2_heads *h, const hs2_cache *k, const char *what);
// The page table's capacity per sequence in *t_cap, or the contiguous layout's.
int check_pages(const hs2_cache *k, const int32_t *page_table, int32_t max_pages, int32_t batch, int64_t *t_cap);

// Tensor map of a cache: (head_dim, heads, slots), boxes of 128 bytes x
// box_rows slots, 128-byte swizzle; the last few are kept.
int cache_map(CUtensorMap *map, const hs2_cache *c, int box_rows);

}  // namespace hs2
