// hs2_api.cu -- the C ABI of libhs2 (declared in include/hs2.h): argument
// validation, workspace layout, TMA descriptors and the launch sequence of
// the full-attention + selection call and of the sparse call.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <mutex>

#include "hs2.h"
#include "hs2_fused_tail.cuh"
#include "hs2_host.h"
#include "hs2_internal.h"

namespace hs2 {

static thread_local char g_err[512] = "";

int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char *what) {
  return fail(HS2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

namespace {
constexpr int kMaxDevices = 64;
constexpr int kMaxCtasPerSm = 4;  // bound used to size the per-unit record slots

}  // namespace

int sm_count() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cache[dev] = n;
  }
  return cache[dev];
}

namespace {

// ---------------------------------------------------------------- TMA encode
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// [num_slots, Hkv, D] cache -> 3-D map (D, Hkv, slots), box (128 bytes, 1, rows), 128-byte swizzle.
int encode_cache_map(CUtensorMap *map, const hs2_cache *c, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(HS2_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const int es = c->dtype == HS2_BF16 ? 2 : 1;
  cuuint64_t dims[3] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->num_kv_heads, (cuuint64_t)c->num_slots};
  cuuint64_t strides[2] = {(cuuint64_t)c->head_dim * es, (cuuint64_t)c->head_dim * c->num_kv_heads * es};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), 1u, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = fn(map, c->dtype == HS2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                  const_cast<void *>(c->data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(HS2_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return HS2_OK;
}

// The tensor map of a cache depends only on its pointer, shape, element type
// and box: the last few are kept, so a decode loop encodes them once.
struct MapKey {
  const void *data;
  int dtype, heads, dim, box, dev;
  int64_t slots;
  bool operator==(const MapKey &o) const {
    return data == o.data && dtype == o.dtype && heads == o.heads && dim == o.dim && box == o.box && dev == o.dev &&
           slots == o.slots;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap map;
  bool used;
};
std::mutex g_map_mu;
MapEntry g_maps[16];
int g_map_next = 0;

}  // namespace

int cache_map(CUtensorMap *map, const hs2_cache *c, int box_rows) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  const MapKey key{c->data, (int)c->dtype, c->num_kv_heads, c->head_dim, box_rows, dev, c->num_slots};
  {
    std::lock_guard<std::mutex> lock(g_map_mu);
    for (const MapEntry &e : g_maps)
      if (e.used && e.key == key) {
        *map = e.map;
        return HS2_OK;
      }
  }
  const int rc = encode_cache_map(map, c, box_rows);
  if (rc) return rc;
  std::lock_guard<std::mutex> lock(g_map_mu);
  g_maps[g_map_next] = MapEntry{key, *map, true};
  g_map_next = (g_map_next + 1) % 16;
  return HS2_OK;
}

namespace {

// ---------------------------------------------------------------- workspace
struct Layout {
  size_t err, prefix, records, logits, scores, above, cand, subcnt, hist, thr, lse, total;
  int R, nsub;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int64_t unit_stride(int64_t t_cap) { return (t_cap + 127) / 128 * 128; }

Layout layout(int B, int Hkv, int G, int D, int64_t t_cap_in) {
  Layout L;
  const size_t U = (size_t)B * Hkv;
  const int64_t t_cap = unit_stride(t_cap_in);  // per-unit arrays keep 16-byte aligned rows
  L.nsub = (int)((t_cap + kSubRange - 1) / kSubRange);
  L.R = sm_count() * kMaxCtasPerSm / Hkv + 2;  // <= 1024 for up to 255 SMs
  size_t o = 0;
  L.err = o;
  o += 256;
  L.prefix = o;
  o = align256(o + (size_t)(B + 1) * 4);
  L.records = o;
  o = align256(o + U * L.R * G * (D + 2) * 4);
  L.logits = o;
  o = align256(o + U * (size_t)t_cap * G * 4);
  L.scores = o;
  o = align256(o + U * (size_t)t_cap * 4);
  L.above = o;
  o = align256(o + U * (size_t)t_cap * 4);
  L.cand = o;
  o = align256(o + U * (size_t)t_cap * 8);
  L.subcnt = o;
  o = align256(o + U * (size_t)L.nsub * 8);
  L.hist = o;  // hist [U][4096], ticket [U], spare [U] back to back
  o = align256(o + U * (kHistBins + 2) * 4);
  L.thr = o;
  o = align256(o + U * 8);
  L.lse = o;
  o = align256(o + U * kMaxGroup * sizeof(double));
  L.total = o;
  return L;
}

FullWs bind(const Layout &L, void *ws, int B, int Hkv) {
  uint8_t *w = static_cast<uint8_t *>(ws);
  const size_t U = (size_t)B * Hkv;
  FullWs f;
  f.err = reinterpret_cast<uint32_t *>(w + L.err);
  f.prefix = reinterpret_cast<int32_t *>(w + L.prefix);
  f.records = reinterpret_cast<float *>(w + L.records);
  f.logits = reinterpret_cast<float *>(w + L.logits);
  f.scores = reinterpret_cast<float *>(w + L.scores);
  f.above = reinterpret_cast<int32_t *>(w + L.above);
  f.cand = reinterpret_cast<uint2 *>(w + L.cand);
  f.subcnt = reinterpret_cast<int2 *>(w + L.subcnt);
  f.hist = reinterpret_cast<uint32_t *>(w + L.hist);
  f.ticket = f.hist + U * kHistBins;
  f.thr = reinterpret_cast<int2 *>(w + L.thr);
  f.lse = reinterpret_cast<double *>(w + L.lse);
  return f;
}

}  // namespace

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool group_ok(int G) { return G == 1 || G == 2 || G == 4 || G == 8 || G == 16 || G == 32; }

// Checks a q/out descriptor against the cache; `what` names it in errors.
int check_heads(const hs2_heads *h, const hs2_cache *k, const char *what) {
  if (!h || !h->data) return fail(HS2_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(h->data)) return fail(HS2_ERR_INVALID_ARG, "%s data is not 16-byte aligned", what);
  if (h->batch < 1 || h->batch > 65535) return fail(HS2_ERR_INVALID_ARG, "%s batch %d out of [1, 65535]", what, h->batch);
  if (h->head_dim != k->head_dim)
    return fail(HS2_ERR_INVALID_ARG, "%s head_dim %d != cache head_dim %d", what, h->head_dim, k->head_dim);
  if (h->num_heads < 1 || h->num_heads % k->num_kv_heads)
    return fail(HS2_ERR_INVALID_ARG, "%s num_heads %d is not a multiple of num_kv_heads %d", what, h->num_heads,
                k->num_kv_heads);
  if (!group_ok(h->num_heads / k->num_kv_heads))
    return fail(HS2_ERR_UNSUPPORTED, "GQA group %d not built (1, 2, 4, 8, 16 or 32)", h->num_heads / k->num_kv_heads);
  if (k->dtype == HS2_F32 && h->num_heads / k->num_kv_heads > 8)
    return fail(HS2_ERR_UNSUPPORTED, "fp32 caches take GQA groups of at most 8 heads");
  const int want = k->dtype == HS2_F32 ? HS2_F32 : HS2_BF16;
  if (h->dtype != want)
    return fail(HS2_ERR_UNSUPPORTED, "%s dtype %d with cache dtype %d (need %s)", what, h->dtype, k->dtype,
                want == HS2_F32 ? "HS2_F32" : "HS2_BF16");
  return HS2_OK;
}

int check_caches(const hs2_cache *k, const hs2_cache *v) {
  if (!k || !v || !k->data || !v->data) return fail(HS2_ERR_INVALID_ARG, "k_cache / v_cache is NULL");
  if (k->dtype != v->dtype || k->num_kv_heads != v->num_kv_heads || k->head_dim != v->head_dim ||
      k->page_size != v->page_size || k->num_slots != v->num_slots)
    return fail(HS2_ERR_INVALID_ARG, "k_cache and v_cache descriptors disagree");
  if (k->dtype != HS2_F32 && k->dtype != HS2_BF16 && k->dtype != HS2_E4M3)
    return fail(HS2_ERR_UNSUPPORTED, "cache dtype %d", k->dtype);
  if (k->head_dim != 64 && k->head_dim != 128) return fail(HS2_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", k->head_dim);
  if (k->dtype == HS2_E4M3 && k->head_dim != 128) return fail(HS2_ERR_UNSUPPORTED, "E4M3 caches need head_dim 128");
  if (k->num_kv_heads < 1 || k->num_kv_heads > 65535) return fail(HS2_ERR_INVALID_ARG, "num_kv_heads %d", k->num_kv_heads);
  if (k->num_slots < 1 || k->num_slots >= (int64_t(1) << 31))
    return fail(HS2_ERR_INVALID_ARG, "num_slots %lld out of [1, 2^31)", (long long)k->num_slots);
  if (k->page_size < 1) return fail(HS2_ERR_INVALID_ARG, "page_size %d", k->page_size);
  if (!aligned16(k->data) || !aligned16(v->data)) return fail(HS2_ERR_INVALID_ARG, "cache data not 16-byte aligned");
  if (k->dtype == HS2_E4M3) {
    if (!k->scale || !v->scale) return fail(HS2_ERR_INVALID_ARG, "E4M3 caches need k and v scales");
    if ((reinterpret_cast<uintptr_t>(k->scale) | reinterpret_cast<uintptr_t>(v->scale)) & 3)
      return fail(HS2_ERR_INVALID_ARG, "scales are misaligned");
  } else if (k->scale || v->scale) {
    return fail(HS2_ERR_INVALID_ARG, "scales are only used with HS2_E4M3 caches");
  }
  return HS2_OK;
}

int check_pages(const hs2_cache *k, const int32_t *page_table, int32_t max_pages, int32_t batch, int64_t *t_cap) {
  if (batch < 1) return fail(HS2_ERR_INVALID_ARG, "batch %d", batch);
  if (batch > kMaxBatchSmem) return fail(HS2_ERR_UNSUPPORTED, "batch %d > %d", batch, kMaxBatchSmem);
  if (page_table) {
    if (max_pages < 1) return fail(HS2_ERR_INVALID_ARG, "max_pages %d with a page table", max_pages);
    *t_cap = (int64_t)max_pages * k->page_size;
  } else {
    if (max_pages != 1) return fail(HS2_ERR_INVALID_ARG, "contiguous layout (no page table) needs max_pages == 1");
    *t_cap = k->page_size;
    if ((int64_t)batch * k->page_size > k->num_slots)
      return fail(HS2_ERR_INVALID_ARG, "contiguous layout needs num_slots >= batch * page_size");
  }
  if (*t_cap > kMaxContext || (int64_t)batch * ((*t_cap + 15) / 16) * k->num_kv_heads >= (int64_t(1) << 31))
    return fail(HS2_ERR_UNSUPPORTED, "context capacity %lld too large (max %lld per sequence)", (long long)*t_cap,
                (long long)kMaxContext);
  return HS2_OK;
}

}  // namespace hs2

using namespace hs2;

namespace {

// Consumer warps, pipeline stages and slices per warp of the attention
// kernel, most preferred first: enough independent work per SM sub-partition
// to hide the MMA and conversion latencies, and enough stages that the bytes
// in flight per SM cover the loaded HBM latency.  A tile must fit the page
// size (one divides the other) in at most 8 page boxes.
bool tile_fits_pages(int tile, int page_size, bool paged) {
  if (!paged) return true;
  if (page_size % tile == 0) return true;
  return tile % page_size == 0 && tile / page_size <= 8;
}

// A warp serves 8 nt query heads, so with more heads per group than that the
// consumer warps split into ceil(G / (8 nt)) head groups and their count must
// divide by it.  Groups of 16 and more heads take nt = 2 where a configuration
// is built for it (each shared-memory fragment then feeds two MMAs).
FullMmaConfig pick_full_config(int D, bool fp8, int page_size, bool paged, int G, int batch) {
  static const FullMmaConfig bf16_128[] = {{4, 3, 2, 1, 0}, {8, 3, 1, 1, 0}, {4, 6, 1, 1, 0}};
  static const FullMmaConfig bf16_64[] = {{8, 6, 1, 1, 0}, {4, 6, 1, 1, 0}};
  static const FullMmaConfig e4m3[] = {{8, 3, 2, 1, 0}, {12, 4, 1, 1, 0}, {8, 6, 1, 1, 0}, {4, 8, 1, 1, 0}};
  // 16 heads per warp: one consumer warp per SM sub-partition with all 255
  // registers measured fastest (MQA at 256K bf16: 136 us against 144 us with
  // 8 warps x 1 slice and 154 us with 8-head warps; at 1M E4M3: 151 us
  // against 160 us with 8-head warps; 8-warp E4M3 variants spilled, 179 us)
  static const FullMmaConfig bf16_128_wide[] = {{4, 3, 2, 2, 0}, {8, 3, 1, 2, 0}};
  static const FullMmaConfig bf16_64_wide[] = {{8, 6, 1, 2, 0}};
  static const FullMmaConfig e4m3_wide[] = {{4, 6, 2, 2, 0}};
  // Groups of 16 or 32 heads over a bf16 cache with d 128 can run both
  // products on tcgen05 (accumulators in tensor memory; "4,3,2,2,1" below).
  // Measured at MQA 256K: attention 133 us against 134 us for the 16-head
  // mma.sync warps (the logit write-back, not the tensor math, bounds it),
  // and the step 3% slower (at 223 KB of shared memory no score CTA fits
  // beside the attention CTA at the kernel boundary), so it is opt-in.
  const bool tc_ok = D == 128 && (G == 16 || G == 32) && full_tc_smem_bytes(batch, fp8) <= 232448 &&
                     tile_fits_pages(128, page_size, paged);
  auto heads_split = [&](const FullMmaConfig &c) { return c.ncw % ((G + 8 * c.nt - 1) / (8 * c.nt)) == 0; };
  auto fits = [&](const FullMmaConfig &c) {
    return heads_split(c) && tile_fits_pages(16 * c.ncw * c.nsl, page_size, paged);
  };
  if (const char *env = getenv("HS2_FULL_CFG")) {  // tuning override: "ncw,nstage[,nsl[,nt[,tc]]]"
    int a = 0, b = 0, c = 1, d = 1, t = 0;
    if (sscanf(env, "%d,%d,%d,%d,%d", &a, &b, &c, &d, &t) >= 2 && a >= 1 && a <= 16 && b >= 1 && b <= 16 &&
        (c == 1 || c == 2) && (d == 1 || (d == 2 && G >= 16)) &&
        (t == 0 || (t == 1 && tc_ok && a == 4 && b == 3 && c == 2 && d == 2))) {
      const FullMmaConfig e{a, b, c, d, t};
      if (fits(e)) return e;
    }
  }
  if (G >= 16) {
    const FullMmaConfig *wide = fp8 ? e4m3_wide : (D == 64 ? bf16_64_wide : bf16_128_wide);
    const int nw = fp8 ? 1 : (D == 64 ? 1 : 2);
    for (int i = 0; i < nw; ++i)
      if (fits(wide[i])) return wide[i];
  }
  const FullMmaConfig *list = fp8 ? e4m3 : (D == 64 ? bf16_64 : bf16_128);
  const int n = fp8 ? 4 : (D == 64 ? 2 : 3);
  for (int i = 0; i < n; ++i)
    if (fits(list[i])) return list[i];
  return list[n - 1];
}

int full_attn_select_impl(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                          const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages, int32_t window,
                          int32_t k_global, int32_t block, hs2_heads *out, int32_t *idx_out, void *workspace,
                          size_t workspace_bytes, void *stream, void *mark_event, bool fused = false,
                          AccumulateParams *accumulate = nullptr);

}  // namespace

extern "C" {

const char *hs2_last_error(void) { return g_err; }

int hs2_version(void) { return 100; }

size_t hs2_full_attn_select_workspace(int32_t batch, int32_t num_kv_heads, int32_t group, int32_t head_dim,
                                      int64_t t_cap) {
  if (batch < 1 || num_kv_heads < 1 || !group_ok(group) || (head_dim != 64 && head_dim != 128) || t_cap < 1 ||
      t_cap > kMaxContext)
    return 0;
  return layout(batch, num_kv_heads, group, head_dim, t_cap).total;
}

int hs2_full_attn_select(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                         const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages, int32_t window,
                         int32_t k_global, hs2_heads *out, int32_t *idx_out, void *workspace,
                         size_t workspace_bytes, void *stream) {
  return hs2_full_attn_select_marked(q, k_cache, v_cache, seq_lens, page_table, max_pages, window, k_global, out,
                                     idx_out, workspace, workspace_bytes, stream, nullptr);
}

int hs2_full_attn_select_marked(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                                const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages,
                                int32_t window, int32_t k_global, hs2_heads *out, int32_t *idx_out,
                                void *workspace, size_t workspace_bytes, void *stream, void *mark_event) {
  return full_attn_select_impl(q, k_cache, v_cache, seq_lens, page_table, max_pages, window, k_global, 0, out,
                               idx_out, workspace, workspace_bytes, stream, mark_event);
}

int hs2_full_attn_select_fused(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                               const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages,
                               int32_t window, int32_t k_global, hs2_heads *out, int32_t *idx_out, void *workspace,
                               size_t workspace_bytes, void *stream) {
  return full_attn_select_impl(q, k_cache, v_cache, seq_lens, page_table, max_pages, window, k_global, 0, out,
                               idx_out, workspace, workspace_bytes, stream, nullptr, true);
}

int hs2_full_attn_select_blocks(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                                const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages,
                                int32_t window, int32_t k_global, int32_t block, hs2_heads *out, int32_t *idx_out,
                                void *workspace, size_t workspace_bytes, void *stream) {
  if (block < 1 || k_global < 0 || k_global % block != 0)
    return fail(HS2_ERR_INVALID_ARG, "block %d must be >= 1 and divide k_global %d", block, k_global);
  return full_attn_select_impl(q, k_cache, v_cache, seq_lens, page_table, max_pages, window, k_global, block, out,
                               idx_out, workspace, workspace_bytes, stream, nullptr);
}

int hs2_full_attn_accumulate(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                             const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages, float decay,
                             int32_t fresh, float *acc, int64_t acc_stride, hs2_heads *out, void *workspace,
                             size_t workspace_bytes, void *stream) {
  AccumulateParams ap{};
  ap.acc = acc;
  ap.acc_stride = acc_stride;
  ap.decay = decay;
  ap.fresh = fresh;
  return full_attn_select_impl(q, k_cache, v_cache, seq_lens, page_table, max_pages, 0, 0, 0, out, nullptr, workspace,
                               workspace_bytes, stream, nullptr, false, &ap);
}

int hs2_full_attn_accumulate_each(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                                  const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages, float decay,
                                  const int32_t *fresh, float *acc, int64_t acc_stride, hs2_heads *out,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  if (!fresh) return fail(HS2_ERR_INVALID_ARG, "fresh is NULL");
  AccumulateParams ap{};
  ap.acc = acc;
  ap.acc_stride = acc_stride;
  ap.decay = decay;
  ap.fresh_each = fresh;
  return full_attn_select_impl(q, k_cache, v_cache, seq_lens, page_table, max_pages, 0, 0, 0, out, nullptr, workspace,
                               workspace_bytes, stream, nullptr, false, &ap);
}

}  // extern "C"

namespace {

// The full layer, then token-level selection (block = 0), block-level selection
// with blocks of `block` positions, or (accumulate) the weights' running sums in
// place of a selection.
int full_attn_select_impl(const hs2_heads *q, const hs2_cache *k_cache, const hs2_cache *v_cache,
                          const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages, int32_t window,
                          int32_t k_global, int32_t block, hs2_heads *out, int32_t *idx_out, void *workspace,
                          size_t workspace_bytes, void *stream, void *mark_event, bool fused,
                          AccumulateParams *accumulate) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if ((rc = check_heads(q, k_cache, "q"))) return rc;
  if ((rc = check_heads(out, k_cache, "out"))) return rc;
  if (out->batch != q->batch || out->num_heads != q->num_heads || out->dtype != q->dtype)
    return fail(HS2_ERR_INVALID_ARG, "out shape/dtype differs from q");
  if (!seq_lens || (!idx_out && !accumulate)) return fail(HS2_ERR_INVALID_ARG, "seq_lens / idx_out is NULL");
  if (accumulate) {
    if (!accumulate->acc || (reinterpret_cast<uintptr_t>(accumulate->acc) & 3))
      return fail(HS2_ERR_INVALID_ARG, "acc is NULL or misaligned");
    if (accumulate->fresh < 0) return fail(HS2_ERR_INVALID_ARG, "fresh %d", accumulate->fresh);
  } else if (window < 0 || k_global < 0 || (int64_t)window + k_global < 1 || (int64_t)window + k_global > kMaxSelect)
    return fail(HS2_ERR_INVALID_ARG, "window %d / k_global %d (need 1 <= window + k_global <= %d)", window,
                k_global, kMaxSelect);
  const int B = q->batch, Hkv = k_cache->num_kv_heads, G = q->num_heads / Hkv, D = k_cache->head_dim;
  const int ps = k_cache->page_size;
  const bool paged = page_table != nullptr;
  int64_t t_cap;
  if (paged) {
    if (max_pages < 1) return fail(HS2_ERR_INVALID_ARG, "max_pages %d with a page table", max_pages);
    t_cap = (int64_t)max_pages * ps;
  } else {
    if (max_pages != 1) return fail(HS2_ERR_INVALID_ARG, "contiguous layout (no page table) needs max_pages == 1");
    t_cap = ps;
    if ((int64_t)B * ps > k_cache->num_slots)
      return fail(HS2_ERR_INVALID_ARG, "contiguous layout needs num_slots >= batch * page_size");
  }
  if (t_cap > kMaxContext || (int64_t)B * ((t_cap + 15) / 16) * Hkv >= (int64_t(1) << 31))
    return fail(HS2_ERR_UNSUPPORTED, "context capacity %lld too large (max %lld per sequence)", (long long)t_cap,
                (long long)kMaxContext);
  if (B > kMaxBatchSmem) return fail(HS2_ERR_UNSUPPORTED, "batch %d > %d", B, kMaxBatchSmem);
  if (accumulate && accumulate->acc_stride < t_cap)
    return fail(HS2_ERR_INVALID_ARG, "acc_stride %lld < capacity %lld", (long long)accumulate->acc_stride,
                (long long)t_cap);
  const bool mma = k_cache->dtype != HS2_F32;
  if (mma && paged && !(ps % 16 == 0 && (ps % 64 == 0 || 64 % ps == 0)))
    return fail(HS2_ERR_UNSUPPORTED, "page_size %d (16, 32 or a multiple of 64)", ps);
  const Layout L = layout(B, Hkv, G, D, t_cap);
  if (!workspace) return fail(HS2_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(HS2_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < L.total)
    return fail(HS2_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, L.total);

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  FullParams p{};
  p.q = q->data;
  p.k = k_cache->data;
  p.v = v_cache->data;
  p.k_scale = k_cache->scale;
  p.v_scale = v_cache->scale;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.B = B;
  p.Hkv = Hkv;
  p.G = G;
  p.D = D;
  p.page_size = ps;
  p.max_pages = paged ? max_pages : 1;
  p.t_cap = t_cap;
  p.ustride = unit_stride(t_cap);
  p.num_slots = k_cache->num_slots;
  p.R = L.R;
  p.c = 1.0f / sqrtf((float)D);
  p.ws = bind(L, workspace, B, Hkv);
  {  // the logits this call writes, bounded by the sequence capacity: small next to the 126 MB L2?
    const double logit_bytes = (double)B * Hkv * (double)t_cap * G * 4.0;
    p.kv_evict_first = logit_bytes <= 48.0 * (1 << 20) ? 1 : 0;
  }
  const int sms = sm_count();
  cudaError_t e;
  const bool fp8 = k_cache->dtype == HS2_E4M3;
  FullMmaConfig cfg{};
  if (!mma) {
    p.tile = full_f32_tile();
    p.N = sms * full_f32_ctas_per_sm();
  } else {
    cfg = pick_full_config(D, fp8, ps, paged, G, B);
    p.tile = 16 * cfg.ncw * cfg.nsl;
    p.N = sms;
  }
  ScoreParams sp{};
  sp.seq_lens = seq_lens;
  sp.page_table = page_table;
  sp.out = out->data;
  sp.out_dtype = out->dtype == HS2_F32 ? 0 : 1;
  sp.idx_out = idx_out;
  sp.B = B;
  sp.Hkv = Hkv;
  sp.G = G;
  sp.D = D;
  sp.page_size = ps;
  sp.max_pages = p.max_pages;
  sp.t_cap = t_cap;
  sp.ustride = p.ustride;
  sp.window = window;
  sp.k_global = k_global;
  sp.N = p.N;
  sp.R = p.R;
  sp.tile = p.tile;
  sp.nsub = L.nsub;
  {  // one wave of the selection kernels over the whole capacity
    const double positions = (double)B * Hkv * (double)t_cap;
    sp.score_chunk = 2048;  // about 4 score CTAs per SM (their register budget)
    while (sp.score_chunk < 65536 && positions / sp.score_chunk > 4.0 * sms) sp.score_chunk *= 2;
    sp.filter_subs = positions / 4096.0 > 5.0 * sms ? 2 : 1;  // 8 warps x 512 positions per sub-range
  }
  sp.c = p.c;
  sp.ncomb = (G * D + 255) / 256;
  sp.ws = p.ws;
  // the fused call: token-level selection on the tensor-core path only
  const bool fuse = fused && mma && block == 0;
  if (fuse && (G >= 16) != (cfg.nt == 2))
    return fail(HS2_ERR_UNSUPPORTED, "fused call: no kernel for %d heads per group with %d-head warps", G, 8 * cfg.nt);
  if (!mma) {
    e = accumulate ? launch_rows_f32(p, p.N, s) : launch_full_f32(p, p.N, s);
    if (e != cudaSuccess) return cuda_fail(e, "full-attention (fp32) launch");
  } else {
    const int box_rows = paged ? (ps < p.tile ? ps : p.tile) : p.tile;
    CUtensorMap tmk, tmv;
    if ((rc = cache_map(&tmk, k_cache, box_rows))) return rc;
    if ((rc = cache_map(&tmv, v_cache, box_rows))) return rc;
    if (fuse) {
      // the grid barrier's arrival counter (word 16 of the flag block) starts at zero
      e = cudaMemsetAsync(p.ws.err + 16, 0, sizeof(uint32_t), s);
      if (e != cudaSuccess) return cuda_fail(e, "clearing the grid-barrier counter");
      e = launch_full_fused(p, sp, tmk, tmv, fp8, cfg, p.N, s);
    } else {
      e = launch_full_mma(p, tmk, tmv, fp8, cfg, p.N, s);
    }
    if (e == cudaErrorInvalidConfiguration)
      return fail(HS2_ERR_UNSUPPORTED, "no %sfull-attention kernel built for ncw=%d nstage=%d nsl=%d nt=%d tc=%d",
                  fuse ? "fused " : "", cfg.ncw, cfg.nstage, cfg.nsl, cfg.nt, cfg.tc);
    if (e != cudaSuccess) return cuda_fail(e, fuse ? "fused full-attention launch" : "full-attention launch");
  }
  if (mark_event) {
    e = cudaEventRecord(static_cast<cudaEvent_t>(mark_event), s);
    if (e != cudaSuccess) return cuda_fail(e, "recording the mark event");
  }
  if (accumulate) {
    accumulate->sp = sp;
    e = launch_accumulate(*accumulate, s);
    return e == cudaSuccess ? HS2_OK : cuda_fail(e, "accumulate launch");
  }
  e = block > 0 ? launch_block_select(sp, block, s) : (fuse ? launch_select_after_score(sp, s) : launch_select(sp, s));
  if (e != cudaSuccess) return cuda_fail(e, "selection launch");
  return HS2_OK;
}

}  // namespace

extern "C" {

int hs2_sparse_attn(const hs2_heads *q_l, const hs2_cache *k_cache, const hs2_cache *v_cache, const int32_t *idx,
                    int32_t idx_stride, hs2_heads *out, void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if ((rc = check_heads(q_l, k_cache, "q_l"))) return rc;
  if ((rc = check_heads(out, k_cache, "out"))) return rc;
  if (out->batch != q_l->batch || out->num_heads != q_l->num_heads || out->dtype != q_l->dtype)
    return fail(HS2_ERR_INVALID_ARG, "out shape/dtype differs from q_l");
  if (!idx) return fail(HS2_ERR_INVALID_ARG, "idx is NULL");
  if (idx_stride < 1 || idx_stride > 4096) return fail(HS2_ERR_UNSUPPORTED, "idx_stride %d out of [1, 4096]", idx_stride);
  SparseParams p{};
  p.q = q_l->data;
  p.k = k_cache->data;
  p.v = v_cache->data;
  p.k_scale = k_cache->scale;
  p.v_scale = v_cache->scale;
  p.idx = idx;
  p.out = out->data;
  p.B = q_l->batch;
  p.Hkv = k_cache->num_kv_heads;
  p.G = q_l->num_heads / p.Hkv;
  p.D = k_cache->head_dim;
  p.L = idx_stride;
  p.c = 1.0f / sqrtf((float)p.D);
  // `warps` warps per CTA take groups of RG = 16 * nsl rows, each warp
  // gathering up to `nbuf` groups at once: rows per CTA = warps * RG * nbuf,
  // one cluster of S CTAs per (sequence, kv head).  nbuf starts at 2 and
  // grows (up to what shared memory holds) while the units' CTAs would not
  // fit in one wave of one CTA per SM or a cluster would exceed 16 CTAs; very
  // long lists then take more rows per CTA than buffers, walked as a rolling
  // pipeline.
  const int units = p.B * p.Hkv * ((p.G + 7) / 8), sms = sm_count();  // clusters: one per 8 query heads
  int warps = 4, nsl = 2, nbuf_env = 0, splits_env = 0;  // (8, 1) measured equal at 32K / 256K, 10% slower at 1M
  if (const char *env = getenv("HS2_SPARSE_CFG")) {  // tuning override: "warps,nsl[,nbuf[,splits]]"
    int a = 0, b2 = 0, c2 = 0, d2 = 0;
    if (sscanf(env, "%d,%d,%d,%d", &a, &b2, &c2, &d2) >= 2 && (a == 4 || a == 8) && (b2 == 1 || b2 == 2)) {
      warps = a;
      nsl = b2;
      nbuf_env = c2;
      splits_env = d2 >= 1 && d2 <= 16 ? d2 : 0;
    }
  }
  const int rg = 16 * nsl;
  // a warp's gather buffer: RG rows of K and V (+ scales); at most 192 KB per CTA
  const int buf_bytes = 2 * rg * p.D * (k_cache->dtype == HS2_E4M3 ? 1 : 2) + (k_cache->dtype == HS2_E4M3 ? 8 * rg : 0);
  int max_nbuf = (192 * 1024) / (warps * buf_bytes);
  max_nbuf = max_nbuf < 1 ? 1 : (max_nbuf > 4 ? 4 : max_nbuf);
  const int per_buf = warps * rg;  // rows per CTA per buffer round
  // two buffers per warp at least (one gather in flight while the other is
  // consumed), more while the CTAs would not fit in one wave
  int nbuf = max_nbuf < 2 ? max_nbuf : 2;
  while (nbuf < max_nbuf && (units * ((idx_stride + per_buf * nbuf - 1) / (per_buf * nbuf)) > sms ||
                             (idx_stride + per_buf * nbuf - 1) / (per_buf * nbuf) > 16))
    ++nbuf;
  // At least as many units as SMs: one CTA per unit walks the whole list with
  // two buffers per warp (the units alone fill the GPU; measured at batch 64,
  // 256 units: 531 against 495 steps/s for 3 CTAs per unit with 3 buffers)
  const bool one_per_unit = units >= sms && splits_env == 0 && nbuf_env == 0;
  if (one_per_unit) nbuf = max_nbuf < 2 ? max_nbuf : 2;
  if (nbuf_env > 0) nbuf = nbuf_env;
  nbuf = nbuf < 1 ? 1 : (nbuf > max_nbuf ? max_nbuf : nbuf);
  int rows = per_buf * nbuf;
  if (one_per_unit) rows = (idx_stride + per_buf - 1) / per_buf * per_buf;
  int S = (idx_stride + rows - 1) / rows;
  while (S > 16) {  // larger lists: more rows per CTA, never more than 16 per cluster
    rows += per_buf;
    S = (idx_stride + rows - 1) / rows;
  }
  if (splits_env > 0) {
    rows = ((idx_stride + splits_env - 1) / splits_env + per_buf - 1) / per_buf * per_buf;
    S = (idx_stride + rows - 1) / rows;
  }
  p.warps = warps;
  p.nsl = nsl;
  p.rows_per_cta = rows;
  p.splits = S;
  p.nbuf = nbuf;
  if (k_cache->dtype == HS2_F32) {
    // fp32 caches: a cluster of up to 16 CTAs per (sequence, kv head), each
    // taking a share of the list's 64-row tiles, as long as the clusters fit
    // one CTA per SM
    const int ntiles = (idx_stride + 63) / 64, per_unit = sms / (p.B * p.Hkv);
    int s32 = per_unit < 1 ? 1 : (per_unit > 16 ? 16 : per_unit);
    if (s32 > ntiles) s32 = ntiles < 1 ? 1 : ntiles;
    p.splits = s32;
  }
  cudaError_t e = launch_sparse_impl(p, k_cache->dtype, k_cache->num_slots, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "sparse-attention launch");
  return HS2_OK;
}

int hs2_workspace_status(void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace || workspace_bytes < 256) return fail(HS2_ERR_WORKSPACE, "workspace is NULL or too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t flag = 0;
  cudaError_t e = cudaMemcpyAsync(&flag, workspace, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, 4, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reading the workspace status");
  if (flag)
    return fail(HS2_ERR_TIMEOUT, "device error flag 0x%x (1: consumer wait, 2: producer wait, 4: record, 8: grid barrier)",
                flag);
  return HS2_OK;
}

size_t hs2_kv_bridge_workspace(int32_t batch, int32_t d_model, int32_t num_kv_heads, int32_t head_dim) {
  if (batch < 1 || batch > 65535 || d_model < 1 || d_model % bridge_row_multiple() || num_kv_heads < 1 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return bridge_workspace_bytes(batch, d_model, num_kv_heads * head_dim);
}

int hs2_kv_bridge_append(const void *hidden, int32_t batch, int32_t d_model, const void *w_k, const void *w_v,
                         const int32_t *seq_lens, const int32_t *page_table, int32_t max_pages,
                         const hs2_cache *k_cache, const hs2_cache *v_cache, void *workspace, size_t workspace_bytes,
                         void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if (!hidden || !w_k || !w_v || !seq_lens) return fail(HS2_ERR_INVALID_ARG, "hidden / w_k / w_v / seq_lens is NULL");
  if (!aligned16(hidden) || !aligned16(w_k) || !aligned16(w_v))
    return fail(HS2_ERR_INVALID_ARG, "hidden / weights not 16-byte aligned");
  if (batch < 1 || batch > 65535) return fail(HS2_ERR_INVALID_ARG, "batch %d", batch);
  if (d_model < 1 || d_model % bridge_row_multiple())
    return fail(HS2_ERR_UNSUPPORTED, "d_model %d (a positive multiple of %d)", d_model, bridge_row_multiple());
  const int ps = k_cache->page_size;
  int64_t t_cap;
  if (page_table) {
    if (max_pages < 1) return fail(HS2_ERR_INVALID_ARG, "max_pages %d with a page table", max_pages);
    t_cap = (int64_t)max_pages * ps;
  } else {
    if (max_pages != 1) return fail(HS2_ERR_INVALID_ARG, "contiguous layout (no page table) needs max_pages == 1");
    t_cap = ps;
    if ((int64_t)batch * ps > k_cache->num_slots)
      return fail(HS2_ERR_INVALID_ARG, "contiguous layout needs num_slots >= batch * page_size");
  }
  const int Hkv = k_cache->num_kv_heads, D = k_cache->head_dim;
  const size_t need = hs2_kv_bridge_workspace(batch, d_model, Hkv, D);
  if (!workspace || workspace_bytes < need)
    return fail(HS2_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(HS2_ERR_WORKSPACE, "workspace not 256-byte aligned");
  BridgeParams p{};
  p.h = static_cast<const __nv_bfloat16 *>(hidden);
  p.wk = static_cast<const __nv_bfloat16 *>(w_k);
  p.wv = static_cast<const __nv_bfloat16 *>(w_v);
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.k = const_cast<void *>(k_cache->data);  // this call writes the new rows
  p.v = const_cast<void *>(v_cache->data);
  p.k_scale = const_cast<float *>(k_cache->scale);
  p.v_scale = const_cast<float *>(v_cache->scale);
  p.kv_dtype = k_cache->dtype;
  p.B = batch;
  p.d_model = d_model;
  p.Hkv = Hkv;
  p.D = D;
  p.N = Hkv * D;
  p.page_size = ps;
  p.max_pages = page_table ? max_pages : 1;
  p.t_cap = t_cap;
  p.num_slots = k_cache->num_slots;
  p.nsplit = bridge_splits(d_model);
  cudaError_t e = launch_bridge(p, workspace, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "KV bridge launch");
  return HS2_OK;
}

int hs2_selftest_bounded_wait(void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace || workspace_bytes < 256) return fail(HS2_ERR_WORKSPACE, "workspace is NULL or too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(HS2_ERR_WORKSPACE, "workspace not 256-byte aligned");
  cudaError_t e = launch_wait_selftest(static_cast<uint32_t *>(workspace), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
  return HS2_OK;
}

int hs2_selftest_grid_barrier(void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace || workspace_bytes < 256) return fail(HS2_ERR_WORKSPACE, "workspace is NULL or too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(HS2_ERR_WORKSPACE, "workspace not 256-byte aligned");
  cudaError_t e = launch_grid_barrier_selftest(static_cast<uint32_t *>(workspace), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
  return HS2_OK;
}

int hs2_copy_peak(void *dst, const void *src, size_t bytes, void *stream) {
  if (!dst || !src || (bytes & 15) || !aligned16(dst) || !aligned16(src))
    return fail(HS2_ERR_INVALID_ARG, "copy needs 16-byte aligned pointers and a multiple of 16 bytes");
  cudaError_t e = launch_copy(dst, src, bytes, sm_count() * 32, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "copy launch");
  return HS2_OK;
}

}  // extern "C"

namespace hs2 {

// One CTA waits on an mbarrier that nothing ever arrives at: the bounded wait
// must give up (after ~10 ms instead of the kernels' ~2 s) and set the
// workspace's sticky flag, then the kernel returns normally.
__global__ void wait_selftest_kernel(uint32_t *err) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1u);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0 && !mbar_wait(&bar, 0u, 20000000LL)) set_error(err, kErrFullWait);
}

cudaError_t launch_wait_selftest(uint32_t *err, cudaStream_t s) {
  wait_selftest_kernel<<<1, 32, 0, s>>>(err);
  return cudaGetLastError();
}

// Two CTAs meet at the fused call's grid barrier sized for three: neither is
// the last arrival, so both give up (after ~10 ms) and set the sticky flag's
// grid-barrier bit, then return.
__global__ void grid_barrier_selftest_kernel(uint32_t *err) {
  __shared__ int flag;
  if (!grid_barrier(err + 16, err + 32, gridDim.x + 1, &flag, 20000000LL) && threadIdx.x == 0)
    set_error(err, kErrGridWait);
}

cudaError_t launch_grid_barrier_selftest(uint32_t *err, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(err + 16, 0, sizeof(uint32_t), s);
  if (e != cudaSuccess) return e;
  grid_barrier_selftest_kernel<<<2, 32, 0, s>>>(err);
  return cudaGetLastError();
}

// Grid-strided 16-byte copy, four loads in flight per thread.  Measured on
// B200 with 2 GiB: 32 CTAs of 256 threads per SM and plain loads/stores
// reach ~6.3 TB/s (read + write); 4 CTAs per SM or streaming (.cs) hints
// stay near 5.9 TB/s.
__global__ void __launch_bounds__(256) copy_kernel(uint4 *__restrict__ dst, const uint4 *__restrict__ src, size_t n) {
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (; i + 3 * stride < n; i += 4 * stride) {
    const uint4 a = src[i], b = src[i + stride], c = src[i + 2 * stride], d = src[i + 3 * stride];
    dst[i] = a;
    dst[i + stride] = b;
    dst[i + 2 * stride] = c;
    dst[i + 3 * stride] = d;
  }
  for (; i < n; i += stride) dst[i] = src[i];
}

int set_last_error(int code, const char *msg) { return fail(code, "%s", msg); }

namespace {
struct SmemAttr {
  const void *kern;
  int dev, bytes;
};
std::mutex g_attr_mu;
SmemAttr g_attr[512];
int g_nattr = 0;
struct WideAttr {
  const void *kern;
  int dev;
};
WideAttr g_wide[128];
int g_nwide = 0;
}  // namespace

cudaError_t allow_wide_clusters_once(const void *kern) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_attr_mu);
  for (int i = 0; i < g_nwide; ++i)
    if (g_wide[i].kern == kern && g_wide[i].dev == dev) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && g_nwide < 128) g_wide[g_nwide++] = WideAttr{kern, dev};
  return e;
}

cudaError_t set_smem_once(const void *kern, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_attr_mu);
  for (int i = 0; i < g_nattr; ++i) {
    if (g_attr[i].kern != kern || g_attr[i].dev != dev) continue;
    if (g_attr[i].bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) g_attr[i].bytes = bytes;
    return e;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && g_nattr < 512) g_attr[g_nattr++] = SmemAttr{kern, dev, bytes};
  return e;
}

bool pdl_enabled() {
  static const bool on = [] {
    const char *env = getenv("HS2_PDL");
    return !(env && env[0] == '0');
  }();
  return on;
}

cudaError_t launch_copy(void *dst, const void *src, size_t bytes, int grid, cudaStream_t s) {
  if (bytes == 0) return cudaSuccess;
  copy_kernel<<<grid, 256, 0, s>>>(static_cast<uint4 *>(dst), static_cast<const uint4 *>(src), bytes / 16);
  return cudaGetLastError();
}

}  // namespace hs2
