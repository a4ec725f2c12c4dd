// hs2_draft_api.cu -- the C ABI of the drafted-token and eviction calls
// (declared in include/hs2.h): argument validation, workspace layout and
// launches.
#include <math.h>

#include <initializer_list>

#include "hs2.h"
#include "hs2_host.h"
#include "hs2_internal.h"

using namespace hs2;

namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int check_tokens(const hs2_tokens *x, const hs2_cache *k, const char *what) {
  if (!x || !x->data) return fail(HS2_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(x->data)) return fail(HS2_ERR_INVALID_ARG, "%s data is not 16-byte aligned", what);
  if (x->batch < 1 || x->tokens < 1) return fail(HS2_ERR_INVALID_ARG, "%s batch %d, tokens %d", what, x->batch, x->tokens);
  if (x->head_dim != k->head_dim)
    return fail(HS2_ERR_INVALID_ARG, "%s head_dim %d != cache head_dim %d", what, x->head_dim, k->head_dim);
  if (x->num_heads < 1 || x->num_heads > 65535) return fail(HS2_ERR_INVALID_ARG, "%s num_heads %d", what, x->num_heads);
  const int want = k->dtype == HS2_F32 ? HS2_F32 : HS2_BF16;
  if (x->dtype != want)
    return fail(HS2_ERR_UNSUPPORTED, "%s dtype %d with cache dtype %d (need %s)", what, x->dtype, k->dtype,
                want == HS2_F32 ? "HS2_F32" : "HS2_BF16");
  const int per16 = want == HS2_F32 ? 4 : 8;
  if (x->token_stride < (int64_t)x->num_heads * x->head_dim || x->token_stride % per16)
    return fail(HS2_ERR_INVALID_ARG, "%s token_stride %lld (at least heads * head_dim, whole 16 bytes)", what,
                (long long)x->token_stride);
  if ((int64_t)x->batch * x->tokens >= (int64_t(1) << 30))
    return fail(HS2_ERR_UNSUPPORTED, "%s batch * tokens too large", what);
  return HS2_OK;
}

struct TreePlan {
  int tile, rows, streams, blocks, groups;
  size_t prefix, records, total;
};

// `small`: the small tiles, where the call's shape has them (fp32 caches, 32 rows)
TreePlan tree_plan(int B, int N, int G, int D, bool f32, bool small) {
  TreePlan t{};
  t.tile = tree_tc_tile();
  t.rows = tree_tc_rows();
  t.streams = f32 ? 1 : 2;
  if (f32) {  // two blocks of few rows take 0.6 to 1.06 of the tiled kernel's time, three would take as long as it
    t.rows = N * G <= 2 * tree_f32_few_rows() ? tree_f32_few_rows() : (N * G <= 32 ? 32 : 64);
    t.tile = t.rows == 32 && small ? 32 : 64;
  }
  const int ctas = sm_count() * (f32 ? tree_f32_ctas_per_sm(D, t.rows, t.tile) : 1), per_block = t.rows * t.streams;
  t.blocks = (N * G + per_block - 1) / per_block;
  t.groups = ctas / t.blocks < 1 ? 1 : (ctas / t.blocks > kMaxTreeGroups ? kMaxTreeGroups : ctas / t.blocks);
  t.prefix = 256;
  t.records = align256(t.prefix + (size_t)(B + 1) * 4);
  t.total = align256(t.records + (size_t)t.groups * kTreeSlots * t.blocks * per_block * (D + 2) * 4);
  return t;
}

bool same(const void *a, const void *b) { return a == b; }

// Memory of an argument; NULL overlaps nothing.
struct Span {
  const void *data;
  uint64_t bytes;
};
bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.data), y = reinterpret_cast<uintptr_t>(b.data);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}
bool overlap(const Span &a, std::initializer_list<Span> others) {
  for (const Span &b : others)
    if (overlap(a, b)) return true;
  return false;
}
Span words(const void *data, int64_t n, int64_t per = 1) { return {data, (uint64_t)n * (uint64_t)per * 4}; }
int elem_bytes(int dtype) { return dtype == HS2_F32 ? 4 : (dtype == HS2_BF16 ? 2 : 1); }
Span span(const hs2_tokens *x) {
  return {x->data, ((uint64_t)((int64_t)x->batch * x->tokens - 1) * x->token_stride + (uint64_t)x->num_heads * x->head_dim) *
                       elem_bytes(x->dtype)};
}
// Whether an element of a is one of b.  Parts of the same wider rows lie between each other without sharing one.
bool overlap(const hs2_tokens *a, const hs2_tokens *b) {
  if (!overlap(span(a), span(b))) return false;
  if (a->token_stride != b->token_stride || a->dtype != b->dtype) return true;
  const int64_t es = elem_bytes(a->dtype), row = a->token_stride * es;
  int64_t off = (int64_t)((reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data)) % row);
  if (off < 0) off += row;
  return off < (int64_t)a->num_heads * a->head_dim * es || off + (int64_t)b->num_heads * b->head_dim * es > row;
}
// K and V (and their scales) of a call that writes them: apart, or pages of one pool that lie whole pages from each
// other (every other page K's and V's), which the page table keeps apart.
int check_written(const hs2_cache *k, const hs2_cache *v, bool paged) {
  auto mixed = [&](const void *a, const void *b, uint64_t slot_bytes) {
    const uint64_t all = (uint64_t)k->num_slots * slot_bytes;
    const int64_t off = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
    return overlap(Span{a, all}, Span{b, all}) && !(paged && off != 0 && off % (int64_t)(slot_bytes * k->page_size) == 0);
  };
  if (mixed(k->data, v->data, (uint64_t)k->num_kv_heads * k->head_dim * elem_bytes(k->dtype)) ||
      mixed(k->scale, v->scale, (uint64_t)k->num_kv_heads * 4))
    return fail(HS2_ERR_INVALID_ARG, "the K and V caches overlap");
  return HS2_OK;
}

}  // namespace

extern "C" {

int hs2_rope_table(const hs2_rope *r, uint64_t *table, float *rot_scale) {
  if (!r || !table || !rot_scale) return fail(HS2_ERR_INVALID_ARG, "rope / table / rot_scale is NULL");
  const int rot = r->rot_dim;
  if (rot < 16 || rot > 128 || rot % 16) return fail(HS2_ERR_UNSUPPORTED, "rot_dim %d (a multiple of 16, at most 128)", rot);
  if (!(r->base > 1.0) || !isfinite(r->base)) return fail(HS2_ERR_INVALID_ARG, "rope base %g", r->base);
  if (r->scaling < HS2_ROPE_PLAIN || r->scaling > HS2_ROPE_BANDS) return fail(HS2_ERR_INVALID_ARG, "rope scaling %d", r->scaling);
  if (r->scaling != HS2_ROPE_PLAIN && (!(r->factor >= 1.0) || !isfinite(r->factor)))
    return fail(HS2_ERR_INVALID_ARG, "rope factor %g", r->factor);
  if (r->scaling >= HS2_ROPE_YARN && (!(r->original_context > 0.0) || !isfinite(r->original_context)))
    return fail(HS2_ERR_INVALID_ARG, "rope original_context %g", r->original_context);
  if (r->scaling == HS2_ROPE_YARN && !(r->beta_fast > r->beta_slow && r->beta_slow > 0.0 && isfinite(r->beta_fast)))
    return fail(HS2_ERR_INVALID_ARG, "rope beta_fast %g, beta_slow %g", r->beta_fast, r->beta_slow);
  if (r->scaling == HS2_ROPE_BANDS &&
      !(r->high_freq_factor > r->low_freq_factor && r->low_freq_factor > 0.0 && isfinite(r->high_freq_factor)))
    return fail(HS2_ERR_INVALID_ARG, "rope low_freq_factor %g, high_freq_factor %g", r->low_freq_factor, r->high_freq_factor);
  const double two_pi = 2.0 * acos(-1.0);
  double base = r->base;
  if (r->scaling == HS2_ROPE_NTK) base *= pow(r->factor, (double)rot / (rot - 2));
  // the pair index at which a head's pairs turn `beta` times in the original context
  auto pair_of = [&](double beta) { return rot * log(r->original_context / (beta * two_pi)) / (2 * log(base)); };
  double lo = 0, hi = 0;
  if (r->scaling == HS2_ROPE_YARN) {
    lo = fmax(floor(pair_of(r->beta_fast)), 0.0);
    hi = fmin(ceil(pair_of(r->beta_slow)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (r->scaling == HS2_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == HS2_ROPE_YARN) {
      const double ramp = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f / r->factor * ramp + f * (1 - ramp);
    }
    if (r->scaling == HS2_ROPE_BANDS) {
      const double turns = r->original_context * f / two_pi;
      const double s =
          fmin(fmax((turns - r->low_freq_factor) / (r->high_freq_factor - r->low_freq_factor), 0.0), 1.0);
      f = (1 - s) * f / r->factor + s * f;
    }
    table[i] = (uint64_t)rint(ldexp(f / two_pi, 64));  // f <= 1: below 2^62
  }
  *rot_scale = r->scaling == HS2_ROPE_YARN ? (float)(0.1 * log(r->factor) + 1.0) : 1.0f;
  return HS2_OK;
}

int hs2_rope_append(const hs2_tokens *q, const hs2_tokens *k, const hs2_tokens *v, const int32_t *positions,
                    const uint64_t *table, int32_t rot_dim, int32_t interleaved, float rot_scale,
                    const int32_t *seq_lens, const int32_t *num_new, const int32_t *page_table, int32_t max_pages,
                    const hs2_cache *k_cache, const hs2_cache *v_cache, void *q_out, void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if ((rc = check_tokens(k, k_cache, "k"))) return rc;
  if ((rc = check_tokens(v, k_cache, "v"))) return rc;
  if (k->num_heads != k_cache->num_kv_heads || v->num_heads != k_cache->num_kv_heads)
    return fail(HS2_ERR_INVALID_ARG, "k / v heads %d / %d, cache heads %d", k->num_heads, v->num_heads, k_cache->num_kv_heads);
  if (v->batch != k->batch || v->tokens != k->tokens) return fail(HS2_ERR_INVALID_ARG, "v batch / tokens differ from k");
  if (q) {
    if ((rc = check_tokens(q, k_cache, "q"))) return rc;
    if (q->batch != k->batch || q->tokens != k->tokens) return fail(HS2_ERR_INVALID_ARG, "q batch / tokens differ from k");
    if (!q_out || !aligned16(q_out)) return fail(HS2_ERR_INVALID_ARG, "q_out is NULL or not 16-byte aligned");
    if (same(q_out, q->data) && q->token_stride != (int64_t)q->num_heads * q->head_dim && q->batch * q->tokens > 1)
      return fail(HS2_ERR_INVALID_ARG, "q_out may be q only when q is contiguous");
  } else if (q_out) {
    return fail(HS2_ERR_INVALID_ARG, "q_out without q");
  }
  if (!positions || !table || !seq_lens) return fail(HS2_ERR_INVALID_ARG, "positions / table / seq_lens is NULL");
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > k_cache->head_dim)
    return fail(HS2_ERR_UNSUPPORTED, "rot_dim %d (a multiple of 16, at most head_dim %d)", rot_dim, k_cache->head_dim);
  int64_t t_cap;
  if ((rc = check_pages(k_cache, page_table, max_pages, k->batch, &t_cap))) return rc;
  if ((rc = check_written(k_cache, v_cache, page_table != nullptr))) return rc;
  if (q) {
    hs2_tokens o = *q;
    o.data = q_out;
    o.token_stride = (int64_t)q->num_heads * q->head_dim;
    if (overlap(&o, k) || overlap(&o, v) || (!same(q_out, q->data) && overlap(&o, q)))
      return fail(HS2_ERR_INVALID_ARG, "q_out overlaps k, v or a part of q");
  }
  RopeParams p{};
  p.q = q ? q->data : nullptr;
  p.k = k->data;
  p.v = v->data;
  p.q_stride = q ? q->token_stride : 0;
  p.k_stride = k->token_stride;
  p.v_stride = v->token_stride;
  p.q_out = q_out;
  p.positions = positions;
  p.table = table;
  p.mscale = rot_scale;
  p.rot = rot_dim;
  p.interleaved = interleaved != 0;
  p.seq_lens = seq_lens;
  p.num_new = num_new;
  p.page_table = page_table;
  p.ck = const_cast<void *>(k_cache->data);
  p.cv = const_cast<void *>(v_cache->data);
  p.k_scale = const_cast<float *>(k_cache->scale);
  p.v_scale = const_cast<float *>(v_cache->scale);
  p.kv_dtype = k_cache->dtype;
  p.B = k->batch;
  p.N = k->tokens;
  p.Hq = q ? q->num_heads : 0;
  p.Hkv = k_cache->num_kv_heads;
  p.D = k_cache->head_dim;
  p.page_size = k_cache->page_size;
  p.max_pages = max_pages;
  p.t_cap = t_cap;
  p.num_slots = k_cache->num_slots;
  const cudaError_t e = launch_rope(p, sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "rope-append launch");
}

size_t hs2_tree_attn_workspace(int32_t batch, int32_t tokens, int32_t num_kv_heads, int32_t group, int32_t head_dim,
                               int32_t kv_dtype) {
  if (batch < 1 || batch > kMaxBatchSmem || tokens < 1 || tokens > kMaxDraft || num_kv_heads < 1 || !group_ok(group) ||
      (head_dim != 64 && head_dim != 128) || kv_dtype < HS2_F32 || kv_dtype > HS2_E4M3)
    return 0;
  // The most that a call of this many tokens and sequences or fewer needs, at any capacity: shorter drafts have fewer
  // row blocks and so more shares.
  const bool f32 = kv_dtype == HS2_F32;
  size_t most = 0;
  for (int n = 1; n <= tokens; ++n)
    for (const bool small : {false, true}) {
      const size_t t = tree_plan(batch, n, group, head_dim, f32, small).total;
      most = t > most ? t : most;
    }
  return most;
}

int hs2_tree_attn(const hs2_tokens *q, const hs2_cache *k_cache, const hs2_cache *v_cache, const int32_t *seq_lens,
                  const int32_t *num_draft, const uint64_t *tree_mask, const int32_t *page_table, int32_t max_pages,
                  hs2_tokens *out, void *workspace, size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if ((rc = check_tokens(q, k_cache, "q"))) return rc;
  if ((rc = check_tokens(out, k_cache, "out"))) return rc;
  if (out->batch != q->batch || out->tokens != q->tokens || out->num_heads != q->num_heads)
    return fail(HS2_ERR_INVALID_ARG, "out shape differs from q");
  if (same(q->data, out->data)) return fail(HS2_ERR_INVALID_ARG, "out is q");
  if (q->tokens > kMaxDraft) return fail(HS2_ERR_UNSUPPORTED, "%d drafted tokens (at most %d)", q->tokens, kMaxDraft);
  const int Hkv = k_cache->num_kv_heads, D = k_cache->head_dim;
  if (q->num_heads % Hkv)
    return fail(HS2_ERR_INVALID_ARG, "q num_heads %d is not a multiple of num_kv_heads %d", q->num_heads, Hkv);
  const int G = q->num_heads / Hkv;
  if (!group_ok(G)) return fail(HS2_ERR_UNSUPPORTED, "GQA group %d not built (1, 2, 4, 8, 16 or 32)", G);
  if (k_cache->dtype == HS2_F32 && G > 8) return fail(HS2_ERR_UNSUPPORTED, "fp32 caches take GQA groups of at most 8 heads");
  if (!seq_lens) return fail(HS2_ERR_INVALID_ARG, "seq_lens is NULL");
  int64_t t_cap;
  if ((rc = check_pages(k_cache, page_table, max_pages, q->batch, &t_cap))) return rc;
  const int ps = k_cache->page_size;
  if (k_cache->dtype != HS2_F32 && page_table && !(ps % 16 == 0 && (ps % 64 == 0 || 64 % ps == 0)))
    return fail(HS2_ERR_UNSUPPORTED, "page_size %d (16, 32 or a multiple of 64)", ps);
  const bool f32 = k_cache->dtype == HS2_F32;
  // short tiles where long ones are too few for the SMs
  const bool small = (t_cap + 63) / 64 * Hkv * q->batch < sm_count();
  const TreePlan plan = tree_plan(q->batch, q->tokens, G, D, f32, small);
  if (!workspace) return fail(HS2_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(HS2_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < plan.total)
    return fail(HS2_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, plan.total);
  if (overlap(q, out)) return fail(HS2_ERR_INVALID_ARG, "out overlaps q");
  uint8_t *w = static_cast<uint8_t *>(workspace);
  TreeParams p{};
  p.q = q->data;
  p.q_stride = q->token_stride;
  p.k = k_cache->data;
  p.v = v_cache->data;
  p.k_scale = k_cache->scale;
  p.v_scale = v_cache->scale;
  p.seq_lens = seq_lens;
  p.num_draft = num_draft;
  p.page_table = page_table;
  p.mask = tree_mask;
  p.out = out->data;
  p.out_stride = out->token_stride;
  p.B = q->batch;
  p.N = q->tokens;
  p.Hq = q->num_heads;
  p.Hkv = Hkv;
  p.G = G;
  p.D = D;
  p.page_size = ps;
  p.max_pages = max_pages;
  p.t_cap = t_cap;
  p.num_slots = k_cache->num_slots;
  p.c2 = (float)(1.4426950408889634074 / sqrt((double)D));
  p.tile = plan.tile;
  p.rows = plan.rows;
  p.streams = plan.streams;
  p.blocks = plan.blocks;
  p.groups = plan.groups;
  p.err = reinterpret_cast<uint32_t *>(w);
  p.prefix = reinterpret_cast<int32_t *>(w + plan.prefix);
  p.records = reinterpret_cast<float *>(w + plan.records);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (f32) {
    e = launch_tree_f32(p, s);
  } else {
    // boxes of consecutive slots: a page's, up to a tile (without pages a sequence's rows are one run)
    p.box = p.tile;
    while (page_table && ps % p.box) p.box /= 2;
    p.page_step = p.tile / ps;
    p.page_off = p.tile % ps;
    CUtensorMap tmk, tmv;
    if ((rc = cache_map(&tmk, k_cache, p.box)) || (rc = cache_map(&tmv, v_cache, p.box))) return rc;
    e = launch_tree_tc(p, tmk, tmv, k_cache->dtype, s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "tree-attention launch");
  e = launch_tree_combine(p, f32, s);
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "tree-attention combine launch");
}

int hs2_tree_accept(const hs2_cache *k_cache, const hs2_cache *v_cache, const int32_t *seq_lens,
                    const int32_t *num_draft, const int32_t *path, const int32_t *path_len, int32_t batch,
                    int32_t max_path, const int32_t *page_table, int32_t max_pages, int32_t *lens_out, void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if (!seq_lens || !path || !path_len || !lens_out)
    return fail(HS2_ERR_INVALID_ARG, "seq_lens / path / path_len / lens_out is NULL");
  if (max_path < 1 || max_path > kMaxDraft) return fail(HS2_ERR_UNSUPPORTED, "max_path %d out of [1, %d]", max_path, kMaxDraft);
  AcceptParams p{};
  if ((rc = check_pages(k_cache, page_table, max_pages, batch, &p.t_cap))) return rc;
  if (overlap(words(lens_out, batch), {words(seq_lens, batch), words(num_draft, batch), words(path_len, batch),
                                       words(path, batch, max_path), words(page_table, batch, max_pages)}))
    return fail(HS2_ERR_INVALID_ARG, "lens_out overlaps seq_lens, num_draft, path, path_len or page_table");
  if ((rc = check_written(k_cache, v_cache, page_table != nullptr))) return rc;
  p.k = const_cast<void *>(k_cache->data);
  p.v = const_cast<void *>(v_cache->data);
  p.k_scale = const_cast<float *>(k_cache->scale);
  p.v_scale = const_cast<float *>(v_cache->scale);
  p.seq_lens = seq_lens;
  p.num_draft = num_draft;
  p.path = path;
  p.path_len = path_len;
  p.page_table = page_table;
  p.lens_out = lens_out;
  p.B = batch;
  p.M = max_path;
  p.Hkv = k_cache->num_kv_heads;
  p.row_bytes = p.Hkv * k_cache->head_dim * elem_bytes(k_cache->dtype);
  p.page_size = k_cache->page_size;
  p.max_pages = max_pages;
  p.num_slots = k_cache->num_slots;
  const cudaError_t e = launch_accept(p, k_cache->dtype == HS2_E4M3, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "tree-accept launch");
}

int hs2_cache_evict(const hs2_cache *k_cache, const hs2_cache *v_cache, const int32_t *seq_lens, int32_t batch,
                    const int32_t *page_table, int32_t max_pages, float *acc, int64_t acc_stride, int32_t budget,
                    int32_t window, int32_t *kept, int32_t *lens_out, void *stream) {
  int rc;
  if ((rc = check_caches(k_cache, v_cache))) return rc;
  if (!seq_lens || !acc || !kept || !lens_out) return fail(HS2_ERR_INVALID_ARG, "seq_lens / acc / kept / lens_out is NULL");
  if (budget < 1 || budget > kMaxContext) return fail(HS2_ERR_INVALID_ARG, "budget %d out of [1, %lld]", budget, (long long)kMaxContext);
  if (window < 0 || window > budget) return fail(HS2_ERR_INVALID_ARG, "window %d out of [0, budget %d]", window, budget);
  if (reinterpret_cast<uintptr_t>(acc) & 3) return fail(HS2_ERR_INVALID_ARG, "acc is misaligned");
  EvictParams p{};
  if ((rc = check_pages(k_cache, page_table, max_pages, batch, &p.t_cap))) return rc;
  if (overlap(words(lens_out, batch), {words(seq_lens, batch), words(page_table, batch, max_pages)}))
    return fail(HS2_ERR_INVALID_ARG, "lens_out overlaps seq_lens or page_table");
  if (acc_stride < p.t_cap)
    return fail(HS2_ERR_INVALID_ARG, "acc_stride %lld < capacity %lld", (long long)acc_stride, (long long)p.t_cap);
  const int64_t units = (int64_t)batch * k_cache->num_kv_heads;
  if (overlap(words(kept, units, budget), {words(seq_lens, batch), words(page_table, batch, max_pages), words(lens_out, batch),
                                           words(acc, units, acc_stride)}))
    return fail(HS2_ERR_INVALID_ARG, "kept overlaps seq_lens, page_table, lens_out or acc");
  if ((rc = check_written(k_cache, v_cache, page_table != nullptr))) return rc;
  p.k = const_cast<void *>(k_cache->data);
  p.v = const_cast<void *>(v_cache->data);
  p.k_scale = const_cast<float *>(k_cache->scale);
  p.v_scale = const_cast<float *>(v_cache->scale);
  p.acc = acc;
  p.acc_stride = acc_stride;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.kept = kept;
  p.lens_out = lens_out;
  p.B = batch;
  p.Hkv = k_cache->num_kv_heads;
  p.budget = budget;
  p.window = window;
  p.head_bytes = k_cache->head_dim * elem_bytes(k_cache->dtype);
  p.page_size = k_cache->page_size;
  p.max_pages = max_pages;
  p.num_slots = k_cache->num_slots;
  const cudaError_t e = launch_evict(p, k_cache->dtype == HS2_E4M3, sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? HS2_OK : cuda_fail(e, "evict launch");
}

}  // extern "C"
