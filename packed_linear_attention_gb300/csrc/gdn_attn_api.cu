// gdn_attn_api.cu — C entry points of the full-attention layers' calls: the checks of their
// arguments and the choice of kernels. Everything is checked before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/gdn.h"
#include "gdn_attn_internal.h"
#include "gdn_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool known_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
size_t item_size(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

gdn_status check_page_size(int32_t p) {
  if (p <= 0) return GDN_ERR_INVALID_ARGUMENT;
  return p == 16 || p == 32 || p == 64 || p == 128 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}
gdn_status check_head_dim(int32_t d) {
  if (d <= 0) return GDN_ERR_INVALID_ARGUMENT;
  return d == 64 || d == 128 || d == 256 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// The cache's sizes (pointers are looked at where the cache is used).
gdn_status check_cache_shape(const gdn_kv_cache* c) {
  if (!c || c->num_pages < 1 || c->num_kv_heads < 1) return GDN_ERR_INVALID_ARGUMENT;
  gdn_status s = check_page_size(c->page_size);
  if (s == GDN_OK) s = check_head_dim(c->head_dim);
  if (s != GDN_OK) return s;
  // below 2^62: three int32 factors, the last at most 128
  if ((double)c->num_pages * c->num_kv_heads * c->page_size > (double)INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
gdn_status check_cache(const gdn_kv_cache* c) {
  const gdn_status s = check_cache_shape(c);
  if (s != GDN_OK) return s;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// Rows of `heads` heads: pointer, alignment and stride.
bool rows_ok(const void* p, int64_t stride, int32_t heads, int32_t head_dim, int32_t dtype) {
  return p && aligned(p, 16) && stride >= (int64_t)heads * head_dim &&
         stride % (int64_t)(16 / item_size(dtype)) == 0 && stride <= (int64_t)1 << 40;
}

struct Span {
  uintptr_t lo, hi;
};
// The bytes that `tokens` rows of a strided tensor reach over.
Span span_of(const void* p, int64_t tokens, int64_t stride, int64_t row, size_t item) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, tokens > 0 ? lo + (uintptr_t)((tokens - 1) * stride + row) * item : lo};
}
bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// Two strided tensors share memory unless their rows lie beside one another in rows of the
// same stride (column ranges of one array).
bool rows_overlap(const void* p, int64_t ps, int64_t prow, const void* q, int64_t qs,
                  int64_t qrow, int64_t tokens, size_t item) {
  if (!overlap(span_of(p, tokens, ps, prow, item), span_of(q, tokens, qs, qrow, item)))
    return false;
  if (ps != qs) return true;
  const int64_t stride = ps * (int64_t)item;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) % stride;
  if (d < 0) d += stride;
  return d < prow * (int64_t)item || d + qrow * (int64_t)item > stride;
}

gdn_status check_rope(const gdn_rope* r) {
  if (!r) return GDN_ERR_INVALID_ARGUMENT;
  const gdn_status s = check_head_dim(r->head_dim);
  if (s != GDN_OK) return s;
  if (r->rotary_dim < 16 || r->rotary_dim > r->head_dim || r->rotary_dim % 16 != 0 ||
      r->num_axes < 1 || r->num_axes > GDN_ROPE_MAX_AXES ||
      (r->pair_layout != GDN_ROPE_HALVES && r->pair_layout != GDN_ROPE_ADJACENT))
    return GDN_ERR_INVALID_ARGUMENT;
  for (int32_t i = 0; i < r->rotary_dim / 2; ++i)
    if (r->axis[i] >= r->num_axes) return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// One tensor of a rotation: in place, or no overlap at all.
bool rope_heads_ok(const void* in, int64_t in_stride, int32_t heads, const void* out,
                   int64_t out_stride, int32_t head_dim, int32_t dtype, int32_t tokens) {
  if (!rows_ok(in, in_stride, heads, head_dim, dtype) ||
      !rows_ok(out, out_stride, heads, head_dim, dtype))
    return false;
  if (in == out && in_stride == out_stride) return true;
  const int64_t row = (int64_t)heads * head_dim;
  return !rows_overlap(in, in_stride, row, out, out_stride, row, tokens, item_size(dtype));
}

// Runs `launch` with the handle's device current.
template <class F>
gdn_status on_device(const gdn_handle* h, F launch) {
  const int device = gdn::handle_device(h);
  int prev = 0;
  if (cudaGetDevice(&prev) != cudaSuccess) return GDN_ERR_CUDA;
  if (prev != device && cudaSetDevice(device) != cudaSuccess) return GDN_ERR_CUDA;
  const int e = launch();
  if (prev != device) cudaSetDevice(prev);
  return e == 0 ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status check_attn(const gdn_attn_config* cfg, const gdn_kv_cache* c, int32_t num_seqs,
                      int32_t num_tokens, int32_t max_q_len, int32_t max_kv_len) {
  if (!cfg) return GDN_ERR_INVALID_ARGUMENT;
  gdn_status s = check_cache_shape(c);
  if (s != GDN_OK) return s;
  if (cfg->num_q_heads < 1 || cfg->num_q_heads % c->num_kv_heads != 0 ||
      !known_dtype(cfg->io_dtype) || !std::isfinite(cfg->scale) || num_seqs < 1 ||
      num_tokens < 0 || max_q_len < 0 || max_kv_len < 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (num_seqs > gdn::kMaxSeqs) return GDN_ERR_UNSUPPORTED;
  // query rows and the split kernel's work items are counted in 32 bits. With fp32 io it takes
  // all rows, with bf16 at most max(kTileRows, group) of a request (split_queries; twice that is
  // counted, so that the rule can move without a call being refused).
  const double group = cfg->num_q_heads / c->num_kv_heads;
  double split_rows = (double)num_tokens * group;
  if (cfg->io_dtype == GDN_BF16)
    split_rows = std::min(split_rows, num_seqs * 2.0 * std::max((double)gdn::kTileRows, group));
  const double items = (split_rows / 8 + num_seqs) * c->num_kv_heads *
                       (max_kv_len / (double)gdn::kSplitTile + 1);
  const double units = ((double)num_tokens * group / gdn::kTileRows + num_seqs) * c->num_kv_heads;
  if ((double)num_tokens * group > (double)INT32_MAX || items >= (double)INT32_MAX ||
      units >= (double)gdn::kMaxUnits)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_plan(gdn_handle* h, int32_t page_size, int32_t num_seqs, int32_t num_tokens,
                       const int32_t* ctx_len, const int32_t* new_len, int32_t* block_table,
                       int32_t max_blocks, int32_t num_pages, const int32_t* free_pages,
                       const int32_t* free_count, int32_t* free_count_out, int32_t* cu_new,
                       int32_t* kv_len, int32_t* positions, int64_t* slots, int32_t* status,
                       void* stream) {
  const gdn_status s = check_page_size(page_size);
  if (s != GDN_OK) return s;
  if (num_seqs < 1 || num_tokens < 0 || max_blocks < 1 || num_pages < 1 || !ctx_len || !new_len ||
      !block_table || !free_pages || !free_count || !free_count_out || !cu_new || !kv_len ||
      (num_tokens > 0 && !slots))
    return GDN_ERR_INVALID_ARGUMENT;
  for (const void* p : {(const void*)ctx_len, (const void*)new_len, (const void*)block_table,
                        (const void*)free_pages, (const void*)free_count,
                        (const void*)free_count_out, (const void*)cu_new, (const void*)kv_len,
                        (const void*)positions, (const void*)status})
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned(slots, 8)) return GDN_ERR_INVALID_ARGUMENT;
  // outputs are written while other blocks still read the inputs (how many entries the free
  // stack has is known on the device alone: its first one is looked at)
  const Span in[] = {span_of(ctx_len, 1, 0, num_seqs, 4), span_of(new_len, 1, 0, num_seqs, 4),
                     span_of(free_pages, 1, 0, 1, 4), span_of(free_count, 1, 0, 1, 4)};
  const Span table = span_of(block_table, 1, 0, (int64_t)num_seqs * max_blocks, 4);
  const Span out[] = {table, span_of(cu_new, 1, 0, num_seqs + 1, 4),
                      span_of(kv_len, 1, 0, num_seqs, 4),
                      span_of(positions, 1, 0, positions ? num_tokens : 0, 4),
                      span_of(slots, 1, 0, slots ? num_tokens : 0, 8)};
  for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
    for (const Span& x : in)
      if (overlap(x, out[i])) return GDN_ERR_INVALID_ARGUMENT;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[j], out[i])) return GDN_ERR_INVALID_ARGUMENT;
  }
  if (num_seqs > gdn::kMaxSeqs) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  const gdn::PlanArgs a = {page_size,  num_seqs,   num_tokens,     max_blocks, num_pages, ctx_len,
                           new_len,    block_table, free_pages,    free_count, free_count_out,
                           cu_new,     kv_len,     positions,      slots,      status};
  return on_device(h, [&] { return gdn::launch_kv_plan(a, stream); });
}

gdn_status gdn_kv_release(gdn_handle* h, int32_t page_size, int32_t num_seqs,
                          const int32_t* kv_len, const int32_t* release, int32_t* block_table,
                          int32_t max_blocks, int32_t num_pages, int32_t* free_pages,
                          int32_t* free_count, int32_t* status, void* stream) {
  const gdn_status s = check_page_size(page_size);
  if (s != GDN_OK) return s;
  if (num_seqs < 1 || max_blocks < 1 || num_pages < 1 || !kv_len || !release || !block_table ||
      !free_pages || !free_count)
    return GDN_ERR_INVALID_ARGUMENT;
  for (const void* p : {(const void*)kv_len, (const void*)release, (const void*)block_table,
                        (const void*)free_pages, (const void*)free_count, (const void*)status})
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARGUMENT;
  if (num_seqs > gdn::kMaxSeqs) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  const gdn::ReleaseArgs a = {page_size, num_seqs,    max_blocks, num_pages,  kv_len,
                              release,   block_table, free_pages, free_count, status};
  return on_device(h, [&] { return gdn::launch_kv_release(a, stream); });
}

gdn_status gdn_rope_init(gdn_rope* rope, int32_t head_dim, int32_t rotary_dim, int32_t num_axes,
                         const int32_t* sections, int32_t axis_layout, int32_t pair_layout,
                         double theta, const double* inv_freq) {
  if (!rope || !sections || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > head_dim ||
      num_axes < 1 ||
      (axis_layout != GDN_ROPE_SECTIONS && axis_layout != GDN_ROPE_INTERLEAVED) ||
      (pair_layout != GDN_ROPE_HALVES && pair_layout != GDN_ROPE_ADJACENT))
    return GDN_ERR_INVALID_ARGUMENT;
  const gdn_status s = check_head_dim(head_dim);
  if (s != GDN_OK) return s;
  if (rotary_dim % 16 != 0 || num_axes > GDN_ROPE_MAX_AXES) return GDN_ERR_UNSUPPORTED;
  const int32_t half = rotary_dim / 2;
  int64_t sum = 0;
  for (int32_t x = 0; x < num_axes; ++x) {
    if (sections[x] < 0) return GDN_ERR_INVALID_ARGUMENT;
    sum += sections[x];
  }
  if (sum != half) return GDN_ERR_INVALID_ARGUMENT;
  if (!inv_freq && !(std::isfinite(theta) && theta >= 1.0)) return GDN_ERR_INVALID_ARGUMENT;
  constexpr long double kTwoPi = 6.283185307179586476925286766559005768L;
  gdn_rope r;
  std::memset(&r, 0, sizeof(r));
  r.head_dim = head_dim;
  r.rotary_dim = rotary_dim;
  r.num_axes = num_axes;
  r.pair_layout = pair_layout;
  int32_t taken[GDN_ROPE_MAX_AXES] = {};
  for (int32_t i = 0; i < half; ++i) {
    // long double: 2^31 positions multiply the fraction's error
    const long double w = inv_freq ? (long double)inv_freq[i]
                                   : std::pow((long double)theta, -2.0L * i / rotary_dim);
    if (!(w >= 0.0L && w < kTwoPi)) return GDN_ERR_INVALID_ARGUMENT;
    const long double turns = std::floor(w / kTwoPi * 18446744073709551616.0L + 0.5L);
    r.turns[i] = turns >= 18446744073709551615.0L ? UINT64_MAX : (uint64_t)turns;
    int32_t x = 0;
    if (axis_layout == GDN_ROPE_SECTIONS) {
      while (taken[x] == sections[x]) ++x;
    } else {
      x = i % num_axes;
      if (x > 0 && taken[x] == sections[x]) x = 0;
    }
    if (axis_layout == GDN_ROPE_SECTIONS || x > 0) ++taken[x];
    r.axis[i] = (uint8_t)x;
  }
  if (axis_layout == GDN_ROPE_INTERLEAVED) {
    // an axis whose pairs do not fit into its turns cannot be laid out in turns
    for (int32_t x = 1; x < num_axes; ++x)
      if (taken[x] != sections[x]) return GDN_ERR_INVALID_ARGUMENT;
  }
  *rope = r;
  return GDN_OK;
}

gdn_status gdn_rope_apply(gdn_handle* h, const gdn_rope* rope, int32_t io_dtype,
                          int32_t num_tokens, const int32_t* positions, int64_t pos_stride,
                          const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                          int64_t q_out_stride, const void* k, int64_t k_stride,
                          int32_t num_k_heads, void* k_out, int64_t k_out_stride, void* stream) {
  const gdn_status s = check_rope(rope);
  if (s != GDN_OK) return s;
  if (!known_dtype(io_dtype) || num_tokens < 0 || num_q_heads < 0 || num_k_heads < 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && num_q_heads + (int64_t)num_k_heads > 0) {
    if (!positions || !aligned(positions, 4) || pos_stride < num_tokens)
      return GDN_ERR_INVALID_ARGUMENT;
    const int32_t d = rope->head_dim;
    if (num_q_heads > 0 && !rope_heads_ok(q, q_stride, num_q_heads, q_out, q_out_stride, d,
                                          io_dtype, num_tokens))
      return GDN_ERR_INVALID_ARGUMENT;
    if (num_k_heads > 0 && !rope_heads_ok(k, k_stride, num_k_heads, k_out, k_out_stride, d,
                                          io_dtype, num_tokens))
      return GDN_ERR_INVALID_ARGUMENT;
    if (num_q_heads > 0 && num_k_heads > 0) {
      const int64_t qr = (int64_t)num_q_heads * d, kr = (int64_t)num_k_heads * d;
      const size_t e = item_size(io_dtype);
      if (rows_overlap(q_out, q_out_stride, qr, k_out, k_out_stride, kr, num_tokens, e) ||
          rows_overlap(q_out, q_out_stride, qr, k, k_stride, kr, num_tokens, e) ||
          rows_overlap(q, q_stride, qr, k_out, k_out_stride, kr, num_tokens, e))
        return GDN_ERR_INVALID_ARGUMENT;
    }
  }
  if (num_q_heads > (1 << 20) || num_k_heads > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  gdn::RopeArgs a = {};
  a.x[0] = {q, q_out, q_stride, q_out_stride, num_q_heads};
  a.x[1] = {k, k_out, k_stride, k_out_stride, num_k_heads};
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.num_tokens = num_tokens;
  return on_device(h, [&] { return gdn::launch_rope(*rope, a, io_dtype == GDN_BF16, stream); });
}

gdn_status gdn_kv_append(gdn_handle* h, const gdn_kv_cache* cache, int32_t io_dtype,
                         int32_t num_tokens, const int64_t* slots, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, const gdn_rope* rope,
                         const int32_t* positions, int64_t pos_stride, const void* q,
                         int64_t q_stride, int32_t num_q_heads, void* q_out,
                         int64_t q_out_stride, int32_t* status, void* stream) {
  gdn_status s = check_cache(cache);
  if (s != GDN_OK) return s;
  if (!known_dtype(io_dtype) || num_tokens < 0 || num_q_heads < 0 || !aligned(status, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  if (rope) {
    s = check_rope(rope);
    if (s != GDN_OK) return s;
    if (rope->head_dim != cache->head_dim) return GDN_ERR_INVALID_ARGUMENT;
  } else if (num_q_heads > 0) {
    return GDN_ERR_INVALID_ARGUMENT;
  }
  const int32_t d = cache->head_dim, hk = cache->num_kv_heads;
  if (num_tokens > 0) {
    if (!slots || !aligned(slots, 8) || !rows_ok(k, k_stride, hk, d, io_dtype) ||
        !rows_ok(v, v_stride, hk, d, io_dtype))
      return GDN_ERR_INVALID_ARGUMENT;
    if (rope && (!positions || !aligned(positions, 4) || pos_stride < num_tokens))
      return GDN_ERR_INVALID_ARGUMENT;
    if (num_q_heads > 0) {
      const int64_t qr = (int64_t)num_q_heads * d, kr = (int64_t)hk * d;
      const size_t e = item_size(io_dtype);
      if (!rope_heads_ok(q, q_stride, num_q_heads, q_out, q_out_stride, d, io_dtype,
                         num_tokens) ||
          rows_overlap(q_out, q_out_stride, qr, k, k_stride, kr, num_tokens, e) ||
          rows_overlap(q_out, q_out_stride, qr, v, v_stride, kr, num_tokens, e))
        return GDN_ERR_INVALID_ARGUMENT;
    }
  }
  if (num_q_heads > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  gdn::AppendArgs a = {};
  a.cache = *cache;
  a.num_tokens = num_tokens;
  a.slots = slots;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.status = status;
  a.rotate = rope != nullptr;
  if (rope) {
    a.rope_args.x[0] = {q, q_out, q_stride, q_out_stride, num_q_heads};
    a.rope_args.positions = positions;
    a.rope_args.pos_stride = pos_stride;
    a.rope_args.num_tokens = num_tokens;
  }
  return on_device(h, [&] { return gdn::launch_kv_append(rope, a, io_dtype == GDN_BF16, stream); });
}

gdn_status gdn_attn_workspace_size(const gdn_attn_config* cfg, const gdn_kv_cache* cache,
                                   int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                                   int32_t max_kv_len, size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARGUMENT;
  const gdn_status s = check_attn(cfg, cache, num_seqs, num_tokens, max_q_len, max_kv_len);
  if (s != GDN_OK) return s;
  *bytes = gdn::attn_workspace(*cfg, *cache);
  return GDN_OK;
}

gdn_status gdn_attn_paged(gdn_handle* h, const gdn_attn_config* cfg, const gdn_kv_cache* cache,
                          int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                          int32_t max_kv_len, const int32_t* cu_q, const int32_t* kv_len,
                          const int32_t* block_table, int32_t max_blocks, const void* q,
                          int64_t q_stride, void* o, int64_t o_stride, float* lse,
                          void* workspace, size_t workspace_bytes, int32_t* status,
                          void* stream) {
  gdn_status s = check_attn(cfg, cache, num_seqs, num_tokens, max_q_len, max_kv_len);
  if (s == GDN_OK) s = check_cache(cache);
  if (s != GDN_OK) return s;
  if (max_blocks < 1 || !cu_q || !kv_len || !block_table || !aligned(cu_q, 4) ||
      !aligned(kv_len, 4) || !aligned(block_table, 4) || !aligned(lse, 4) || !aligned(status, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0) {
    if (!rows_ok(q, q_stride, cfg->num_q_heads, cache->head_dim, cfg->io_dtype) ||
        !rows_ok(o, o_stride, cfg->num_q_heads, cache->head_dim, cfg->io_dtype))
      return GDN_ERR_INVALID_ARGUMENT;
    const int64_t row = (int64_t)cfg->num_q_heads * cache->head_dim;
    const size_t e = item_size(cfg->io_dtype);
    if (rows_overlap(q, q_stride, row, o, o_stride, row, num_tokens, e))
      return GDN_ERR_INVALID_ARGUMENT;
    if (lse) {
      const Span l = span_of(lse, 1, 0, (int64_t)num_tokens * cfg->num_q_heads, 4);
      if (overlap(l, span_of(q, num_tokens, q_stride, row, e)) ||
          overlap(l, span_of(o, num_tokens, o_stride, row, e)))
        return GDN_ERR_INVALID_ARGUMENT;
    }
  }
  if (!workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < gdn::attn_workspace(*cfg, *cache)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0 || max_q_len == 0) return GDN_OK;
  gdn::AttnArgs a = {};
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.q_stride = q_stride;
  a.o_stride = o_stride;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.block_table = block_table;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.max_blocks = max_blocks;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.hkv = cache->num_kv_heads;
  a.group = cfg->num_q_heads / cache->num_kv_heads;
  a.by_group = gdn::FastDiv((uint32_t)a.group);
  while ((1 << a.page_shift) < a.page_size) ++a.page_shift;
  a.head_dim = cache->head_dim;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.max_q_len = max_q_len;
  a.max_kv_len = max_kv_len;
  a.causal = cfg->causal ? 1 : 0;
  a.scale_log2 = cfg->scale * 1.4426950408889634f;
  a.status = status;
  a.partials = static_cast<float*>(workspace);
  a.counter = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) +
                                         gdn::attn_workspace(*cfg, *cache) - 256);
  return on_device(h, [&] { return gdn::launch_attn(a, *cache, cfg->io_dtype == GDN_BF16, stream); });
}

}  // extern "C"

namespace gdn {

size_t attn_workspace(const gdn_attn_config& cfg, const gdn_kv_cache& c) {
  const size_t n = split_workspace(cfg, c);
  return (n + 255) / 256 * 256 + 256;  // and the tile kernel's counter
}

// Longest request, in queries, that the split kernel takes. It passes over a request's tokens
// once for every 16 rows (query heads of a group, query by query), on all SMs together; the tile
// kernel once for every 128, a unit to an SM. So the split kernel is the faster one while the
// passes are few: up to about 64 for each round of units over the SMs at head_dim 256, 128 below.
// Measured with 2,000 cached tokens, split / tile in us of a call: 32 requests of 16 query and 2
// key/value heads (D 256) 47 / 45 with 16 rows, 57 / 45 with 32, 83 / 46 with 64; 4 such requests
// 21 / 37, 27 / 38, 43 / 39 and 42 / 41 with 128; 32 of 32 and 8 heads (D 128) 52 / 62 with 16,
// 86 / 62 with 32.
// One query of a group of 16 always counts as few.
int split_queries(const AttnArgs& a, int sms) {
  const int64_t units = (int64_t)a.num_seqs * a.hkv;
  const int64_t passes = (a.head_dim == 256 ? 64 : 128) * ((units + sms - 1) / sms);
  const int64_t rows = std::min<int64_t>(std::max<int64_t>(16 * (passes / units), 16), kTileRows);
  return std::max<int>(1, (int)(rows / a.group));
}

int launch_attn(const AttnArgs& args, const gdn_kv_cache& c, bool bf16, void* stream) {
  AttnArgs a = args;
  int sms = 0;
  const int e = device_sms(&sms);
  if (e != 0) return e;
  sms = std::min(sms, kMaxSms);
  // fp32 queries need more than the tile kernel's operands hold
  a.split_q = bf16 ? split_queries(a, sms) : a.max_q_len;
  // The kernels write different rows and may run at the same time; the counter of the second is
  // cleared in front of both.
  const bool tiles = a.max_q_len > a.split_q;
  int r = 0;
  if (tiles)
    r = (int)cudaMemsetAsync(a.counter, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream));
  if (r == 0) r = launch_attn_split(a, c, bf16, sms, stream);
  return r != 0 || !tiles ? r : launch_attn_tile(a, c, sms, stream);
}

}  // namespace gdn
