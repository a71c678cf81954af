// gdn_step_api.cu — C entry points of the calls around the recurrent layers (convolution, selective
// scan, norm, sampling): the checks of their arguments. Everything is checked before anything is
// enqueued; the handle comes last, so that a call without one shows what else is wrong with it.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/gdn.h"
#include "gdn_args.h"
#include "gdn_internal.h"
#include "gdn_step_internal.h"

namespace {

using namespace gdn::args;

// The host fields of a pack of requests; its device arrays where `arrays`.
gdn_status check_requests(const gdn_requests* r, bool arrays) {
  if (!r || r->num_seqs < 1 || r->num_tokens < 0 || r->max_len < 0 || r->num_slots < 1 ||
      r->num_ckpt < 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (arrays) {
    if (!r->cu || !aligned(r->cu, 4) || !aligned(r->slot_idx, 4) || !aligned(r->start_zero, 4) ||
        !aligned(r->ckpt_cu, 4) || !aligned(r->ckpt_pos, 4) ||
        (r->ckpt_cu && r->num_ckpt > 0 && !r->ckpt_pos) || (!r->slot_idx && r->num_seqs > r->num_slots))
      return GDN_ERR_INVALID_ARGUMENT;
  }
  return r->num_seqs > gdn::kMaxRequests || r->num_tokens > gdn::kMaxRows ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

bool row_ok(const void* p, int64_t stride, int32_t n, int32_t dtype) {
  return rows_ok(p, stride, 1, n, dtype);
}

// Two arrays of rows: the same one (in place), or none of the other's memory.
bool same_or_apart(const void* p, int64_t ps, const void* q, int64_t qs, int64_t row, int64_t tokens,
                   size_t item) {
  return (p == q && ps == qs) || !rows_overlap(p, ps, row, q, qs, row, tokens, item);
}

Span whole(const void* p, int64_t items, size_t item) { return span_of(p, 1, 0, items, item); }

gdn_status check_conv(const gdn_conv_config* c) {
  if (!c || c->channels < 1 || c->width < 1 || !known_dtype(c->io_dtype) || !c->weight ||
      !aligned(c->weight, 4) || !aligned(c->bias, 4) ||
      (c->activation != GDN_ACT_NONE && c->activation != GDN_ACT_SILU))
    return GDN_ERR_INVALID_ARGUMENT;
  return c->width < 2 || c->width > 4 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn_status check_ssm(const gdn_ssm_config* c, bool arrays) {
  if (!c || c->channels < 1 || c->num_groups < 1 || c->channels % c->num_groups != 0 ||
      c->state_dim < 1 || !known_dtype(c->io_dtype))
    return GDN_ERR_INVALID_ARGUMENT;
  // a's rows and the states' are read 16 bytes at a time
  if (arrays && (!c->a || !aligned(c->a, 16) || !aligned(c->d, 4) || !aligned(c->delta_bias, 4)))
    return GDN_ERR_INVALID_ARGUMENT;
  return c->state_dim > 128 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

// The rows of a scan: each array by itself, and y against the others.
bool ssm_rows_ok(const gdn_ssm_config& c, const gdn_ssm_rows* r, int64_t tokens) {
  if (!r) return false;
  if (tokens == 0) return true;
  const size_t e = item_size(c.io_dtype);
  const int64_t ch = c.channels, gn = (int64_t)c.num_groups * c.state_dim;
  if (!row_ok(r->x, r->x_stride, c.channels, c.io_dtype) ||
      !row_ok(r->delta, r->delta_stride, c.channels, c.io_dtype) ||
      !row_ok(r->y, r->y_stride, c.channels, c.io_dtype) ||
      (r->z && !row_ok(r->z, r->z_stride, c.channels, c.io_dtype)))
    return false;
  for (const auto& [p, s] : {std::pair<const void*, int64_t>{r->b, r->b_stride}, {r->c, r->c_stride}}) {
    if (!p || !aligned(p, e) || s < gn || s > (int64_t)1 << 40) return false;
    if (rows_overlap(r->y, r->y_stride, ch, p, s, gn, tokens, e)) return false;
  }
  return same_or_apart(r->y, r->y_stride, r->x, r->x_stride, ch, tokens, e) &&
         same_or_apart(r->y, r->y_stride, r->delta, r->delta_stride, ch, tokens, e) &&
         (!r->z || same_or_apart(r->y, r->y_stride, r->z, r->z_stride, ch, tokens, e));
}

// A pool of states and the checkpoints beside it.
gdn_status check_states(const void* pool, int64_t slots, const void* ckpt, int64_t num_ckpt,
                        int64_t state, size_t item) {
  if (!pool || !aligned(pool, 16) || !aligned(ckpt, 16) || (num_ckpt > 0 && !ckpt))
    return GDN_ERR_INVALID_ARGUMENT;
  if (num_ckpt > 0 && overlap(whole(pool, slots * state, item), whole(ckpt, num_ckpt * state, item)))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// What the kernels' grids take: blocks in all, and of a row's channels.
bool grid_ok(int32_t channels, double blocks) {
  return channels <= (1 << 18) && blocks <= (double)INT32_MAX;
}

// Bytes of `units` end states, and of them with their sums of dt: the workspace.
void scan_bytes(const gdn_ssm_config& cfg, int64_t units, size_t* ends, size_t* bytes) {
  *ends = ((size_t)units * cfg.channels * cfg.state_dim * 4 + 255) / 256 * 256;
  *bytes = std::max<size_t>(256, *ends + ((size_t)units * cfg.channels * 4 + 255) / 256 * 256);
}

}  // namespace

extern "C" {

gdn_status gdn_conv_packed(gdn_handle* h, const gdn_conv_config* cfg, const gdn_requests* req,
                           const void* x, int64_t x_stride, void* y, int64_t y_stride,
                           void* state_pool, void* ckpt_states, int32_t* status, void* stream) {
  gdn_status s = check_conv(cfg);
  if (s == GDN_OK) s = check_requests(req, true);
  if (s != GDN_OK) return s;
  const size_t e = item_size(cfg->io_dtype);
  const int64_t state = (int64_t)(cfg->width - 1) * cfg->channels, tokens = req->num_tokens;
  const int32_t num_ckpt = req->ckpt_cu ? req->num_ckpt : 0;
  s = check_states(state_pool, req->num_slots, ckpt_states, num_ckpt, state, e);
  if (s != GDN_OK) return s;
  if (!aligned(status, 4)) return GDN_ERR_INVALID_ARGUMENT;
  if (tokens > 0) {
    if (!row_ok(x, x_stride, cfg->channels, cfg->io_dtype) ||
        !row_ok(y, y_stride, cfg->channels, cfg->io_dtype) ||
        rows_overlap(x, x_stride, cfg->channels, y, y_stride, cfg->channels, tokens, e))
      return GDN_ERR_INVALID_ARGUMENT;
    const Span pool = whole(state_pool, req->num_slots * state, e);
    const Span ckpt = whole(ckpt_states, num_ckpt * state, e);
    const Span in = span_of(x, tokens, x_stride, cfg->channels, e);
    const Span out = span_of(y, tokens, y_stride, cfg->channels, e);
    if (overlap(in, pool) || overlap(out, pool) || overlap(in, ckpt) || overlap(out, ckpt))
      return GDN_ERR_INVALID_ARGUMENT;
  }
  // one block for every 32 rows and 512 channels at least (four channels of 128 threads)
  if (!grid_ok(cfg->channels, (tokens / 32.0 + req->num_seqs) * (cfg->channels / 512.0 + 1))) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  const gdn::ConvArgs a = {*cfg, *req, x, y, x_stride, y_stride, state_pool, ckpt_states, status};
  return on_device(h, [&] { return gdn::launch_conv_packed(a, stream); });
}

gdn_status gdn_conv_step(gdn_handle* h, const gdn_conv_config* cfg, int32_t batch, const void* x,
                         int64_t x_stride, void* y, int64_t y_stride, void* state_pool,
                         int32_t num_slots, const int32_t* slot_idx, int32_t* status, void* stream) {
  gdn_status s = check_conv(cfg);
  if (s != GDN_OK) return s;
  if (batch < 0 || num_slots < 1 || !aligned(status, 4)) return GDN_ERR_INVALID_ARGUMENT;
  const size_t e = item_size(cfg->io_dtype);
  const int64_t state = (int64_t)(cfg->width - 1) * cfg->channels;
  s = check_states(state_pool, num_slots, nullptr, 0, state, e);
  if (s != GDN_OK) return s;
  if (batch > 0) {
    if (!slot_idx || !aligned(slot_idx, 4) || !row_ok(x, x_stride, cfg->channels, cfg->io_dtype) ||
        !row_ok(y, y_stride, cfg->channels, cfg->io_dtype) ||
        !same_or_apart(y, y_stride, x, x_stride, cfg->channels, batch, e))
      return GDN_ERR_INVALID_ARGUMENT;
    const Span pool = whole(state_pool, num_slots * state, e);
    if (overlap(pool, span_of(x, batch, x_stride, cfg->channels, e)) ||
        overlap(pool, span_of(y, batch, y_stride, cfg->channels, e)))
      return GDN_ERR_INVALID_ARGUMENT;
  }
  if (!grid_ok(cfg->channels, (double)batch * (cfg->channels / 512.0 + 1))) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  gdn::ConvArgs a = {*cfg, {}, x, y, x_stride, y_stride, state_pool, nullptr, status};
  a.req.num_tokens = batch;
  a.req.num_slots = num_slots;
  a.req.slot_idx = slot_idx;
  return on_device(h, [&] { return gdn::launch_conv_step(a, stream); });
}

gdn_status gdn_ssm_workspace_size(const gdn_ssm_config* cfg, const gdn_requests* req,
                                  size_t* bytes) {
  gdn_status s = check_ssm(cfg, false);
  if (s == GDN_OK) s = check_requests(req, false);
  if (s != GDN_OK) return s;
  if (!bytes) return GDN_ERR_INVALID_ARGUMENT;
  size_t ends;
  scan_bytes(*cfg, gdn::ssm_most_units(*cfg, *req), &ends, bytes);
  return GDN_OK;
}

gdn_status gdn_ssm_packed(gdn_handle* h, const gdn_ssm_config* cfg, const gdn_requests* req,
                          const gdn_ssm_rows* rows, float* state_pool, float* ckpt_states,
                          void* workspace, size_t workspace_bytes, int32_t* status,
                          void* stream) {
  gdn_status s = check_ssm(cfg, true);
  if (s == GDN_OK) s = check_requests(req, true);
  if (s != GDN_OK) return s;
  const int64_t state = (int64_t)cfg->channels * cfg->state_dim, tokens = req->num_tokens;
  const int32_t num_ckpt = req->ckpt_cu ? req->num_ckpt : 0;
  s = check_states(state_pool, req->num_slots, ckpt_states, num_ckpt, state, 4);
  if (s != GDN_OK) return s;
  if (!aligned(status, 4) || !ssm_rows_ok(*cfg, rows, tokens)) return GDN_ERR_INVALID_ARGUMENT;
  const int32_t segment = gdn::ssm_segment(*cfg, *req);
  const int64_t units = gdn::ssm_units(*req, segment);
  size_t ends, need;
  scan_bytes(*cfg, units, &ends, &need);
  if (!workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARGUMENT;
  const Span pool = whole(state_pool, req->num_slots * state, 4);
  const Span ckpt = whole(ckpt_states, num_ckpt * state, 4);
  const Span work = whole(workspace, (int64_t)need, 1);
  if (overlap(work, pool) || overlap(work, ckpt)) return GDN_ERR_INVALID_ARGUMENT;
  if (tokens > 0) {
    const size_t e = item_size(cfg->io_dtype);
    const int64_t gn = (int64_t)cfg->num_groups * cfg->state_dim;
    const Span all[] = {span_of(rows->x, tokens, rows->x_stride, cfg->channels, e),
                        span_of(rows->delta, tokens, rows->delta_stride, cfg->channels, e),
                        span_of(rows->y, tokens, rows->y_stride, cfg->channels, e),
                        span_of(rows->b, tokens, rows->b_stride, gn, e),
                        span_of(rows->c, tokens, rows->c_stride, gn, e),
                        rows->z ? span_of(rows->z, tokens, rows->z_stride, cfg->channels, e) : Span{0, 0}};
    for (const Span& a : all)
      if (overlap(a, pool) || overlap(a, ckpt) || overlap(a, work)) return GDN_ERR_INVALID_ARGUMENT;
  }
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  // blocks: of a group's channels 16 at least
  if (!grid_ok(cfg->channels, (double)(req->num_seqs + units) * (cfg->channels / 16.0 + cfg->num_groups)))
    return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  gdn::SsmArgs a = {*cfg, *req, *rows, state_pool, ckpt_states, static_cast<float*>(workspace),
                    reinterpret_cast<float*>(static_cast<char*>(workspace) + ends), segment,
                    (int32_t)units, status};
  return on_device(h, [&] { return gdn::launch_ssm_packed(a, stream); });
}

gdn_status gdn_ssm_step(gdn_handle* h, const gdn_ssm_config* cfg, int32_t batch,
                        const gdn_ssm_rows* rows, float* state_pool, int32_t num_slots,
                        const int32_t* slot_idx, int32_t* status, void* stream) {
  gdn_status s = check_ssm(cfg, true);
  if (s != GDN_OK) return s;
  const int64_t state = (int64_t)cfg->channels * cfg->state_dim;
  if (batch < 0 || num_slots < 1 || !aligned(status, 4)) return GDN_ERR_INVALID_ARGUMENT;
  s = check_states(state_pool, num_slots, nullptr, 0, state, 4);
  if (s != GDN_OK) return s;
  if (!ssm_rows_ok(*cfg, rows, batch)) return GDN_ERR_INVALID_ARGUMENT;
  if (batch > 0) {
    if (!slot_idx || !aligned(slot_idx, 4)) return GDN_ERR_INVALID_ARGUMENT;
    const Span pool = whole(state_pool, num_slots * state, 4);
    const size_t e = item_size(cfg->io_dtype);
    const int64_t gn = (int64_t)cfg->num_groups * cfg->state_dim;
    if (overlap(pool, span_of(rows->x, batch, rows->x_stride, cfg->channels, e)) ||
        overlap(pool, span_of(rows->delta, batch, rows->delta_stride, cfg->channels, e)) ||
        overlap(pool, span_of(rows->y, batch, rows->y_stride, cfg->channels, e)) ||
        overlap(pool, span_of(rows->b, batch, rows->b_stride, gn, e)) ||
        overlap(pool, span_of(rows->c, batch, rows->c_stride, gn, e)) ||
        (rows->z && overlap(pool, span_of(rows->z, batch, rows->z_stride, cfg->channels, e))))
      return GDN_ERR_INVALID_ARGUMENT;
  }
  if (!grid_ok(cfg->channels, batch)) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  gdn::SsmArgs a = {*cfg, {}, *rows, state_pool, nullptr, nullptr, nullptr, 0, 0, status};
  a.req.num_tokens = batch;
  a.req.num_slots = num_slots;
  a.req.slot_idx = slot_idx;
  return on_device(h, [&] { return gdn::launch_ssm_step(a, stream); });
}

gdn_status gdn_rms_norm(gdn_handle* h, const gdn_norm_config* cfg, int32_t num_tokens,
                        const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, void* sum, int64_t sum_stride, const void* gate,
                        int64_t gate_stride, void* y, int64_t y_stride, void* codes,
                        int64_t codes_stride, float* scales, void* stream) {
  if (!cfg || cfg->num_heads < 1 || cfg->dim < 1 || !known_dtype(cfg->io_dtype) ||
      cfg->scale_group < 0 || !(cfg->eps >= 0.f) || !std::isfinite(cfg->eps) ||
      !std::isfinite(cfg->weight_offset) || !aligned(cfg->weight, 16) || num_tokens < 0)
    return GDN_ERR_INVALID_ARGUMENT;
  const int32_t group = cfg->scale_group, d = cfg->dim, heads = cfg->num_heads;
  const int64_t row = (int64_t)heads * d;
  if (group > 0 && d % group != 0) return GDN_ERR_INVALID_ARGUMENT;
  // a call of no rows may come with no arrays
  if (num_tokens > 0 && ((codes == nullptr) != (scales == nullptr) || (!y && !codes) || (sum && !residual)))
    return GDN_ERR_INVALID_ARGUMENT;
  if (row > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (num_tokens > 0) {
    const size_t e = item_size(cfg->io_dtype);
    const int32_t io = cfg->io_dtype, n = (int32_t)row;
    struct Rows {
      const void* p;
      int64_t stride;
    };
    const Rows in[] = {{x, x_stride}, {residual, residual_stride}, {gate, gate_stride}};
    const Rows out[] = {{sum, sum_stride}, {y, y_stride}};
    if (!x) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : in)
      if (r.p && !row_ok(r.p, r.stride, n, io)) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : out)
      if (r.p && !row_ok(r.p, r.stride, n, io)) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& o : out)
      for (const Rows& i : in)
        if (o.p && i.p && !same_or_apart(o.p, o.stride, i.p, i.stride, row, num_tokens, e))
          return GDN_ERR_INVALID_ARGUMENT;
    if (sum && y && rows_overlap(sum, sum_stride, row, y, y_stride, row, num_tokens, e))
      return GDN_ERR_INVALID_ARGUMENT;
    if (codes) {
      if (!aligned(codes, 16) || codes_stride < row || codes_stride % 16 != 0 ||
          codes_stride > (int64_t)1 << 40 || !aligned(scales, 4))
        return GDN_ERR_INVALID_ARGUMENT;
      const Span c = span_of(codes, num_tokens, codes_stride, row, 1);
      const Span s = whole(scales, (int64_t)num_tokens * (group ? row / group : 1), 4);
      if (overlap(c, s)) return GDN_ERR_INVALID_ARGUMENT;
      for (const Rows& r : {in[0], in[1], in[2], out[0], out[1]}) {
        if (!r.p) continue;
        const Span a = span_of(r.p, num_tokens, r.stride, row, e);
        if (overlap(a, c) || overlap(a, s)) return GDN_ERR_INVALID_ARGUMENT;
      }
    }
  }
  if ((group != 0 && group != 32 && group != 64 && group != 128) ||
      (heads > 1 && d != 64 && d != 128 && d != 256) || row > gdn::kMaxNormRow)
    return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  const gdn::NormArgs a = {*cfg, num_tokens, x, residual, gate, sum, y, codes, x_stride,
                           residual_stride, gate_stride, sum_stride, y_stride, codes_stride, scales};
  return on_device(h, [&] { return gdn::launch_rms_norm(a, stream); });
}

gdn_status gdn_sample(gdn_handle* h, int32_t io_dtype, int32_t num_rows, int32_t vocab,
                      const void* logits, int64_t stride, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p,
                      const float* u, int32_t* token, float* logprob, int32_t* status,
                      void* stream) {
  if (!known_dtype(io_dtype) || num_rows < 0 || vocab < 1 || !aligned(status, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  if (num_rows > 0) {
    const size_t e = item_size(io_dtype);
    if (!logits || !aligned(logits, e) || stride < vocab || stride > (int64_t)1 << 40 || !u || !token)
      return GDN_ERR_INVALID_ARGUMENT;
    const Span in[] = {span_of(logits, num_rows, stride, vocab, e), whole(u, num_rows, 4),
                       whole(temperature, temperature ? num_rows : 0, 4),
                       whole(top_k, top_k ? num_rows : 0, 4), whole(top_p, top_p ? num_rows : 0, 4),
                       whole(min_p, min_p ? num_rows : 0, 4)};
    const Span t = whole(token, num_rows, 4), l = whole(logprob, logprob ? num_rows : 0, 4);
    for (const void* p : {(const void*)u, (const void*)temperature, (const void*)top_k,
                          (const void*)top_p, (const void*)min_p, (const void*)token,
                          (const void*)logprob})
      if (!aligned(p, 4)) return GDN_ERR_INVALID_ARGUMENT;
    for (const Span& i : in)
      if (overlap(i, t) || overlap(i, l)) return GDN_ERR_INVALID_ARGUMENT;
    if (overlap(t, l)) return GDN_ERR_INVALID_ARGUMENT;
  }
  if (vocab > gdn::kMaxVocab || num_rows > (1 << 24)) return GDN_ERR_UNSUPPORTED;
  if (!h) return GDN_ERR_INVALID_ARGUMENT;
  const gdn::SampleArgs a = {io_dtype, num_rows, vocab, logits, stride, temperature, top_k,
                             top_p,    min_p,    u,     token,  logprob, status};
  return on_device(h, [&] { return gdn::launch_sample(a, stream); });
}

}  // extern "C"
