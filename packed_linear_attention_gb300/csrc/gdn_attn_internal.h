// gdn_attn_internal.h — structures shared by the full-attention kernels (step plan, rotary
// embedding, cache append, paged attention) and their C entry points.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"

namespace gdn {

constexpr int kMaxSeqs = 4096;  // requests of one plan or attention call (prefix sums in smem)

struct PlanArgs {
  int32_t page_size, num_seqs, num_tokens, max_blocks, num_pages;
  const int32_t *ctx_len, *new_len;
  int32_t* block_table;
  const int32_t *free_pages, *free_count;
  int32_t *free_count_out, *cu_new, *kv_len, *positions;
  int64_t* slots;
  int32_t* status;
};
int launch_kv_plan(const PlanArgs& a, void* stream);

struct ReleaseArgs {
  int32_t page_size, num_seqs, max_blocks, num_pages;
  const int32_t *kv_len, *release;
  int32_t *block_table, *free_pages, *free_count, *status;
};
int launch_kv_release(const ReleaseArgs& a, void* stream);

// The heads of one tensor (q or k) of a rotation; in == out with equal strides is in place.
struct RopeHeads {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;  // elements
  int32_t heads;
};
struct RopeArgs {
  RopeHeads x[2];
  const int32_t* positions;
  int64_t pos_stride;
  int32_t num_tokens;
};
int launch_rope(const gdn_rope& rope, const RopeArgs& a, bool bf16, void* stream);

struct AppendArgs {
  gdn_kv_cache cache;
  int32_t num_tokens;
  const int64_t* slots;
  const void *k, *v;
  int64_t k_stride, v_stride;
  int32_t* status;
  bool rotate;    // k is rotated with rope_args.positions (and q, when rope_args.x[0].heads)
  RopeArgs rope_args;
};
int launch_kv_append(const gdn_rope* rope, const AppendArgs& a, bool bf16, void* stream);

// Paged attention. Every request's queries are taken as rows r = query * group + head of one
// key/value head (group = query heads per key/value head).
// n / d for n in [0, 2^31) as a product and a shift: m = ceil(2^(31 + s) / d), s = ceil(log2 d),
// is off by less than 2^s / d, at most one in n m / 2^(31 + s) before the floor's next step.
struct FastDiv {
  uint32_t d = 1, m = 0, s = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    while ((1u << s) < d) ++s;
    if (s > 0) m = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int32_t operator()(int32_t n) const {
    return s == 0 ? n : (int32_t)(__umulhi((uint32_t)n, m) >> (s - 1));
  }
#endif
};

struct AttnArgs {
  const void* q;
  void* o;
  float* lse;
  int64_t q_stride, o_stride;  // elements
  const int32_t *cu_q, *kv_len, *block_table;
  const float *k_scale, *v_scale;
  int32_t max_blocks, num_pages, page_size, page_shift, hkv, group, head_dim;
  FastDiv by_group;            // rows to queries
  int32_t num_seqs, num_tokens, max_q_len, max_kv_len;
  int32_t causal;
  float scale_log2;            // score scale times log2(e)
  // Requests of at most split_q queries go to the split kernel (gdn_attn_split.cu), longer ones
  // to the tile kernel (gdn_attn_tile.cu); split_queries in gdn_attn_api.cu has the rule.
  int32_t split_q;
  int32_t* status;
  float* partials;             // workspace of the split kernel
  int32_t* counter;            // workspace of the tile kernel: units taken
};
// Value scales enter the exponents, not the accumulator. With s a token's score (log2) and z = s +
// log2(its value scale) + kScaleShift, a row keeps two running maxima over the tokens that it sees:
// ms of s, to which its softmax sum refers, and mz of z, to which the accumulator does. P is
// 2^(z - mz), so that the row's largest weight (probability times value scale) fills the f16 range
// whatever the scales of other pages are; the sum takes P times 2^(mz - ms + s - z), one factor
// for 16 tokens. Both maxima are looked at when a z passes mz by kLazyMax (log2 units), or when a
// scale lies 2^kNear below the row's (mz - ms); in between scores stay below ms + kLazyMax + kNear.
// For a scale that far below, the exponent is raised to at least -kFar - ms + s: P is 0 in f16 all
// the same, and the probability is not lost from the sum. The shift brings scales of ordinary
// values (2^-6) to z = s. Scales below 2^-100 (the append's least) count as 0: their tokens have the
// exponent of 2^-100 and zeros for values. Scales above 2^120 (its largest) count as that.
constexpr float kScaleShift = 6.f;
constexpr float kLazyMax = 8.f, kNear = 40.f, kFar = 45.f;
constexpr float kNoMax = -3.402823466e38f;  // maxima of a row that has seen no token (finite, so
                                            // that differences are no NaN)
constexpr float kMinValueScale = 7.8886090522101181e-31f;  // 2^-100
constexpr float kMaxValueScale = 1.3292279957849159e36f;   // 2^120

constexpr int kSplitTile = 64;     // cached tokens of a work item of the split kernel
constexpr int kTileRows = 128;     // query rows of a unit of the tile kernel
// Units of the tile kernel in one call: 32 requests' sum fits 32 bits. (2^26 units of 128 rows of
// 64 bf16 values would be a terabyte of queries.)
constexpr int kMaxUnits = 1 << 26;

// Longest request: tokens are numbered in 32 bits, by batches of 512 and a batch ahead. (A cache
// has fewer than 2^31 tokens in all.)
constexpr int32_t kMaxKvLen = INT32_MAX - 4096;

constexpr int kMaxSms = 160;       // the workspace is sized without asking the device

size_t attn_workspace(const gdn_attn_config& cfg, const gdn_kv_cache& c);
int launch_attn(const AttnArgs& a, const gdn_kv_cache& c, bool bf16, void* stream);
// Workspace bytes of the split kernel's partial results.
size_t split_workspace(const gdn_attn_config& cfg, const gdn_kv_cache& c);
int launch_attn_split(const AttnArgs& a, const gdn_kv_cache& c, bool bf16, int num_sms,
                      void* stream);
int launch_attn_tile(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, void* stream);
// uint8 map over the cache's rows ([pages * heads * page_size] x head_dim) with boxes of
// box_rows rows x 128 bytes (64 for head_dim 64), swizzled by as much (gdn_tma.cu).
bool make_cache_map(CUtensorMap* m, const void* base, const gdn_kv_cache& c, int box_rows);
// SM count of the current device (asked once per device).
int device_sms(int* out);

#ifdef __CUDACC__
// Request b's range, made safe: first row, queries, cached tokens. Raises `bad` when the
// caller's numbers had to be cut. Both ends are cut to [0, num_tokens] before the subtraction,
// which would wrap for an end far below 0. (For the host too, where its test runs it.)
struct AttnSeq {
  int32_t row0, q_len, kv_len;
};
__host__ __device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b, bool& bad) {
  const int32_t r0 = a.cu_q[b], r1 = a.cu_q[b + 1], kv = a.kv_len[b];
  AttnSeq s;
  s.row0 = min(max(r0, 0), a.num_tokens);
  s.q_len = min(max(min(max(r1, 0), a.num_tokens) - s.row0, 0), a.max_q_len);
  const int64_t room = (int64_t)a.max_blocks * a.page_size;
  s.kv_len = (int32_t)min((int64_t)min(max(kv, 0), min(a.max_kv_len, kMaxKvLen)), room);
  bad = bad || s.row0 != r0 || s.q_len != (int64_t)r1 - r0 || s.kv_len != kv;
  return s;
}
// Cached tokens that query i of the request sees.
__host__ __device__ __forceinline__ int32_t attn_limit(const AttnArgs& a, const AttnSeq& s,
                                                       int32_t i) {
  return a.causal ? min(max(s.kv_len - s.q_len + i + 1, 0), s.kv_len) : s.kv_len;
}

// Sum of two counts of work items (or units), held at kTooMany. The host check keeps those of
// requests in order below it; requests whose rows overlap can ask for more, and get none.
constexpr int32_t kTooMany = INT32_MAX;
__host__ __device__ __forceinline__ int32_t add_items(int32_t x, int32_t y) {
  const uint32_t sum = (uint32_t)x + (uint32_t)y;
  return sum < (uint32_t)kTooMany ? (int32_t)sum : kTooMany;
}

__device__ __forceinline__ void raise_status(int32_t* status, int32_t code) {
  if (status) atomicMax(status, code);
}
#endif

}  // namespace gdn
