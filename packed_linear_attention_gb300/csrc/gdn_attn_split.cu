// gdn_attn_split.cu — attention of few queries over the paged e4m3 cache, the work split over
// the cached tokens.
//
// A unit is (request, key/value head, up to 8 NT query rows); its work items are the 64-token
// tiles of the request's cache. All units' items form one line that is cut into equal pieces,
// one for each resident block, whatever the requests' lengths: one user's 32K context and a
// ragged batch both fill every SM, and no host lengths are needed (each block finds its piece
// from a prefix sum over the requests). A block that covers a unit's whole range writes the
// output; pieces of a unit that was cut leave (max, sum, accumulator) in the workspace and a
// second kernel joins them in order, so the result does not depend on timing.
//
// Bound: HBM (16 query and 2 key/value heads of 256, one query each: 128 requests of 128 to 16,384
// tokens 164 us, 89% of the measured copy rate; one of 32,768 tokens 19 us of which the read is 5
// and the rest two launches, the pipeline's start and the join). A cached token is read once for
// all query rows of its head, up to 16. One producer warp
// keeps the stages' TMA copies in flight (page ids and scales are fetched 512 tokens ahead);
// four consumer warps take 16 tokens of every tile each, with running maximum, sum and
// accumulator of their own, merged when the piece ends.
//
// Products run transposed on m16n8k16 f16 warp MMAs (the tensor rate is not the bound here,
// and 8 query rows fill n = 8 exactly):
//   S^T (16 tokens x 8 rows) = K (16 x D) Q^T      O^T (D x 8 rows) += V^T P^T
// e4m3 values are f16 values, so K and V enter exactly. The contraction index of S may be
// permuted alike in K and Q, so a thread takes its K operand as whole 16-byte chunks of a
// token's row; V^T is read with transposing 16-bit ldmatrix (two channels to an element) and
// one byte permutation. The queries are scaled by a power of two per row into the f16 range
// (bf16 fits exactly); fp32 queries and probabilities are two f16 terms.
// The running maxima (of scores and of exponents with the value scales, see kScaleShift in
// gdn_attn_internal.h) are only raised when one is passed by 8 (in log2 units): until then
// weights stay below 2^8 and no cross-lane reduction is needed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gdn_attn_internal.h"
#include "gdn_internal.h"
#include "ptx_sm103.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kWarps = 4;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);     // and the producer warp
constexpr int kTile = kSplitTile;
constexpr int kGroups = kTile / 16;             // 16-token groups of a tile, one per warp
constexpr int kCtasPerSm = 2;
constexpr int kMaxStages = 8;
constexpr uint32_t kWaitLimit = 1u << 20;       // a poll that fails takes 0.8 us: about a second
constexpr float kProbScale = 64.f;              // weights times this and a scale's fraction: at
                                                // most 2^15 in f16
constexpr float kOutShift = 6.f + kScaleShift;  // log2 of kProbScale and the scales' shift
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kStatusTimeout = GDN_ERR_DEVICE_TIMEOUT;
constexpr size_t kSmemPerCta = 112 * 1024;      // two blocks share an SM's 227 KB

#define GDN_INF __int_as_float(0x7f800000)

struct SplitParams {
  AttnArgs a;
  CUtensorMap tk, tv;
  float* part;        // [2 workers][RB (D + 4)]: rows, then their maxima (z, s) and sum
  int32_t stages;
  uint32_t off_q, off_red, off_pre;  // shared-memory map after the stages
};

__device__ __forceinline__ uint32_t e4m3_to_half2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ uint32_t lo_half2(uint32_t w) { return e4m3_to_half2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_half2(uint32_t w) { return e4m3_to_half2((uint16_t)(w >> 16)); }
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of 64 rows as TMA wrote it:
// regions of 128 bytes a row under the 128-byte swizzle, or rows of 64 bytes under the 64-byte
// one.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {
  if constexpr (D == 64) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
  else return (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

struct __align__(16) GroupMeta {
  float ks;       // key scale; below 0: the group's page is absent
  float lv;       // exponent of the value scale, shifted
  float pv;       // its fraction, in [1, 2), times kProbScale; 0 for no value
};

template <int NT>
struct SmemHead {
  uint64_t full[kMaxStages], empty[kMaxStages];
  GroupMeta meta[kMaxStages][kGroups];
  float row_scale[8 * NT];
  int32_t row_limit[8 * NT];
  float mz[kWarps][8 * NT], ms[kWarps][8 * NT], l[kWarps][8 * NT];
  int32_t scan[8];
  int32_t dead;
};

// Waits for a phase with a bound; after any wait of the block gave up, none waits again, so
// that every loop still runs its course and no thread is left at a barrier.
__device__ __forceinline__ void wait_or_die(uint64_t* bar, uint32_t parity, volatile int32_t* dead,
                                            int32_t* status) {
  if (mbar_try_wait(bar, parity)) return;
  if (*dead) return;
  if (!mbar_wait_bounded(bar, parity, kWaitLimit)) {
    *dead = 1;
    raise_status(status, kStatusTimeout);
  }
}

// One piece of a unit.
struct Segment {
  int32_t seq, head, row_tile;
  int32_t t0, t1, tiles;  // tiles [t0, t1) of `tiles`
};

template <int RB>
__device__ __forceinline__ int32_t seq_items(const AttnArgs& a, const AttnSeq& s) {
  if (s.q_len == 0 || s.q_len > a.split_q) return 0;
  return a.hkv * ((s.q_len * a.group + RB - 1) / RB) * max(1, (s.kv_len + kTile - 1) / kTile);
}

// The segment that begins at item `w` and ends at or before item `w1`.
template <int RB>
__device__ __forceinline__ Segment find_segment(const AttnArgs& a, const int32_t* pre, int32_t w,
                                                int32_t w1, AttnSeq& s) {
  int32_t lo = 0, hi = a.num_seqs - 1;
  while (lo < hi) {  // the last request whose items begin at or before w
    const int32_t mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= w) lo = mid;
    else hi = mid - 1;
  }
  bool bad = false;
  s = attn_seq(a, lo, bad);
  const int32_t row_tiles = (s.q_len * a.group + RB - 1) / RB;
  Segment g;
  g.seq = lo;
  g.tiles = max(1, (s.kv_len + kTile - 1) / kTile);
  const int32_t x = w - pre[lo], unit = x / g.tiles;
  g.head = unit / row_tiles;
  g.row_tile = unit % row_tiles;
  g.t0 = x % g.tiles;
  g.t1 = min(g.tiles, g.t0 + (w1 - w));
  return g;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// T: type of q and o. NT: tiles of 8 query rows.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
split_kernel(const __grid_constant__ SplitParams p) {
  constexpr int RB = 8 * NT;
  constexpr int kTerms = std::is_same<T, float>::value ? 2 : 1;
  constexpr int kSteps = D / 16;          // k steps of S, and 16-channel chunks of O
  constexpr int kRed = D + 8;             // row stride of the merge buffer
  constexpr uint32_t kTileBytes = kTile * D;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ SmemHead<NT> sm;
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint2* qfrag = reinterpret_cast<uint2*>(smem + p.off_q);  // [terms][NT][kSteps][32]
  float* red = reinterpret_cast<float*>(smem + p.off_red);  // [RB][kRed]
  int32_t* pre = reinterpret_cast<int32_t*>(smem + p.off_pre);  // [num_seqs + 1]

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the second kernel may come
  // ---- prefix sums of the requests' items (every block for itself)
  {
    const int per = (a.num_seqs + kThreads - 1) / kThreads, b0 = tid * per;
    const int b1 = min(a.num_seqs, b0 + per);
    int32_t sum = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const AttnSeq s = attn_seq(a, b, bad);
      sum = add_items(sum, seq_items<RB>(a, s));
    }
    if (bad && blockIdx.x == 0) raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = add_items(inc, y);
    }
    if (lane == 31) sm.scan[warp] = inc;
    if (tid == 0) {
      sm.dead = 0;
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&sm.full[s], 1);
        mbar_init(&sm.empty[s], kWarps);
      }
      fence_mbar_init();
    }
    __syncthreads();
    int32_t at = inc - sum;
    for (int w = 0; w < warp; ++w) at = add_items(at, sm.scan[w]);
    for (int b = b0; b < b1; ++b) {
      pre[b] = at;
      at = add_items(at, seq_items<RB>(a, attn_seq(a, b, bad)));
    }
    if (b1 == a.num_seqs && b0 < b1) pre[a.num_seqs] = at;
    __syncthreads();
  }
  // G workers share W items
  const int64_t W = pre[a.num_seqs] == kTooMany ? 0 : pre[a.num_seqs],
                G = min((int64_t)gridDim.x, W);
  if (blockIdx.x >= G) return;
  const int32_t w0 = (int32_t)(W * blockIdx.x / G), w1 = (int32_t)(W * (blockIdx.x + 1) / G);
  uint32_t it = 0;  // tiles since the start: stage and phase
  const int S = p.stages;

  if (warp == kWarps) {
    // ---- producer
    const int box_rows = min(a.page_size, kTile), per_box = box_rows / 16;
    const uint32_t box_bytes = (uint32_t)box_rows * D;
    for (int32_t w = w0; w < w1;) {
      AttnSeq s;
      const Segment g = find_segment<RB>(a, pre, w, w1, s);
      w += g.t1 - g.t0;
      const int32_t* table = a.block_table + (int64_t)g.seq * a.max_blocks;
      for (int32_t tb = g.t0; tb < g.t1; tb += 8) {  // 8 tiles' pages and scales, one group a lane
        const int32_t tok = tb * kTile + lane * 16;
        int32_t id = -1;
        float ks = -1.f, vs = 0.f;
        if (tok < s.kv_len && tok < g.t1 * kTile) {
          id = table[tok >> a.page_shift];
          if (id >= 0 && id < a.num_pages) {
            ks = a.k_scale[(int64_t)id * a.hkv + g.head];
            vs = a.v_scale[(int64_t)id * a.hkv + g.head];
            if (!(ks >= 0.f)) ks = 0.f;  // not a scale: the group counts as zeros
          } else {
            id = -1;
            raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
          }
        }
        const uint32_t vb = __float_as_uint(fminf(fmaxf(vs, kMinValueScale), kMaxValueScale));
        const int lv = (int)(vb >> 23) - 127 + (int)kScaleShift;
        const GroupMeta group = {ks, (float)lv,
                                 vs >= kMinValueScale  // what is no scale counts as 0
                                     ? __uint_as_float((vb & 0x7FFFFFu) | 0x3F800000u) * kProbScale
                                     : 0.f};
        for (int j = 0; j < 8 && tb + j < g.t1; ++j, ++it) {
          const int st = it % S;
          wait_or_die(&sm.empty[st], ((it / S) & 1u) ^ 1u, &sm.dead, a.status);
          const int first = j * kGroups;
          if (lane >= first && lane < first + kGroups) sm.meta[st][lane - first] = group;
          // one lane per box: the lanes that hold its first group
          const bool box = lane >= first && lane < first + kGroups &&
                           (lane - first) % per_box == 0 && id >= 0;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], 2 * boxes * box_bytes);
          __syncwarp();
          if (box) {
            uint8_t* dk = smem + (uint32_t)st * 2 * kTileBytes;
            const int32_t y = (int32_t)(((int64_t)id * a.hkv + g.head) * a.page_size +
                                        (tok & (a.page_size - 1)));
            const uint32_t row = (uint32_t)(lane - first) * 16;
#pragma unroll
            for (int r = 0; r < (D + 127) / 128; ++r) {
              const uint32_t at = r * (kTile * 128) + row * (D == 64 ? 64 : 128);
              tma_load_2d(dk + at, &p.tk, 128 * r, y, &sm.full[st]);
              tma_load_2d(dk + kTileBytes + at, &p.tv, 128 * r, y, &sm.full[st]);
            }
          }
        }
      }
    }
    // after a wait gave up, copies may still be in flight: let them land
    if (sm.dead)
      for (int k = 0; k < S && k < (int)it; ++k) {
        const uint32_t i = it - 1 - k;
        mbar_wait_bounded(&sm.full[i % S], (i / S) & 1u, kWaitLimit);
      }
    return;
  }

  // ---- consumers
  const int c = lane & 3, n8 = lane >> 2;
  for (int32_t w = w0; w < w1;) {
    AttnSeq s;
    const Segment g = find_segment<RB>(a, pre, w, w1, s);
    w += g.t1 - g.t0;
    const int32_t rows = s.q_len * a.group, r0 = g.row_tile * RB;
    // queries of the unit as f16 operands, a row per warp and round
    for (int r = warp; r < RB; r += kWarps) {
      const int32_t row = r0 + r;
      const bool live = row < rows;
      const int32_t i = live ? a.by_group(row) : 0;
      const T* src = static_cast<const T*>(a.q) + (int64_t)(s.row0 + i) * a.q_stride +
                     (int64_t)(g.head * a.group + (live ? (row - a.by_group(row) * a.group) : 0)) * D;
      constexpr int kQuads = (D / 4 + 31) / 32;
      float x[kQuads][4];
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int quad = lane + 32 * k;
        x[k][0] = x[k][1] = x[k][2] = x[k][3] = 0.f;
        if (live && quad < D / 4) load4(src + 4 * quad, x[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[k][e]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // power of two that brings the row's largest magnitude to [2^13, 2^14)
      int ex = (int)(__float_as_uint(amax) >> 23) - 127;
      ex = ex == 128 ? 13 : max(ex, -100);  // a row with an infinity keeps its values
      const float up = __uint_as_float((uint32_t)(13 - ex + 127) << 23);
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int quad = lane + 32 * k;
        if (quad < D / 4) {
          // element 4 quad + 2 f + e sits in chunk quad / 4, word i = quad % 4 of the chunk
          const int chunk = quad >> 2, word = quad & 3;
          const int step = D == 64 ? word : (chunk >> 3) * 8 + (chunk & 1) * 4 + word;
          const int ln = (r & 7) * 4 + (D == 64 ? chunk : (chunk & 7) >> 1);
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = x[k][e] * up;
          uint2 h = make_uint2(f16x2(y[0], y[1]), f16x2(y[2], y[3]));
          qfrag[((r >> 3) * kSteps + step) * 32 + ln] = h;
          if constexpr (kTerms == 2) {
            const float2 h0 = half2_floats(h.x), h1 = half2_floats(h.y);
            qfrag[((NT + (r >> 3)) * kSteps + step) * 32 + ln] =
                make_uint2(f16x2(y[0] - h0.x, y[1] - h0.y), f16x2(y[2] - h1.x, y[3] - h1.y));
          }
        }
      }
      if (lane == 0) {
        sm.row_scale[r] = a.scale_log2 * __uint_as_float((uint32_t)(ex - 13 + 127) << 23);
        sm.row_limit[r] = live ? attn_limit(a, s, i) : s.kv_len;
      }
    }
    named_sync(1, 32 * kWarps);
    float rs[NT][2];
    int32_t lim[NT][2];
    const int32_t min_limit = sm.row_limit[0];  // limits rise with the row
    const int32_t max_limit = attn_limit(a, s, (min(rows, r0 + RB) - 1) / a.group);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rs[t][e] = sm.row_scale[8 * t + 2 * c + e];
        lim[t][e] = sm.row_limit[8 * t + 2 * c + e];
      }

    float O[kSteps][NT][4];
    float mz[NT][2], apart[NT][2], l[NT][2];  // apart: mz - ms
    float most = kNoMax;                      // largest apart of this thread's rows
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mz[t][0] = mz[t][1] = kNoMax;
      apart[t][0] = apart[t][1] = l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[k][t][e] = 0.f;
    }

    for (int32_t t = g.t0; t < g.t1; ++t, ++it) {
      const int st = it % S;
      wait_or_die(&sm.full[st], (it / S) & 1u, &sm.dead, a.status);
      const int32_t j0 = t * kTile + 16 * warp;
      const GroupMeta meta = sm.meta[st][warp];
      if (j0 < max_limit && meta.ks >= 0.f) {
        const uint32_t sk = smem_u32(smem) + (uint32_t)st * 2 * kTileBytes, sv = sk + kTileBytes;
        // ---- S^T = K Q^T, two accumulator chains
        float acc[2][NT][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[x][n][e] = 0.f;
#pragma unroll
        for (int q = 0; q < kSteps / 4; ++q) {  // chunks of 16 channels: 4 k steps each
          const int chunk = D == 64 ? c : (q >> 1) * 8 + 2 * c + (q & 1);
          uint32_t ka[4], kb[4];
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(ka[0]), "=r"(ka[1]), "=r"(ka[2]), "=r"(ka[3])
                       : "r"(sk + tile_offset<D>(16 * warp + n8, chunk)));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(kb[0]), "=r"(kb[1]), "=r"(kb[2]), "=r"(kb[3])
                       : "r"(sk + tile_offset<D>(16 * warp + n8 + 8, chunk)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 4 * q + i;
            const uint32_t A[4] = {lo_half2(ka[i]), lo_half2(kb[i]), hi_half2(ka[i]),
                                   hi_half2(kb[i])};
#pragma unroll
            for (int x = 0; x < kTerms; ++x)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint2 b = qfrag[((x * NT + n) * kSteps + step) * 32 + lane];
                const uint32_t B[2] = {b.x, b.y};
                mma_f16_16816(acc[step & 1][n], A, B);
              }
          }
        }
        // ---- exponents, running maxima, weights
        float z4[NT][4];
        bool over = most > meta.lv + kNear;
        const bool masked = j0 + 16 > min_limit;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float z = fmaf(acc[0][n][e] + acc[1][n][e], meta.ks * rs[n][e & 1], meta.lv);
            if (masked && j0 + n8 + (e >= 2 ? 8 : 0) >= lim[n][e & 1]) z = -GDN_INF;
            z4[n][e] = z;
            over = over || z > mz[n][e & 1] + kLazyMax;
          }
        if (__any_sync(0xffffffffu, over)) {
          most = kNoMax;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float z = fmaxf(z4[n][e], z4[n][e + 2]);
              z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 4));
              z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 8));
              z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 16));
              const float was = mz[n][e] - apart[n][e], ms = fmaxf(z - meta.lv, was);
              l[n][e] *= ex2(was - ms);
              z = fmaxf(z, mz[n][e]);
              const float f = ex2(mz[n][e] - z);
              mz[n][e] = z;
              apart[n][e] = z - ms;
              most = fmaxf(most, z - ms);
              const float up = fmaxf(apart[n][e] - kFar - meta.lv, 0.f);  // a scale far below
              z4[n][e] += up;
              z4[n][e + 2] += up;
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                O[k][n][e] *= f;
                O[k][n][e + 2] *= f;
              }
            }
        }
        uint32_t B[kTerms][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float pr = ex2(z4[n][e] - mz[n][e & 1]);
            l[n][e & 1] = fmaf(pr, ex2(fminf(apart[n][e & 1] - meta.lv, kFar)), l[n][e & 1]);
            y[e] = pr * meta.pv;
          }
          const uint32_t h0 = f16x2(y[0], y[1]), h1 = f16x2(y[2], y[3]);
          B[0][n][0] = movmatrix_trans(h0);
          B[0][n][1] = movmatrix_trans(h1);
          if constexpr (kTerms == 2) {
            const float2 z0 = half2_floats(h0), z1 = half2_floats(h1);
            B[kTerms - 1][n][0] = movmatrix_trans(f16x2(y[0] - z0.x, y[1] - z0.y));
            B[kTerms - 1][n][1] = movmatrix_trans(f16x2(y[2] - z1.x, y[3] - z1.y));
          }
        }
        // ---- O^T += V^T P^T
        // rows past the cached tokens hold anything: they are taken as zeros
        const int32_t left = s.kv_len - j0;
        uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
        if (left < 16) {
          mlo = (2 * c < left ? 0x0000ffffu : 0u) | (2 * c + 1 < left ? 0xffff0000u : 0u);
          mhi = (2 * c + 8 < left ? 0x0000ffffu : 0u) | (2 * c + 9 < left ? 0xffff0000u : 0u);
        }
        const int vrow = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), vch = lane >> 4;
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t r4[4];
          ldmatrix_x4_trans(r4, sv + tile_offset<D>(vrow, k + vch));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = __byte_perm(r4[2 * h] & mlo, 0, 0x3120);
            const uint32_t z = __byte_perm(r4[2 * h + 1] & mhi, 0, 0x3120);
            const uint32_t A[4] = {lo_half2(x), hi_half2(x), lo_half2(z), hi_half2(z)};
#pragma unroll
            for (int xx = 0; xx < kTerms; ++xx)
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16_16816(O[k + h][n], A, B[xx][n]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
    }

    // ---- merge the four warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[n][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (n8 == 0) {
          sm.mz[warp][8 * n + 2 * c + e] = mz[n][e];
          sm.ms[warp][8 * n + 2 * c + e] = mz[n][e] - apart[n][e];
          sm.l[warp][8 * n + 2 * c + e] = x;
        }
      }
    named_sync(1, 32 * kWarps);
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = sm.mz[0][8 * n + 2 * c + e];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) M = fmaxf(M, sm.mz[x][8 * n + 2 * c + e]);
        f[n][e] = ex2(mz[n][e] - M);
      }
    for (int x = 0; x < kWarps; ++x) {  // in a fixed order
      if (warp == x) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2* at = reinterpret_cast<float2*>(red + (8 * n + 2 * c + e) * kRed + 16 * k +
                                                     2 * n8);
              float2 y = make_float2(O[k][n][e] * f[n][e], O[k][n][e + 2] * f[n][e]);
              if (x > 0) {
                const float2 z = *at;
                y.x += z.x;
                y.y += z.y;
              }
              *at = y;
            }
      }
      named_sync(1, 32 * kWarps);
    }
    // ---- write the output, or the piece
    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
    float* part = p.part + ((int64_t)2 * blockIdx.x + (g.t0 > 0 ? 0 : 1)) * (RB * (D + 4));
    for (int r = warp; r < RB; r += kWarps) {
      const int32_t row = r0 + r;
      if (row >= rows) break;
      float MZ = sm.mz[0][r], MS = sm.ms[0][r];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) {
        MZ = fmaxf(MZ, sm.mz[x][r]);
        MS = fmaxf(MS, sm.ms[x][r]);
      }
      float L = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) L += sm.l[x][r] * ex2(sm.ms[x][r] - MS);
      const float inv = !whole ? 1.f : L == 0.f ? 0.f : ex2(MZ - MS - kOutShift) / L;
      const int64_t tok = s.row0 + a.by_group(row);
      const int head = g.head * a.group + (row - a.by_group(row) * a.group);
      for (int quad = lane; quad < D / 4; quad += 32) {
        const float4 v = *reinterpret_cast<const float4*>(red + r * kRed + 4 * quad);
        const float y[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        if (whole) store4(static_cast<T*>(a.o) + tok * a.o_stride + (int64_t)head * D + 4 * quad, y);
        else store4(part + r * D + 4 * quad, y);
      }
      if (lane == 0) {
        if (!whole) {
          *reinterpret_cast<float4*>(part + RB * D + 4 * r) = make_float4(MZ, MS, L, 0.f);
        } else if (a.lse) {
          a.lse[tok * (a.hkv * a.group) + head] = L == 0.f ? -GDN_INF : (MS + log2f(L)) * kLn2;
        }
      }
    }
    named_sync(1, 32 * kWarps);  // the next unit writes the shared arrays again
  }
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxWorkers = kCtasPerSm * kMaxSms;
constexpr int kMaxJoinBlocks = 16384, kBlockRows = 512;

// Joins the pieces of the units that were cut. Where there are few rows (at most kBlockRows; one
// long context: 152 pieces of 8 rows) a block joins 64 columns of a row, else a warp a row.
// Which units were cut, and where, follows from the lengths alone, so every block works it out
// while the first kernel still runs. Measured: 128 requests of 128 to 16,384 tokens 175 us with
// blocks and 167 us with warps; one of 32,768 tokens 20 us with blocks, 50 us with warps.
template <typename T, int D, int RB, bool kBlocks>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(AttnArgs a, const float* part, int workers) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the tile kernel may come
  extern __shared__ int32_t join_smem[];
  __shared__ int32_t scan[kJoinWarps][2];
  constexpr int kTeams = kBlocks ? 1 : kJoinWarps;  // rows that a block has in hand at a time
  constexpr int kTeam = kJoinThreads / kTeams;       // threads of one
  __shared__ float weight[kTeams][kMaxWorkers];
  __shared__ float red[kJoinWarps];
  __shared__ float4 sum[kBlocks ? kJoinThreads : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_seqs;
  int32_t* pre = join_smem;       // [n + 1] items before a request
  int32_t* unit0 = pre + n + 1;   // [n + 1] units before it
  {
    const int per = (n + kJoinThreads - 1) / kJoinThreads, b0 = tid * per, b1 = min(n, b0 + per);
    bool bad = false;
    auto units_of = [&](const AttnSeq& s) {
      return s.q_len == 0 || s.q_len > a.split_q ? 0 : a.hkv * ((s.q_len * a.group + RB - 1) / RB);
    };
    int32_t items = 0, units = 0;
    for (int b = b0; b < b1; ++b) {
      const AttnSeq s = attn_seq(a, b, bad);
      items = add_items(items, seq_items<RB>(a, s));
      units = add_items(units, units_of(s));
    }
    int32_t x = items, y = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x = add_items(x, u);
        y = add_items(y, v);
      }
    }
    if (lane == 31) {
      scan[warp][0] = x;
      scan[warp][1] = y;
    }
    __syncthreads();
    x -= items;
    y -= units;
    for (int w = 0; w < warp; ++w) {
      x = add_items(x, scan[w][0]);
      y = add_items(y, scan[w][1]);
    }
    for (int b = b0; b < b1; ++b) {
      pre[b] = x;
      unit0[b] = y;
      const AttnSeq s = attn_seq(a, b, bad);
      x = add_items(x, seq_items<RB>(a, s));
      y = add_items(y, units_of(s));
    }
    if (b1 == n && b0 < b1) {
      pre[n] = x;
      unit0[n] = y;
    }
    __syncthreads();
  }
  const int64_t W = pre[n], G = min((int64_t)workers, W);
  const int64_t jobs = W == kTooMany ? 0 : (int64_t)unit0[n] * RB;
  const int me = tid % kTeam;             // this thread in its row's team
  float* const w = weight[tid / kTeam];
  auto worker_of = [&](int64_t item) {
    int64_t k = item * G / W;
    while (W * (k + 1) / G <= item) ++k;
    while (W * k / G > item) --k;
    return (int)k;
  };
  auto reduce = [&](float x, bool take_max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = take_max ? fmaxf(x, y) : x + y;
    }
    if constexpr (kBlocks) {
      __syncthreads();
      if (lane == 0) red[warp] = x;
      __syncthreads();
      x = red[0];
#pragma unroll
      for (int v = 1; v < kJoinWarps; ++v) x = take_max ? fmaxf(x, red[v]) : x + red[v];
    }
    return x;
  };
  bool waited = false;
  for (int64_t job = (int64_t)blockIdx.x * kTeams + tid / kTeam; job < jobs;
       job += (int64_t)gridDim.x * kTeams) {
    const int32_t u = (int32_t)(job / RB), r = (int32_t)(job % RB);
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {  // the last request whose units begin at or before u
      const int32_t mid = (lo + hi + 1) >> 1;
      if (unit0[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    bool bad = false;
    const AttnSeq s = attn_seq(a, lo, bad);
    const int32_t row_tiles = (s.q_len * a.group + RB - 1) / RB, k = u - unit0[lo];
    const int32_t row = k % row_tiles * RB + r;
    if (row >= s.q_len * a.group) continue;  // the whole team, here and below
    const int64_t tiles = max(1, (s.kv_len + kTile - 1) / kTile), item = pre[lo] + k * tiles;
    const int w0 = worker_of(item), count = worker_of(item + tiles - 1) - w0 + 1;
    if (count == 1) continue;  // written by its worker
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are written
    waited = true;
    // piece i: the second slot of the first worker, then the first slots of the next ones
    auto piece = [&](int i) {
      return part + ((int64_t)2 * (w0 + i) + (i == 0 ? 1 : 0)) * (RB * (D + 4));
    };
    constexpr int kStats = (kMaxWorkers + kTeam - 1) / kTeam;
    float4 st[kStats];
    float MZ = kNoMax, MS = kNoMax, L = 0.f;
#pragma unroll
    for (int x = 0; x < kStats; ++x) {
      const int i = me + x * kTeam;
      st[x] = make_float4(kNoMax, kNoMax, 0.f, 0.f);
      if (i < count) st[x] = *reinterpret_cast<const float4*>(piece(i) + RB * D + 4 * r);
      MZ = fmaxf(MZ, st[x].x);
      MS = fmaxf(MS, st[x].y);
    }
    MZ = reduce(MZ, true);
    MS = reduce(MS, true);
#pragma unroll
    for (int x = 0; x < kStats; ++x) {
      const int i = me + x * kTeam;
      if (i < count) w[i] = ex2(st[x].x - MZ);
      L += st[x].z * ex2(st[x].y - MS);
    }
    __syncwarp();
    L = reduce(L, false);
    const float inv = L == 0.f ? 0.f : ex2(MZ - MS - kOutShift) / L;
    const int32_t query = a.by_group(row);
    const int64_t tok = s.row0 + query;
    const int head = k / row_tiles * a.group + row - query * a.group;
    T* out = static_cast<T*>(a.o) + tok * a.o_stride + (int64_t)head * D;
    auto add = [&](float4& y, int i, int at) {
      const float4 v = *reinterpret_cast<const float4*>(piece(i) + r * D + at);
      const float f = w[i];
      y.x += v.x * f; y.y += v.y * f; y.z += v.z * f; y.w += v.w * f;
    };
    auto put = [&](const float4& y, int at) {
      const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
      store4(out + at, z);
    };
    if constexpr (kBlocks) {  // 16 threads for 64 columns, 16 sets of pieces
      const int at = 64 * blockIdx.y + 4 * (tid & 15), set = tid >> 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int i = set; i < count; i += kJoinThreads / 16) add(y, i, at);
      sum[tid] = y;
      __syncthreads();
      if (set == 0) {
#pragma unroll
        for (int x = 1; x < kJoinThreads / 16; ++x) {
          const float4 v = sum[16 * x + tid];
          y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
        }
        put(y, at);
      }
      __syncthreads();  // weights and sums are written again
    } else {
      for (int at = 4 * lane; at < D; at += 128) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i < count; ++i) add(y, i, at);
        put(y, at);
      }
      __syncwarp();
    }
    if (me == 0 && blockIdx.y == 0 && a.lse)
      a.lse[tok * (a.hkv * a.group) + head] = L == 0.f ? -GDN_INF : (MS + log2f(L)) * kLn2;
  }
  // what follows in the stream waits for this kernel: let it stand for the first one too
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Row tiles of 8 in a unit. Two fit the registers up to D = 128 (12 bytes of spills in bf16); at
// D = 256 the accumulator alone takes 128 of the 168, and 360 bytes spill. Four do not fit at 128:
// 32 requests of 32 rows behind 2,000 tokens (8 key/value heads) took 142 us with four and 93 with
// two passes of two.
constexpr int kMaxRowTiles = 2;

template <typename T, int D, int NT>
int launch(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, cudaStream_t stream) {
  constexpr int RB = 8 * NT;
  constexpr int kTerms = std::is_same<T, float>::value ? 2 : 1;
  SplitParams p;
  p.a = a;
  const int box = std::min(c.page_size, kTile);
  if (!make_cache_map(&p.tk, c.k, c, box) || !make_cache_map(&p.tv, c.v, c, box))
    return (int)cudaErrorInvalidValue;
  // one block per SM slot, no more than there can be items
  const int64_t units = ((int64_t)a.num_tokens * a.group + RB - 1) / RB + a.num_seqs;
  const int64_t items = units * a.hkv *
                        std::max<int64_t>(1, ((int64_t)a.max_kv_len + kTile - 1) / kTile);
  const int workers = (int)std::min<int64_t>((int64_t)kCtasPerSm * num_sms, items);
  p.part = a.partials;
  const size_t q = (size_t)kTerms * NT * D * 16, red = sizeof(float) * RB * (D + 8);
  const size_t fixed = q + red + align_up(sizeof(int32_t) * (a.num_seqs + 1), 16) + 1024 +
                       sizeof(SmemHead<NT>);
  const size_t stage = 2 * (size_t)kTile * D;
  p.stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(2, (kSmemPerCta - fixed) / stage));
  p.off_q = (uint32_t)(p.stages * stage);
  p.off_red = p.off_q + (uint32_t)q;
  p.off_pre = p.off_red + (uint32_t)red;
  const size_t smem = p.off_pre + sizeof(int32_t) * (a.num_seqs + 1) + 1024;
  static std::atomic<int> ready[kMaxDevices];
  int e = configure_once(ready, [] {
    return (int)cudaFuncSetAttribute(split_kernel<T, D, NT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
  });
  if (e != 0) return e;
  split_kernel<T, D, NT><<<workers, kThreads, smem, stream>>>(p);
  if ((e = (int)cudaGetLastError()) != 0 || workers == 1) return e;
  cudaLaunchConfig_t cfg = {};
  // a unit's rows are at most those of the longest request that this kernel takes
  const int64_t longest = ((int64_t)std::min(a.max_q_len, a.split_q) * a.group + RB - 1) / RB;
  const int64_t jobs = std::min(units, a.num_seqs * longest) * a.hkv * RB;
  const bool blocks = jobs <= kBlockRows;
  cfg.gridDim = blocks ? dim3((unsigned)jobs, D / 64)
                       : dim3((unsigned)std::min<int64_t>((jobs + kJoinWarps - 1) / kJoinWarps,
                                                          kMaxJoinBlocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = sizeof(int32_t) * 2 * (a.num_seqs + 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // its launch overlaps the first kernel's end
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)(blocks ? cudaLaunchKernelEx(&cfg, join_kernel<T, D, RB, true>, a,
                                           (const float*)p.part, workers)
                      : cudaLaunchKernelEx(&cfg, join_kernel<T, D, RB, false>, a,
                                           (const float*)p.part, workers));
}

}  // namespace

size_t split_workspace(const gdn_attn_config& cfg, const gdn_kv_cache& c) {
  const size_t workers = (size_t)kCtasPerSm * kMaxSms;
  return 2 * workers * 8 * kMaxRowTiles * (c.head_dim + 4) * sizeof(float);
}

int launch_attn_split(const AttnArgs& a, const gdn_kv_cache& c, bool bf16, int num_sms,
                      void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)std::min(a.max_q_len, a.split_q) * a.group;
  auto tiles = [&](auto type, auto dim) {
    using T = decltype(type);
    constexpr int D = decltype(dim)::value;
    if (rows <= 8) return launch<T, D, 1>(a, c, num_sms, s);
    return launch<T, D, kMaxRowTiles>(a, c, num_sms, s);
  };
  auto dims = [&](auto type) {
    if (c.head_dim == 64) return tiles(type, std::integral_constant<int, 64>());
    if (c.head_dim == 128) return tiles(type, std::integral_constant<int, 128>());
    return tiles(type, std::integral_constant<int, 256>());
  };
  return bf16 ? dims(__nv_bfloat16()) : dims(float());
}

}  // namespace gdn
