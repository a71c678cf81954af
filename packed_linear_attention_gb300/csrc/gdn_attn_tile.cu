// gdn_attn_tile.cu — attention of prompts (many queries) over the paged e4m3 cache, on the
// tcgen05 tensor cores.
//
// A unit is (request, key/value head, 128 query rows), the rows of a head group's queries one
// after another (row = query * group + head), so that a key/value tile serves every query head
// of its group. Per tile of BN cached tokens (64 for heads of 256, else 128):
//   S (128 x BN)  = Q K^T                        running maximum m and sum l per row
//   O (128 x D)  += P V,  P = 2^(S - m)
//
// Operands. K enters as it lies in the cache: e4m3 tiles come by TMA into the swizzled layout
// that kind::f8f6f4 reads, and Q is split into two e4m3 terms, q 2^k = hi + lo (hi to four
// significant bits, lo the rest; the row's power of two brings its largest value to [128,
// 256)): a bf16 value has eight bits, so the two terms are exact down to 2^-10 of the row's
// largest value and off by at most 2^-18 of it below. Two e4m3 products cost what one f16
// product costs, and no K tile is converted. Such a split of P would lose the small
// probabilities of a long context, so P is f16 (from registers to TMEM, as the A operand) and
// V is widened to f16 in shared memory (exact).
// The maximum is raised only when a score passes it by 2^8 (see gdn_attn_split.cu); value
// scales enter P as ratios to the largest that the unit has met.
//
// Block: 18 warps. 0-7 softmax (a row is shared by two threads, one for each half of the tile's
// columns) and epilogue; 8-15 Q and V operands; 16 the TMA producer and unit scheduler; 17 the
// MMA issuer. S is double buffered: S(i + 1) runs under the softmax of tile i, P V(i) under
// that of tile i + 1. Units come from a counter, heaviest rows of a request first.
// Every wait is bounded; after one gave up the block's warps leave at their unit's end.
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

constexpr int kRows = kTileRows;          // query rows of a unit (the MMA's M)
constexpr int kSoftWarps = 8, kAuxWarps = 8;
constexpr int kProducer = kSoftWarps + kAuxWarps, kIssuer = kProducer + 1;
constexpr int kWarps = kIssuer + 1, kThreads = 32 * kWarps;
constexpr int kSoftThreads = 32 * kSoftWarps, kAuxThreads = 32 * kAuxWarps;
constexpr int kMeta = 8;                  // ring of tile scales
constexpr int kCoarse = kMaxSeqs / 32;    // prefix sums are kept for every 32 requests
constexpr uint32_t kWaitLimit = 1u << 24;
constexpr float kLazyMax = 8.f;
constexpr float kProbScale = 128.f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSoftBar = 2;               // named barrier of the softmax warps

#define GDN_INF __int_as_float(0x7f800000)

// Byte offset of 16-byte chunk `chunk` of row `row` in an e4m3 operand tile of `rows` rows.
template <int D>
__device__ __forceinline__ uint32_t f8_offset(int row, int chunk, int rows) {
  if constexpr (D == 64) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
  else return (chunk >> 3) * (rows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
template <int D>
__device__ __forceinline__ uint64_t f8_desc(uint32_t addr) {
  return D == 64 ? smem_desc_sw64(addr, 16, 512) : smem_desc_sw128(addr, 16, 1024);
}

struct Unit {
  int32_t seq, row0, q_len, kv_len;  // the request (seq < 0: no more units)
  int32_t head, first;               // key/value head; first row of the unit
  int32_t tiles, pad;
};

template <int G>
struct TileMeta {
  float ks[G];    // key scale of each 16-token group; negative: its page is absent
  float vr[G];    // value scale / vref * kProbScale
  float vref;     // largest value scale of the unit so far
  float vfac;     // what the accumulator is multiplied by as vref grew
};

template <int G>
struct Smem {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t sfull[2], pfull[2], odone[2], hfull[2];
  uint64_t qfull, qempty, ofree, drain;
  uint64_t mfull[kMeta];
  uint64_t ufull[2], uempty[2];
  Unit unit[2];
  TileMeta<G> meta[kMeta];
  float exchange[2][kRows];
  int8_t row_exp[2][kRows];  // power of two of a row of Q (two units' worth)
  int32_t coarse[kCoarse + 1];
  uint32_t tmem;
  int32_t dead;
};

template <int D>
struct Shape {
  static constexpr int BN = D == 256 ? 64 : 128;
  static constexpr int kGroups = BN / 16;
  static constexpr int SK = 4;                                  // K stages
  static constexpr int SV = D == 256 ? 2 : D == 128 ? 3 : 4;    // V stages (e4m3)
  static constexpr uint32_t kTileBytes = BN * D;                // one e4m3 tile
  static constexpr uint32_t kQBytes = kRows * D;                // one term of Q
  static constexpr uint32_t kHBytes = 2 * BN * D;               // a V tile in f16
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * kQBytes;
  static constexpr uint32_t OFF_V = OFF_K + SK * kTileBytes;
  static constexpr uint32_t OFF_H = OFF_V + SV * kTileBytes;
  static constexpr uint32_t OFF_SM = OFF_H + 2 * kHBytes;
  static constexpr uint32_t kSmem = OFF_SM + sizeof(Smem<kGroups>);
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
  static constexpr uint32_t kRowPitch = D == 64 ? 64 : 128;     // bytes of a row in a region
  // TMEM columns: S twice, P twice (f16, two to a column), O
  static constexpr uint32_t TM_S = 0, TM_P = 2 * BN, TM_O = D == 256 ? 256 : 384;
};

struct TileParams {
  AttnArgs a;
  CUtensorMap tk, tv;
  int32_t* counter;   // units taken
};

// A whole warp waits for a phase; one answer for the warp. After any wait of the block gave up,
// none waits again.
template <class S>
__device__ __forceinline__ bool wait_or_die(uint64_t* bar, uint32_t parity, S& sm,
                                            int32_t* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    volatile int32_t* dead = &sm.dead;
    WaitClock clk;
    for (uint32_t i = 0; !ok; ++i) {
      if ((i & 15u) == 0u && *dead) break;
      if (i >= kWaitLimit || clk.expired(i)) {
        *dead = 1;
        raise_status(status, GDN_ERR_DEVICE_TIMEOUT);
        break;
      }
      ok = mbar_try_wait(bar, parity);
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ int32_t seq_units(const AttnArgs& a, const AttnSeq& s) {
  if (s.q_len <= a.split_q) return 0;
  return a.hkv * ((s.q_len * a.group + kRows - 1) / kRows);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t e4m3_to_half2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ uint16_t half2_to_e4m3(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tile_kernel(const __grid_constant__ TileParams p) {
  using Sh = Shape<D>;
  constexpr int BN = Sh::BN;
  extern __shared__ __align__(1024) uint8_t smem[];  // no static shared memory in front of it
  Smem<Sh::kGroups>& sm = *reinterpret_cast<Smem<Sh::kGroups>*>(smem + Sh::OFF_SM);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzles need it; the declaration asks for it
    raise_status(a.status, GDN_ERR_CUDA);
    return;
  }

  // ---- set-up: barriers, tensor memory, units before every 32nd request
  if (tid == 0) {
    sm.dead = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.kfull[i], 1);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.vfull[i], 1);
      mbar_init(&sm.vempty[i], kAuxWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pfull[i], kSoftWarps);
      mbar_init(&sm.odone[i], 1);
      mbar_init(&sm.hfull[i], kAuxWarps);
      mbar_init(&sm.ufull[i], 1);
      mbar_init(&sm.uempty[i], kSoftWarps + kAuxWarps + 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&sm.mfull[i], 1);
    mbar_init(&sm.qfull, kAuxWarps);
    mbar_init(&sm.qempty, 1);
    mbar_init(&sm.ofree, kSoftWarps);
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
  }
  const int chunks = (a.num_seqs + 31) / 32;
  bool bad = false;
  for (int c = warp; c < chunks; c += kWarps) {
    const int b = 32 * c + lane;
    int32_t n = b < a.num_seqs ? seq_units(a, attn_seq(a, b, bad)) : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sm.coarse[c + 1] = n;
  }
  if (bad && blockIdx.x == 0) raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
  if (warp == kIssuer) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    int32_t at = 0;
    sm.coarse[0] = 0;
    for (int c = 1; c <= chunks; ++c) sm.coarse[c] = at += sm.coarse[c];
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem;
  const int32_t total = sm.coarse[chunks];

  // Takes the next unit of the block's list (every role but the producer).
  uint32_t nu = 0;
  auto next_unit = [&](Unit& u) {
    const int slot = nu & 1;
    if (!wait_or_die(&sm.ufull[slot], (nu >> 1) & 1u, sm, a.status)) return false;
    u = sm.unit[slot];
    ++nu;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.uempty[slot]);
    return u.seq >= 0;
  };

  if (warp == kProducer) {
    // ---- units, pages and scales, TMA copies
    const int box_rows = min(a.page_size, BN), per_box = box_rows / 16;
    const uint32_t box_bytes = (uint32_t)box_rows * D;
    constexpr int kBatchTiles = 32 / Sh::kGroups;
    uint32_t it = 0;
    for (uint32_t n = 0;; ++n) {
      int32_t x = 0;
      if (lane == 0) x = atomicAdd(p.counter, 1);
      x = __shfl_sync(0xffffffffu, x, 0);
      Unit u = {-1, 0, 0, 0, 0, 0, 0, 0};
      if (x < total) {
        int lo = 0, hi = chunks - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (sm.coarse[mid] <= x) lo = mid;
          else hi = mid - 1;
        }
        const int b = 32 * lo + lane;
        bool cut = false;
        AttnSeq s = {0, 0, 0};
        int32_t mine = 0;
        if (b < a.num_seqs) {
          s = attn_seq(a, b, cut);
          mine = seq_units(a, s);
        }
        int32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const int32_t y = x - sm.coarse[lo];
        const int src = __ffs(__ballot_sync(0xffffffffu, inc > y)) - 1;
        u.seq = 32 * lo + src;
        u.row0 = __shfl_sync(0xffffffffu, s.row0, src);
        u.q_len = __shfl_sync(0xffffffffu, s.q_len, src);
        u.kv_len = __shfl_sync(0xffffffffu, s.kv_len, src);
        const int32_t k = y - __shfl_sync(0xffffffffu, inc - mine, src);
        const int32_t row_tiles = (u.q_len * a.group + kRows - 1) / kRows;
        u.head = k / row_tiles;
        u.first = (row_tiles - 1 - k % row_tiles) * kRows;  // the rows that see most come first
        const int32_t last = min(u.q_len * a.group, u.first + kRows) - 1;
        const AttnSeq q = {u.row0, u.q_len, u.kv_len};
        u.tiles = (attn_limit(a, q, last / a.group) + BN - 1) / BN;
        // the queries on their way to L2, before their turn
        const int32_t t0 = u.first / a.group, t1 = last / a.group;
        for (int32_t t = t0 + lane; t <= t1; t += 32)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           static_cast<const __nv_bfloat16*>(a.q) +
                           (int64_t)(u.row0 + t) * a.q_stride + (int64_t)u.head * a.group * D),
                       "r"(a.group * D * 2)
                       : "memory");
      }
      const int slot = n & 1;
      if (!wait_or_die(&sm.uempty[slot], ((n >> 1) & 1u) ^ 1u, sm, a.status)) break;
      if (lane == 0) {
        sm.unit[slot] = u;
        mbar_arrive(&sm.ufull[slot]);
      }
      if (u.seq < 0) break;
      const int32_t* table = a.block_table + (int64_t)u.seq * a.max_blocks;
      float vref = 0.f;
      for (int32_t tb = 0; tb < u.tiles; tb += kBatchTiles) {
        const int32_t tok = tb * BN + lane * 16;
        int32_t id = -1;
        float ks = -1.f, vs = 0.f;
        if (tok < u.kv_len && tok < u.tiles * BN) {
          id = table[tok / a.page_size];
          if (id >= 0 && id < a.num_pages) {
            ks = a.k_scale[(int64_t)id * a.hkv + u.head];
            vs = a.v_scale[(int64_t)id * a.hkv + u.head];
            if (!(ks >= 0.f)) ks = 0.f;
            if (!(vs >= 0.f)) vs = 0.f;
          } else {
            id = -1;
            raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
          }
        }
        for (int j = 0; j < kBatchTiles && tb + j < u.tiles; ++j, ++it) {
          const int first = j * Sh::kGroups;
          const bool mine = lane >= first && lane < first + Sh::kGroups;
          const bool box = mine && (lane - first) % per_box == 0 && id >= 0;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
          const float top = __uint_as_float(
              __reduce_max_sync(0xffffffffu, mine ? __float_as_uint(vs) : 0u));
          const float fac = top > vref ? vref / top : 1.f;
          vref = fmaxf(vref, top);
          const int ms = it % kMeta, kst = it % Sh::SK, vst = it % Sh::SV;
          if (!wait_or_die(&sm.kempty[kst], ((it / Sh::SK) & 1u) ^ 1u, sm, a.status)) break;
          if (mine) {
            sm.meta[ms].ks[lane - first] = ks;
            sm.meta[ms].vr[lane - first] = vref > 0.f ? vs / vref * kProbScale : 0.f;
          }
          if (lane == 0) {
            sm.meta[ms].vref = vref;
            sm.meta[ms].vfac = fac;
          }
          const int32_t y = (int32_t)(((int64_t)id * a.hkv + u.head) * a.page_size +
                                      tok % a.page_size);
          const uint32_t at = (uint32_t)(lane - first) * 16 * Sh::kRowPitch;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.mfull[ms]);
            mbar_arrive_expect_tx(&sm.kfull[kst], boxes * box_bytes);
          }
          __syncwarp();
          if (box)
#pragma unroll
            for (int r = 0; r < (D + 127) / 128; ++r)
              tma_load_2d(smem + Sh::OFF_K + kst * Sh::kTileBytes + r * (BN * 128) + at, &p.tk,
                          128 * r, y, &sm.kfull[kst]);
          const bool go = wait_or_die(&sm.vempty[vst], ((it / Sh::SV) & 1u) ^ 1u, sm, a.status);
          if (lane == 0) mbar_arrive_expect_tx(&sm.vfull[vst], go ? boxes * box_bytes : 0u);
          __syncwarp();
          if (box && go)
#pragma unroll
            for (int r = 0; r < (D + 127) / 128; ++r)
              tma_load_2d(smem + Sh::OFF_V + vst * Sh::kTileBytes + r * (BN * 128) + at, &p.tv,
                          128 * r, y, &sm.vfull[vst]);
        }
      }
    }
    if (sm.dead) {  // copies may be in flight: let them land
      for (uint32_t k = 0; k < Sh::SK && k < it; ++k)
        mbar_wait_bounded(&sm.kfull[(it - 1 - k) % Sh::SK], ((it - 1 - k) / Sh::SK) & 1u, kWaitLimit);
      for (uint32_t k = 0; k < Sh::SV && k < it; ++k)
        mbar_wait_bounded(&sm.vfull[(it - 1 - k) % Sh::SV], ((it - 1 - k) / Sh::SV) & 1u, kWaitLimit);
    }
  } else if (warp == kIssuer) {
    // ---- MMA issue
    constexpr uint32_t id_s = idesc_f16(kRows, BN, 0, 0), id_o = idesc_f16(kRows, D, 0, 1);
    const uint64_t q_desc = f8_desc<D>(smem_u32(smem) + Sh::OFF_Q);
    const uint64_t h_desc = smem_desc_sw128(smem_u32(smem) + Sh::OFF_H, BN * 128, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tbase, 0), el = elect_lane();
    uint32_t g = 0, units = 0, nq = 0;
    Unit u;
    while (next_unit(u)) {
      if (u.tiles == 0) continue;
      bool ok = wait_or_die(&sm.qfull, nq & 1u, sm, a.status);
      ++nq;
      auto issue_s = [&](uint32_t j, bool last) {  // j: tile number since the start
        const int st = j % Sh::SK;
        ok = ok && wait_or_die(&sm.kfull[st], (j / Sh::SK) & 1u, sm, a.status);
        tc_fence_after();
        if (ok) {
          const uint64_t kd = q_desc + (Sh::OFF_K + st * Sh::kTileBytes) / 16;
          const uint32_t d = tm + Sh::TM_S + (j & 1u) * BN;
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              warp_mma_f8_ss(
                  el, d, q_desc + (term * Sh::kQBytes + (k >> 2) * (kRows * 128) + (k & 3) * 32) / 16,
                  kd + ((k >> 2) * (BN * 128) + (k & 3) * 32) / 16, id_s, term + k > 0);
          if (el) {
            mma_commit(&sm.kempty[st]);
            mma_commit(&sm.sfull[j & 1u]);
            if (last) mma_commit(&sm.qempty);
          }
        }
        __syncwarp();
      };
      const int32_t tiles = __shfl_sync(0xffffffffu, u.tiles, 0);
      issue_s(g, tiles == 1);
      if (tiles > 1) issue_s(g + 1, tiles == 2);
      for (int32_t i = 0; i < tiles && ok; ++i, ++g) {
        const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
        ok = wait_or_die(&sm.hfull[b], ph, sm, a.status) &&
             wait_or_die(&sm.pfull[b], ph, sm, a.status) &&
             (i > 0 || wait_or_die(&sm.ofree, (units & 1u) ^ 1u, sm, a.status));
        tc_fence_after();
        if (ok) {
          const uint64_t hd = h_desc + b * (Sh::kHBytes / 16);
          const uint32_t pa = tm + Sh::TM_P + b * (BN / 2);
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            warp_mma_f16_ts(el, tm + Sh::TM_O, pa + 8 * k, hd + k * (2048 / 16), id_o,
                            i > 0 || k > 0);
          if (el) mma_commit(&sm.odone[b]);
        }
        __syncwarp();
        if (i + 2 < tiles) issue_s(g + 2, i + 3 == tiles);
      }
      ++units;
      if (!ok) break;
    }
    // what was issued has completed before the block's memory goes
    if (el) mma_commit(&sm.drain);
    mbar_wait_bounded(&sm.drain, 0, kWaitLimit);
  } else if (warp >= kSoftWarps) {
    // ---- operands: Q of the unit, then its V tiles
    const int aw = warp - kSoftWarps, at = tid - kSoftThreads;
    uint32_t g = 0, nq = 0;
    Unit u;
    while (next_unit(u)) {
      if (u.tiles == 0) continue;
      const int32_t rows = u.q_len * a.group;
      constexpr int kPer = D / 32;  // elements of a lane
      bool ok = wait_or_die(&sm.qempty, (nq & 1u) ^ 1u, sm, a.status);
      const float sign = a.scale_log2 < 0.f ? -1.f : 1.f;
      constexpr int kBatch = 8;
      for (int rb = 0; rb < kRows / kAuxWarps && ok; rb += kBatch) {
        uint32_t w[kBatch][kPer / 2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int32_t row = u.first + aw * (kRows / kAuxWarps) + rb + k;
          const bool live = row < rows;
          const int32_t i = live ? row / a.group : 0, hd = live ? row - i * a.group : 0;
          const uint32_t* src = reinterpret_cast<const uint32_t*>(
              static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(u.row0 + i) * a.q_stride +
              (int64_t)(u.head * a.group + hd) * D + lane * kPer);
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e) w[k][e] = 0;
          if (live) {
            if constexpr (kPer == 8) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              w[k][0] = v.x; w[k][1] = v.y; w[k][2] = v.z; w[k][3] = v.w;
            } else if constexpr (kPer == 4) {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              w[k][0] = v.x; w[k][1] = v.y;
            } else {
              w[k][0] = *src;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int r = aw * (kRows / kAuxWarps) + rb + k;
          // largest magnitude: bf16 bit patterns without their signs order like integers
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e)
            top = __vmaxu2(top, w[k][e] & 0x7fff7fffu);
          top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
          int ex = (int)(top >> 7) - 127;        // [128, 256) after the scaling
          const bool wild = ex == 128;           // an infinity or NaN: the row is NaN
          ex = wild ? 7 : max(ex, -100);
          const float up = wild ? __int_as_float(0x7fffffff)
                                : sign * __uint_as_float((uint32_t)(7 - ex + 127) << 23);
          uint32_t hi[(kPer + 3) / 4], lo[(kPer + 3) / 4];
#pragma unroll
          for (int e = 0; e < (kPer + 3) / 4; ++e) hi[e] = lo[e] = 0;
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e) {
            const uint32_t h = f16x2(__uint_as_float(w[k][e] << 16) * up,
                                     __uint_as_float(w[k][e] & 0xffff0000u) * up);
            const uint16_t c = half2_to_e4m3(h);
            const uint32_t back = e4m3_to_half2(c);
            const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&h),
                                         *reinterpret_cast<const __half2*>(&back));
            hi[e >> 1] |= (uint32_t)c << (16 * (e & 1));
            lo[e >> 1] |= (uint32_t)half2_to_e4m3(h2_bits(rest)) << (16 * (e & 1));
          }
          const int d0 = lane * kPer;
          uint8_t* dst = smem + Sh::OFF_Q + f8_offset<D>(r, d0 >> 4, kRows) + (d0 & 15);
          if constexpr (kPer == 8) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + Sh::kQBytes) = make_uint2(lo[0], lo[1]);
          } else if constexpr (kPer == 4) {
            *reinterpret_cast<uint32_t*>(dst) = hi[0];
            *reinterpret_cast<uint32_t*>(dst + Sh::kQBytes) = lo[0];
          } else {
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)hi[0];
            *reinterpret_cast<uint16_t*>(dst + Sh::kQBytes) = (uint16_t)lo[0];
          }
          if (lane == 0) sm.row_exp[nq & 1u][r] = (int8_t)(ex - 7);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfull);
      ++nq;
      for (int32_t t = 0; t < u.tiles && ok; ++t, ++g) {
        const int st = g % Sh::SV;
        const uint32_t b = g & 1u;
        ok = wait_or_die(&sm.vfull[st], (g / Sh::SV) & 1u, sm, a.status) &&
             wait_or_die(&sm.odone[b], ((g >> 1) & 1u) ^ 1u, sm, a.status);  // P V(g - 2) is done
        const auto& m = sm.meta[g % kMeta];
        const uint8_t* src = smem + Sh::OFF_V + st * Sh::kTileBytes;
        uint8_t* dst = smem + Sh::OFF_H + b * Sh::kHBytes;
        constexpr int kChunks = BN * D / 16 / kAuxThreads;
        uint4 v[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int x = k * kAuxThreads + at, tok = x % BN, chunk = x / BN;
          v[k] = *reinterpret_cast<const uint4*>(src + f8_offset<D>(tok, chunk, BN));
          // places past the cached tokens, or without a page, hold anything: zeros
          if (t * BN + tok >= u.kv_len || m.ks[tok >> 4] < 0.f) v[k] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int x = k * kAuxThreads + at, tok = x % BN, chunk = x / BN;
          const uint32_t s4[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[2 * e] = e4m3_to_half2((uint16_t)s4[e]);
            h[2 * e + 1] = e4m3_to_half2((uint16_t)(s4[e] >> 16));
          }
          *reinterpret_cast<uint4*>(dst + sw128_offset(tok, 16 * chunk, BN)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + sw128_offset(tok, 16 * chunk + 8, BN)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.hfull[b]);
          mbar_arrive(&sm.vempty[st]);
        }
      }
      if (!ok) break;
    }
  } else {
    // ---- softmax and epilogue
    const int half = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    constexpr int kCols = BN / 2;      // columns of a thread
    uint32_t g = 0, nq = 0;
    Unit u;
    while (true) {
      const bool more = next_unit(u);
      // the warps leave together, so that none is left at their barrier
      if (named_any(kSoftBar, kSoftThreads, !more)) break;
      const int32_t rows = u.q_len * a.group, row = u.first + r;
      const bool live = row < rows;
      const int32_t query = live ? row / a.group : 0;
      const AttnSeq s = {u.row0, u.q_len, u.kv_len};
      const int32_t limit = live ? attn_limit(a, s, query) : u.kv_len;
      const int32_t min_limit = attn_limit(a, s, u.first / a.group);
      float m = -GDN_INF, l = 0.f, vref = 0.f;
      float rs = 0.f;
      for (int32_t i = 0; i < u.tiles; ++i, ++g) {
        const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
        wait_or_die(&sm.mfull[g % kMeta], (g / kMeta) & 1u, sm, a.status);
        wait_or_die(&sm.sfull[b], ph, sm, a.status);
        tc_fence_after();
        if (i == 0)
          rs = fabsf(a.scale_log2) *
               __uint_as_float((uint32_t)(sm.row_exp[nq & 1u][r] + 127) << 23);
        const auto& meta = sm.meta[g % kMeta];
        uint32_t x[kCols];
#pragma unroll
        for (int c = 0; c < kCols; c += 32)
          tmem_ld32(tbase + lane_off + Sh::TM_S + b * BN + half * kCols + c,
                    reinterpret_cast<uint32_t(&)[32]>(x[c]));
        tmem_ld_wait();
        vref = meta.vref;
        const int32_t j0 = i * BN + half * kCols;
        float top = -GDN_INF;
        const bool masked = (i + 1) * BN > min_limit;
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          const float ks = meta.ks[half * (kCols / 16) + q], f = ks * rs;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float2 y = mul2(make_float2(__uint_as_float(x[16 * q + e]),
                                        __uint_as_float(x[16 * q + e + 1])),
                            make_float2(f, f));
            if (masked) {
              if (j0 + 16 * q + e >= limit || ks < 0.f) y.x = -GDN_INF;
              if (j0 + 16 * q + e + 1 >= limit || ks < 0.f) y.y = -GDN_INF;
            } else if (ks < 0.f) {
              y.x = y.y = -GDN_INF;
            }
            top = fmaxf(top, fmaxf(y.x, y.y));
            x[16 * q + e] = __float_as_uint(y.x);
            x[16 * q + e + 1] = __float_as_uint(y.y);
          }
        }
        const float vfac = meta.vfac;
        if (named_any(kSoftBar, kSoftThreads, top > m + kLazyMax || (vfac != 1.f && i > 0))) {
          // a new maximum for the rows, the accumulator and sum follow
          sm.exchange[half][r] = top;
          named_sync(kSoftBar, kSoftThreads);
          const float both = fmaxf(fmaxf(sm.exchange[0][r], sm.exchange[1][r]), m);
          const float f = both == -GDN_INF ? 1.f : ex2(m - both);
          m = both;
          l *= f;
          if (i > 0) {
            wait_or_die(&sm.odone[b ^ 1u], ((g - 1) >> 1) & 1u, sm, a.status);  // P V(g - 1)
            tc_fence_after();
            const float fo = f * vfac;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t o[16];
              const uint32_t ad = tbase + lane_off + Sh::TM_O + half * (D / 2) + c;
              tmem_ld16(ad, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
              tmem_st16(ad, o);
            }
            tmem_st_wait();
          }
        }
        const float mu = m == -GDN_INF ? 0.f : m;
        float2 sum = make_float2(0.f, 0.f);
        uint32_t ph16[kCols / 2];
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          const float vr = meta.vr[half * (kCols / 16) + q];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 z = add2(make_float2(__uint_as_float(x[16 * q + e]),
                                              __uint_as_float(x[16 * q + e + 1])),
                                  make_float2(-mu, -mu));
            const float2 pr = make_float2(ex2(z.x), ex2(z.y));
            sum = add2(sum, pr);
            const float2 pw = mul2(pr, make_float2(vr, vr));
            ph16[8 * q + e / 2] = f16x2(pw.x, pw.y);
          }
        }
        l += sum.x + sum.y;
        if (g >= 2) {  // P V(g - 2) has read this buffer
          wait_or_die(&sm.odone[b], ph ^ 1u, sm, a.status);
        }
        const uint32_t pa = tbase + lane_off + Sh::TM_P + b * (BN / 2) + half * (kCols / 2);
        if constexpr (kCols == 64) tmem_st32(pa, reinterpret_cast<uint32_t(&)[32]>(ph16));
        else tmem_st16(pa, reinterpret_cast<uint32_t(&)[16]>(ph16));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[b]);
      }
      // ---- output
      if (u.tiles > 0) {
        ++nq;
        const uint32_t last = g - 1;
        sm.exchange[half][r] = l;
        named_sync(kSoftBar, kSoftThreads);
        l = sm.exchange[0][r] + sm.exchange[1][r];
        wait_or_die(&sm.odone[last & 1u], (last >> 1) & 1u, sm, a.status);
        tc_fence_after();
      }
      const float inv = l == 0.f ? 0.f : vref / (l * kProbScale);
      const int64_t tok = u.row0 + query;
      const int hq = u.head * a.group + (row - query * a.group);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + tok * a.o_stride +
                           (int64_t)hq * D + half * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t o[32];
        if (u.tiles > 0) {
          tmem_ld32(tbase + lane_off + Sh::TM_O + half * (D / 2) + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 y =
                  __floats2bfloat162_rn(__uint_as_float(o[e + 2 * k]) * inv,
                                        __uint_as_float(o[e + 2 * k + 1]) * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && half == 0 && a.lse)
        a.lse[tok * (a.hkv * a.group) + hq] = l == 0.f ? -GDN_INF : (m + log2f(l)) * kLn2;
      if (u.tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ofree);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
int launch(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, cudaStream_t stream) {
  using Sh = Shape<D>;
  TileParams p;
  p.a = a;
  const int box = std::min(c.page_size, Sh::BN);
  if (!make_cache_map(&p.tk, c.k, c, box) || !make_cache_map(&p.tv, c.v, c, box))
    return (int)cudaErrorInvalidValue;
  p.counter = a.counter;
  static std::atomic<int> ready[kMaxDevices];
  constexpr int kSmem = (int)Sh::kSmem;
  int e = configure_once(ready, [] {
    return (int)cudaFuncSetAttribute(tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmem);
  });
  if (e != 0) return e;
  if ((e = (int)cudaMemsetAsync(p.counter, 0, sizeof(int32_t), stream)) != 0) return e;
  const int64_t units =
      (((int64_t)a.num_tokens * a.group + kRows - 1) / kRows + a.num_seqs) * a.hkv;
  tile_kernel<D><<<(unsigned)std::min<int64_t>(units, num_sms), kThreads, kSmem, stream>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_attn_tile(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.head_dim == 64) return launch<64>(a, c, num_sms, s);
  if (c.head_dim == 128) return launch<128>(a, c, num_sms, s);
  return launch<256>(a, c, num_sms, s);
}

}  // namespace gdn
