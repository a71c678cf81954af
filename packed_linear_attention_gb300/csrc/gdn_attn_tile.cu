// gdn_attn_tile.cu — attention of prompts (many queries) over the paged e4m3 cache, on the
// tcgen05 tensor cores.
//
// A unit is (request, key/value head, 128 query rows), the rows of a head group's queries one
// after another (row = query * group + head), so that a key/value tile serves every query head
// of its group. Per tile of BN = 64 cached tokens:
//   S (128 x BN)  = Q K^T                        running maximum m and sum l per row
//   O (128 x D)  += P V,  P = 2^(S - m)
//
// Operands. K enters as it lies in the cache: e4m3 tiles come by TMA into the swizzled layout
// that kind::f8f6f4 reads. Q stays in tensor memory for the whole unit and is split into two
// e4m3 terms, q 2^k = hi + lo (hi to four significant bits, lo the rest; the row's power of two
// brings its largest value to [128, 256)): a bf16 value has eight bits, so the two terms are
// exact down to 2^-10 of the row's largest value and off by at most 2^-17 of it below. Two e4m3
// products cost what one f16 product costs, and no K tile is converted. Such a split of P would lose the small
// probabilities of a long context, so P is f16 (from registers to TMEM, as the A operand) and
// V is widened to f16 on its way from the cache to shared memory (exact). Shared memory is what
// a tile would be bound by otherwise: with Q and a staged e4m3 V read from it, a tile of 64
// tokens at D = 256 moved 208 KB through 128 bytes a clock against 1,024 clocks of products;
// this way it moves 112 KB.
// The running maxima (of scores and of exponents with the value scales, see kScaleShift in
// gdn_attn_internal.h) are raised only when one is passed by 8 (see gdn_attn_split.cu).
//
// Block: 20 warps. 0-3 and 4-7 softmax, tile by tile in turns, a row to a thread: the latency
// of a tile (tensor memory loads, 64 exponentials, the store of P) is then two tiles long. Only
// the running maxima pass from one group to the other, warp by warp, through shared memory and
// a pair of named barriers. 8-15 operands: V tiles, and the next unit's Q, whose bf16 rows
// a bulk copy brings to shared memory while this unit runs and which moves to tensor memory
// when its last S is done; 16 the producer (pages, scales, K tiles); 17 issues S, 18 P V (the
// twenty products of a tile, issued one after another between the waits of both, took one warp
// longer than the tensor pipe); 19 takes the units and copies their rows of Q, so that they are
// there when the unit before ends.
// S is free again as soon as a group holds it in registers. Units come from a counter, heaviest
// rows of a request first.
// Every wait is bounded; after one gave up the block's warps leave at their unit's end.
//
// Bound and measured (16 query and 2 key/value heads of 256, causal). 4 x 8,192 tokens: 1,470 us
// for 2.20 TFLOP, 80% of the measured bf16 peak. A tile takes 1,530 clocks where its products
// take 1,024: tensor memory holds one S beside O and Q, so S(j + 1) waits until S(j) is read, and
// P V stands in the same queue. 32 x 1,024 tokens: 312 us, 47%; a unit has 8.5 tiles, and its
// start and end (Q to two terms, the output, the next first scores) take as long as six. 32 and 8
// heads of 128, 8 requests of 190 to 1,789 tokens behind up to 1,537: 243 us, 42%; the products take 512
// clocks of a tile, the two softmax groups 1,200. Half of the issue slots and 42% of the ALU are
// taken, so instructions of any role cost time: page arithmetic in the operand warps cost 5% of
// the first case. Tried and dropped: a second S at D <= 128 (no change), tiles of 128 tokens there
// (265 us: scores read twice), V tiles taken in turns by two operand groups with the next unit's Q
// converted between them (1,572, 383 and 283 us in the order of the cases: 7 KB more code).
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
constexpr int kProducer = kSoftWarps + kAuxWarps, kIssuerS = kProducer + 1, kIssuerO = kProducer + 2,
              kScheduler = kProducer + 3;
constexpr int kWarps = 20, kThreads = 32 * kWarps;
// Registers of a thread: 640 threads are launched with 96; the softmax warps take what the
// others give (256 * 120 + 256 * 88 + 128 * 64 = 640 * 96).
constexpr int kSoftRegs = 120, kAuxRegs = 88, kMiscRegs = 64;
static_assert(256 * kSoftRegs + 256 * kAuxRegs + 128 * kMiscRegs == kThreads * 96, "registers");
constexpr int kSoftThreads = 32 * kSoftWarps, kAuxThreads = 32 * kAuxWarps;
// Scales and pages are looked up for a batch of tiles at a time, a 16-token group to a lane. The
// ring holds 16 batches: at least 16 tiles, more than the roles are apart (K stages and four).
constexpr int kBatch = 8, kBatches = 16;
constexpr int kLead = 16;                 // K tiles of a unit left to load when the next is taken
constexpr int kCoarse = kMaxSeqs / 32;    // prefix sums are kept for every 32 requests
constexpr float kProbShift = 7.f;  // P = 2^(z - m + this), at most 2^15 in f16
constexpr float kOutShift = kProbShift + kScaleShift;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSoftBar = 2, kAuxBar = 3;  // named barriers of the softmax and operand warps
constexpr int kPairBar = 4;               // 4-11: a pair of softmax warps, either direction
constexpr int BN = 64;                    // cached tokens of a tile
constexpr int kGroups = BN / 16;

#define GDN_INF __int_as_float(0x7f800000)

template <int D>
__device__ __forceinline__ uint64_t f8_desc(uint32_t addr) {
  return D == 64 ? smem_desc_sw64(addr, 16, 512) : smem_desc_sw128(addr, 16, 1024);
}

struct Unit {
  int32_t seq, row0, q_len, kv_len;  // the request (seq < 0: no more units)
  int32_t head, first;               // key/value head; first row of the unit
  int32_t tiles, pad;
};

struct __align__(16) TileMeta {
  float ks[kGroups];    // key scale of each 16-token group
  float lv[kGroups];    // log2 of its value scale, shifted
  int32_t row[kGroups]; // the group's first row of values in the cache; negative: zeros
  uint32_t absent;      // bit g: group g is absent; bit 4 + g: its values are zeros
  float lvmin;          // least lv of the groups that are there
  uint32_t pad[2];
};

constexpr int kMaxStages = 8;
// P V products are counted on a ring of four barriers: a softmax group that waits for the
// product of tile j - 1 knows that of tile j - 4 done, so no phase can be taken for another.
constexpr int kDone = 4;
struct Smem {
  uint64_t kfull[kMaxStages], kempty[kMaxStages];
  uint64_t pfull[2], sfull[2], odone[kDone], hfull[4];
  uint64_t sfree, qfull, qempty, ofree, drain[2], rawfull, rawempty;
  uint64_t mfull[kBatches];
  uint64_t ufull[2], uempty[2], unext;
  Unit unit[2];
  TileMeta meta[kBatches][kBatch];
  float2 m[kRows];           // running maxima on their way between the softmax groups
  float exchange_l[2][kRows];
  uint16_t exchange_q[2][kRows];
  int8_t row_exp[2][kRows];  // power of two of a row of Q (two units' worth)
  int32_t coarse[kCoarse + 1];
  uint32_t tmem;
  int32_t dead;
};

template <int D>
struct Shape {
  static constexpr int SK = D == 256 ? 4 : 8;                   // K stages
  static constexpr int NH = D == 256 ? 2 : 4;                   // V tiles in f16
  static constexpr uint32_t kTileBytes = BN * D;                // one e4m3 tile
  static constexpr uint32_t kHBytes = 2 * BN * D;
  static constexpr uint32_t kRawPitch = 2 * D + 16;             // a bf16 row of Q: odd in 16 bytes
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_H = OFF_K + SK * kTileBytes;
  static constexpr uint32_t OFF_RAW = OFF_H + NH * kHBytes;
  static constexpr uint32_t OFF_OUT = OFF_RAW + kRows * kRawPitch;  // a warp's rows on their way out
  static constexpr uint32_t OFF_SM = OFF_OUT + kSoftWarps * 2048;
  static constexpr uint32_t kSmem = OFF_SM + sizeof(Smem);
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
  static constexpr uint32_t kRowPitch = D == 64 ? 64 : 128;     // bytes of a row in a region
  // TMEM columns: O, the two terms of Q (four elements a column), S, P twice (f16, two a column)
  static constexpr uint32_t TM_O = 0, TM_Q = D, TM_S = D + D / 2, TM_P = TM_S + BN;
  static_assert(TM_P + BN <= 512, "tensor memory");
};

struct TileParams {
  AttnArgs a;
  CUtensorMap tk;
  const void* v;      // the cache's values
  int32_t* counter;   // units taken
};

// A lane's wait for a phase (wait_or_die: one answer for the warp). At most 2^20 polls, of which one
// that fails takes 0.8 us (measured), so about a second; after any wait of the block gave up,
// none waits again. One short loop in assembly: there are twenty of these, the kernel's roles
// share one instruction cache, and as C++ each took up to 1 KB of it.
__device__ __forceinline__ uint32_t wait_lane(uint64_t* bar, uint32_t parity, Smem& sm,
                                              int32_t* status) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 n, d;\n"
      " mov.u32 n, %5;\n"
      "POLL:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " @p bra DONE;\n"
      " ld.volatile.shared.b32 d, [%3];\n"
      " setp.ne.u32 q, d, 0;\n"
      " @q bra DONE;\n"
      " sub.u32 n, n, 1;\n"
      " setp.ne.u32 q, n, 0;\n"
      " @q bra POLL;\n"
      " st.volatile.shared.b32 [%3], 1;\n"
      " setp.ne.u64 q, %4, 0;\n"
      " @q red.global.max.s32 [%4], %6;\n"
      "DONE:\n"
      " selp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(&sm.dead)), "l"(status), "n"(1 << 20),
        "n"((int)GDN_ERR_DEVICE_TIMEOUT)
      : "memory");
  return ok;
}
__device__ __forceinline__ bool wait_or_die(uint64_t* bar, uint32_t parity, Smem& sm,
                                            int32_t* status) {
  return __all_sync(0xffffffffu, wait_lane(bar, parity, sm, status));
}
// For the softmax warps, which run their unit's course whether or not a wait gave up.
__device__ __forceinline__ void wait_on(uint64_t* bar, uint32_t parity, Smem& sm,
                                        int32_t* status) {
  wait_lane(bar, parity, sm, status);
  __syncwarp();
}

// The same for what must have landed before the block ends, also after a wait gave up.
__device__ __noinline__ void wait_landed(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 20); ++i)
    if (mbar_try_wait(bar, parity)) return;
}

__device__ __forceinline__ int32_t seq_units(const AttnArgs& a, const AttnSeq& s) {
  if (s.q_len <= a.split_q) return 0;
  return a.hkv * ((s.q_len * a.group + kRows - 1) / kRows);
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A warp's part in a two-warp barrier: announce, or wait for the other's announcement.
__device__ __forceinline__ void pair_arrive(int id) {
  asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void pair_wait(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __nv_bfloat162 bf16x2(uint32_t x) {
  return *reinterpret_cast<const __nv_bfloat162*>(&x);
}
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
  extern __shared__ __align__(1024) uint8_t smem[];  // no static shared memory in front of it
  Smem& sm = *reinterpret_cast<Smem*>(smem + Sh::OFF_SM);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzles need it; the declaration asks for it
    raise_status(a.status, GDN_ERR_CUDA);
    return;
  }

  // ---- set-up: barriers, tensor memory, units before every 32nd request
  if (tid == 0) {
    sm.dead = 0;
#pragma unroll 1
    for (int i = 0; i < Sh::SK; ++i) {
      mbar_init(&sm.kfull[i], 1);
      mbar_init(&sm.kempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.pfull[i], kSoftWarps / 2);
      mbar_init(&sm.ufull[i], 1);
      mbar_init(&sm.uempty[i], kSoftWarps + kAuxWarps + 3);
    }
    for (int i = 0; i < kDone; ++i) mbar_init(&sm.odone[i], 1);
    for (int i = 0; i < Sh::NH; ++i) mbar_init(&sm.hfull[i], kAuxWarps);
#pragma unroll 1
    for (int i = 0; i < kBatches; ++i) mbar_init(&sm.mfull[i], 1);
    mbar_init(&sm.sfull[0], 1);  // a barrier for each softmax group: it waits for every second S
    mbar_init(&sm.sfull[1], 1);
    mbar_init(&sm.sfree, kSoftWarps / 2);
    mbar_init(&sm.qfull, kAuxWarps);
    mbar_init(&sm.qempty, 1);
    mbar_init(&sm.ofree, kSoftWarps);
    mbar_init(&sm.rawfull, 1);
    mbar_init(&sm.unext, 1);
    mbar_init(&sm.rawempty, kAuxWarps);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    fence_mbar_init();
  }
  const int chunks = (a.num_seqs + 31) / 32;
  bool bad = false;
#pragma unroll 1
  for (int c = warp; c < chunks; c += kWarps) {
    const int b = 32 * c + lane;
    int32_t n = b < a.num_seqs ? seq_units(a, attn_seq(a, b, bad)) : 0;
    n = __reduce_add_sync(0xffffffffu, n);  // each below kMaxUnits
    if (lane == 0) sm.coarse[c + 1] = n;
  }
  if (bad && blockIdx.x == 0) raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
  if (warp == kIssuerS) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    int32_t at = 0;
    sm.coarse[0] = 0;
#pragma unroll 1
    for (int c = 1; c <= chunks; ++c) sm.coarse[c] = at = add_items(at, sm.coarse[c]);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem;
  const int32_t total = sm.coarse[chunks] == kTooMany ? 0 : sm.coarse[chunks];

  // Takes the next unit of the block's list (every role but the scheduler).
  uint32_t nu = 0;
  auto see_unit = [&] {
    return wait_or_die(&sm.ufull[nu & 1], (nu >> 1) & 1u, sm, a.status) &&
           *(volatile int32_t*)&sm.unit[nu & 1].seq >= 0;
  };
  auto take_unit = [&](Unit& u) {
    u = sm.unit[nu & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.uempty[nu & 1]);
    ++nu;
  };
  auto next_unit = [&](Unit& u) {
    if (!see_unit()) return false;
    take_unit(u);
    return true;
  };

  if (warp >= kProducer) {
    give_registers<kMiscRegs>();
    if (warp == kProducer) {
      // ---- pages and scales, K tiles
      const int box_rows = min(a.page_size, BN), per_box = box_rows / 16;
      const uint32_t box_bytes = (uint32_t)box_rows * D;
      static_assert(kBatch * kGroups == 32, "a group to a lane");
      uint32_t it = 0, nb = 0;
      Unit u;
      while (next_unit(u)) {
        if (u.tiles == 0) {
          if (lane == 0) mbar_arrive(&sm.unext);
          continue;
        }
        const int32_t* table = a.block_table + (int64_t)u.seq * a.max_blocks;
        const int32_t end = min(u.kv_len, u.tiles * BN);
        auto page_of = [&](int32_t tok) { return tok < end ? table[tok >> a.page_shift] : -1; };
        auto scales_of = [&](int32_t tok, int32_t& id, float& ks, float& vs) {
          ks = vs = 0.f;
          if (id >= 0 && id < a.num_pages) {
            ks = a.k_scale[(int64_t)id * a.hkv + u.head];
            vs = a.v_scale[(int64_t)id * a.hkv + u.head];
          } else {
            if (tok < end) raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
            id = -1;
          }
        };
        float ks, vs;
        int32_t id = page_of(16 * lane);
        scales_of(16 * lane, id, ks, vs);
        bool ok = true;
#pragma unroll 1
        for (int32_t tb = 0; tb < u.tiles && ok; tb += kBatch, ++nb) {
          if (lane == 0 && tb + kLead >= u.tiles && (tb == 0 || tb + kLead - kBatch < u.tiles))
            mbar_arrive(&sm.unext);
          const int32_t tok = tb * BN + lane * 16;
          ks = ks >= 0.f ? ks : 0.f;  // values that are no scales count as zeros
          const bool empty = !(vs >= kMinValueScale);
          const uint32_t gone = __ballot_sync(0xffffffffu, id < 0);
          const int32_t y = (int32_t)(((int64_t)id * a.hkv + u.head) * a.page_size +
                                      (tok & (a.page_size - 1)));
          TileMeta& m = sm.meta[nb % kBatches][lane >> 2];
          m.ks[lane & 3] = ks;
          const float lv =
              id < 0 ? 127.f
                     : __log2f(fminf(fmaxf(vs, kMinValueScale), kMaxValueScale)) + kScaleShift;
          float least = fminf(lv, __shfl_xor_sync(0xffffffffu, lv, 1));
          least = fminf(least, __shfl_xor_sync(0xffffffffu, least, 2));
          m.lv[lane & 3] = lv;
          m.row[lane & 3] = id < 0 || empty ? -1 : y;
          const uint32_t zeros = __ballot_sync(0xffffffffu, empty);
          if ((lane & 3) == 0) {
            m.absent = ((gone >> lane) & 15u) | ((zeros >> lane) & 15u) << 4;
            m.lvmin = least;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.mfull[nb % kBatches]);
          const bool box = (lane & (per_box - 1)) == 0 && id >= 0;
          const uint32_t boxes = __ballot_sync(0xffffffffu, box);
          const uint32_t at = (uint32_t)(lane & 3) * 16 * Sh::kRowPitch;
          int32_t next_id = page_of(tok + kBatch * BN);
#pragma unroll 1
          for (int j = 0; j < kBatch && tb + j < u.tiles; ++j, ++it) {
            const int kst = it % Sh::SK;
            ok = wait_or_die(&sm.kempty[kst], ((it / Sh::SK) & 1u) ^ 1u, sm, a.status);
            if (!ok) break;
            if (lane == 0)
              mbar_arrive_expect_tx(&sm.kfull[kst],
                                    __popc((boxes >> (kGroups * j)) & 15u) * box_bytes);
            __syncwarp();
            if (box && (lane >> 2) == j) {
              uint8_t* dst = smem + Sh::OFF_K + kst * Sh::kTileBytes + at;
#pragma unroll
              for (int r = 0; r < (D + 127) / 128; ++r)
                tma_load_2d(dst + r * (BN * 128), &p.tk, 128 * r, y, &sm.kfull[kst]);
            }
          }
          id = next_id;
          scales_of(tok + kBatch * BN, id, ks, vs);
        }
        if (!ok) break;
      }
      if (sm.dead) {  // copies may be in flight: let them land
#pragma unroll 1
        for (uint32_t k = 0; k < Sh::SK && k < it; ++k) {
          const uint32_t x = it - 1 - k;
          wait_landed(smem_u32(&sm.kfull[x % Sh::SK]), (x / Sh::SK) & 1u);
        }
      }
    } else if (warp == kScheduler) {
      // ---- units and their rows of Q
      uint32_t raws = 0;
      for (uint32_t n = 0; n <= (uint32_t)total; ++n) {
        // not long before its time, so that the last units go to the blocks that are free first
        if (n > 0 && !wait_or_die(&sm.unext, (n - 1) & 1u, sm, a.status)) break;
        int32_t x = lane == 0 ? atomicAdd(p.counter, 1) : 0;
        x = __shfl_sync(0xffffffffu, x, 0);
        Unit u = {-1, 0, 0, 0, 0, 0, 0, 0};
        int32_t last = 0;
        if (x < total) {
          int lo = 0, hi = chunks - 1;
#pragma unroll 1
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
#pragma unroll 1
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
          last = min(u.q_len * a.group, u.first + kRows) - 1;
          const AttnSeq q = {u.row0, u.q_len, u.kv_len};
          u.tiles = (attn_limit(a, q, a.by_group(last)) + BN - 1) / BN;
        }
        const int slot = n & 1;
        if (!wait_or_die(&sm.uempty[slot], ((n >> 1) & 1u) ^ 1u, sm, a.status)) break;
        if (lane == 0) {
          sm.unit[slot] = u;
          mbar_arrive(&sm.ufull[slot]);
        }
        if (u.seq < 0) break;
        if (u.tiles == 0) continue;
        // the unit's rows of Q, one copy each, when the last unit's have moved on
        if (!wait_or_die(&sm.rawempty, (raws & 1u) ^ 1u, sm, a.status)) break;
        ++raws;
        if (lane == 0)
          mbar_arrive_expect_tx(&sm.rawfull, (uint32_t)(last - u.first + 1) * 2 * D);
        __syncwarp();
#pragma unroll 1
        for (int32_t r = u.first + lane; r <= last; r += 32) {
          const int32_t i = a.by_group(r), h = r - i * a.group;
          bulk_load(smem + Sh::OFF_RAW + (r - u.first) * Sh::kRawPitch,
                    static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(u.row0 + i) * a.q_stride +
                        (int64_t)(u.head * a.group + h) * D,
                    2 * D, &sm.rawfull);
        }
      }
      if (sm.dead && raws > 0) wait_landed(smem_u32(&sm.rawfull), (raws - 1) & 1u);
      // this kernel reads nothing of the ones before it in the call, but it must not end first
      asm volatile("griddepcontrol.wait;" ::: "memory");
    } else if (warp == kIssuerS) {
      // ---- S = Q K^T
      constexpr uint32_t id_s = idesc_f16(kRows, BN, 0, 0);
      const uint64_t k_desc = f8_desc<D>(smem_u32(smem) + Sh::OFF_K);
      const uint32_t tm = __shfl_sync(0xffffffffu, tbase, 0), el = elect_lane();
      uint32_t g = 0, nq = 0;
      Unit u;
      while (next_unit(u)) {
        const int32_t tiles = __shfl_sync(0xffffffffu, u.tiles, 0);
        if (tiles == 0) continue;
        bool ok = wait_or_die(&sm.qfull, nq & 1u, sm, a.status);
        ++nq;
#pragma unroll 1
        for (int32_t i = 0; i < tiles && ok; ++i) {
          const uint32_t j = g + i;  // tile number since the start
          const uint32_t st = j % Sh::SK;
          ok = wait_or_die(&sm.kfull[st], (j / Sh::SK) & 1u, sm, a.status) &&
               wait_or_die(&sm.sfree, (j & 1u) ^ 1u, sm, a.status);
          tc_fence_after();
          if (ok) {
            const uint64_t kd = k_desc + (uint32_t)(st * (Sh::kTileBytes / 16));
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                warp_mma_f8_ts(el, tm + Sh::TM_S, tm + Sh::TM_Q + term * (D / 4) + 8 * k,
                               kd + ((k >> 2) * (BN * 128) + (k & 3) * 32) / 16, id_s,
                               term + k > 0);
            if (el) {
              mma_commit(&sm.kempty[st]);
              mma_commit(&sm.sfull[j & 1u]);
              if (i + 1 == tiles) mma_commit(&sm.qempty);
            }
          }
          __syncwarp();
        }
        g += tiles;
        if (!ok) break;
      }
      // what was issued has completed before the block's memory goes
      if (el) mma_commit(&sm.drain[0]);
      wait_landed(smem_u32(&sm.drain[0]), 0);
    } else if (warp == kIssuerO) {
      // ---- O += P V
      constexpr uint32_t id_o = idesc_f16(kRows, D, 0, 1);
      const uint64_t h_desc = smem_desc_sw128(smem_u32(smem) + Sh::OFF_H, BN * 128, 1024);
      const uint32_t tm = __shfl_sync(0xffffffffu, tbase, 0), el = elect_lane();
      uint32_t g = 0, nq = 0;
      Unit u;
      while (next_unit(u)) {
        const int32_t tiles = __shfl_sync(0xffffffffu, u.tiles, 0);
        if (tiles == 0) continue;
        bool ok = wait_or_die(&sm.ofree, (nq & 1u) ^ 1u, sm, a.status);
        ++nq;
#pragma unroll 1
        for (int32_t i = 0; i < tiles && ok; ++i) {
          const uint32_t j = g + i, b = j & 1u, hb = j % Sh::NH;
          ok = wait_or_die(&sm.hfull[hb], (j / Sh::NH) & 1u, sm, a.status) &&
               wait_or_die(&sm.pfull[b], (j >> 1) & 1u, sm, a.status);
          tc_fence_after();
          if (ok) {
            const uint64_t hd = h_desc + (uint32_t)(hb * (Sh::kHBytes / 16));
            const uint32_t pa = tm + Sh::TM_P + b * (BN / 2);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              warp_mma_f16_ts(el, tm + Sh::TM_O, pa + 8 * k, hd + k * (2048 / 16), id_o,
                              i > 0 || k > 0);
            if (el) mma_commit(&sm.odone[j % kDone]);
          }
          __syncwarp();
        }
        g += tiles;
        if (!ok) break;
      }
      if (el) mma_commit(&sm.drain[1]);
      wait_landed(smem_u32(&sm.drain[1]), 0);
    }
  } else if (warp >= kSoftWarps) {
    // ---- operands: Q of a unit, then its V tiles
    give_registers<kAuxRegs>();
    const int aw = warp - kSoftWarps, at = tid - kSoftThreads;
    uint32_t g = 0, nq = 0, nb = 0;
    Unit u;
    // a thread's place in V tiles: 16 channels of every (256 * 16 / D)-th token. Eight lanes
    // take four chunks of two neighbouring tokens, whose f16 chunks fall on distinct banks.
    constexpr int kChunks = D / 16, kStep = kAuxThreads / kChunks, kV = BN / kStep;
    const int vc = (at & 3) | ((at >> 3) & (kChunks / 4 - 1)) << 2;
    const int vt = ((at >> 2) & 1) | (at >> 3) / (kChunks / 4) << 1;
    const uint32_t h0 = sw128_offset(vt, 16 * vc, BN), h1 = sw128_offset(vt, 16 * vc + 8, BN);
    static_assert(kStep % 8 == 0, "the swizzle repeats from step to step");
    const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + 16 * vc;
    // and in Q: half of a row
    const int qr = 32 * (warp & 3) + lane, qhalf = aw >> 2;
    uint8_t* raw = smem + Sh::OFF_RAW + qr * Sh::kRawPitch + qhalf * D;
    bool more = next_unit(u);
    while (true) {
      if (named_any(kAuxBar, kAuxThreads, !more)) break;  // these warps leave together
      if (u.tiles > 0) {
        bool ok = true;
        // V tiles: a tile's loads are on their way while the one before is stored
        uint4 v[kV];
#pragma unroll 1
        for (int32_t t = -1; t < u.tiles && ok; ++t) {
          uint4 cur[kV];
#pragma unroll
          for (int k = 0; k < kV; ++k) cur[k] = v[k];
          if (t + 1 < u.tiles) {
            const uint32_t mb = nb + (uint32_t)(t + 1) / kBatch;
            if ((t + 1) % kBatch == 0)
              ok = wait_or_die(&sm.mfull[mb % kBatches], (mb / kBatches) & 1u, sm, a.status);
            const TileMeta& m = sm.meta[mb % kBatches][(t + 1) % kBatch];
            auto row = [&](int k) {
              return *reinterpret_cast<const uint4*>(
                  vbase + (int64_t)(m.row[(vt + k * kStep) >> 4] + ((vt + k * kStep) & 15)) * D);
            };
            if (ok && m.absent == 0 && (t + 2) * BN <= u.kv_len) {
#pragma unroll
              for (int k = 0; k < kV; ++k) v[k] = row(k);
            } else {  // zeros past the cached tokens and without a page
              const int32_t left = ok ? u.kv_len - (t + 1) * BN - vt : 0;
#pragma unroll
              for (int k = 0; k < kV; ++k) {
                v[k] = make_uint4(0, 0, 0, 0);
                if (k * kStep < left && m.row[(vt + k * kStep) >> 4] >= 0) v[k] = row(k);
              }
            }
          }
          if (t < 0) {  // Q, while the first V tile is on its way
            ok = wait_or_die(&sm.rawfull, nq & 1u, sm, a.status) && ok;
            int ex;
            {
              const bool live = u.first + qr < u.q_len * a.group;
              // largest magnitude of the row, NaN if there is one
              __nv_bfloat162 big = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
              for (int c = 0; c < D; c += 16) {
                const uint4 w = *reinterpret_cast<const uint4*>(raw + c);
                big = __hmax2_nan(big, __habs2(bf16x2(w.x)));
                big = __hmax2_nan(big, __habs2(bf16x2(w.y)));
                big = __hmax2_nan(big, __habs2(bf16x2(w.z)));
                big = __hmax2_nan(big, __habs2(bf16x2(w.w)));
              }
              uint32_t top = *reinterpret_cast<const uint32_t*>(&big);
              sm.exchange_q[qhalf][qr] = (uint16_t)max(top & 0xffffu, top >> 16);
              named_sync(kAuxBar, kAuxThreads);
              top = max(sm.exchange_q[0][qr], sm.exchange_q[1][qr]);
              ex = (int)(top >> 7) - 127;            // [128, 256) after the scaling
              const bool wild = live && ex == 128;   // an infinity or NaN: the row is NaN
              ex = wild ? 7 : max(ex, -100);
              if (!live) ex = 7;
              float up = wild ? __int_as_float(0x7fffffff)
                              : __uint_as_float((uint32_t)(7 - ex + 127) << 23);
              if (a.scale_log2 < 0.f) up = -up;
              const __nv_bfloat162 up2 = __floats2bfloat162_rn(up, up);  // exact: a power of two
              if (!live) {  // the row may hold anything
#pragma unroll 1
                for (int c = 0; c < D; c += 16)
                  *reinterpret_cast<uint4*>(raw + c) = make_uint4(0, 0, 0, 0);
              }
              // in place: eight values become eight e4m3 codes of each term
#pragma unroll 2
              for (int c = 0; c < D; c += 16) {
                uint4* at8 = reinterpret_cast<uint4*>(raw + c);
                const uint4 v = *at8;
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 y = __hmul2(bf16x2(w[e]), up2);
                  const uint32_t yb = *reinterpret_cast<const uint32_t*>(&y);
                  const uint32_t h =
                      f16x2(__uint_as_float(yb << 16), __uint_as_float(yb & 0xffff0000u));
                  const uint16_t k = half2_to_e4m3(h);
                  const uint32_t back = e4m3_to_half2(k);
                  const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&h),
                                               *reinterpret_cast<const __half2*>(&back));
                  hi[e >> 1] |= (uint32_t)k << (16 * (e & 1));
                  lo[e >> 1] |= (uint32_t)half2_to_e4m3(h2_bits(rest)) << (16 * (e & 1));
                }
                *at8 = make_uint4(hi[0], hi[1], lo[0], lo[1]);
              }
            }
            // to tensor memory, when the S products of the unit before have read theirs
            ok = wait_or_die(&sm.qempty, (nq & 1u) ^ 1u, sm, a.status) && ok;
            tc_fence_after();
            if (qhalf == 0) sm.row_exp[nq & 1u][qr] = (int8_t)(ex - 7);  // nor does one read this
            {
              const uint32_t tq = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + Sh::TM_Q +
                                  qhalf * (D / 8);
#pragma unroll 1
              for (int c = 0; c < D / 64; ++c) {  // 32 elements: eight columns of each term
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint4 w = *reinterpret_cast<const uint4*>(raw + 64 * c + 16 * e);
                  hi[2 * e] = w.x; hi[2 * e + 1] = w.y; lo[2 * e] = w.z; lo[2 * e + 1] = w.w;
                }
                tmem_st8(tq + 8 * c, hi);
                tmem_st8(tq + D / 4 + 8 * c, lo);
              }
            }
            tmem_st_wait();
            tc_fence_before();
            fence_proxy_async_smem();  // the next rows come by the async proxy
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sm.qfull);
              mbar_arrive(&sm.rawempty);
            }
            ++nq;
            continue;
          }
          const uint32_t j = g + t, hb = j % Sh::NH;
          if (j >= Sh::NH) {  // P V(j - NH) has read this buffer
            const uint32_t o = j - Sh::NH;
            ok = wait_or_die(&sm.odone[o % kDone], (o / kDone) & 1u, sm, a.status) && ok;
          }
          uint8_t* dst = smem + Sh::OFF_H + hb * Sh::kHBytes;
#pragma unroll
          for (int k = 0; k < kV; ++k) {
            const uint32_t s4[4] = {cur[k].x, cur[k].y, cur[k].z, cur[k].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[2 * e] = e4m3_to_half2((uint16_t)s4[e]);
              h[2 * e + 1] = e4m3_to_half2((uint16_t)(s4[e] >> 16));
            }
            *reinterpret_cast<uint4*>(dst + h0 + k * kStep * 128) =
                make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + h1 + k * kStep * 128) =
                make_uint4(h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.hfull[hb]);
        }
        g += u.tiles;
        nb += (u.tiles + kBatch - 1) / kBatch;
      }
      more = next_unit(u);
    }
  } else {
    // ---- softmax (tiles of this group's parity) and epilogue
    take_registers<kSoftRegs>();
    const uint32_t grp = warp >> 2;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t t_row = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
    const int from_other = kPairBar + 2 * (warp & 3) + (int)grp,
              to_other = kPairBar + 2 * (warp & 3) + (int)(grp ^ 1u);
    const float scale = fabsf(a.scale_log2);
    uint32_t g = 0, nq = 0, nb = 0;
    Unit u;
    // the warps leave together, so that none is left at a barrier
    bool more = see_unit();
    more = !named_any(kSoftBar, kSoftThreads, !more);
    while (more) {
      take_unit(u);
      const int32_t rows = u.q_len * a.group, row = u.first + r;
      const bool live = row < rows;
      const int32_t query = live ? a.by_group(row) : 0;
      const AttnSeq s = {u.row0, u.q_len, u.kv_len};
      const int32_t limit = live ? attn_limit(a, s, query) : u.kv_len;
      const int32_t min_limit = attn_limit(a, s, a.by_group(u.first));
      float mz = kNoMax, ms = kNoMax, l = 0.f, rs = 0.f;
      const uint32_t first = (g & 1u) ^ grp;  // this group's first tile of the unit
      for (int32_t i = (int32_t)first; i < u.tiles; i += 2) {
        const uint32_t j = g + i, b = grp;  // tile number since the start; its P buffer
        const uint32_t mb = nb + (uint32_t)i / kBatch;
        if (i % kBatch < 2)  // this group's first tile of the batch
          wait_on(&sm.mfull[mb % kBatches], (mb / kBatches) & 1u, sm, a.status);
        // the tile's scales, while S is on its way
        const TileMeta& meta = sm.meta[mb % kBatches][i % kBatch];
        const float4 ks4 = *reinterpret_cast<const float4*>(meta.ks);
        const float4 lv4 = *reinterpret_cast<const float4*>(meta.lv);
        const uint32_t absent = meta.absent;
        const float lvmin = meta.lvmin;
        wait_on(&sm.sfull[grp], (j >> 1) & 1u, sm, a.status);
        tc_fence_after();
        if (i == (int32_t)first)
          rs = scale * __uint_as_float((uint32_t)(sm.row_exp[nq & 1u][r] + 127) << 23);
        uint32_t x[BN];
        tmem_ld32(t_row + Sh::TM_S, reinterpret_cast<uint32_t(&)[32]>(x[0]));
        tmem_ld32(t_row + Sh::TM_S + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sfree);
        if ((i + 1) * BN > min_limit || absent != 0) {
#pragma unroll
          for (int q = 0; q < kGroups; ++q) {
            const int32_t room = (absent >> q) & 1u ? 0 : limit - i * BN - 16 * q;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e >= room) x[16 * q + e] = 0xff800000u;
          }
        }
        // the tile's largest exponents: within a group of 16 tokens before the group's scales
        const float ksq[kGroups] = {ks4.x, ks4.y, ks4.z, ks4.w};
        float lvq[kGroups] = {lv4.x, lv4.y, lv4.z, lv4.w};
        float f[kGroups], zq[kGroups];
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          f[q] = fmaxf(ksq[q] * rs, 1e-37f);  // above 0: what is masked stays -inf
          float y = __uint_as_float(x[16 * q]), y2 = __uint_as_float(x[16 * q + 1]);
#pragma unroll
          for (int e = 2; e < 16; e += 4) {  // two chains of three-input maxima
            y = max3(y, __uint_as_float(x[16 * q + e]), __uint_as_float(x[16 * q + e + 1]));
            if (e + 2 < 16)
              y2 = max3(y2, __uint_as_float(x[16 * q + e + 2]), __uint_as_float(x[16 * q + e + 3]));
          }
          y = fmaxf(y, y2);
          zq[q] = fmaf(y, f[q], lvq[q]);
        }
        const float top = fmaxf(fmaxf(zq[0], zq[1]), fmaxf(zq[2], zq[3]));
        if (i > 0) {
          pair_wait(from_other);
          const float was = ms;
          const float2 m = sm.m[r];
          mz = m.x;
          ms = m.y;
          l *= ex2(was - ms);
        }
        float apart = mz - ms;
        if (__any_sync(0xffffffffu, top > mz + kLazyMax || lvmin < apart - kNear)) {
          // new maxima for these rows, the accumulator and sum follow
          float top_s = ms;
#pragma unroll
          for (int q = 0; q < kGroups; ++q) top_s = fmaxf(top_s, zq[q] - lvq[q]);
          const float top_z = fmaxf(top, mz);
          const float fm = ex2(mz - top_z);
          l *= ex2(ms - top_s);
          ms = top_s;
          mz = top_z;
          apart = mz - ms;
#pragma unroll
          for (int q = 0; q < kGroups; ++q) lvq[q] = fmaxf(lvq[q], apart - kFar);
          if (i > 0 && __any_sync(0xffffffffu, fm != 1.f)) {
            const uint32_t o = j - 1;  // P V of the tile before
            wait_on(&sm.odone[o % kDone], (o / kDone) & 1u, sm, a.status);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t y[16];
              tmem_ld16(t_row + Sh::TM_O + c, y);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * fm);
              tmem_st16(t_row + Sh::TM_O + c, y);
            }
            tmem_st_wait();
          }
        }
        if (i + 1 < u.tiles) {
          sm.m[r] = make_float2(mz, ms);
          pair_arrive(to_other);
        }
        // P = 2^(z - mz + kProbShift)
        const float mu = mz - kProbShift;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ph[16];
#pragma unroll
          for (int q = 2 * h; q < 2 * h + 2; ++q) {
            const float off = lvq[q] - mu, fq = f[q];
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 16 * q; e < 16 * q + 16; e += 2) {
              float2 z = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              z = fma2(z, make_float2(fq, fq), make_float2(off, off));
              const float2 pr = make_float2(ex2(z.x), ex2(z.y));
              sum = add2(sum, pr);
              ph[e / 2 - 16 * h] = f16x2(pr.x, pr.y);
            }
            l = fmaf(sum.x + sum.y, ex2(apart - kProbShift - lvq[q]), l);
          }
          if (h == 0 && j >= 2) {  // P V(j - 2) has read this group's buffer
            const uint32_t o = j - 2;
            wait_on(&sm.odone[o % kDone], (o / kDone) & 1u, sm, a.status);
            tc_fence_after();
          }
          tmem_st16(t_row + Sh::TM_P + b * (BN / 2) + 16 * h, ph);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[b]);
      }
      g += u.tiles;
      nb += (u.tiles + kBatch - 1) / kBatch;
      // ---- output: the groups' sums meet, each writes half of the row. What needs only the sums
      // is done while the last P V runs, and the look for the next unit falls into it.
      const uint32_t last = g - 1;
      if (u.tiles > 0) {
        ++nq;
        if ((last & 1u) == grp) sm.m[r] = make_float2(mz, ms);  // who has the final maxima
        named_sync(kSoftBar, kSoftThreads);
        const float2 m = sm.m[r];
        sm.exchange_l[grp][r] = l * ex2(ms - m.y);
        mz = m.x;
        ms = m.y;
      }
      more = see_unit();
      more = !named_any(kSoftBar, kSoftThreads, !more);
      if (u.tiles > 0) l = sm.exchange_l[0][r] + sm.exchange_l[1][r];
      const float inv = l == 0.f ? 0.f : __fdividef(ex2(mz - ms - kOutShift), l);
      if (live && grp == 0 && a.lse)
        a.lse[(int64_t)(u.row0 + query) * (a.hkv * a.group) + u.head * a.group + row -
              query * a.group] = l == 0.f ? -GDN_INF : (ms + __log2f(l)) * kLn2;
      // through shared memory, 32 columns at a time, so that four lanes store 64 consecutive
      // bytes of a row (a thread storing its own row would touch 32 lines with every store)
      uint8_t* stage = smem + Sh::OFF_OUT + warp * 2048;
      __nv_bfloat16* out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int32_t ro = u.first + 32 * (warp & 3) + 8 * k + (lane >> 2);
        const int32_t qo = a.by_group(ro);
        out[k] = ro < rows ? static_cast<__nv_bfloat16*>(a.o) +
                                 (int64_t)(u.row0 + qo) * a.o_stride +
                                 (int64_t)(u.head * a.group + ro - qo * a.group) * D +
                                 grp * (D / 2) + 8 * (lane & 3)
                           : nullptr;
      }
      if (u.tiles > 0) {
        wait_on(&sm.odone[last % kDone], (last / kDone) & 1u, sm, a.status);
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t o[32];
        if (u.tiles > 0) {
          tmem_ld32(t_row + Sh::TM_O + grp * (D / 2) + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 z = mul2(make_float2(__uint_as_float(o[8 * e + 2 * k]),
                                              __uint_as_float(o[8 * e + 2 * k + 1])),
                                  make_float2(inv, inv));
            const __nv_bfloat162 y = __floats2bfloat162_rn(z.x, z.y);
            w[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = 8 * k + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(
              stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
          if (out[k]) *reinterpret_cast<uint4*>(out[k] + c) = w;
        }
        __syncwarp();
      }
      if (u.tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ofree);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerS) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
int launch(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, cudaStream_t stream) {
  using Sh = Shape<D>;
  TileParams p;
  p.a = a;
  const int box = std::min(c.page_size, BN);
  if (!make_cache_map(&p.tk, c.k, c, box)) return (int)cudaErrorInvalidValue;
  p.v = c.v;
  p.counter = a.counter;
  static std::atomic<int> ready[kMaxDevices];
  constexpr int kSmem = (int)Sh::kSmem;
  int e = configure_once(ready, [] {
    return (int)cudaFuncSetAttribute(tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmem);
  });
  if (e != 0) return e;
  const int64_t units =
      (((int64_t)a.num_tokens * a.group + kRows - 1) / kRows + a.num_seqs) * a.hkv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(units, num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // blocks may start as the kernels before leave SMs free
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, tile_kernel<D>, p);
}

}  // namespace

int launch_attn_tile(const AttnArgs& a, const gdn_kv_cache& c, int num_sms, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.head_dim == 64) return launch<64>(a, c, num_sms, s);
  if (c.head_dim == 128) return launch<128>(a, c, num_sms, s);
  return launch<256>(a, c, num_sms, s);
}

}  // namespace gdn
