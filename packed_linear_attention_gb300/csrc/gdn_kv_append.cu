// gdn_kv_append.cu — rotary embedding with several position axes, and the append that
// quantises keys and values into the paged e4m3 cache.
//
// Rotation. Pair i turns by position * f_i, f_i in turns per position held as a 64-bit binary
// fraction: the low 64 bits of the integer product position * F_i are the angle modulo a turn,
// with no rounding that grows with the position. Its top bits, rounded, name the quarter turn;
// the rest, at most an eighth of a turn, is one fp32 number, and the Taylor series of sine and
// cosine to r^9 and r^10 leave less than 2^-28. Both kernels are bound by HBM
// (every element is read and written once); a thread of the rotation takes the same pairs of
// several heads of a token, so that the sine and cosine are formed once for them. Measured: 18
// heads of 256 of 32,768 tokens 101 us, 6.0 TB/s, 88% of the measured copy rate.
//
// Append. A unit is a run of rows that land in one page, for one head: keys by one half of a
// block's 512 threads and values by the other, eight elements of a row a thread. The run's rows
// are copied to shared memory at once, asynchronously, and stay there as they came while its
// largest magnitude is found; the rotation is cheap enough to be done twice (its sines and
// cosines are formed once for the run, by all threads, while the rows are on their way; the other
// half of a pair is read beside, since a row never leaves a warp). Only runs longer than eight
// bf16 or four fp32 rows a thread read their first rows a second time. With power-of-two scales
// the division is exact, and a later, larger scale only moves the exponents of the codes that are
// already there. No
// unit list is needed: a row begins a run when its slot opens a page or does not follow the
// previous row's slot. Measured: 32 x 1,024 tokens, 16 query heads rotated beside 2 + 2 heads of
// 256, 129 us, 4.9 TB/s, 73% of the copy rate; keys and values alone 37 us, 15 more rotated,
// where a block's chain of slots, rows, maximum and store is what bounds it (two blocks an SM).
// Rows in registers took 137 us, three blocks an SM 152 (spills), and asking for the rows before
// the slots are known changed nothing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gdn_attn_internal.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHalf = 256;               // threads for the keys, and as many for the values
constexpr int kAppendThreads = 2 * kHalf;
constexpr int kMinExp = -100;            // exponent of the smallest scale

struct RopeDev {  // gdn_rope without what the kernels do not need
  uint64_t turns[GDN_ROPE_MAX_PAIRS];
  uint8_t axis[GDN_ROPE_MAX_PAIRS];
  int32_t head_dim, rotary_dim, adjacent, num_axes;
};

// Eight consecutive elements of a tensor, as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  static constexpr int kRows = 8, kParts = 1;  // rows that a thread of the append stages
  uint4 w;
  __device__ void fetch(const uint4* p, int) { w = p[0]; }
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Raw8<float> {
  static constexpr int kRows = 4, kParts = 2;
  float4 a, b;
  __device__ void fetch(const uint4* p, int step) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + step);
  }
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// The table in shared memory: lanes look up different pairs, which constant memory would serve
// one after another (8 us of a 79 us append).
struct Turns {
  uint64_t turns[GDN_ROPE_MAX_PAIRS];
  uint8_t axis[GDN_ROPE_MAX_PAIRS];
  __device__ void load(const RopeDev& r, int tid, int threads) {  // ends with the block together
    for (int i = tid; i < r.rotary_dim / 2; i += threads) {
      turns[i] = r.turns[i];
      axis[i] = r.axis[i];
    }
    __syncthreads();
  }
};

// cos and sin of pair i at position `at` of its axis.
__device__ __forceinline__ void pair_angle(const Turns& r, int i, int32_t at, float& c, float& s) {
  const uint64_t turn = (uint64_t)(int64_t)at * r.turns[i];
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  // the rest in 2^-34 turns, in [-2^31, 2^31], times 2 pi 2^-34
  const float x = (float)(int32_t)((int64_t)(turn - ((uint64_t)quarter << 62)) >> 30) *
                  (6.283185307179586f / 17179869184.f);
  const float z = x * x;
  float p = fmaf(z, 1.f / 362880, -1.f / 5040);
  p = fmaf(z, p, 1.f / 120);
  p = fmaf(z, p, -1.f / 6);
  const float sn = fmaf(x * z, p, x);
  float q = fmaf(z, -1.f / 3628800, 1.f / 40320);
  q = fmaf(z, q, -1.f / 720);
  q = fmaf(z, q, 1.f / 24);
  q = fmaf(z, q, -0.5f);
  const float cs = fmaf(z, q, 1.f);
  c = quarter & 1 ? sn : cs;
  s = quarter & 1 ? cs : sn;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter & 2) s = -s;
}

// One thread: 16 elements of every head of a token in [head0, head1), the heads of x[0]
// followed by those of x[1]. Item i < R/16 are the pairs 8i..8i+7 (elements 8i.. and
// R/2 + 8i.. in the halves layout, 16i.. in the adjacent one), the later items copy.
template <typename T>
__device__ __forceinline__ void rope_heads(const RopeDev& r, const Turns& table,
                                           const RopeArgs& a, int64_t token, int item, int head0,
                                           int head1) {
  const int D = r.head_dim, R = r.rotary_dim;
  const bool turn = 16 * item < R;
  const int lo = turn && !r.adjacent ? 8 * item : 16 * item;
  const int hi = turn && !r.adjacent ? lo + R / 2 : lo + 8;
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      pair_angle(table, 8 * item + e,
                 __ldg(a.positions + table.axis[8 * item + e] * a.pos_stride + token), c[e], s[e]);
  }
#pragma unroll 4
  for (int h = head0; h < head1; ++h) {
    const bool second = h >= a.x[0].heads;
    const RopeHeads& x = second ? a.x[1] : a.x[0];
    const int hh = second ? h - a.x[0].heads : h;
    const T* in = static_cast<const T*>(x.in) + token * x.in_stride + (int64_t)hh * D;
    T* out = static_cast<T*>(x.out) + token * x.out_stride + (int64_t)hh * D;
    if (!turn && in == out) continue;  // in place: nothing to copy
    Raw8<T> u, v;
    // plain loads: in place, another item's store may follow, but never to these elements
    u.load(in + lo);
    v.load(in + hi);
    if (turn) {
      float p[8], q[8];
      u.get(p);
      v.get(q);
      if (r.adjacent) {  // (p0 p1) (p2 p3) ... then q's pairs
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = p[2 * e], y0 = p[2 * e + 1], x1 = q[2 * e], y1 = q[2 * e + 1];
          p[2 * e] = x0 * c[e] - y0 * s[e];
          p[2 * e + 1] = y0 * c[e] + x0 * s[e];
          q[2 * e] = x1 * c[4 + e] - y1 * s[4 + e];
          q[2 * e + 1] = y1 * c[4 + e] + x1 * s[4 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = p[e], y0 = q[e];
          p[e] = x0 * c[e] - y0 * s[e];
          q[e] = y0 * c[e] + x0 * s[e];
        }
      }
      u.set(p);
      v.set(q);
    }
    u.store(out + lo);
    v.store(out + hi);
  }
}

// Block `block` of a rotation over num_tokens tokens, `slices` slices of the heads.
template <typename T>
__device__ __forceinline__ void rope_block(const RopeDev& r, Turns& table, const RopeArgs& a,
                                           int64_t block, int slices, int threads, int tid) {
  table.load(r, tid, threads);
  const int items = r.head_dim / 16, heads = a.x[0].heads + a.x[1].heads;
  const int64_t g = block / slices * threads + tid;
  const int64_t token = g / items;
  if (token >= a.num_tokens) return;
  const int slice = (int)(block % slices), per = (heads + slices - 1) / slices;
  rope_heads<T>(r, table, a, token, (int)(g % items), slice * per, min(heads, (slice + 1) * per));
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeDev r, const __grid_constant__ RopeArgs a, int slices) {
  __shared__ Turns table;
  rope_block<T>(r, table, a, blockIdx.x, slices, kRopeThreads, threadIdx.x);
}

// Two fp32 values as e4m3 codes (nearest even, NaN kept, larger magnitudes to 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Exponent of the least power of two s with amax <= 448 s = 1.75 * 2^8 s, amax finite >= 0.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinExp);  // zeros and subnormals among them
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ void copy16_async(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

struct AppendDev {
  AppendArgs a;
  int32_t rows_per_block;  // rows whose runs a block handles
  int32_t append_blocks;   // the others rotate q
  int32_t rope_slices;
};

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, 2)
append_kernel(const __grid_constant__ AppendDev p, const __grid_constant__ RopeDev r) {
  const AppendArgs& a = p.a;
  const int tid = threadIdx.x;
  __shared__ Turns table;
  // the two kinds of blocks in turns: the append waits for memory where the rotation fills it
  // (32 x 1,024 tokens: 152 us with the append's blocks first, 137 in turns)
  const int64_t before = (int64_t)blockIdx.x * p.append_blocks / gridDim.x;
  if (((int64_t)blockIdx.x + 1) * p.append_blocks / gridDim.x == before) {
    rope_block<T>(r, table, a.rope_args, blockIdx.x - before, p.rope_slices, kAppendThreads, tid);
    return;
  }
  constexpr int kVec = D / 8;              // threads of a row
  constexpr int kRows = kHalf / kVec;      // rows of a pass
  constexpr int kBatch = Raw8<T>::kRows, kParts = Raw8<T>::kParts;
  __shared__ int64_t s_slot[1 + 256];      // slots from the row in front of the block's on
  __shared__ int32_t s_pos[GDN_ROPE_MAX_AXES][256];  // positions of the rows from row0 on
  __shared__ int s_start[128];
  __shared__ int s_nstart, s_n;
  __shared__ uint32_t s_amax[2];
  __shared__ uint32_t s_nan[4];            // rows of v that hold a NaN
  extern __shared__ uint4 stage[];         // [kBatch][kParts][thread]: rows as they came
  float2* s_turn = reinterpret_cast<float2*>(stage + kBatch * kParts * kAppendThreads);
  // cos, sin: [rows of a batch][R / 2]
  const int P = a.cache.page_size, H = a.cache.num_kv_heads;
  const int head = (int)(before % H);
  const int64_t row0 = before / H * p.rows_per_block;
  const int64_t nslots = (int64_t)a.cache.num_pages * P;
  const bool is_v = tid >= kHalf;
  const int lt = tid & (kHalf - 1), vec = lt % kVec, sub = lt / kVec;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + (int64_t)head * D + 8 * vec;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int R = a.rotate ? r.rotary_dim : 0, half = R / 2;
  // this thread's chunk in the rotation: its first pair and, in the halves layout, the lane that
  // copies the pairs' other elements
  const bool rot = !is_v && 8 * vec < R, low = 8 * vec < half;
  const int pair0 = r.adjacent ? 4 * vec : low ? 8 * vec : 8 * vec - half;
  const int lane = tid & 31;
  const int other = rot && !r.adjacent ? (low ? lane + half / 8 : lane - half / 8) : lane;

  // the block's slots and a page's worth behind them: runs begin here and may end there
  if (tid <= p.rows_per_block + P) {
    const int64_t row = row0 + tid - 1;
    s_slot[tid] = row >= 0 && row < a.num_tokens ? a.slots[row] : -1;
  }
  if (tid == 0) s_nstart = 0;
  if (R) {
    for (int x = tid >> 8; x < r.num_axes; x += kAppendThreads / 256) {
      const int i = tid & 255;
      if (i < p.rows_per_block + P && row0 + i < a.num_tokens)
        s_pos[x][i] = a.rope_args.positions[x * a.rope_args.pos_stride + row0 + i];
    }
    table.load(r, tid, kAppendThreads);
  } else {
    __syncthreads();
  }
  if (tid < p.rows_per_block) {
    const int64_t slot = s_slot[tid + 1];
    if (slot >= nslots)
      raise_status(a.status, GDN_ERR_INVALID_ARGUMENT);
    else if (slot >= 0 && ((slot & (P - 1)) == 0 || s_slot[tid] != slot - 1))
      s_start[atomicAdd(&s_nstart, 1)] = tid;
  }
  __syncthreads();
  const int nstart = s_nstart;
#pragma unroll 1
  for (int u = 0; u < nstart; ++u) {  // in any order: the runs are independent
    const int at0 = s_start[u];
    const int64_t row = row0 + at0, slot = s_slot[at0 + 1];
    const int off = (int)(slot & (P - 1));
    const int64_t page = (slot - off) / P;
    if (tid == 0) s_n = P - off;
    if (tid < 2) s_amax[tid] = 0;
    if (tid < 4) s_nan[tid] = 0;
    __syncthreads();
    if (tid > 0 && tid < P - off && s_slot[at0 + 1 + tid] != slot + tid) atomicMin(&s_n, tid);
    __syncthreads();
    const int n = s_n;
    const int passes = (n + kRows - 1) / kRows, batches = (passes + kBatch - 1) / kBatch;

    auto load = [&](int b) {  // rows b kBatch kRows + j kRows + sub
#pragma unroll 2
      for (int j = 0; j < kBatch; ++j) {
        const int i = (b * kBatch + j) * kRows + sub;
        const char* from = reinterpret_cast<const char*>(src + (row + i) * stride);
#pragma unroll
        for (int x = 0; x < kParts; ++x)
          if (i < n) copy16_async(stage + (j * kParts + x) * kAppendThreads + tid, from + 16 * x);
      }
    };
    auto landed = [&] {  // a row is copied and read by the same warp
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    };
    auto turns = [&](int b) {  // cos and sin of the batch's rows (all threads)
      if (!R) return;
      const int i0 = b * kBatch * kRows, rows = min(n - i0, kBatch * kRows);
      __syncthreads();  // the batch before has been read
      const int teams = kAppendThreads / half;
      if (tid < teams * half) {
        const int e = tid % half;
#pragma unroll 1
        for (int i = tid / half; i < rows; i += teams) {
          float c, s;
          pair_angle(table, e, s_pos[table.axis[e]][at0 + i0 + i], c, s);
          s_turn[i * half + e] = make_float2(c, s);
        }
      }
      __syncthreads();
    };
    // the eight elements of the batch's row j, rotated
    auto values = [&](int j, float (&x)[8]) {
      const uint4* at = stage + j * kParts * kAppendThreads + tid;
      Raw8<T> w;
      w.fetch(at, kAppendThreads);
      w.get(x);
      if (!rot) return;
      const float2* t = s_turn + (j * kRows + sub) * half + pair0;
      if (r.adjacent) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = x[2 * e], y0 = x[2 * e + 1];
          x[2 * e] = x0 * t[e].x - y0 * t[e].y;
          x[2 * e + 1] = y0 * t[e].x + x0 * t[e].y;
        }
      } else {
        float y[8];
        w.fetch(at + other - lane, kAppendThreads);
        w.get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = low ? -t[e].y : t[e].y;
          x[e] = x[e] * t[e].x + y[e] * s;
        }
      }
    };
    float amax = 0.f;
#pragma unroll 1
    for (int b = 0; b < batches; ++b) {
      if (b > 0) __syncwarp();  // the batch before has been read
      load(b);
      turns(b);
      landed();
#pragma unroll 2
      for (int j = 0; j < kBatch; ++j) {
        const int i = (b * kBatch + j) * kRows + sub;
        if (i < n) {
          float x[8];
          values(j, x);
          bool nan = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float m = fabsf(x[e]);
            nan = nan || m != m;
            if (m < __int_as_float(0x7f800000)) amax = fmaxf(amax, m);
          }
          if (is_v && nan) atomicOr(&s_nan[i >> 5], 1u << (i & 31));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) atomicMax(&s_amax[is_v], __float_as_uint(amax));
    __syncthreads();
    float* sp = (is_v ? a.cache.v_scale : a.cache.k_scale) + page * H + head;
    uint8_t* codes = static_cast<uint8_t*>(is_v ? a.cache.v : a.cache.k) +
                     ((page * H + head) * P) * (int64_t)D + 8 * vec;
    const float need = exp2_int(scale_exp(__uint_as_float(s_amax[is_v])));
    float scale = need;
    if (off > 0) {
      const float old = *sp;
      scale = fmaxf(old, need);
      if (scale > old) {  // the rows in front move to the larger scale
        const float f = old / scale;
#pragma unroll 1
        for (int i = sub; i < off; i += kRows) {
          uint2* c = reinterpret_cast<uint2*>(codes + (int64_t)i * D);
          const uint2 z2 = *c;
          uint32_t z[4] = {z2.x & 0xFFFFu, z2.x >> 16, z2.y & 0xFFFFu, z2.y >> 16};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = from_e4m3x2(z[e]);
            z[e] = e4m3x2(y.x * f, y.y * f);
          }
          *c = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
        }
      }
    }
    const float inv = 1.f / scale;  // exact: a power of two (or the caller's own old scale)
    auto store = [&](int b) {
#pragma unroll 2
      for (int j = 0; j < kBatch; ++j) {
        const int i = (b * kBatch + j) * kRows + sub;
        if (i < n) {
          float x[8];
          values(j, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv;
          if ((s_nan[i >> 5] >> (i & 31)) & 1u) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              x[e] = !is_v ? __int_as_float(0x7fffffff) : x[e] == x[e] ? x[e] : 0.f;
          }
          *reinterpret_cast<uint2*>(codes + (int64_t)(off + i) * D) =
              make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16,
                         e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
        }
      }
    };
    // the last batch's rows are still there; the others are loaded again
#pragma unroll 1
    for (int b = batches - 1;;) {
      store(b);
      if (--b < 0) break;
      __syncwarp();
      load(b);
      turns(b);
      landed();
    }
    __syncthreads();  // every thread has read the old scale and the flags
    if (lt == 0) *sp = scale;
  }
}

RopeDev device_rope(const gdn_rope& rope) {
  RopeDev r;
  for (int i = 0; i < GDN_ROPE_MAX_PAIRS; ++i) {
    r.turns[i] = rope.turns[i];
    r.axis[i] = rope.axis[i];
  }
  r.head_dim = rope.head_dim;
  r.rotary_dim = rope.rotary_dim;
  r.num_axes = rope.num_axes;
  r.adjacent = rope.pair_layout == GDN_ROPE_ADJACENT;
  return r;
}

// Slices of the heads: one while the tokens alone fill the SMs, else up to one per head, so
// that a decode step's few tokens still spread over the GPU.
int rope_slices(int64_t threads, int heads) {
  constexpr int64_t kFill = 152 * 1024;
  int s = 1;
  while (s < heads && threads * s < kFill) s *= 2;
  return std::min(s, heads);
}

}  // namespace

int launch_rope(const gdn_rope& rope, const RopeArgs& a, bool bf16, void* stream) {
  const int heads = a.x[0].heads + a.x[1].heads;
  if (a.num_tokens == 0 || heads == 0) return 0;
  const int64_t threads = (int64_t)a.num_tokens * (rope.head_dim / 16);
  const int slices = rope_slices(threads, heads);
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads * slices;
  if (blocks > INT32_MAX) return (int)cudaErrorInvalidValue;
  const RopeDev r = device_rope(rope);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (bf16) rope_kernel<__nv_bfloat16><<<(unsigned)blocks, kRopeThreads, 0, s>>>(r, a, slices);
  else rope_kernel<float><<<(unsigned)blocks, kRopeThreads, 0, s>>>(r, a, slices);
  return (int)cudaGetLastError();
}

int launch_kv_append(const gdn_rope* rope, const AppendArgs& a, bool bf16, void* stream) {
  if (a.num_tokens == 0) return 0;
  AppendDev p;
  p.a = a;
  const int H = a.cache.num_kv_heads;
  // rows per block: a page's worth when that still fills the SMs, else fewer
  int rows = a.cache.page_size;
  while (rows > 1 && ((int64_t)a.num_tokens + rows - 1) / rows * H < 2 * 152) rows /= 2;
  p.rows_per_block = rows;
  const int64_t append = ((int64_t)a.num_tokens + rows - 1) / rows * H;
  int64_t turn = 0;
  p.rope_slices = 1;
  RopeDev r = {};
  if (rope) r = device_rope(*rope);
  if (a.rotate && a.rope_args.x[0].heads > 0) {
    const int64_t threads = (int64_t)a.num_tokens * (rope->head_dim / 16);
    p.rope_slices = rope_slices(threads, a.rope_args.x[0].heads);
    turn = (threads + kAppendThreads - 1) / kAppendThreads * p.rope_slices;
  }
  if (append + turn > INT32_MAX) return (int)cudaErrorInvalidValue;
  p.append_blocks = (int32_t)append;
  const unsigned blocks = (unsigned)(append + turn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int e = 0;
  auto run = [&](auto type, auto dim) {
    using T = decltype(type);
    constexpr int D = decltype(dim)::value;
    // the rows of a batch: at most a page's
    const int batch = std::min(a.cache.page_size, Raw8<T>::kRows * (kHalf / (D / 8)));
    const size_t smem = sizeof(uint4) * Raw8<T>::kRows * Raw8<T>::kParts * kAppendThreads +
                        (a.rotate ? sizeof(float2) * batch * (r.rotary_dim / 2) : 0);
    static std::atomic<int> ready[kMaxDevices];
    e = configure_once(ready, [] {
      return (int)cudaFuncSetAttribute(append_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 192 * 1024);
    });
    if (e == 0) append_kernel<T, D><<<blocks, kAppendThreads, smem, s>>>(p, r);
  };
  auto pick = [&](auto type) {
    if (a.cache.head_dim == 64) run(type, std::integral_constant<int, 64>());
    else if (a.cache.head_dim == 128) run(type, std::integral_constant<int, 128>());
    else run(type, std::integral_constant<int, 256>());
  };
  if (bf16) pick(__nv_bfloat16());
  else pick(float());
  return e != 0 ? e : (int)cudaGetLastError();
}

}  // namespace gdn
