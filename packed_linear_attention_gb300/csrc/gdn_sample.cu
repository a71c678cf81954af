// gdn_sample.cu — a token from every row of logits: temperature, top-k, top-p and min-p, then the
// inverse of the kept tokens' cumulative weights at a given random number.
//
// A row belongs to one cluster of blocks: each holds a slice of it in shared memory, so the logits
// are read from memory once, however many passes the filters take. Nothing is sorted: every filter
// keeps a beginning of the order (falling logits, equal ones by rising index), so it is enough to
// find the last token kept. The tokens are counted in bins of their distance from the maximum. For
// top-k the counts say which bin it is in; for top-p they bound the weights to about 1.5% and say
// between which bins. The tokens there, when few, are ranked against one another, else their bits
// are cut into 2,048 finer bins, until they are few or all equal.
//
// Weights are integers, 2^44 for the maximum, so that their sums are exact and depend on no order:
// exp((l - m) / T) = 2^-y, and 2^-y is a table entry times 1 + a polynomial of the last 1/32 of y.
// l - m and y carry a second fp32 term, since errors of 2^-24 would move borders that u or
// top_p may fall next to: weights are right to 2^-28. Seven roundings of 2^-31 to 2^-30.5 of the weight
// each (table entry, its fp32 form, r, the polynomial, r times it, the product, the sum) are 2^-28.15;
// 24 million random ones were within 2^-28.6.
#include <cooperative_groups.h>

#include <algorithm>

#include "gdn_internal.h"
#include "gdn_step_internal.h"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

using u32 = uint32_t;
using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kBinsOf = kBins / kThreads;  // bins of a thread
static_assert(kBinsOf == 4, "a thread's counts are read 16 bytes at a time");
constexpr int kList = 128;                               // tokens ranked against one another
constexpr float kRange = 44.f;                           // 2^-44 of the maximum: weight 1
constexpr int kMaxCluster = 8;
constexpr size_t kMostMemory = 227 * 1024;               // shared memory of a block, and of an SM

// 2^(31 - j/32), j = 0 .. 31, as a whole number and as fp32. One entry a bank: lanes may look up what
// they like.
struct Powers {
  u32 whole[32], factor[32];
};
constexpr double root_of(double x) {
  double r = x;
  for (int i = 0; i < 60; ++i) r = 0.5 * (r + x / r);
  return r;
}
constexpr Powers make_powers() {
  double step = 0.5;  // 2^(-1/32): five square roots of a half
  for (int i = 0; i < 5; ++i) step = root_of(step);
  Powers t = {};
  double p = 2147483648.0;
  for (int j = 0; j < 32; ++j, p *= step) {
    t.whole[j] = (u32)(p + 0.5);
    // bits of the fp32 number nearest to p in [2^30, 2^31]: 24 bits from 2^7 (or 2^8) on
    const double unit = j == 0 ? 256.0 : 128.0;
    const u32 m = (u32)(p / unit + 0.5);
    t.factor[j] = ((j == 0 ? 158u : 157u) << 23) + (m - (1u << 23));
  }
  return t;
}
__device__ const Powers kPowers = make_powers();

struct Entry {
  u64 weight;
  u32 key, at;
};
struct List {
  Entry mine[kList], all[kList];
  u32 count;
};
struct Found {
  u64 before_weight;
  u32 bin, before, count;
};
struct alignas(16) Shared {  // the slice lies behind it, read 16 bytes at a time
  u32 count[kBins];  // tokens at each distance from the maximum
  union {
    u32 finer[kBins];
    List list;
  };
  Powers table;
  u64 box[2];         // what the cluster's blocks tell one another, in turns
  u64 warp_weight[kWarps];
  u32 warp_count[kWarps];
  Found found;
  u32 window[2];
  int row;
  Entry chosen;       // the last token kept
};
static_assert(sizeof(Shared) % 16 == 0, "the slice's vectors are aligned");

// x times `total` for x in [0, 1), rounded down or up: exact, in whole numbers (fp64 arithmetic is
// two lanes a clock here).
__device__ __forceinline__ u64 share(float x, u64 total, bool up) {
  const u32 bits = __float_as_uint(x), e = bits >> 23;
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;  // x = m 2^-s
  const int s = 150 - max((int)e, 1);                                   // 24 .. 149
  const u64 hi = __umul64hi(m, total), lo = m * total;
  if (s >= 128) return up && (hi | lo) ? 1 : 0;
  u64 q, rest;
  if (s >= 64) {
    q = s == 64 ? hi : hi >> (s - 64);
    rest = lo | (s == 64 ? 0 : hi << (128 - s));
  } else {
    q = lo >> s | hi << (64 - s);
    rest = lo << (64 - s);
  }
  return q + (up && rest ? 1 : 0);
}

// Orders logits as unsigned numbers: 32 bits of an fp32 value, 16 of a bf16 one. A value is as far
// from 2^31 as its magnitude's bits say, so the two zeros share a key and neighbouring keys are
// neighbouring values: a bound may be any key, and comparing values is the same as comparing keys.
template <typename T>
__device__ __forceinline__ u32 key_of(float x) {
  const u32 b = __float_as_uint(x), k = b >> 31 ? 0u - b : b + 0x80000000u;
  return sizeof(T) == 2 ? k >> 16 : k;
}
template <typename T>
__device__ __forceinline__ float value_of(u32 key) {
  const u32 k = sizeof(T) == 4 ? key : key << 16;
  return __uint_as_float(k >> 31 ? k - 0x80000000u : 0u - k);
}

// Weights of one row.
struct Weights {
  float top, hi, lo;   // the maximum; log2(e) / temperature
  const Powers* table;

  // -log2 of the weight, y + rest; kRange or more (or NaN): weight 0
  __device__ __forceinline__ float distance(float l, float& rest) const {
    const float d = top - l, b = d - top;
    const float err = (top - (d - b)) - (l + b);  // top - l = d + err
    const float y = d * hi;
    rest = fmaf(err, hi, fmaf(d, lo, fmaf(d, hi, -y)));
    return y;
  }
  __device__ __forceinline__ float distance(float l) const {
    return (top - l) * hi;
  }
  // No branches: a thread's elements are worked out side by side.
  __device__ __forceinline__ u64 operator()(float l) const {
    float rest;
    const float y = distance(l, rest), held = fminf(y, kRange);
    constexpr float kMagic = 0x1.8p23f;  // 32 y to the nearest whole number, in the low bits
    const float shifted = fmaf(held, 32.f, kMagic);
    const u32 n = __float_as_uint(shifted) & 0x7ffu;
    const float r = fmaf(shifted - kMagic, -1.f / 32.f, held) + rest;  // the difference is exact
    // 2^-r - 1, |r| <= 1/64: powers of r ln 2 over factorials, the next one below 2^-39
    float q = fmaf(r, 0.0096181291f, -0.0555041087f);
    q = fmaf(r, q, 0.2402265070f);
    q = fmaf(r, q, -0.6931471806f);
    const u32 w = table->whole[n & 31] +
                  (u32)__float2int_rn(__uint_as_float(table->factor[n & 31]) * (r * q));
    return y < kRange ? (u64)w << 13 >> (n >> 5) : 0;
  }
  // The same for two logits with the same roundings, half of the instructions in pairs.
  __device__ __forceinline__ void two(float l0, float l1, u64 (&w)[2]) const {
    const f32x2 l = pair(l0, l1), t = both(top), minus = both(-1.f);
    const f32x2 d = fma2(l, minus, t), b = add2(d, both(-top));
    const f32x2 err = fma2(add2(l, b), minus, fma2(fma2(b, minus, d), minus, t));
    const f32x2 y = mul2(d, both(-hi));
    const f32x2 rest = fma2(err, both(hi), fma2(d, both(lo), fma2(d, both(hi), y)));
    float y0, y1;  // the distances, negated
    unpair(y, y0, y1);
    const f32x2 held = pair(fmaxf(y0, -kRange), fmaxf(y1, -kRange));
    constexpr float kMagic = 0x1.8p23f;
    const f32x2 shifted = fma2(held, both(-32.f), both(kMagic));
    float s0, s1;
    unpair(shifted, s0, s1);
    const u32 n0 = __float_as_uint(s0) & 0x7ffu, n1 = __float_as_uint(s1) & 0x7ffu;
    const f32x2 r = fma2(fma2(add2(shifted, both(-kMagic)), both(1.f / 32.f), held), minus, rest);
    f32x2 q = fma2(r, both(0.0096181291f), both(-0.0555041087f));
    q = fma2(r, q, both(0.2402265070f));
    q = fma2(r, q, both(-0.6931471806f));
    const f32x2 f = pair(__uint_as_float(table->factor[n0 & 31]), __uint_as_float(table->factor[n1 & 31]));
    float e0, e1;
    unpair(mul2(f, mul2(r, q)), e0, e1);
    const u32 w0 = table->whole[n0 & 31] + (u32)__float2int_rn(e0);
    const u32 w1 = table->whole[n1 & 31] + (u32)__float2int_rn(e1);
    w[0] = y0 > -kRange ? (u64)w0 << 13 >> (n0 >> 5) : 0;
    w[1] = y1 > -kRange ? (u64)w1 << 13 >> (n1 >> 5) : 0;
  }
};

// A block's part of a row. A thread owns `each` neighbouring vectors (an odd number of them, so that
// the lanes' reads do not meet in a bank): sums over threads run in the order of the row.
template <typename T>
struct Slice {
  static constexpr int N = Vec<T>::N;
  const Vec<T>* data;
  int vecs, per_thread;
  u32 first;      // place of the block's first element in the row
  // f(value, place) for every element
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const int v1 = min(vecs, ((int)threadIdx.x + 1) * per_thread);
    for (int v = threadIdx.x * per_thread; v < v1; ++v) {
      float x[N];
      unpack(data[v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) f(x[i], first + v * N + i);
    }
  }
  // f(two values, place of the first) for every two elements
  template <class F>
  __device__ __forceinline__ void twos(F f) const {
    const int v1 = min(vecs, ((int)threadIdx.x + 1) * per_thread);
    for (int v = threadIdx.x * per_thread; v < v1; ++v) {
      float x[N];
      unpack(data[v], x);
#pragma unroll
      for (int i = 0; i < N; i += 2) f(x[i], x[i + 1], first + v * N + i);
    }
  }
  // f(value, place) for the elements that are wanted, where they are few: looked for side by side,
  // then taken one by one.
  template <class Want, class F>
  __device__ __forceinline__ void some(Want want, F f) const {
    const int v1 = min(vecs, ((int)threadIdx.x + 1) * per_thread);
    for (int v = threadIdx.x * per_thread; v < v1; ++v) {
      float x[N];
      unpack(data[v], x);
      u32 mask = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) mask |= want(x[i], first + v * N + i) ? 1u << i : 0;
      while (mask) {
        const int i = __ffs(mask) - 1;
        mask &= mask - 1;
        f(to_f32(reinterpret_cast<const T*>(data + v)[i]), first + v * N + i);
      }
    }
  }
};

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ u64 warp_upto(u64 v) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// Everything below is called by all threads of all blocks of a cluster.
template <typename T>
struct Row {
  cg::cluster_group cluster;
  Shared& sh;
  Slice<T> slice;
  Weights weight;
  int turn = 0;

  __device__ __forceinline__ Row(Shared& s) : cluster(cg::this_cluster()), sh(s) {}

  // The row of cluster j: rows with top-p, which take the longest, come first.
  __device__ __forceinline__ int place_of(const SampleArgs& p, int j) {
    const int per = (p.num_rows + kThreads - 1) / kThreads;
    const int first = min(p.num_rows, (int)threadIdx.x * per), last = min(p.num_rows, first + per);
    const auto is_long = [&](int n) {
      return p.top_p[n] < 1.f && !(p.temperature && p.temperature[n] == 0.f);
    };
    int mine = 0;
    for (int n = first; n < last; ++n) mine += is_long(n);
    u64 all;
    const int front = (int)scan((u64)mine, all), others = first - front;
    const bool want = j < (int)all;
    const int from = want ? front : (int)all + others, have = want ? mine : last - first - mine;
    if (from <= j && j < from + have) {
      int at = from;
      for (int n = first; n < last; ++n)
        if (is_long(n) == want && at++ == j) sh.row = n;
    }
    __syncthreads();
    return sh.row;
  }

  // Every block's value (thread 0's): lane r of every warp has block r's, others 0. Read side by side:
  // a read from another block takes about 300 ns.
  __device__ __forceinline__ u64 exchange(u64 mine) {
    if (threadIdx.x == 0) sh.box[turn] = mine;
    cluster.sync();
    const unsigned lane = threadIdx.x % 32;
    const u64 v = lane < cluster.num_blocks() ? *cluster.map_shared_rank(&sh.box[turn], lane) : 0;
    turn ^= 1;
    return v;
  }
  __device__ __forceinline__ u64 in_front(u64 of_block) {  // of exchanged values, those of the blocks in front
    return warp_sum(threadIdx.x % 32 < cluster.block_rank() ? of_block : 0);
  }

  // Sum in front of this thread, and of the whole block.
  __device__ __forceinline__ u64 scan(u64 v, u64& all) {
    const u64 upto = warp_upto(v);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    __syncthreads();
    if (lane == 31) sh.warp_weight[warp] = upto;
    __syncthreads();
    const u64 w = warp_upto(lane < kWarps ? sh.warp_weight[lane] : 0);
    all = __shfl_sync(0xffffffffu, w, kWarps - 1);
    const u64 front = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp > 0 ? front : 0) + upto - v;
  }
  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_weight[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_sum(threadIdx.x % 32 < kWarps ? sh.warp_weight[threadIdx.x % 32] : 0);
  }
  __device__ __forceinline__ u64 cluster_sum(u64 v) {
    return warp_sum(exchange(block_sum(v)));
  }
  __device__ __forceinline__ static u64 warp_max(u64 x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const u64 o = __shfl_xor_sync(0xffffffffu, x, off);
      x = o > x ? o : x;
    }
    return x;
  }
  __device__ __forceinline__ u64 block_max(u64 v) {
    v = warp_max(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_weight[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_max(threadIdx.x % 32 < kWarps ? sh.warp_weight[threadIdx.x % 32] : 0);
  }

  __device__ __forceinline__ static float bins_of(float y) { return y * (kBins / kRange); }
  __device__ __forceinline__ static u32 bin_of(float y) {
    return min((u32)bins_of(y), (u32)kBins - 1);
  }

  // The cluster's counts of this thread's bins.
  __device__ __forceinline__ void counts(u32* mine, u32 (&c)[kBinsOf]) {
    uint4 o[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      o[r] = make_uint4(0, 0, 0, 0);
      if (r < cluster.num_blocks())
        o[r] = reinterpret_cast<const uint4*>(cluster.map_shared_rank(mine, r))[threadIdx.x];
    }
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) c[i] = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      c[0] += o[r].x;
      c[1] += o[r].y;
      c[2] += o[r].z;
      c[3] += o[r].w;
    }
  }

  // The bin at which the cumulative count reaches goal (`before`: what lies in front of the bins), and
  // the tokens in all; nothing found: bin kBins.
  __device__ __forceinline__ Found find(const u32 (&c)[kBinsOf], u32 before, u64 goal, u64& all) {
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) sum += c[i];
    u64 at = scan(sum, all) + before;
    if (threadIdx.x == 0) sh.found.bin = kBins;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      if (at < goal && goal <= at + c[i]) sh.found = {0, (u32)(threadIdx.x * kBinsOf + i), (u32)at, c[i]};
      at += c[i];
    }
    __syncthreads();
    return sh.found;
  }

  // The tokens in front of the bins first .. last, and in them.
  __device__ __forceinline__ Found tokens(const u32 (&c)[kBinsOf], u32 first, u32 last) {
    u64 v = 0;  // front and inside, 32 bits each
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      const u32 b = threadIdx.x * kBinsOf + i;
      v += b < first ? (u64)c[i] << 32 : b <= last ? c[i] : 0;
    }
    v = block_sum(v);
    return {0, first, (u32)(v >> 32), (u32)v};
  }

  // The bins first .. last, one of which the cumulative weight reaches goal in, from bounds of the
  // bins' weights: goal lies between least(sums of lo, of hi) and most(...).
  template <class Goal>
  __device__ __forceinline__ void window(const u64 (&lo)[kBinsOf], const u64 (&hi)[kBinsOf], u64 before,
                                         Goal goal, u32& first, u32& last) {
    u64 sum_hi = 0, sum_lo = 0, all_hi, all_lo, least, most;
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      sum_hi += hi[i];
      sum_lo += lo[i];
    }
    u64 at_hi = scan(sum_hi, all_hi) + before, at_lo = scan(sum_lo, all_lo) + before;
    goal(all_lo, all_hi, least, most);
    if (threadIdx.x == 0) {
      sh.window[0] = 0;
      sh.window[1] = kBins - 1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      if (at_hi < least && least <= at_hi + hi[i]) sh.window[0] = threadIdx.x * kBinsOf + i;
      if (at_lo < most && most <= at_lo + lo[i]) sh.window[1] = threadIdx.x * kBinsOf + i;
      at_hi += hi[i];
      at_lo += lo[i];
    }
    __syncthreads();
    first = sh.window[0];
    last = sh.window[1];
  }

  // The first place at which the cumulative g passes target, given this thread's sum of g and what
  // lies in front of it. One warp finds it and runs `got` on one of its lanes.
  template <class G, class Got>
  __device__ __forceinline__ void select(u64 target, u64 front, u64 sum, G g, Got got) {
    constexpr int N = Slice<T>::N;
    const u32 owner = __ballot_sync(0xffffffffu, front <= target && target < front + sum);
    if (owner == 0) return;
    const int lane = threadIdx.x % 32, src = __ffs(owner) - 1;
    u64 at = __shfl_sync(0xffffffffu, front, src);
    const int v0 = (threadIdx.x - lane + src) * slice.per_thread;
    const int items = (min(slice.vecs, v0 + slice.per_thread) - v0) * N;
    const T* data = reinterpret_cast<const T*>(slice.data + v0);
    for (int i0 = 0; i0 < items; i0 += 32) {
      const int i = i0 + lane;
      const u32 place = slice.first + v0 * N + i;
      const u64 w = i < items ? g(to_f32(data[i]), place) : 0;
      const u64 upto = at + warp_upto(w);
      if (upto - w <= target && target < upto) got(place, w);
      at = __shfl_sync(0xffffffffu, upto, 31);
      if (target < at) return;
    }
  }

  // f(weight, value) for all tokens, or for those that are wanted, about `count` of the cluster's. A weight of its
  // own takes a lane some 60 instructions with the others waiting, one of two 22: where every eighth
  // token is wanted, all are worked out.
  template <class F>
  __device__ __forceinline__ void weigh_all(F f) const {
    slice.twos([&](float x0, float x1, u32) {
      u64 w[2];
      weight.two(x0, x1, w);
      f(w[0], x0);
      f(w[1], x1);
    });
  }
  template <class Want, class F>
  __device__ __forceinline__ void weigh(u32 count, Want want, F f) const {
    if (count / 4 < (u32)(slice.vecs * Slice<T>::N / 32) * cluster.num_blocks()) {
      slice.some(want, [&](float x, u32) { f(weight(x), x); });
      return;
    }
    slice.twos([&](float x0, float x1, u32 at) {
      u64 w[2];
      weight.two(x0, x1, w);
      if (want(x0, at)) f(w[0], x0);
      if (want(x1, at + 1)) f(w[1], x1);
    });
  }
  // The weight of the keys above `low`, up to `high`, about `count` tokens.
  __device__ __forceinline__ u64 weight_between(u32 count, u32 low, u32 high) {
    u64 sum = 0;
    const float v0 = value_of<T>(low), v1 = value_of<T>(high);
    weigh(count, [&](float x, u32) { return x > v0 && x <= v1; }, [&](u64 w, float) { sum += w; });
    return cluster_sum(sum);
  }

  // The keys lo .. hi whose distances lie in the bins first .. last: distances fall as keys rise. One
  // warp looks for either end, in 32 places at a time.
  __device__ __forceinline__ void keys_of(u32 first, u32 last, u32& hi, u32& lo) {
    const u32 top = key_of<T>(weight.top);
    const float to = last < kBins - 1 ? (float)(last + 1) : INFINITY;
    // at the least key for which it holds, at `top` if for none below
    const auto least = [&](auto holds) {
      u32 a = key_of<T>(-INFINITY) + 1, b = top;
      while (a < b) {
        const u32 step = (b - a) / 32 + 1, k = (u32)min((u64)b, a + (u64)(threadIdx.x % 32) * step);
        const u32 yes = __ballot_sync(0xffffffffu, k == b || holds(weight.distance(value_of<T>(k))));
        const u32 n = yes ? __ffs(yes) - 1 : 32;
        const u32 end = (u32)min((u64)b, a + (u64)n * step);
        if (n > 0) a = (u32)min((u64)b, a + (u64)(n - 1) * step + 1);
        if (n < 32) b = end;
      }
      return a;
    };
    if (threadIdx.x < 64) {
      u32 k;
      if (threadIdx.x < 32) {
        k = least([&](float y) { return y < kRange && bins_of(y) < to; });
      } else {
        k = first == 0 ? top : least([&](float y) { return bins_of(y) < (float)first; }) - 1;
      }
      if (threadIdx.x % 32 == 0) sh.window[threadIdx.x / 32] = k;
    }
    __syncthreads();
    lo = sh.window[0];
    hi = sh.window[1];
  }
  // The finer bins of the keys lo .. hi.
  __device__ __forceinline__ static int shift_of(u32 lo, u32 hi) {
    return max(0, 21 - __clz(hi - lo));  // (hi - lo) >> shift is below 2,048
  }
  __device__ __forceinline__ void clear_finer() {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.finer[i] = 0;
    __syncthreads();
  }

  // The last token kept, whose key lies in lo .. hi: the one at which the count (or weight) of the order
  // reaches goal. f: what lies in front of those keys, and the tokens in them. `counted`: the finer bins
  // hold their counts.
  __device__ __forceinline__ Entry resolve(u32 lo, u32 hi, Found f, bool by_weight, u64 goal,
                                           bool counted) {
    float above = value_of<T>(lo), below = value_of<T>(hi);
    const auto member = [&](float x, u32) { return x >= above && x <= below; };
    while (f.count > kList && lo < hi) {  // the keys left are halved at least
      const int shift = shift_of(lo, hi);
      if (!counted) {
        clear_finer();
        slice.each([&](float x, u32 at) {
          if (member(x, at)) atomicAdd(&sh.finer[(hi - key_of<T>(x)) >> shift], 1u);
        });
      }
      counted = false;
      cluster.sync();
      u32 c[kBinsOf], b0, b1;
      u64 front = 0;  // this thread's part of the weight in front of bin b0
      counts(sh.finer, c);
      if (by_weight) {
        // a bin's weights lie between those of its ends, to twice their own error
        u64 least[kBinsOf], most[kBinsOf];
#pragma unroll
        for (int i = 0; i < kBinsOf; ++i) {
          const u32 k = hi - ((threadIdx.x * kBinsOf + i) << shift);
          const u64 w0 = c[i] ? weight(value_of<T>(k)) : 0;
          const u64 w1 = c[i] ? weight(value_of<T>(max(lo, k - ((1u << shift) - 1)))) : 0;
          most[i] = c[i] * (w0 + (shift ? (w0 >> 26) + 2 : 0));
          least[i] = c[i] * (w1 - (shift ? min(w1, (w1 >> 26) + 2) : 0));
        }
        window(least, most, f.before_weight, [&](u64, u64, u64& a, u64& b) { a = b = goal; }, b0, b1);
#pragma unroll
        for (int i = 0; i < kBinsOf; ++i) front += threadIdx.x * kBinsOf + i < b0 ? most[i] : 0;
      } else {
        u64 all;
        b0 = b1 = find(c, f.before, goal, all).bin;
      }
      b1 = min(b1, (hi - lo) >> shift);
      const Found in = tokens(c, b0, b1);
      f.before += in.before;
      f.count = in.count;
      const u32 top = hi, span = hi - lo;
      lo = max(lo, hi - (b1 << shift) - ((1u << shift) - 1));
      hi -= b0 << shift;
      // a bin of one key has its weight times its count
      if (by_weight) f.before_weight += shift ? weight_between(in.before, hi, top) : block_sum(front);
      if (hi - lo > span / 2) {  // bounds too wide to tell: halve the keys by exact sums
        const u32 mid = lo + (hi - lo) / 2;
        const float v0 = value_of<T>(mid), v1 = value_of<T>(hi);
        u32 here = 0;
        slice.each([&](float x, u32) { here += x > v0 && x <= v1; });
        const u64 n = cluster_sum(here);
        const u64 w = by_weight ? weight_between((u32)n, mid, hi) : n;
        if ((by_weight ? f.before_weight : f.before) + w >= goal) {
          lo = mid + 1;
          f.count = (u32)n;
        } else {
          hi = mid;
          f.before += (u32)n;
          f.before_weight += by_weight ? w : 0;
          f.count -= (u32)n;
        }
      }
      above = value_of<T>(lo);
      below = value_of<T>(hi);
      cluster.sync();  // the bins have been read
    }
    if (f.count <= kList) {
      if (threadIdx.x == 0) sh.list.count = 0;
      __syncthreads();
      slice.some(member, [&](float x, u32 at) {
        sh.list.mine[atomicAdd(&sh.list.count, 1u)] = {by_weight ? weight(x) : 1, key_of<T>(x), at};
      });
      cluster.sync();
      // the lists one behind another: entry threadIdx.x of them all
      const unsigned lane = threadIdx.x % 32;
      const u32 n = lane < cluster.num_blocks() ? cluster.map_shared_rank(&sh.list, lane)->count : 0;
      u32 from = 0, i = threadIdx.x;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const u32 k = __shfl_sync(0xffffffffu, n, r);
        if (from == (u32)r && i >= k) {
          i -= k;
          ++from;
        }
      }
      if (threadIdx.x < f.count) sh.list.all[threadIdx.x] = cluster.map_shared_rank(&sh.list, from)->mine[i];
      __syncthreads();
      // four threads an entry
      constexpr int kPer = kThreads / kList;
      const u32 mine = threadIdx.x / kPer;
      const Entry me = sh.list.all[min(mine, f.count - 1)];
      u64 front = 0;
      for (u32 j = threadIdx.x % kPer; j < f.count; j += kPer) {
        const Entry o = sh.list.all[j];
        front += o.key > me.key || (o.key == me.key && o.at < me.at) ? o.weight : 0;
      }
#pragma unroll
      for (int off = 1; off < kPer; off <<= 1) front += __shfl_xor_sync(0xffffffffu, front, off);
      front += by_weight ? f.before_weight : f.before;
      if (mine < f.count && threadIdx.x % kPer == 0 && front < goal && goal <= front + me.weight)
        sh.chosen = me;
      __syncthreads();
    } else {  // all equal: the first of them, by place
      u64 n = goal - f.before;
      if (by_weight) {
        const u64 each = weight(value_of<T>(lo));
        n = (goal - f.before_weight + each - 1) / each;
      }
      u32 mine = 0;
      u64 all;
      slice.each([&](float x, u32) { mine += x == above; });
      const u64 inside = scan(mine, all);
      const u64 front = in_front(exchange(all));
      select(n - 1, front + inside, mine, [&](float x, u32) { return (u64)(x == above); },
             [&](u32 at, u64) {
               for (unsigned r = 0; r < cluster.num_blocks(); ++r)
                 *cluster.map_shared_rank(&sh.chosen, r) = {0, lo, at};
             });
      cluster.sync();
    }
    return sh.chosen;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs p, int vecs_of_block, bool ordered) {
  extern __shared__ __align__(16) unsigned char memory[];
  constexpr int N = Vec<T>::N;
  Shared& sh = *reinterpret_cast<Shared*>(memory);
  Vec<T>* data = reinterpret_cast<Vec<T>*>(memory + sizeof(Shared));
  Row<T> row(sh);
  const unsigned rank = row.cluster.block_rank(), blocks = row.cluster.num_blocks();
  const int r = ordered ? row.place_of(p, blockIdx.x / blocks) : blockIdx.x / blocks;
  const int V = p.vocab;
  const T* logits = static_cast<const T*>(p.logits) + (int64_t)r * p.stride;
  // places count from the 16-byte boundary at or in front of the row
  const int shift = (int)(reinterpret_cast<uintptr_t>(logits) % 16 / sizeof(T));
  const int vecs = (shift + V + N - 1) / N, v0 = rank * vecs_of_block;
  const int mine = max(0, min(vecs_of_block, vecs - v0));

  // the slice; what lies outside the row is -inf
  for (int v = threadIdx.x; v < mine; v += kThreads) {
    const int i0 = (v0 + v) * N - shift;
    const u32 to = (u32)__cvta_generic_to_shared(data + v);
    if (i0 >= 0 && i0 + N <= V) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(logits + i0) : "memory");
    } else {
      T* e = reinterpret_cast<T*>(data + v);
      for (int i = 0; i < N; ++i)
        e[i] = i0 + i >= 0 && i0 + i < V ? logits[i0 + i] : from_f32<T>(-INFINITY);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (threadIdx.x < 32) {
    sh.table.whole[threadIdx.x] = kPowers.whole[threadIdx.x];
    sh.table.factor[threadIdx.x] = kPowers.factor[threadIdx.x];
  }
  const float temp = p.temperature ? p.temperature[r] : 1.f;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float u = p.u[r];
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  row.slice = {data, mine, ((mine + kThreads - 1) / kThreads) | 1, (u32)v0 * N};

  // the maximum and its first place
  float most = -INFINITY;
  u32 most_at = 0xffffffffu;
  row.slice.each([&](float x, u32 at) {
    if (x > most) {
      most = x;
      most_at = at;
    }
  });
  u64 best = most > -INFINITY ? (u64)key_of<T>(most) << 32 | (u32)~most_at : 0;
  best = row.block_max(best);
  best = Row<T>::warp_max(row.exchange(best));
  const float top = best == 0 ? -INFINITY : value_of<T>((u32)(best >> 32));
  const bool bad = best == 0 || !(temp >= 0.f) || top_p != top_p || min_p != min_p || u != u;
  if (bad || temp == 0.f) {
    if (rank == 0 && threadIdx.x == 0) {
      if (bad) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
      p.token[r] = bad ? -1 : (int32_t)(~(u32)best) - shift;
      if (p.logprob) p.logprob[r] = bad ? -INFINITY : 0.f;
    }
    row.cluster.sync();  // no block leaves while another reads its box
    return;
  }
  // log2(e) / temperature as two fp32 terms: the quotient and its remainder's
  constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = (float)(1.4426950408889634074 - kLog2e);
  float hi = __fdiv_rn(kLog2e, temp);
  float lo = __fdiv_rn(fmaf(-hi, temp, kLog2e) + kLog2eRest, temp);
  if (!(hi <= 1e30f)) hi = 1e30f;
  if (hi == 1e30f || temp > 1e30f) lo = 0.f;
  row.weight = {top, hi, lo, &sh.table};
  if (top == INFINITY) {  // such logits share the row: zeros among -inf, all with weight 1
    for (int v = threadIdx.x; v < mine; v += kThreads) {
      T* e = reinterpret_cast<T*>(data + v);
      for (int i = 0; i < N; ++i) e[i] = from_f32<T>(to_f32(e[i]) == INFINITY ? 0.f : -INFINITY);
    }
    row.weight = {0.f, 1.f, 0.f, &sh.table};
    __syncthreads();
  }

  // the last token that top-k and top-p keep; until then every one is
  bool cut = false;
  u32 num_kept = (u32)V;  // about as many, or more
  float last_value = -INFINITY;
  u32 last_at = 0xffffffffu;
  const auto cut_at = [&](const Entry& e) {
    cut = true;
    last_value = value_of<T>(e.key);
    last_at = e.at;
  };
  const auto inside_of = [&](float x, u32 at) {
    return x > last_value || (x == last_value && at <= last_at);
  };
  u64 floor_weight = 0;
  const auto kept = [&](float x, u32 at) -> u64 {
    const u64 w = row.weight(x);
    return inside_of(x, at) && w >= floor_weight ? w : 0;
  };
  const bool by_k = top_k > 0 && top_k < V, by_p = top_p < 1.f;
  if (by_k || by_p) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.count[i] = 0;
    __syncthreads();
    row.slice.each([&](float x, u32) {
      const float y = row.weight.distance(x);
      if (y < kRange) atomicAdd(&sh.count[Row<T>::bin_of(y)], 1u);
    });
    row.cluster.sync();
    u32 c[kBinsOf];
    u64 all;
    u32 limit = kBins - 1;  // the last bin with a token kept, where top-k cuts one
    row.counts(sh.count, c);
    if (by_k) {
      const Found f = row.find(c, 0, (u64)top_k, all);
      if (all > (u64)top_k) {
        u32 lo, hi;
        row.keys_of(f.bin, f.bin, hi, lo);
        cut_at(row.resolve(lo, hi, f, false, (u64)top_k, false));
        limit = f.bin;
        num_kept = (u32)top_k;
      }
    }
    if (by_p) {
      // a bin's weights lie between 2^44 times 2^-(its ends), to 2^-16 (a distance is off by 2^-18);
      // of the last bin some tokens may be left out
      u64 most[kBinsOf], least[kBinsOf];
#pragma unroll
      for (int i = 0; i < kBinsOf; ++i) {
        const u32 b = threadIdx.x * kBinsOf + i;
        const float y = (float)b * (kRange / kBins);
        most[i] = b <= limit ? c[i] * ((u64)(exp2f(44.f - y) * (1.f + 0x1p-16f)) + 1) : 0;
        least[i] = b < limit || !cut
                       ? c[i] * (u64)(exp2f(44.f - y - kRange / kBins) * (1.f - 0x1p-16f)) : 0;
      }
      const auto share_of = [&](u64 total) {
        return top_p > 0.f ? max(share(top_p, total, true), (u64)1) : 1;
      };
      u32 first, last;
      row.window(least, most, 0, [&](u64 lo, u64 hi, u64& a, u64& b) {
        a = share_of(lo);
        b = share_of(hi);
      }, first, last);
      last = min(last, limit);
      Found f = row.tokens(c, first, last);
      u32 key_lo, key_hi;
      row.keys_of(first, last, key_hi, key_lo);
      const float above = value_of<T>(key_lo), below = value_of<T>(key_hi);
      u64 front = 0, total = 0;
      const auto add = [&](u64 w, float x) {
        total += w;
        front += x > below ? w : 0;
      };
      if (cut) {
        row.weigh(num_kept, inside_of, add);
      } else {
        row.clear_finer();
        const int shift = Row<T>::shift_of(key_lo, key_hi);
        row.weigh_all([&](u64 w, float x) {
          add(w, x);
          if (x >= above && x <= below) atomicAdd(&sh.finer[(key_hi - key_of<T>(x)) >> shift], 1u);
        });
      }
      f.before_weight = row.cluster_sum(front);
      num_kept = min(num_kept, f.before + f.count);
      const u64 goal = share_of(row.cluster_sum(total));
      cut_at(row.resolve(key_lo, key_hi, f, true, goal, !cut));
    }
  }
  if (min_p > 0.f) floor_weight = min_p < 1.f ? share(min_p, 1ull << 44, true) : 1ull << 44;
  u64 sum = 0;
  const auto add = [&](u64 w, float) { sum += w >= floor_weight ? w : 0; };
  if (cut) row.weigh(num_kept, inside_of, add);
  else row.weigh_all(add);
  u64 all;
  const u64 inside = row.scan(sum, all), of_block = row.exchange(all);
  const u64 front = row.in_front(of_block), total = warp_sum(of_block);
  const u64 target = u > 0.f ? (u < 1.f ? share(u, total, false) : total - 1) : 0;
  row.select(target, front + inside, sum, kept, [&](u32 at, u64 w) {
    p.token[r] = (int32_t)at - shift;
    if (p.logprob) {
      // the quotient's fp32 value, and what that leaves
      const double q = (double)w / (double)total;
      const float f = (float)q;
      p.logprob[r] = logf(f) + (float)(q - (double)f) / f;
    }
  });
  row.cluster.sync();  // no block leaves while another reads its box
}

template <typename T>
int launch(const SampleArgs& a, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int vecs = (a.vocab + N - 1) / N + 1;  // one more where the row starts off a boundary
  const auto share = [&](int blocks) { return (vecs + blocks - 1) / blocks; };
  const auto memory = [&](int blocks) { return sizeof(Shared) + (size_t)share(blocks) * 16; };
  // Eight blocks a row, unless fewer still give every SM two (256 rows of 151,936 bf16 logits, top-p:
  // 372 us with eight, 237 with four; fp32, of which four leave an SM one block: 427 and 419, without
  // a filter 119 and 132) or the row is short.
  int blocks = kMaxCluster;
  while (blocks > 1 && (vecs <= kThreads || ((int64_t)a.num_rows * blocks / 2 >= 2 * 152 &&
                                             2 * (memory(blocks / 2) + 1024) <= kMostMemory + 1024)))
    blocks /= 2;
  const int of_block = share(blocks);
  // Rows are put in order where not all run at once, and a thread looks at few of them (256 bf16 rows, a
  // quarter of them with top-p: 158 us as they stand, 139 in order; all with top-p: 233 and 236).
  const bool ordered = a.top_p && (int64_t)a.num_rows * blocks > 2 * 152 && a.num_rows <= 8 * kThreads;
  const size_t bytes = memory(blocks);
  static std::atomic<int> done[kMaxDevices];
  const int e = configure_once(done, [] {
    return (int)cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kMostMemory);
  });
  if (e != 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_rows * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)blocks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, of_block, ordered);
}

}  // namespace

int launch_sample(const SampleArgs& a, void* stream) {
  if (a.num_rows == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace gdn
