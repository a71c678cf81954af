// gdn_sample.cu — a token from every row of logits: temperature, top-k, top-p and min-p, then the
// inverse of the kept tokens' cumulative weights at a given random number.
//
// A row belongs to one cluster of blocks: each holds a slice of it in shared memory, so the logits
// are read from memory once, however many passes the filters take. Nothing is sorted: every filter
// keeps a beginning of the order (falling logits, equal ones by rising index), so it is enough to
// find the last token kept. A histogram over the distance from the maximum gives its bin; the
// bin's tokens, when few, are ranked against one another, else their bits are cut into 2,048 finer
// bins, until they are few or all equal.
//
// Weights are integers, 2^44 for the maximum, so that their sums are exact and depend on no order:
// exp((l - m) / T) = 2^-y, and 2^-y is a table entry times 1 + a polynomial of the last 1/64 of y.
// l - m and y carry a second fp32 term, since errors of 2^-24 would move borders that u or
// top_p may fall next to: weights are right to 2^-30 (2^-32 from the polynomial, the rest from y).
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
constexpr int kList = kThreads;                          // tokens ranked against one another
constexpr float kRange = 44.f;                           // 2^-44 of the maximum: weight 1
constexpr int kMaxCluster = 8;

struct Bins {
  u64 weight[kBins];
  u32 count[kBins];
};
struct Entry {
  u64 weight;
  u32 key, at;
};
struct List {
  Entry mine[kList], all[kList];
  u32 count;
};
struct Found {
  u64 before_weight, weight;
  u32 bin, before, count;
};
struct Shared {
  Bins bins;
  union {
    Bins finer;
    List list;
  };
  u64 table[64];      // 2^(36 - j/64)
  float factor[64];   // the same
  u64 box[2];         // what the cluster's blocks tell one another, in turns
  u64 warp_weight[kWarps];
  u32 warp_count[kWarps];
  Found found;
  Entry chosen;       // weight: of all tokens up to the chosen one
};

// Orders floats as unsigned numbers (-0 as 0).
__device__ __forceinline__ u32 key_of(float x) {
  const u32 b = __float_as_uint(x + 0.f);
  return b ^ ((u32)((int32_t)b >> 31) | 0x80000000u);
}

// Weights of one row.
struct Weights {
  float top, hi, lo;   // the maximum; log2(e) / temperature
  bool infinite;       // the maximum is +inf: such logits share the row
  const u64* table;
  const float* factor;

  // -log2 of the weight, y + rest; kRange or more (or NaN): weight 0
  __device__ __forceinline__ float distance(float l, float& rest) const {
    if (infinite) {
      rest = 0.f;
      return l == top ? 0.f : 2.f * kRange;
    }
    const float d = top - l, b = d - top;
    const float err = (top - (d - b)) - (l + b);  // top - l = d + err
    const float y = d * hi;
    rest = fmaf(err, hi, fmaf(d, lo, fmaf(d, hi, -y)));
    return y;
  }
  __device__ __forceinline__ float distance(float l) const {
    return infinite ? (l == top ? 0.f : 2.f * kRange) : (top - l) * hi;
  }
  __device__ __forceinline__ u64 operator()(float l) const {
    float rest;
    const float y = distance(l, rest);
    if (!(y < kRange)) return 0;
    const int n = (int)(y * 64.f);
    const float r = fmaf((float)n, -1.f / 64.f, y) + rest;  // the difference is exact
    // 2^-r - 1, r < 1/64: powers of r ln 2 over factorials, the next one below 2^-38
    float q = fmaf(r, 0.0096181291f, -0.0555041087f);
    q = fmaf(r, q, 0.2402265070f);
    q = fmaf(r, q, -0.6931471806f);
    q *= r;
    const int j = n & 63;
    const u64 w = table[j] + (u64)(int64_t)__float2int_rn(factor[j] * q);
    return (w << 8) >> (n >> 6);
  }
};

template <typename T>
struct Slice {
  static constexpr int N = Vec<T>::N;
  const Vec<T>* data;
  int vecs;       // of this block
  u32 first;      // place of its first element in the row
  // f(value, place) for every element
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
      float x[N];
      unpack(data[v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) f(x[i], first + v * N + i);
    }
  }
};

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
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

  // Every block's value (thread 0's), combined by f in the blocks' order.
  template <class F>
  __device__ __forceinline__ void exchange(u64 mine, F f) {
    if (threadIdx.x == 0) sh.box[turn] = mine;
    cluster.sync();
    for (unsigned r = 0; r < cluster.num_blocks(); ++r)
      f(r, *cluster.map_shared_rank(&sh.box[turn], r));
    turn ^= 1;
  }

  __device__ __forceinline__ u64 block_sum(u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_weight[threadIdx.x / 32] = v;
    __syncthreads();
    u64 s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sh.warp_weight[w];
    return s;
  }
  __device__ __forceinline__ u64 block_max(u64 v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const u64 o = __shfl_xor_sync(0xffffffffu, v, off);
      v = o > v ? o : v;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_weight[threadIdx.x / 32] = v;
    __syncthreads();
    u64 s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s = sh.warp_weight[w] > s ? sh.warp_weight[w] : s;
    return s;
  }

  __device__ __forceinline__ void clear(Bins& b) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      b.weight[i] = 0;
      b.count[i] = 0;
    }
    __syncthreads();
  }

  // Sums in front of this thread (exclusive), and of the whole block.
  __device__ __forceinline__ void scan(u32 c, u64 w, u32& before_c, u64& before_w, u32& all_c,
                                       u64& all_w) {
    u32 upc = c;
    u64 upw = w;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u32 a = __shfl_up_sync(0xffffffffu, upc, off);
      const u64 b = __shfl_up_sync(0xffffffffu, upw, off);
      if (lane >= off) {
        upc += a;
        upw += b;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sh.warp_count[warp] = upc;
      sh.warp_weight[warp] = upw;
    }
    __syncthreads();
    before_c = upc - c;
    before_w = upw - w;
    all_c = 0;
    all_w = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) {
        before_c += all_c;
        before_w += all_w;
      }
      all_c += sh.warp_count[i];
      all_w += sh.warp_weight[i];
    }
  }

  // The cluster's bins: the sums of all, and the first bin at which the count (or weight) reaches
  // a target, which may follow from the sums.
  template <class Target>
  __device__ __forceinline__ Found find(Bins& mine, bool by_weight, u32 before, u64 before_weight,
                                        Target target, u32& all_c, u64& all_w) {
    u32 c[kBinsOf] = {}, sum_c = 0, at_c;
    u64 w[kBinsOf] = {}, sum_w = 0, at_w;
    for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
      const Bins& b = *cluster.map_shared_rank(&mine, r);
#pragma unroll
      for (int i = 0; i < kBinsOf; ++i) {
        c[i] += b.count[threadIdx.x * kBinsOf + i];
        w[i] += b.weight[threadIdx.x * kBinsOf + i];
      }
    }
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      sum_c += c[i];
      sum_w += w[i];
    }
    scan(sum_c, sum_w, at_c, at_w, all_c, all_w);
    const u64 goal = target(all_c, all_w);
    at_c += before;
    at_w += before_weight;
#pragma unroll
    for (int i = 0; i < kBinsOf; ++i) {
      const u64 front = by_weight ? at_w : at_c, back = front + (by_weight ? w[i] : c[i]);
      if (front < goal && goal <= back)
        sh.found = {at_w, w[i], (u32)(threadIdx.x * kBinsOf + i), at_c, c[i]};
      at_c += c[i];
      at_w += w[i];
    }
    __syncthreads();
    return sh.found;
  }

  // The first place at which the cumulative g passes target (total: what it passes in the end).
  template <class G>
  __device__ __forceinline__ bool select(u64 target, u64 before, G g, u32& place, u64& value) {
    constexpr int N = Slice<T>::N;
    for (int v0 = 0; v0 < slice.vecs; v0 += kThreads) {
      const int v = v0 + threadIdx.x;
      float x[N];
      u64 w[N], sum = 0, at, all;
      if (v < slice.vecs) unpack(slice.data[v], x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        w[i] = v < slice.vecs ? g(x[i], slice.first + v * N + i) : 0;
        sum += w[i];
      }
      u32 none, none2;
      scan(0, sum, none, at, none2, all);
      at += before;
      if (at <= target && target < at + sum) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (at <= target && target < at + w[i]) {
            place = slice.first + v * N + i;
            value = w[i];
            return true;
          }
          at += w[i];
        }
      }
      before += all;
      if (target < before) return false;  // another thread has it
    }
    return false;
  }

  // The last token kept, when the bin `f` of the first histogram holds it: the one at which the
  // count (or weight) of the order reaches goal. at: its place; weight: of all up to it.
  __device__ __forceinline__ Entry resolve(Found f, bool by_weight, u64 goal) {
    u32 hi = 0, lo = 0xffffffffu;
    slice.each([&](float x, u32) {
      const float y = weight.distance(x);
      if (y < kRange && bin_of(y) == f.bin) {
        const u32 k = key_of(x);
        hi = max(hi, k);
        lo = min(lo, k);
      }
    });
    u32 inv = __reduce_max_sync(0xffffffffu, ~lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.warp_weight[threadIdx.x / 32] = (u64)hi << 32 | inv;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      hi = max(hi, (u32)(sh.warp_weight[w] >> 32));
      inv = max(inv, (u32)sh.warp_weight[w]);
    }
    exchange((u64)hi << 32 | inv, [&](unsigned, u64 o) {
      hi = max(hi, (u32)(o >> 32));
      inv = max(inv, (u32)o);
    });
    lo = ~inv;
    while (f.count > kList && lo < hi) {
      const int shift = max(0, 21 - __clz(hi - lo));  // (hi - lo) >> shift is below 2,048
      clear(sh.finer);
      slice.each([&](float x, u32) {
        const u32 k = key_of(x);
        if (k >= lo && k <= hi) {
          atomicAdd(&sh.finer.count[(hi - k) >> shift], 1u);
          atomicAdd(&sh.finer.weight[(hi - k) >> shift], weight(x));
        }
      });
      cluster.sync();
      u32 c;
      u64 w;
      f = find(sh.finer, by_weight, f.before, f.before_weight, [&](u32, u64) { return goal; }, c, w);
      hi -= f.bin << shift;
      lo = max(lo, hi - ((1u << shift) - 1));
      cluster.sync();  // the bins have been read
    }
    if (f.count <= kList) {
      if (threadIdx.x == 0) sh.list.count = 0;
      __syncthreads();
      slice.each([&](float x, u32 at) {
        const u32 k = key_of(x);
        if (k >= lo && k <= hi) sh.list.mine[atomicAdd(&sh.list.count, 1u)] = {weight(x), k, at};
      });
      cluster.sync();
      u32 i = threadIdx.x;
      for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
        const List& l = *cluster.map_shared_rank(&sh.list, r);
        const u32 n = l.count;
        if (i < n) {
          sh.list.all[threadIdx.x] = l.mine[i];
          break;
        }
        i -= n;
      }
      __syncthreads();
      if (threadIdx.x < f.count) {
        const Entry me = sh.list.all[threadIdx.x];
        u64 c = f.before, w = f.before_weight;
        for (u32 j = 0; j < f.count; ++j) {
          const Entry o = sh.list.all[j];
          if (o.key > me.key || (o.key == me.key && o.at < me.at)) {
            ++c;
            w += o.weight;
          }
        }
        const u64 front = by_weight ? w : c, back = front + (by_weight ? me.weight : 1);
        if (front < goal && goal <= back) sh.chosen = {w + me.weight, me.key, me.at};
      }
      __syncthreads();
    } else {  // all equal: the first of them, by place
      const u64 each = f.weight / f.count;
      const u64 n = by_weight ? (goal - f.before_weight + each - 1) / each : goal - f.before;
      u64 mine = 0, before = 0;
      slice.each([&](float x, u32) { mine += key_of(x) == lo; });
      mine = block_sum(mine);
      exchange(mine, [&](unsigned r, u64 o) { before += r < cluster.block_rank() ? o : 0; });
      u32 at;
      u64 one;
      if (before < n && n <= before + mine &&
          select(n - 1, before, [&](float x, u32) { return (u64)(key_of(x) == lo); }, at, one))
        for (unsigned r = 0; r < cluster.num_blocks(); ++r)
          *cluster.map_shared_rank(&sh.chosen, r) = {f.before_weight + n * each, lo, at};
      cluster.sync();
    }
    return sh.chosen;
  }

  __device__ __forceinline__ static u32 bin_of(float y) {
    return min((u32)(y * (kBins / kRange)), (u32)kBins - 1);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs p, int vecs_of_block) {
  extern __shared__ __align__(16) unsigned char memory[];
  constexpr int N = Vec<T>::N;
  Shared& sh = *reinterpret_cast<Shared*>(memory);
  Vec<T>* data = reinterpret_cast<Vec<T>*>(memory + sizeof(Shared));
  Row<T> row(sh);
  const unsigned rank = row.cluster.block_rank(), blocks = row.cluster.num_blocks();
  const int r = blockIdx.x / blocks;
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
  if (threadIdx.x < 64) {
    const double t = exp2(36.0 - threadIdx.x / 64.0);
    sh.table[threadIdx.x] = (u64)__double2ll_rn(t);
    sh.factor[threadIdx.x] = (float)t;
  }
  const float temp = p.temperature ? p.temperature[r] : 1.f;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  const int top_k = p.top_k ? p.top_k[r] : 0;
  const float u = p.u[r];
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  row.slice = {data, mine, (u32)v0 * N};

  // the maximum and its first place
  u64 best = 0;
  for (int v = threadIdx.x; v < mine; v += kThreads) {
    float x[N];
    unpack(data[v], x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (x[i] == x[i]) {
        const u64 k = (u64)key_of(x[i]) << 32 | (u32)~(u32)((v0 + v) * N + i);
        best = k > best ? k : best;
      }
    }
  }
  best = row.block_max(best);
  row.exchange(best, [&](unsigned, u64 o) { best = o > best ? o : best; });
  const u32 bits = (u32)(best >> 32);
  const float top = best == 0 ? -INFINITY
                              : __uint_as_float(bits ^ ((u32)((int32_t)~bits >> 31) | 0x80000000u));
  const bool bad = !(top > -INFINITY) || !(temp >= 0.f) || top_p != top_p || min_p != min_p || u != u;
  const bool out = rank == 0 && threadIdx.x == 0;
  if (bad || temp == 0.f) {
    if (out) {
      if (bad) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
      p.token[r] = bad ? -1 : (int32_t)(~(u32)best) - shift;
      if (p.logprob) p.logprob[r] = bad ? -INFINITY : 0.f;
    }
    row.cluster.sync();  // no block leaves while another reads its box
    return;
  }
  const double rate = fmin(1.4426950408889634074 / (double)temp, 1e30);
  const float hi = (float)rate;
  row.weight = {top, hi, (float)(rate - (double)hi), top == INFINITY, sh.table, sh.factor};

  // the last token that top-k and top-p keep; until then every one is
  u32 last_key = 0, last_at = 0xffffffffu;
  const bool by_k = top_k > 0 && top_k < V, by_p = top_p < 1.f;
  if (by_k || by_p) {
    row.clear(sh.bins);
    row.slice.each([&](float x, u32) {
      const float y = row.weight.distance(x);
      if (y < kRange) {
        const u32 b = Row<T>::bin_of(y);
        atomicAdd(&sh.bins.count[b], 1u);
        atomicAdd(&sh.bins.weight[b], row.weight(x));
      }
    });
    row.cluster.sync();
    u32 count;
    u64 total;
    if (by_k) {
      const Found f = row.find(sh.bins, false, 0, 0, [&](u32, u64) { return (u64)top_k; }, count, total);
      if (count > (u32)top_k) {
        const Entry e = row.resolve(f, false, top_k);
        last_key = e.key;
        last_at = e.at;
        total = e.weight;
      }
    }
    if (by_p) {
      u64 goal = 0, all_weight;
      const Found f = row.find(
          sh.bins, true, 0, 0,
          [&](u32, u64 all) {
            const u64 of = by_k ? total : all;
            const double g = ceil((double)top_p * (double)of);
            goal = g < 1.0 ? 1 : min((u64)g, of);
            return goal;
          },
          count, all_weight);
      const Entry e = row.resolve(f, true, goal);
      last_key = e.key;
      last_at = e.at;
    }
  }
  const double least = ceil(fmin((double)min_p, 1.0) * 17592186044416.0);  // 2^44
  const u64 floor_weight = least > 1.0 ? (u64)least : 1;
  const auto kept = [&](float x, u32 at) -> u64 {
    const u32 k = key_of(x);
    if (k < last_key || (k == last_key && at > last_at)) return 0;
    const u64 w = row.weight(x);
    return w >= floor_weight ? w : 0;
  };
  u64 sum = 0, before = 0, total = 0;
  row.slice.each([&](float x, u32 at) { sum += kept(x, at); });
  sum = row.block_sum(sum);
  row.exchange(sum, [&](unsigned i, u64 o) {
    if (i < rank) before += o;
    total += o;
  });
  const double goal = u > 0.f ? (double)u * (double)total : 0.0;
  const u64 target = goal >= (double)total ? total - 1 : min((u64)goal, total - 1);
  u32 at;
  u64 w;
  if (before <= target && target < before + sum && row.select(target, before, kept, at, w)) {
    p.token[r] = (int32_t)at - shift;
    if (p.logprob) p.logprob[r] = (float)log((double)w / (double)total);
  }
  row.cluster.sync();  // no block leaves while another reads its box
}

template <typename T>
int launch(const SampleArgs& a, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int vecs = (a.vocab + N - 1) / N + 1;  // one more where the row starts off a boundary
  const int blocks = vecs <= kThreads ? 1 : kMaxCluster;
  const int of_block = (vecs + blocks - 1) / blocks;
  const size_t bytes = sizeof(Shared) + (size_t)of_block * 16;
  static std::atomic<int> done[kMaxDevices];
  const int e = configure_once(done, [] {
    const size_t most = sizeof(Shared) + ((size_t)(kMaxVocab / N + 1 + kMaxCluster - 1) / kMaxCluster) * 16;
    return (int)cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)most);
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
  return (int)cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, of_block);
}

}  // namespace

int launch_sample(const SampleArgs& a, void* stream) {
  if (a.num_rows == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace gdn
